// Attention over a paged cache: the entry points (pfop_attention_paged).
#include "attention_runs.cuh"

namespace {

using namespace pf;

int pages_log(int page_size) {
  int l = 0;
  while ((1 << l) < page_size && l < 30) ++l;
  return l;
}

// What the call and the size query share.  (page ids are device data: the
// kernel looks at them)
int check_paged(int Hq, int Hkv, int hd, const pfop_attn_run* runs, int n_runs, bool tree, int words, int64_t* total) {
  const int rc = check_runs(Hq, Hkv, hd, runs, n_runs, -1, total);
  if (rc != PF_OK) return rc;
  if (tree) {
    if (words < 1 || words > MASK_WORDS_MAX) return runs_fail(PF_E_ARG, "mask_words outside [1, 4]");
    for (int r = 0; r < n_runs; ++r)
      if (runs[r].n_rows > 64 * words) return runs_fail(PF_E_ARG, "a run has more rows than its mask has bits");
  }
  return PF_OK;
}

}  // namespace

extern "C" int pfop_attention_paged(const void* q_dev, const void* k_dev, const void* v_dev, int32_t n_pages,
                                    int32_t page_size, int32_t Hq, int32_t Hkv, int32_t hd, const pfop_attn_run* runs,
                                    int32_t n_runs, const int32_t* table_dev, int64_t n_entries,
                                    const uint64_t* mask_dev, int32_t mask_words, void* out_dev, void* work_dev,
                                    int64_t work_bytes, void* stream) {
  if (page_size < 8 || (page_size & (page_size - 1)) != 0)
    return runs_fail(PF_E_ARG, "page_size must be a power of two, at least 8");
  if (n_pages < 0 || int64_t(n_pages) * page_size > (int64_t(1) << 31) - 1024)
    return runs_fail(PF_E_ARG, "n_pages negative or more than 2^31 - 1024 cells");
  const bool tree = mask_dev != nullptr;
  int64_t total = 0;
  const int rc = check_paged(Hq, Hkv, hd, runs, n_runs, tree, mask_words, &total);
  if (rc != PF_OK) return rc;
  const int page_log = pages_log(page_size);
  for (int r = 0; r < n_runs; ++r) {
    const int64_t end = static_cast<int64_t>(runs[r].pos0) + runs[r].n_rows;
    if (runs[r].n_rows > 0 && runs[r].cell0 + ((end + page_size - 1) >> page_log) > n_entries)
      return runs_fail(PF_E_ARG, "a run past the table's entries");
  }
  if (total == 0) return PF_OK;
  if (!q_dev || !k_dev || !v_dev || !table_dev || !out_dev || !work_dev || n_pages == 0)
    return runs_fail(PF_E_ARG, "null buffer, or no pages");
  if (((reinterpret_cast<uintptr_t>(q_dev) | reinterpret_cast<uintptr_t>(k_dev) | reinterpret_cast<uintptr_t>(v_dev)) & 15) ||
      (reinterpret_cast<uintptr_t>(out_dev) & 31))
    return runs_fail(PF_E_ARG, "q, k and v must be 16-byte aligned, out 32-byte aligned");
  if ((reinterpret_cast<uintptr_t>(mask_dev) & 7) || (reinterpret_cast<uintptr_t>(table_dev) & 3))
    return runs_fail(PF_E_ARG, "mask must be 8-byte aligned, the table 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(work_dev) & 255) return runs_fail(PF_E_ARG, "the scratch must be 256-byte aligned");
  RunsPlan p;
  if (!(tree ? make_plan<true>(p, runs, n_runs, Hq, Hkv, hd) : make_plan<false>(p, runs, n_runs, Hq, Hkv, hd)))
    return runs_fail(PF_E_ARG, TOO_MUCH);
  if (work_bytes < WORK_HEADER + p.state_bytes) return runs_fail(PF_E_ARG, "the scratch is smaller than these runs need");
  int* err = static_cast<int*>(work_dev);
  const int64_t n_cells = int64_t(n_pages) << page_log;
  const RunPages pages{table_dev, n_pages, page_log, static_cast<int>(n_cells), err + BAD_PAGE_AT};
  auto go = [&](auto launch) {
    return launch(p, static_cast<const __half*>(q_dev), static_cast<const __half*>(k_dev),
                  static_cast<const __half*>(v_dev), n_cells, static_cast<int>(total), mask_dev, mask_words,
                  static_cast<__nv_bfloat16*>(out_dev), static_cast<uint8_t*>(work_dev) + WORK_HEADER, err,
                  err + FLAGS_AT, pages, static_cast<cudaStream_t>(stream));
  };
  const cudaError_t e = hd == 256 ? (tree ? go(launch_runs<256, 2, true, RunPages>) : go(launch_runs<256, 2, false, RunPages>))
                        : p.cl == 2 ? (tree ? go(launch_runs<64, 2, true, RunPages>) : go(launch_runs<64, 2, false, RunPages>))
                                    : (tree ? go(launch_runs<64, 1, true, RunPages>) : go(launch_runs<64, 1, false, RunPages>));
  if (e != cudaSuccess) return runs_fail(PF_E_CUDA, std::string("paged attention launch: ") + cudaGetErrorString(e));
  return PF_OK;
}

extern "C" int64_t pfop_attention_paged_work_bytes(int32_t Hq, int32_t Hkv, int32_t hd, const pfop_attn_run* runs,
                                                   int32_t n_runs) {
  return pfop_attention_work_bytes(Hq, Hkv, hd, runs, n_runs);
}

extern "C" int pfop_attention_paged_status(void* work_dev, void* stream) {
  if (!work_dev) return runs_fail(PF_E_ARG, "null scratch");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int h[2] = {0, 0};
  static_assert(BAD_PAGE_AT == 1, "one copy brings both words");
  cudaError_t e = cudaMemcpyAsync(h, work_dev, sizeof(h), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && (h[0] || h[1])) {
    // over before this returns, since the next call may come on any stream
    e = cudaMemsetAsync(work_dev, 0, WORK_HEADER, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  if (e != cudaSuccess) return runs_fail(PF_E_CUDA, std::string("attention status: ") + cudaGetErrorString(e));
  if (h[0]) return runs_fail(PF_E_DEVICE_TIMEOUT, "attention gave up a bounded wait, code " + std::to_string(h[0]));
  if (h[1]) return runs_fail(PF_E_ARG, "a page id outside the cache");
  return PF_OK;
}
