// Attention over runs of a contiguous cache: the entry points
// (pfop_attention_packed, pfop_attention_tree).
#include "attention_runs.cuh"

namespace {

using namespace pf;

int run_attention(bool tree, const void* q, const void* k, const void* v, int64_t n_cells, int Hq, int Hkv, int hd,
                  const pfop_attn_run* runs, int n_runs, const uint64_t* mask, int words, void* out, void* work,
                  int64_t work_bytes, cudaStream_t s) {
  if (n_cells < 0 || n_cells > (int64_t(1) << 31) - 1024) return runs_fail(PF_E_ARG, "n_cells outside [0, 2^31 - 1024]");
  int64_t total = 0;
  int rc = check_runs(Hq, Hkv, hd, runs, n_runs, n_cells, &total);
  if (rc != PF_OK) return rc;
  if (tree) {
    if (words < 1 || words > MASK_WORDS_MAX) return runs_fail(PF_E_ARG, "mask_words outside [1, 4]");
    for (int r = 0; r < n_runs; ++r)
      if (runs[r].n_rows > 64 * words) return runs_fail(PF_E_ARG, "a run has more rows than its mask has bits");
  }
  if (total == 0) return PF_OK;
  if (!q || !k || !v || !out || !work || (tree && !mask)) return runs_fail(PF_E_ARG, "null buffer");
  if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15) ||
      (reinterpret_cast<uintptr_t>(out) & 31))
    return runs_fail(PF_E_ARG, "q, k and v must be 16-byte aligned, out 32-byte aligned");
  if (tree && (reinterpret_cast<uintptr_t>(mask) & 7)) return runs_fail(PF_E_ARG, "mask must be 8-byte aligned");
  if (reinterpret_cast<uintptr_t>(work) & 255) return runs_fail(PF_E_ARG, "the scratch must be 256-byte aligned");
  RunsPlan p;
  if (!(tree ? make_plan<true>(p, runs, n_runs, Hq, Hkv, hd) : make_plan<false>(p, runs, n_runs, Hq, Hkv, hd)))
    return runs_fail(PF_E_ARG, TOO_MUCH);
  if (work_bytes < WORK_HEADER + p.state_bytes) return runs_fail(PF_E_ARG, "the scratch is smaller than these runs need");
  int* err = static_cast<int*>(work);
  uint8_t* states = static_cast<uint8_t*>(work) + WORK_HEADER;
  auto go = [&](auto launch) {
    return launch(p, static_cast<const __half*>(q), static_cast<const __half*>(k), static_cast<const __half*>(v),
                  n_cells, static_cast<int>(total), mask, words, static_cast<__nv_bfloat16*>(out), states, err, err + FLAGS_AT,
                  NoPages{}, s);
  };
  const cudaError_t e = hd == 256   ? (tree ? go(launch_runs<256, 2, true, NoPages>) : go(launch_runs<256, 2, false, NoPages>))
                        : p.cl == 2 ? (tree ? go(launch_runs<64, 2, true, NoPages>) : go(launch_runs<64, 2, false, NoPages>))
                                    : (tree ? go(launch_runs<64, 1, true, NoPages>) : go(launch_runs<64, 1, false, NoPages>));
  if (e != cudaSuccess) return runs_fail(PF_E_CUDA, std::string("attention launch: ") + cudaGetErrorString(e));
  return PF_OK;
}

}  // namespace

extern "C" int pfop_attention_packed(const void* q_dev, const void* k_dev, const void* v_dev, int64_t n_cells,
                                     int32_t Hq, int32_t Hkv, int32_t hd, const pfop_attn_run* runs, int32_t n_runs,
                                     void* out_dev, void* work_dev, int64_t work_bytes, void* stream) {
  return run_attention(false, q_dev, k_dev, v_dev, n_cells, Hq, Hkv, hd, runs, n_runs, nullptr, 0, out_dev, work_dev,
                       work_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" int pfop_attention_tree(const void* q_dev, const void* k_dev, const void* v_dev, int64_t n_cells,
                                   int32_t Hq, int32_t Hkv, int32_t hd, const pfop_attn_run* runs, int32_t n_runs,
                                   const uint64_t* mask_dev, int32_t mask_words, void* out_dev, void* work_dev,
                                   int64_t work_bytes, void* stream) {
  return run_attention(true, q_dev, k_dev, v_dev, n_cells, Hq, Hkv, hd, runs, n_runs, mask_dev, mask_words, out_dev,
                       work_dev, work_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" int64_t pfop_attention_work_bytes(int32_t Hq, int32_t Hkv, int32_t hd, const pfop_attn_run* runs,
                                             int32_t n_runs) {
  int64_t total = 0;
  const int rc = check_runs(Hq, Hkv, hd, runs, n_runs, -1, &total);
  if (rc != PF_OK) return rc;
  if (total == 0) return WORK_HEADER;
  RunsPlan a, b;
  if (!make_plan<false>(a, runs, n_runs, Hq, Hkv, hd)) return runs_fail(PF_E_ARG, TOO_MUCH);
  // a tree's rows all see the whole context: runs that no tree has are not
  // counted as one, and what only the tree call refuses it refuses itself
  bool tree = true;
  for (int r = 0; r < n_runs; ++r) tree = tree && runs[r].n_rows <= 64 * MASK_WORDS_MAX;
  const bool both = tree && make_plan<true>(b, runs, n_runs, Hq, Hkv, hd);
  return WORK_HEADER + std::max(a.state_bytes, both ? b.state_bytes : 0);
}

extern "C" int pfop_attention_status(void* work_dev, void* stream) {
  if (!work_dev) return runs_fail(PF_E_ARG, "null scratch");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int h = 0;
  cudaError_t e = cudaMemcpyAsync(&h, work_dev, 4, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && h) {
    // flags of a call that gave up too; over before this returns, since the next call may come on any stream
    e = cudaMemsetAsync(work_dev, 0, WORK_HEADER, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  if (e != cudaSuccess) return runs_fail(PF_E_CUDA, std::string("attention status: ") + cudaGetErrorString(e));
  if (h) return runs_fail(PF_E_DEVICE_TIMEOUT, "attention gave up a bounded wait, code " + std::to_string(h));
  return PF_OK;
}
