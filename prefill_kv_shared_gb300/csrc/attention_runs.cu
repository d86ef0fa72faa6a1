// Attention of several sequences' rows in one call (pfop_attention_packed,
// pfop_attention_tree): causal over each sequence's own keys, or over a
// context and a tree of drafted tokens.
#include "../../include/prefill_ops.h"
#include "attn.cuh"
#include "common.cuh"
#include "kernels.h"

#include <string>

namespace pf {

constexpr int RUNS_MAX = 128;

// the call's runs, passed in the kernel's parameters
struct RunTable {
  int n_runs = 0;
  int row0[RUNS_MAX];  // first packed row
  int n[RUNS_MAX], pos0[RUNS_MAX], cell0[RUNS_MAX];
};

// A warp per (row, query head): lane owns HD/32 dims, keys in ascending
// order, one online softmax.
template <int HD, bool TREE>
__global__ void __launch_bounds__(256) attn_runs_kernel(const __grid_constant__ RunTable rt, const __half* q,
                                                        const __half* k, const __half* v, int Hq, int Hkv,
                                                        const uint64_t* mask, int words, int total,
                                                        __nv_bfloat16* out) {
  constexpr int PER = HD / 32;
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int64_t pair = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int t = static_cast<int>(pair / Hq), h = static_cast<int>(pair % Hq);
  if (t >= total) return;
  int r = 0;
  while (r + 1 < rt.n_runs && rt.row0[r + 1] <= t) ++r;
  const int i = t - rt.row0[r], n = rt.n[r], pos0 = rt.pos0[r];
  const int kvh = h / (Hq / Hkv);
  float qf[PER], o[PER];
  for (int d = 0; d < PER; ++d) {
    qf[d] = __half2float(q[(static_cast<size_t>(t) * Hq + h) * HD + lane * PER + d]) * attn_c<HD>();
    o[d] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int keys = TREE ? pos0 + n : pos0 + i + 1;
  for (int j = 0; j < keys; ++j) {
    if (TREE && j >= pos0) {
      const int d = j - pos0;
      if (!(mask[static_cast<size_t>(t) * words + d / 64] >> (d % 64) & 1)) continue;
    }
    const size_t row = (static_cast<size_t>(rt.cell0[r] + j) * Hkv + kvh) * HD + lane * PER;
    float s = 0.f;
    for (int d = 0; d < PER; ++d) s = __fmaf_rn(qf[d], __half2float(k[row + d]), s);
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    const float mn = fmaxf(m, s);
    const float a = m == -INFINITY ? 0.f : ex2_approx(m - mn);
    const float p = mn == -INFINITY ? 0.f : ex2_approx(s - mn);
    l = l * a + p;
    for (int d = 0; d < PER; ++d) o[d] = o[d] * a + p * __half2float(v[row + d]);
    m = mn;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  for (int d = 0; d < PER; ++d)
    out[(static_cast<size_t>(t) * Hq + h) * HD + lane * PER + d] = __float2bfloat16(o[d] * inv);
}

}  // namespace pf

namespace {

using namespace pf;

constexpr int64_t WORK_HEADER = 256;  // the error word, alone in its lines

int fail(int code, const std::string& m) {
  set_op_error(m);
  return code;
}

// The checks that both calls and the size query share; *total = the runs' rows.
int check_runs(int Hq, int Hkv, int hd, const pfop_attn_run* runs, int n_runs, int64_t n_cells, int64_t* total) {
  if (hd != 64 && hd != 256) return fail(PF_E_ARG, "head_dim must be 64 or 256");
  if (Hq < 1 || Hkv < 1 || Hq > 1024 || Hq % Hkv != 0 || Hq / Hkv > 16 || 16 % (Hq / Hkv) != 0)
    return fail(PF_E_ARG, "n_head must be a multiple of n_head_kv with a group size dividing 16, at most 1024");
  if (n_runs < 0 || n_runs > RUNS_MAX) return fail(PF_E_ARG, "n_runs outside [0, 128]");
  if (n_runs > 0 && !runs) return fail(PF_E_ARG, "runs is null");
  int64_t t = 0;
  for (int r = 0; r < n_runs; ++r) {
    if (runs[r].n_rows < 0 || runs[r].pos0 < 0 || runs[r].cell0 < 0) return fail(PF_E_ARG, "a negative run field");
    t += runs[r].n_rows;
    const int64_t end = static_cast<int64_t>(runs[r].pos0) + runs[r].n_rows;
    if (end > (int64_t(1) << 30)) return fail(PF_E_ARG, "a run past position 2^30");
    if (n_cells >= 0 && runs[r].n_rows > 0 && runs[r].cell0 + end > n_cells)
      return fail(PF_E_ARG, "a run past the cache's cells");
  }
  if (t > (1 << 20)) return fail(PF_E_ARG, "more than 2^20 rows");
  *total = t;
  return PF_OK;
}

int run_attention(bool tree, const void* q, const void* k, const void* v, int64_t n_cells, int Hq, int Hkv, int hd,
                  const pfop_attn_run* runs, int n_runs, const uint64_t* mask, int words, void* out, void* work,
                  int64_t work_bytes, cudaStream_t s) {
  if (n_cells < 0 || n_cells > (int64_t(1) << 31) - 1024) return fail(PF_E_ARG, "n_cells outside [0, 2^31 - 1024]");
  int64_t total = 0;
  int rc = check_runs(Hq, Hkv, hd, runs, n_runs, n_cells, &total);
  if (rc != PF_OK) return rc;
  if (tree) {
    if (words < 1 || words > 4) return fail(PF_E_ARG, "mask_words outside [1, 4]");
    for (int r = 0; r < n_runs; ++r)
      if (runs[r].n_rows > 64 * words) return fail(PF_E_ARG, "a run has more rows than its mask has bits");
  }
  if (total == 0) return PF_OK;
  if (!q || !k || !v || !out || !work || (tree && !mask)) return fail(PF_E_ARG, "null buffer");
  if ((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) |
       reinterpret_cast<uintptr_t>(out)) & 15)
    return fail(PF_E_ARG, "q, k, v and out must be 16-byte aligned");
  if (tree && (reinterpret_cast<uintptr_t>(mask) & 7)) return fail(PF_E_ARG, "mask must be 8-byte aligned");
  if (reinterpret_cast<uintptr_t>(work) & 255) return fail(PF_E_ARG, "the scratch must be 256-byte aligned");
  if (work_bytes < WORK_HEADER) return fail(PF_E_ARG, "the scratch is smaller than these runs need");
  RunTable rt;
  int row = 0;
  for (int r = 0; r < n_runs; ++r) {
    if (runs[r].n_rows > 0) {
      const int i = rt.n_runs++;
      rt.row0[i] = row;
      rt.n[i] = runs[r].n_rows;
      rt.pos0[i] = runs[r].pos0;
      rt.cell0[i] = runs[r].cell0;
    }
    row += runs[r].n_rows;
  }
  const dim3 grid(static_cast<unsigned>((total * Hq + 7) / 8));
  auto go = [&](auto kernel) {
    return launch_k(kernel, grid, dim3(256), 0, s, 1, rt, static_cast<const __half*>(q), static_cast<const __half*>(k),
                    static_cast<const __half*>(v), Hq, Hkv, mask, words, static_cast<int>(total),
                    static_cast<__nv_bfloat16*>(out));
  };
  const cudaError_t e = hd == 256 ? (tree ? go(attn_runs_kernel<256, true>) : go(attn_runs_kernel<256, false>))
                                  : (tree ? go(attn_runs_kernel<64, true>) : go(attn_runs_kernel<64, false>));
  if (e != cudaSuccess) return fail(PF_E_CUDA, std::string("attention launch: ") + cudaGetErrorString(e));
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
  return rc != PF_OK ? rc : WORK_HEADER;
}

extern "C" int pfop_attention_status(void* work_dev, void* stream) {
  if (!work_dev) return fail(PF_E_ARG, "null scratch");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int h = 0;
  cudaError_t e = cudaMemcpyAsync(&h, work_dev, 4, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && h) e = cudaMemsetAsync(work_dev, 0, 4, s);
  if (e != cudaSuccess) return fail(PF_E_CUDA, std::string("attention status: ") + cudaGetErrorString(e));
  if (h) return fail(PF_E_DEVICE_TIMEOUT, "attention gave up a bounded wait, code " + std::to_string(h));
  return PF_OK;
}
