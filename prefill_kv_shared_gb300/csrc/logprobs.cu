// Log probabilities of given tokens, entropy and the most probable
// alternatives of rows of logits (pfop_logprobs).
//
// With m = max x, d = x - m, s = sum e^d: log p[v] = d[v] - log s and
// entropy = log s - (sum e^d d) / s; terms with e^d = 0 add nothing (d may
// be -inf there).
#include "../../include/prefill_ops.h"
#include "common.cuh"
#include "kernels.h"

#include <string>

namespace pf {

constexpr int LP_THREADS = 256;
constexpr int LP_TOP_MAX = 32;

struct LogprobArgs {
  const void* logits;
  int64_t ld;
  int vocab;
  const int* tok;
  int n_top;
  float *logp, *entropy;
  int* top_id;
  float* top_logp;
};

__device__ __forceinline__ float lp_load(const float* p) { return *p; }
__device__ __forceinline__ float lp_load(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// sum over the block, the same value in every thread (fixed order)
__device__ __forceinline__ float lp_block_sum(float v, float* red) {
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
  for (int w = 0; w < LP_THREADS / 32; ++w) t += red[w];
  return t;
}

// A value and its id as one key: larger values first, then smaller ids.
__device__ __forceinline__ unsigned long long lp_key(float x, int id) {
  const uint32_t b = __float_as_uint(x + 0.f);  // -0 counts as 0
  const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (static_cast<unsigned long long>(o) << 32) | (0xffffffffu - static_cast<uint32_t>(id));
}

template <class T>
__global__ void __launch_bounds__(LP_THREADS) logprobs_kernel(const LogprobArgs a) {
  __shared__ float red[LP_THREADS / 32];
  __shared__ unsigned long long best;
  pdl_launch();
  pdl_wait();
  const int r = blockIdx.x;
  const T* x = static_cast<const T*>(a.logits) + static_cast<int64_t>(r) * a.ld;
  float m = -INFINITY;
  for (int v = threadIdx.x; v < a.vocab; v += LP_THREADS) m = fmaxf(m, lp_load(x + v));
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = m;
  __syncthreads();
  for (int w = 0; w < LP_THREADS / 32; ++w) m = fmaxf(m, red[w]);
  float s = 0.f, s1 = 0.f;
  for (int v = threadIdx.x; v < a.vocab; v += LP_THREADS) {
    const float d = lp_load(x + v) - m, e = expf(d);
    s += e;
    if (e != 0.f) s1 += e * d;
  }
  s = lp_block_sum(s, red);
  s1 = lp_block_sum(s1, red);
  const bool ok = s >= 1.f;  // false where s is NaN: a NaN, +inf, or only -inf
  const float nan = __int_as_float(0x7fc00000), log_s = logf(s);
  if (threadIdx.x == 0) {
    if (a.logp) {
      const int t = a.tok[r];
      a.logp[r] = ok && t >= 0 && t < a.vocab ? lp_load(x + t) - m - log_s : nan;
    }
    if (a.entropy) a.entropy[r] = ok ? log_s - s1 / s : nan;
  }
  unsigned long long last = ~0ull;
  for (int i = 0; i < a.n_top; ++i) {
    if (threadIdx.x == 0) best = 0;
    __syncthreads();
    unsigned long long b = 0;
    for (int v = threadIdx.x; v < a.vocab; v += LP_THREADS) {
      const unsigned long long key = lp_key(lp_load(x + v), v);
      if (key < last && key > b) b = key;
    }
    atomicMax(&best, b);
    __syncthreads();
    last = best;
    if (threadIdx.x == 0) {
      const int id = static_cast<int>(0xffffffffu - static_cast<uint32_t>(last));
      a.top_id[static_cast<int64_t>(r) * a.n_top + i] = ok ? id : -1;
      a.top_logp[static_cast<int64_t>(r) * a.n_top + i] = ok ? lp_load(x + id) - m - log_s : nan;
    }
    __syncthreads();
  }
}

}  // namespace pf

extern "C" int pfop_logprobs(int32_t ltype, const void* logits_dev, int64_t ld, int32_t rows, int32_t vocab,
                             const int32_t* tok_dev, int32_t n_top, float* logp_dev, float* entropy_dev,
                             int32_t* top_id_dev, float* top_logp_dev, void* stream) {
  using namespace pf;
  auto fail = [](int code, const std::string& m) {
    set_op_error(m);
    return code;
  };
  if (ltype != PF_L_F32 && ltype != PF_L_BF16) return fail(PF_E_ARG, "ltype");
  if (rows < 0 || vocab < 1 || vocab >= (1 << 30) || ld < vocab) return fail(PF_E_ARG, "rows, vocab or ld");
  if (n_top < 0 || n_top > LP_TOP_MAX || n_top > vocab) return fail(PF_E_ARG, "n_top outside [0, min(32, vocab)]");
  if (rows == 0) return PF_OK;
  if (!logits_dev || (tok_dev == nullptr) != (logp_dev == nullptr) || (n_top > 0 && (!top_id_dev || !top_logp_dev)))
    return fail(PF_E_ARG, "missing buffer");
  const uintptr_t out = reinterpret_cast<uintptr_t>(tok_dev) | reinterpret_cast<uintptr_t>(logp_dev) |
                        reinterpret_cast<uintptr_t>(entropy_dev) |
                        (n_top > 0 ? reinterpret_cast<uintptr_t>(top_id_dev) | reinterpret_cast<uintptr_t>(top_logp_dev) : 0);
  if ((out & 3) || (reinterpret_cast<uintptr_t>(logits_dev) & (ltype == PF_L_F32 ? 3 : 1)))
    return fail(PF_E_ARG, "misaligned buffer");
  const LogprobArgs a{logits_dev, ld, vocab, tok_dev, n_top, logp_dev, entropy_dev, top_id_dev, top_logp_dev};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      ltype == PF_L_F32 ? launch_k(logprobs_kernel<float>, dim3(rows), dim3(LP_THREADS), 0, s, 1, a)
                        : launch_k(logprobs_kernel<__nv_bfloat16>, dim3(rows), dim3(LP_THREADS), 0, s, 1, a);
  if (e != cudaSuccess) return fail(PF_E_CUDA, std::string("log probabilities launch: ") + cudaGetErrorString(e));
  return PF_OK;
}
