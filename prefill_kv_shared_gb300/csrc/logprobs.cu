// Log probabilities of given tokens, entropy and the most probable
// alternatives of rows of logits (pfop_logprobs).
//
// With m = max x, t = (x - m) log2 e, s = sum 2^t and h = sum 2^t t over the
// vocabulary: log p[v] = (x[v] - m) - log s and entropy = log s - ln 2 h / s.
// One pass over the row: a thread keeps its own m, s, h (when m moves by d:
// s <- 2^-d s, h <- 2^-d (h - d s)), joined over the block and the cluster.
// t is held at -200 or above, so that a masked logit (-inf, or the type's
// lowest value) adds 2^t t = 0 and not 0 * inf; a NaN stays a NaN and marks
// the row as one without a distribution.
//
// The alternatives need no second look at the whole row: the n-th largest of
// the maxima of 32 groups of threads is not above the n-th largest value, so
// only threads whose own maximum reaches it read their logits again (from
// L2) and list those that do: a few dozen of a row as a rule, whose ranks
// are then counted.  Where the list overflows (many equal values, as in a
// row that is mostly masked) a radix select finds the n-th value and the
// lowest ids at it.
//
// Bound by the row's bytes from HBM for many rows, by latency for few: then
// a cluster of up to 8 CTAs takes a row, a slice each, and rank 0 joins
// their sums and lists through distributed shared memory.
#include "../../include/prefill_ops.h"
#include "common.cuh"
#include "kernels.h"

#include <string>

namespace pf {

constexpr int LP_THREADS = 256;
constexpr int LP_WARPS = LP_THREADS / 32;
constexpr int LP_TOP_MAX = 32;
constexpr int LP_GROUPS = LP_THREADS / 8;  // 32: one per lane
constexpr int LP_CAND = 512;               // listed candidates
constexpr int LP_CLUSTER_MAX = 8;
constexpr int LP_CTAS_PER_SM = 5;          // 48 registers a thread
constexpr float LP_LOG2E = 1.4426950408889634f, LP_LN2 = 0.6931471805599453f;
static_assert(LP_GROUPS == 32 && LP_TOP_MAX <= LP_GROUPS, "a lane per group");

struct LogprobArgs {
  const void* logits;
  int64_t ld;
  int vocab, slice;  // slice: logits per CTA of a cluster, a multiple of 8
  const int* tok;
  int n_top;
  float *logp, *entropy;
  int* top_id;
  float* top_logp;
};

__device__ __forceinline__ float lp_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lp_max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// 16 bytes of logits as floats
template <class T>
struct LpVec;
template <>
struct LpVec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4& r, float* v) {
    v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y), v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
};
template <>
struct LpVec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void get(const uint4& r, float* v) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
};

// values in order as unsigned numbers (-0 as 0), and back
__device__ __forceinline__ uint32_t lp_order(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float lp_value(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
// a value and its id as one key: larger values first, then lower ids
__device__ __forceinline__ unsigned long long lp_key(uint32_t order, int id) {
  return (static_cast<unsigned long long>(order) << 32) | (0xffffffffu - static_cast<uint32_t>(id));
}

// running maximum and sums
struct LpSums {
  float m = -INFINITY, s = 0.f, h = 0.f;
  __device__ __forceinline__ void raise(float to) {
    if (to > m) {
      if (m != -INFINITY) {
        const float d = (to - m) * LP_LOG2E, w = lp_ex2(-d);
        h = w * (h - d * s);
        s *= w;
        if (w == 0.f) s = h = s != s ? s : 0.f;  // d may be inf
      }
      m = to;
    }
  }
  __device__ __forceinline__ void join(float om, float os, float oh) {
    LpSums o;
    o.m = om, o.s = os, o.h = oh;
    raise(om);
    o.raise(m);
    s += o.s;
    h += o.h;
  }
};

// A thread's logits of the slice x[0 .. n): vectors tid, tid + 256, .. of the
// 16-byte aligned middle and one logit of each ragged end.  BATCH vectors
// are in flight; body(values, first id of each vector, count) per batch.
template <class T>
struct LpSlice {
  static constexpr int VN = LpVec<T>::N;
  const T* x;
  int n, head, nvec;
  __device__ LpSlice(const T* p, int len) : x(p), n(len) {
    const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    head = min(len, mis ? VN - mis : 0);
    nvec = (len - head) / VN;
  }
  // f(value, id in the slice) for this thread's logits, one at a time
  template <class F>
  __device__ __forceinline__ void each(F&& f) const {
    const int t = threadIdx.x;
    if (t < head) f(LpVec<T>::one(x + t), t);
    for (int v = t; v < nvec; v += LP_THREADS) {
      const int id = head + v * VN;
      float e[VN];
      LpVec<T>::get(__ldcg(reinterpret_cast<const uint4*>(x + id)), e);
#pragma unroll
      for (int i = 0; i < VN; ++i) f(e[i], id + i);
    }
    const int tail = head + nvec * VN;
    if (t < n - tail) f(LpVec<T>::one(x + tail + t), tail + t);
  }
  __device__ __forceinline__ void sums(LpSums& a) const {
    constexpr int BATCH = 4;
    const int t = threadIdx.x;
    auto add = [&](const float* e, int cnt) {
      float mx = e[0];
#pragma unroll
      for (int i = 1; i < BATCH * VN; ++i)
        if (i < cnt) mx = fmaxf(mx, e[i]);
      a.raise(mx);
      // x - m first: m log2 e alone may overflow
      const float m = a.m == -INFINITY ? 0.f : a.m;
      float s0 = 0.f, s1 = 0.f, h0 = 0.f, h1 = 0.f;
#pragma unroll
      for (int i = 0; i < BATCH * VN; i += 2) {
        if (i < cnt) {
          const float t0 = lp_max_nan((e[i] - m) * LP_LOG2E, -200.f), e0 = lp_ex2(t0);
          s0 += e0;
          h0 = __fmaf_rn(e0, t0, h0);
        }
        if (i + 1 < cnt) {
          const float t1 = lp_max_nan((e[i + 1] - m) * LP_LOG2E, -200.f), e1 = lp_ex2(t1);
          s1 += e1;
          h1 = __fmaf_rn(e1, t1, h1);
        }
      }
      a.s += s0 + s1;
      a.h += h0 + h1;
    };
    const uint4* xv = reinterpret_cast<const uint4*>(x + head);
    int v = t;
    for (; v + (BATCH - 1) * LP_THREADS < nvec; v += BATCH * LP_THREADS) {
      uint4 r[BATCH];
#pragma unroll
      for (int b = 0; b < BATCH; ++b) r[b] = __ldcg(xv + v + b * LP_THREADS);
      float e[BATCH * VN];
#pragma unroll
      for (int b = 0; b < BATCH; ++b) LpVec<T>::get(r[b], e + b * VN);
      add(e, BATCH * VN);
    }
    for (; v < nvec; v += LP_THREADS) {
      float e[BATCH * VN];
      LpVec<T>::get(__ldcg(xv + v), e);
      add(e, VN);
    }
    const int tail = head + nvec * VN;
    float e[BATCH * VN];
    if (t < head) {
      e[0] = LpVec<T>::one(x + t);
      add(e, 1);
    }
    if (t < n - tail) {
      e[0] = LpVec<T>::one(x + tail + t);
      add(e, 1);
    }
  }
};

struct LpShared {
  unsigned long long top[LP_TOP_MAX];                   // the CTA's best, in order
  unsigned long long all[LP_CLUSTER_MAX * LP_TOP_MAX];  // rank 0: the cluster's
  unsigned long long cand[LP_CAND];
  float4 sums[LP_CLUSTER_MAX];  // rank 0: m, s, h of each CTA
  float m[LP_WARPS], s[LP_WARPS], h[LP_WARPS];
  float group[LP_GROUPS];
  int hist[256];
  int count, prefix, left, found, warp_count[LP_WARPS];
};

// The n best of sh.cand[0 .. cnt) (all different) into dst, in order: a
// candidate's rank is the number of larger ones.
__device__ __forceinline__ void lp_rank(const unsigned long long* cand, int cnt, int n, unsigned long long* dst) {
  for (int i = threadIdx.x; i < cnt; i += LP_THREADS) {
    const unsigned long long k = cand[i];
    int r = 0;
    for (int j = 0; j < cnt; ++j) r += cand[j] > k ? 1 : 0;
    if (r < n) dst[r] = k;
  }
}

// The n best of a slice with too many candidates for the list: the n-th
// largest value by four passes over 8 bits of its order each, the larger
// ones, and the lowest ids at that value.
template <class T>
__device__ __noinline__ void lp_select(const LpSlice<T>& sl, int id0, int n, LpShared& sh) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t prefix = 0;
  int left = n;  // of the values with this prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += LP_THREADS) sh.hist[i] = 0;
    __syncthreads();
    sl.each([&](float v, int) {
      const uint32_t o = lp_order(v);
      if (shift == 24 || o >> (shift + 8) == prefix) atomicAdd(&sh.hist[o >> shift & 255], 1);
    });
    __syncthreads();
    if (warp == 0) {
      // lane: bins 8 lane .. + 7; those above it
      int own = 0;
      for (int i = 0; i < 8; ++i) own += sh.hist[8 * lane + i];
      int above = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_down_sync(0xffffffffu, above, o);
        if (lane + o < 32) above += v;
      }
      above -= own;
      if (above < left && above + own >= left) {
        int a = above;
        for (int i = 7; i >= 0; --i) {
          const int c = sh.hist[8 * lane + i];
          if (a + c >= left) {
            sh.prefix = static_cast<int>(prefix << 8 | static_cast<uint32_t>(8 * lane + i));
            sh.left = left - a;
            break;
          }
          a += c;
        }
      }
    }
    __syncthreads();
    prefix = static_cast<uint32_t>(sh.prefix);
    left = sh.left;
    __syncthreads();
  }
  // prefix: the n-th value; `left` of those equal to it are wanted
  if (tid == 0) sh.count = 0;
  __syncthreads();
  sl.each([&](float v, int i) {
    const uint32_t o = lp_order(v);
    if (o > prefix) sh.cand[atomicAdd(&sh.count, 1)] = lp_key(o, id0 + i);
  });
  __syncthreads();
  const int larger = sh.count;  // n - left
  int found = 0;
  for (int base = 0; base < sl.n && found < left; base += LP_THREADS) {
    const int i = base + tid;
    const bool eq = i < sl.n && lp_order(LpVec<T>::one(sl.x + i)) == prefix;
    const unsigned b = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) sh.warp_count[warp] = __popc(b);
    __syncthreads();
    int at = found, total = found;
    for (int w = 0; w < LP_WARPS; ++w) {
      if (w < warp) at += sh.warp_count[w];
      total += sh.warp_count[w];
    }
    at += __popc(b & ((1u << lane) - 1u));
    if (eq && at < left) sh.cand[larger + at] = lp_key(prefix, id0 + i);
    found = total;
    __syncthreads();
  }
  lp_rank(sh.cand, n, n, sh.top);
}

template <class T>
__global__ void __launch_bounds__(LP_THREADS, LP_CTAS_PER_SM) logprobs_kernel(const LogprobArgs a, int cluster) {
  __shared__ LpShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = static_cast<int>(blockIdx.x) / cluster, rank = static_cast<int>(blockIdx.x) % cluster;
  const T* x = static_cast<const T*>(a.logits) + static_cast<int64_t>(r) * a.ld;
  const int id0 = rank * a.slice;
  const LpSlice<T> sl(x + id0, min(a.vocab - id0, a.slice));
  pdl_launch();
  // no CTA writes into another before that one runs: arrive now, wait there
  if (cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  if (tid == 0) sh.count = 0;
  pdl_wait();

  LpSums q;
  sl.sums(q);
  const float own = q.m;
  // the block's sums
  {
    float g = own;  // the group's maximum
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
    if ((lane & 7) == 0) sh.group[tid >> 3] = g;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float om = __shfl_xor_sync(0xffffffffu, q.m, o), os = __shfl_xor_sync(0xffffffffu, q.s, o),
                  oh = __shfl_xor_sync(0xffffffffu, q.h, o);
      q.join(om, os, oh);
    }
    if (lane == 0) sh.m[warp] = q.m, sh.s[warp] = q.s, sh.h[warp] = q.h;
  }
  __syncthreads();
  const int n = a.n_top;
  if (n > 0) {
    // the n-th largest of the groups' maxima (every warp for itself)
    const float g = sh.group[lane];
    int rk = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float o = __shfl_sync(0xffffffffu, g, i);
      rk += (o > g || (o == g && i < lane)) ? 1 : 0;
    }
    const float tau = __shfl_sync(0xffffffffu, g, __ffs(__ballot_sync(0xffffffffu, rk == n - 1)) - 1);
    if (own >= tau) {
      const uint32_t ot = lp_order(tau);
      sl.each([&](float v, int i) {
        const uint32_t o = lp_order(v);
        if (o >= ot) {
          const int at = atomicAdd(&sh.count, 1);
          if (at < LP_CAND) sh.cand[at] = lp_key(o, id0 + i);
        }
      });
    }
    __syncthreads();
    const int cnt = sh.count;
    if (cnt <= LP_CAND) {
      lp_rank(sh.cand, cnt, n, sh.top);
    } else {
      __syncthreads();  // every thread has read the count
      lp_select(sl, id0, n, sh);
    }
  }
  const unsigned long long* top = sh.top;
  LpSums z;
  if (cluster > 1) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (warp == 0) {
      // the CTA's sums, to rank 0
      LpSums b;
      for (int w = 0; w < LP_WARPS; ++w) b.join(sh.m[w], sh.s[w], sh.h[w]);
      if (lane == 0) {
        const uint32_t at = map_to_rank(smem_u32(&sh.sums[rank]), 0);
        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(b.m), "f"(b.s), "f"(b.h), "f"(0.f)
                     : "memory");
      }
    }
    __syncthreads();  // the CTA's list is complete
    if (tid < n) {
      const uint32_t at = map_to_rank(smem_u32(&sh.all[rank * n + tid]), 0);
      asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(at), "l"(sh.top[tid]) : "memory");
    }
    cluster_sync_all();
    if (rank != 0) return;
    for (int c = 0; c < cluster; ++c) z.join(sh.sums[c].x, sh.sums[c].y, sh.sums[c].z);
    if (n > 0) {
      lp_rank(sh.all, cluster * n, n, sh.cand);
      top = sh.cand;
    }
  } else {
    for (int w = 0; w < LP_WARPS; ++w) z.join(sh.m[w], sh.s[w], sh.h[w]);
  }
  __syncthreads();
  const bool ok = z.s >= 1.f && z.m < INFINITY;  // false for a NaN too: a NaN, +inf, or only -inf
  const float nan = __int_as_float(0x7fc00000), log_s = logf(z.s);
  if (tid < n) {
    const unsigned long long k = top[tid];
    const int64_t at = static_cast<int64_t>(r) * n + tid;
    a.top_id[at] = ok ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(k)) : -1;
    a.top_logp[at] = ok ? lp_value(static_cast<uint32_t>(k >> 32)) - z.m - log_s : nan;
  }
  if (tid == LP_THREADS - 1 && a.logp) {
    const int t = a.tok[r];
    a.logp[r] = ok && t >= 0 && t < a.vocab ? LpVec<T>::one(x + t) - z.m - log_s : nan;
  }
  if (tid == LP_THREADS - 2 && a.entropy) a.entropy[r] = ok ? log_s - LP_LN2 * (z.h / z.s) : nan;
}

// CTAs per row: as many as the GPU holds at once, each with at least
// LP_SLICE_MIN logits.
constexpr int LP_SLICE_MIN = 2048;

template <class T>
static cudaError_t launch_logprobs(LogprobArgs a, int rows, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  int cluster = LP_CLUSTER_MAX;
  while (cluster > 1 && (static_cast<int64_t>(rows) * cluster > static_cast<int64_t>(LP_CTAS_PER_SM) * sms || a.vocab / cluster < LP_SLICE_MIN))
    cluster /= 2;
  a.slice = ((a.vocab + cluster - 1) / cluster + 7) / 8 * 8;
  return launch_k(logprobs_kernel<T>, dim3(static_cast<unsigned>(rows) * cluster), dim3(LP_THREADS), 0, s, cluster, a,
                  cluster);
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
  const LogprobArgs a{logits_dev, ld, vocab, 0, tok_dev, n_top, logp_dev, entropy_dev, top_id_dev, top_logp_dev};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      ltype == PF_L_F32 ? launch_logprobs<float>(a, rows, s) : launch_logprobs<__nv_bfloat16>(a, rows, s);
  if (e != cudaSuccess) return fail(PF_E_CUDA, std::string("log probabilities launch: ") + cudaGetErrorString(e));
  return PF_OK;
}
