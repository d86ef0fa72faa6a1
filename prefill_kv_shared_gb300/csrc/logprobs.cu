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
// only threads whose own maximum reaches it go over their logits again and
// list those that do: a few dozen of a row as a rule, whose ranks are then
// counted.  Where the list overflows (many equal values, as in a row that is
// mostly masked) a radix select finds the n-th value and the lowest ids at it.
//
// A CTA takes a row, or a cluster of up to 8 a slice each (rank 0 joins their
// sums and lists through distributed shared memory).  A slice of up to 64 KB
// is brought into shared memory by one bulk copy, which keeps the HBM busy
// with no registers held and makes the second look cheap; longer slices are
// read through registers, and again from L2.  Bound by the row's bytes for
// many rows, by latency for few.
#include "../../include/prefill_ops.h"
#include "common.cuh"
#include "kernels.h"

#include <string>

namespace pf {

constexpr int LP_THREADS = 256;
constexpr int LP_WARPS = LP_THREADS / 32;
constexpr int LP_TOP_MAX = 32;
constexpr int LP_GROUP = LP_THREADS / 32;  // threads of a group
constexpr int LP_CAND = 512;               // listed candidates
constexpr int LP_CLUSTER_MAX = 8;
constexpr int LP_SMEM_SLICE = 65536;       // bytes of a slice held in shared memory
constexpr int LP_CTAS_PER_SM = 3;          // by 64 KB slices
constexpr float LP_LOG2E = 1.4426950408889634f, LP_LN2 = 0.6931471805599453f;
static_assert(LP_TOP_MAX <= 32 && LP_GROUP <= 32, "a lane per group");

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
  // the sums against a maximum `to` >= m
  __device__ __forceinline__ void rebase(float to) {
    const float d = (to - m) * LP_LOG2E, w = lp_ex2(-d);
    // w 0 (nothing seen yet, or d infinite): a NaN stays, else nothing is left
    const float z = s != s ? s : 0.f;
    h = w == 0.f || m == -INFINITY ? z : w * (h - d * s);
    s = w == 0.f || m == -INFINITY ? z : w * s;
    m = to;
  }
  __device__ __forceinline__ void raise(float to) {
    if (to > m) rebase(to);
  }
  // over the warp, the same in every lane
  __device__ __forceinline__ void join() {
    float to = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, o));
    rebase(to);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      h += __shfl_xor_sync(0xffffffffu, h, o);
    }
  }
};

__device__ __forceinline__ uint64_t lp_pack(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 lp_unpack(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}

// A thread's logits of the slice x[0 .. n) (SM: in shared memory, else in
// global): vectors tid, tid + LP_THREADS, .. of the 16-byte aligned middle
// and one logit of each ragged end.
template <class T, bool SM>
struct LpSlice {
  static constexpr int VN = LpVec<T>::N;
  static constexpr int BATCH = 4;  // vectors taken at once
  const T* x;
  int n, head, nvec;
  __device__ LpSlice(const T* p, int len, int mis) : x(p), n(len) {
    head = min(len, mis ? VN - mis : 0);
    nvec = (len - head) / VN;
  }
  __device__ __forceinline__ uint4 vec(int v) const {
    const uint4* p = reinterpret_cast<const uint4*>(x + head) + v;
    return SM ? *p : __ldcg(p);
  }
  // f(value, id in the slice) for the logits of at least tau among those of
  // thread t, its vectors dealt out over the warp
  template <class F>
  __device__ __forceinline__ void from(int t, float tau, F&& f) const {
    const int lane = threadIdx.x & 31;
    auto one = [&](float v, int i) {
      if (v >= tau) f(v, i);
    };
    for (int v = t + lane * LP_THREADS; v < nvec; v += 32 * LP_THREADS) {
      float e[VN];
      LpVec<T>::get(vec(v), e);
      float mx = e[0];
#pragma unroll
      for (int i = 1; i < VN; ++i) mx = fmaxf(mx, e[i]);
      if (mx >= tau) {
#pragma unroll
        for (int i = 0; i < VN; ++i) one(e[i], head + v * VN + i);
      }
    }
    const int tail = head + nvec * VN;
    if (lane == 0 && t < head) one(LpVec<T>::one(x + t), t);
    if (lane == 0 && t < n - tail) one(LpVec<T>::one(x + tail + t), tail + t);
  }
  // f(value, id in the slice) for all of them
  template <class F>
  __device__ __forceinline__ void each(F&& f) const {
    const int t = threadIdx.x;
    if (t < head) f(LpVec<T>::one(x + t), t);
    int v = t;
    for (; v < nvec; v += BATCH * LP_THREADS) {
      uint4 r[BATCH];
#pragma unroll
      for (int b = 0; b < BATCH; ++b) r[b] = v + b * LP_THREADS < nvec ? vec(v + b * LP_THREADS) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        if (v + b * LP_THREADS >= nvec) break;
        float e[VN];
        LpVec<T>::get(r[b], e);
#pragma unroll
        for (int i = 0; i < VN; ++i) f(e[i], head + (v + b * LP_THREADS) * VN + i);
      }
    }
    const int tail = head + nvec * VN;
    if (t < n - tail) f(LpVec<T>::one(x + tail + t), tail + t);
  }
  template <int CNT>
  static __device__ __forceinline__ void add(LpSums& a, const float* e) {
    float mx = e[0];
#pragma unroll
    for (int i = 1; i < CNT; ++i) mx = fmaxf(mx, e[i]);
    a.raise(mx);
    // x - m first: m log2 e alone may overflow
    const float m = a.m == -INFINITY ? 0.f : a.m;
    if constexpr (CNT == 1) {
      const float t = lp_max_nan((e[0] - m) * LP_LOG2E, -200.f), w = lp_ex2(t);
      a.s += w;
      a.h = __fmaf_rn(w, t, a.h);
    } else {
      // two logits an instruction
      const uint64_t nm = lp_pack(-m, -m), c = lp_pack(LP_LOG2E, LP_LOG2E);
      uint64_t s[2] = {0ull, 0ull}, h[2] = {0ull, 0ull};
#pragma unroll
      for (int i = 0; i < CNT; i += 2) {
        uint64_t d = lp_pack(e[i], e[i + 1]);
        asm("add.rn.f32x2 %0, %0, %1;" : "+l"(d) : "l"(nm));
        asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(d) : "l"(c));
        float2 t = lp_unpack(d);
        t.x = lp_max_nan(t.x, -200.f);
        t.y = lp_max_nan(t.y, -200.f);
        const uint64_t w = lp_pack(lp_ex2(t.x), lp_ex2(t.y)), tt = lp_pack(t.x, t.y);
        const int q = (i >> 1) & 1;
        asm("add.rn.f32x2 %0, %0, %1;" : "+l"(s[q]) : "l"(w));
        asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(h[q]) : "l"(w), "l"(tt));
      }
      const float2 s0 = lp_unpack(s[0]), s1 = lp_unpack(s[1]), h0 = lp_unpack(h[0]), h1 = lp_unpack(h[1]);
      a.s += (s0.x + s0.y) + (s1.x + s1.y);
      a.h += (h0.x + h0.y) + (h1.x + h1.y);
    }
  }
  __device__ __forceinline__ void sums(LpSums& a) const {
    const int t = threadIdx.x;
    int v = t;
    if constexpr (SM) {
      for (; v + (BATCH - 1) * LP_THREADS < nvec; v += BATCH * LP_THREADS) {
        float e[BATCH * VN];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) LpVec<T>::get(vec(v + b * LP_THREADS), e + b * VN);
        add<BATCH * VN>(a, e);
      }
    } else if (v + (BATCH - 1) * LP_THREADS < nvec) {
      // the next batch is on its way while this one is taken
      uint4 r[BATCH];
#pragma unroll
      for (int b = 0; b < BATCH; ++b) r[b] = vec(v + b * LP_THREADS);
      for (;;) {
        const int w = v + BATCH * LP_THREADS;
        const bool more = w + (BATCH - 1) * LP_THREADS < nvec;
        float e[BATCH * VN];
#pragma unroll
        for (int b = 0; b < BATCH; ++b) LpVec<T>::get(r[b], e + b * VN);
        if (more) {
#pragma unroll
          for (int b = 0; b < BATCH; ++b) r[b] = vec(w + b * LP_THREADS);
        }
        add<BATCH * VN>(a, e);
        v = w;
        if (!more) break;
      }
    }
    for (; v < nvec; v += LP_THREADS) {
      float e[VN];
      LpVec<T>::get(vec(v), e);
      add<VN>(a, e);
    }
    const int tail = head + nvec * VN;
    if (t < head) {
      const float e = LpVec<T>::one(x + t);
      add<1>(a, &e);
    }
    if (t < n - tail) {
      const float e = LpVec<T>::one(x + tail + t);
      add<1>(a, &e);
    }
  }
};

struct LpShared {
  unsigned long long top[LP_TOP_MAX];                   // the CTA's best, in order
  unsigned long long all[LP_CLUSTER_MAX * LP_TOP_MAX];  // rank 0: the cluster's
  unsigned long long cand[LP_CAND];
  float4 sums[LP_CLUSTER_MAX];  // rank 0: m, s, h of each CTA
  float m[LP_WARPS], s[LP_WARPS], h[LP_WARPS];
  float group[32];
  int hist[256];
  float tau;
  int queue[LP_THREADS];  // threads that reach tau
  int queued, count, prefix, left, warp_count[LP_WARPS];
  uint64_t landed;  // barrier of the slice's copy
};

// The n best of sh.cand[0 .. cnt) (all different) into dst, in order: a
// candidate's rank is the number of larger ones.
__device__ __forceinline__ void lp_rank(const unsigned long long* cand, int cnt, int n, unsigned long long* dst) {
  for (int i = threadIdx.x; i < cnt; i += LP_THREADS) {
    const unsigned long long k = cand[i];
    int r = 0;
#pragma unroll 8
    for (int j = 0; j < cnt; ++j) r += cand[j] > k ? 1 : 0;
    if (r < n) dst[r] = k;
  }
}

// The n best of a slice with too many candidates for the list: the n-th
// largest value by four passes over 8 bits of its order each, the larger
// ones, and the lowest ids at that value.
template <class T, bool SM>
__device__ __noinline__ void lp_select(const LpSlice<T, SM>& sl, int id0, int n, LpShared& sh) {
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

template <class T, bool SM>
__global__ void __launch_bounds__(LP_THREADS, SM ? LP_CTAS_PER_SM : 2) logprobs_kernel(const LogprobArgs a, int cluster) {
  __shared__ LpShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r = static_cast<int>(blockIdx.x) / cluster, rank = static_cast<int>(blockIdx.x) % cluster;
  const T* x = static_cast<const T*>(a.logits) + static_cast<int64_t>(r) * a.ld;
  const int id0 = rank * a.slice;
  const int len = min(a.vocab - id0, a.slice);
  const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(x + id0) & 15) / sizeof(T));
  extern __shared__ __align__(16) uint8_t lp_slice[];
  // the copy keeps the logits' alignment
  const LpSlice<T, SM> sl(SM ? reinterpret_cast<const T*>(lp_slice) + mis : x + id0, len, mis);
  pdl_launch();
  // no CTA writes into another before that one runs: arrive now, wait there
  if (cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  if (tid == 0) {
    sh.count = sh.queued = 0;
    if (SM) {
      mbar_init(&sh.landed, 1);
      fence_mbar_init();
    }
  }
  bool landed = true;
  if constexpr (SM) {
    __syncthreads();
    pdl_wait();
    T* d = reinterpret_cast<T*>(lp_slice) + mis;
    if (tid == 0) {
      const uint32_t bytes = static_cast<uint32_t>(sl.nvec) * 16u;
      mbar_arrive_expect_tx(&sh.landed, bytes);
      if (bytes) bulk_load(d + sl.head, x + id0 + sl.head, bytes, &sh.landed);
    }
    const int tail = sl.head + sl.nvec * LpVec<T>::N;
    if (tid < sl.head) d[tid] = x[id0 + tid];
    if (tid < len - tail) d[tail + tid] = x[id0 + tail + tid];
    // a copy that never lands (the bounded wait gives up) makes the row one without a distribution
    if (warp == 0) landed = mbar_wait(&sh.landed, 0, nullptr, PF_DEV_TIMEOUT_PRODUCER);
    landed = __syncthreads_and(landed);
  } else {
    pdl_wait();
  }

  // the asked token's logit, well before it is needed
  int tok = -1;
  float x_tok = 0.f;
  if (tid == 0 && rank == 0 && a.logp) {
    tok = a.tok[r];
    if (tok >= 0 && tok < a.vocab) x_tok = LpVec<T>::one(x + tok);
  }
  LpSums q;
  if (landed)
    sl.sums(q);
  else
    q.s = __int_as_float(0x7fc00000);
  const float own = q.m;
  // the warp's sums, and the maxima of the 32 groups of threads
  {
    float g = own;
#pragma unroll
    for (int o = 1; o < LP_GROUP; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
    if (tid % LP_GROUP == 0) sh.group[tid / LP_GROUP] = g;
    q.join();
    if (lane == 0) sh.m[warp] = q.m, sh.s[warp] = q.s, sh.h[warp] = q.h;
  }
  __syncthreads();
  const int n = a.n_top;
  if (n > 0 && landed) {
    if (warp == 0) {
      // the n-th largest of the groups' maxima
      const float g = sh.group[lane];
      int rk = 0;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float o = __shfl_sync(0xffffffffu, g, i);
        rk += (o > g || (o == g && i < lane)) ? 1 : 0;
      }
      if (rk == n - 1) sh.tau = g;
    }
    __syncthreads();
    const float tau = sh.tau;
    if (own >= tau) sh.queue[atomicAdd(&sh.queued, 1)] = tid;
    __syncthreads();
    for (int i = warp; i < sh.queued; i += LP_WARPS)
      sl.from(sh.queue[i], tau, [&](float v, int at_id) {
        const int at = atomicAdd(&sh.count, 1);
        if (at < LP_CAND) sh.cand[at] = lp_key(lp_order(v), id0 + at_id);
      });
    __syncthreads();
    const int cnt = sh.count;
    if (cnt <= LP_CAND) {
      lp_rank(sh.cand, cnt, n, sh.top);
    } else {
      __syncthreads();  // every thread has read the count
      lp_select(sl, id0, n, sh);
    }
    __syncthreads();  // the list is complete
  }
  // From here one warp a CTA: the CTA's sums (lane w: warp w's), then the
  // cluster's
  if (warp != 0 && cluster == 1) return;
  const unsigned long long* top = sh.top;
  LpSums z;
  if (warp == 0) {
    if (lane < LP_WARPS) z.m = sh.m[lane], z.s = sh.s[lane], z.h = sh.h[lane];
    z.join();
  }
  if (cluster > 1) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (warp == 0) {
      if (lane == 0) {
        const uint32_t at = map_to_rank(smem_u32(&sh.sums[rank]), 0);
        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(z.m), "f"(z.s), "f"(z.h), "f"(0.f)
                     : "memory");
      }
      if (lane < n) {
        const uint32_t at = map_to_rank(smem_u32(&sh.all[rank * n + lane]), 0);
        asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(at), "l"(sh.top[lane]) : "memory");
      }
    }
    cluster_sync_all();
    if (rank != 0) return;
    if (n > 0) {
      lp_rank(sh.all, cluster * n, n, sh.cand);
      top = sh.cand;
      __syncthreads();
    }
    if (warp != 0) return;
    z = LpSums();
    if (lane < cluster) z.m = sh.sums[lane].x, z.s = sh.sums[lane].y, z.h = sh.sums[lane].z;
    z.join();
  }
  const bool ok = z.s >= 1.f && z.m < INFINITY;  // false for a NaN too: a NaN, +inf, or only -inf
  const float nan = __int_as_float(0x7fc00000), log_s = logf(z.s);
  if (lane < n) {
    const unsigned long long k = top[lane];
    const int64_t at = static_cast<int64_t>(r) * n + lane;
    a.top_id[at] = ok ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(k)) : -1;
    a.top_logp[at] = ok ? lp_value(static_cast<uint32_t>(k >> 32)) - z.m - log_s : nan;
  }
  if (lane == 0 && a.logp) a.logp[r] = ok && tok >= 0 && tok < a.vocab ? x_tok - z.m - log_s : nan;
  if (lane == 31 && a.entropy) a.entropy[r] = ok ? log_s - LP_LN2 * (z.h / z.s) : nan;
}

// CTAs per row: enough that a slice fits shared memory, and for few rows as
// many as leave a slice of LP_SLICE_MIN logits and still run at once (three
// a SM with full slices).
constexpr int LP_SLICE_MIN = 2048;

template <class T>
static cudaError_t launch_logprobs(LogprobArgs a, int rows, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  int cluster = 1;
  while (cluster < LP_CLUSTER_MAX && a.vocab / (2 * cluster) >= LP_SLICE_MIN &&
         (static_cast<int64_t>(a.vocab) * sizeof(T) > static_cast<int64_t>(LP_SMEM_SLICE) * cluster ||
          static_cast<int64_t>(rows) * 2 * cluster <= static_cast<int64_t>(LP_CTAS_PER_SM) * sms))
    cluster *= 2;
  a.slice = ((a.vocab + cluster - 1) / cluster + 7) / 8 * 8;
  const dim3 grid(static_cast<unsigned>(rows) * cluster);
  const int64_t bytes = static_cast<int64_t>(a.slice) * sizeof(T);
  if (bytes > LP_SMEM_SLICE) return launch_k(logprobs_kernel<T, false>, grid, dim3(LP_THREADS), 0, s, cluster, a, cluster);
  e = smem_opt_in<logprobs_kernel<T, true>>(LP_SMEM_SLICE + 16);
  if (e != cudaSuccess) return e;
  return launch_k(logprobs_kernel<T, true>, grid, dim3(LP_THREADS), static_cast<size_t>(bytes) + 16, s, cluster, a,
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
