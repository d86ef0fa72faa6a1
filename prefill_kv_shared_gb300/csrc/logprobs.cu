// Log probabilities of given tokens, entropy and the most probable
// alternatives of rows of logits (pfop_logprobs).
//
// With m = max x, t = (x - m) log2 e, s = sum 2^t and h = sum 2^t t over the
// vocabulary: log p[v] = (x[v] - m) - log s and entropy = log s - ln 2 h / s.
// One pass over the row: a thread keeps its own m, s, h (when m moves by d:
// s <- 2^-d s, h <- 2^-d (h - d s)), joined over the block and the cluster.
// A masked logit (-inf, or the type's lowest value) has to add 2^t t = 0 and
// not 0 * inf: once a thread has met one it holds t at -200 or above.  A NaN
// stays a NaN and marks the row as one without a distribution.
//
// The alternatives need no second look at the whole row: the n-th largest of
// the maxima of 64 groups of threads is not above the n-th largest value, so
// only what reaches it is listed, a few dozen logits as a rule, whose ranks
// are then counted.  A thread keeps where its largest step of 16 logits began
// and the next largest step's maximum: mostly that one step is all that has
// to be read again.  (Reading all of such a thread's logits again took 127 us
// instead of 109 for 3000 rows of 50257 fp32 logits, which have left L2 by
// then.)  Where the list overflows (many equal values, as in a row that is
// mostly masked) a radix select finds the n-th value and the lowest ids at it.
//
// A CTA takes a row, or a cluster of up to 8 a slice each (rank 0 joins their
// sums and lists through distributed shared memory).  The logits come in bulk
// copies of 2 KB, two on their way for every warp: no registers are held and
// no warp waits for another until the row's end.  (Whole 64 KB slices in
// shared memory, three to an SM, left too few rows in flight: 512 rows of
// 32768 fp32 logits 21.7 us, now 14.6.)
//
// Bound by the row's bytes for many rows, and by what a CTA does once a row
// (launch, first copy, joins, ranks: about 4 us), by latency for few.  32768
// logits, 5 or 8 alternatives: 1 row fp32 4.5 us; 512 rows fp32 14.6 us, 4.6
// TB/s; 4096 rows bf16 58 us, 4.6 TB/s (61 with three in ten masked).
#include "../../include/prefill_ops.h"
#include "common.cuh"
#include "kernels.h"

#include <string>

namespace pf {

constexpr int LP_TOP_MAX = 32;
constexpr int LP_GROUPS = 64;  // of a CTA's threads, whose maxima are compared
// Alternatives found from 32 pairs of groups; more from the 64 groups: the
// n-th of 32 has 44 logits at or above it for n = 24 and 130 for n = 32, where
// the list now and then overflowed (26 us instead of 8 for 8 rows).
constexpr int LP_PAIRS_MAX = 24;
constexpr int LP_CAND = 256;   // listed candidates
constexpr int LP_CLUSTER_MAX = 8;
constexpr int LP_CHUNK_LOG = 7, LP_CHUNK_VECS = 1 << LP_CHUNK_LOG;  // 16-byte vectors of a warp's copy
constexpr int LP_STAGES = 2;        // copies a warp has on their way
// W: warps of a CTA
constexpr int lp_ring_bytes(int w) { return w * LP_STAGES * LP_CHUNK_VECS * 16; }
constexpr int lp_ctas_per_sm(int w) { return 32 / w; }
constexpr float LP_LOG2E = 1.4426950408889634f, LP_LN2 = 0.6931471805599453f;
static_assert(LP_GROUPS == 64 && LP_PAIRS_MAX <= 32 && LP_TOP_MAX <= 32 && LP_CLUSTER_MAX * LP_TOP_MAX <= LP_CAND, "a lane per alternative, a list for a cluster's");

struct LogprobArgs {
  const void* logits;
  int64_t ld;
  int rows, vocab, slice;  // slice: logits per CTA of a cluster, a multiple of 8
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
__device__ __forceinline__ float lp_max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
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
  // one more logit
  __device__ __forceinline__ void take(float x) {
    if (x > m) rebase(x);
    // x - m first: m log2 e alone may overflow
    const float t = lp_max_nan((x - (m == -INFINITY ? 0.f : m)) * LP_LOG2E, -200.f), w = lp_ex2(t);
    s += w;
    h = __fmaf_rn(w, t, h);
  }
  // CNT more, none above m.  HOLD false: without holding t at -200, a fifth
  // of the work of the ALU pipe; where h then comes out as a NaN (2^t t =
  // 0 * -inf) they are not added and the answer is false.
  template <int CNT, bool HOLD>
  __device__ __forceinline__ bool add(const float* e) {
    const float at = m == -INFINITY ? 0.f : m;
    // two logits an instruction
    const uint64_t nm = lp_pack(-at, -at), c = lp_pack(LP_LOG2E, LP_LOG2E);
    uint64_t s2[2] = {0ull, 0ull}, h2[2] = {0ull, 0ull};
#pragma unroll
    for (int i = 0; i < CNT; i += 2) {
      uint64_t d = lp_pack(e[i], e[i + 1]);
      asm("add.rn.f32x2 %0, %0, %1;" : "+l"(d) : "l"(nm));
      asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(d) : "l"(c));
      float2 t = lp_unpack(d);
      if (HOLD) {
        t.x = lp_max_nan(t.x, -200.f);
        t.y = lp_max_nan(t.y, -200.f);
        d = lp_pack(t.x, t.y);
      }
      const uint64_t w = lp_pack(lp_ex2(t.x), lp_ex2(t.y));
      const int q = (i >> 1) & 1;
      asm("add.rn.f32x2 %0, %0, %1;" : "+l"(s2[q]) : "l"(w));
      asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(h2[q]) : "l"(w), "l"(d));
    }
    const float2 s0 = lp_unpack(s2[0]), s1 = lp_unpack(s2[1]), h0 = lp_unpack(h2[0]), h1 = lp_unpack(h2[1]);
    const float ho = (h0.x + h0.y) + (h1.x + h1.y);
    if (!HOLD && ho != ho) return false;
    s += (s0.x + s0.y) + (s1.x + s1.y);
    h += ho;
    return true;
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

// A CTA's logits x[0 .. n): one a thread at each ragged end, and between them
// 16-byte aligned vectors, LP_CHUNK bytes of them at a time to a warp, the
// warps in turn.
template <class T, int W>
struct LpSlice {
  static constexpr int VN = LpVec<T>::N;
  static constexpr int TAKE = 16 / VN;  // vectors of a step: 16 logits
  const T* x;
  int n, head, nvec;
  int chunk_log;  // 1 << chunk_log vectors are a chunk, at least 32
  __device__ LpSlice(const T* p, int len) : x(p), n(len) {
    const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    head = min(len, mis ? VN - mis : 0);
    nvec = (len - head) / VN;
    // a small slice is dealt out to all threads (else half its groups would be empty)
    chunk_log = nvec <= 32 * W ? 5 : nvec <= 64 * W ? 6 : LP_CHUNK_LOG;
  }
  __device__ __forceinline__ const uint4* vecs() const { return reinterpret_cast<const uint4*>(x + head); }
  __device__ __forceinline__ int chunks() const { return (nvec + (1 << chunk_log) - 1) >> chunk_log; }
  // vectors of a step that one place stands for: those of 16 logits, in a small slice one
  __device__ __forceinline__ int step_log() const { return chunk_log < LP_CHUNK_LOG ? 0 : TAKE == 4 ? 2 : 1; }
  // f(value, id in the slice) for the logits of vector v that are at least tau
  template <class F>
  __device__ __forceinline__ void look(int v, float tau, F&& f) const {
    if (v >= nvec) return;
    float e[VN];
    LpVec<T>::get(__ldcg(vecs() + v), e);
    float mx = e[0];
#pragma unroll
    for (int i = 1; i < VN; ++i) mx = fmaxf(mx, e[i]);
    if (mx < tau) return;
#pragma unroll
    for (int i = 0; i < VN; ++i)
      if (e[i] >= tau) f(e[i], head + v * VN + i);
  }
  // The logits of at least tau: of the steps that begin at vectors
  // few[0 .. n_few), and all of the threads many[0 .. n_many)'s
  template <class F>
  __device__ __forceinline__ void from(const int* few, int n_few, const int* many, int n_many, float tau, F&& f) const {
    const int per_log = chunk_log - 5;  // 1 << per_log vectors of a chunk are a thread's
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int sl = step_log(), steps = n_few << sl;
    // vectors dealt out over the CTA, then those of a thread over a warp
    const int per_thread = ((chunks() + W - 1) / W) << per_log;
    int i = threadIdx.x, q = warp, k = lane;
#pragma unroll 1
    for (;;) {  // (one copy of the code: what is run once a row costs its fetching)
      int v;
      if (i < steps) {
        v = few[i >> sl] + 32 * (i & ((1 << sl) - 1));
        i += (32 * W);
      } else if (q < n_many) {
        const int t = many[q];
        v = k < per_thread ? (((t >> 5) + W * (k >> per_log)) << chunk_log) + (k & ((1 << per_log) - 1)) * 32 + (t & 31) : nvec;
        k += 32;
        if (k >= per_thread) k = lane, q += W;
      } else {
        break;
      }
      look(v, tau, f);
    }
    const int t = threadIdx.x, tail = head + nvec * VN;
    auto one = [&](float v, int i) {
      if (v >= tau) f(v, i);
    };
    if (t < head) one(LpVec<T>::one(x + t), t);
    if (t < n - tail) one(LpVec<T>::one(x + tail + t), tail + t);
  }
  // f(value, id in the slice) for all of them
  template <class F>
  __device__ __forceinline__ void each(F&& f) const {
    constexpr int BATCH = 4;  // vectors in flight
    const int t = threadIdx.x;
    if (t < head) f(LpVec<T>::one(x + t), t);
    for (int v = t; v < nvec; v += BATCH * (32 * W)) {
      uint4 r[BATCH];
#pragma unroll
      for (int b = 0; b < BATCH; ++b)
        r[b] = v + b * (32 * W) < nvec ? __ldcg(vecs() + v + b * (32 * W)) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        if (v + b * (32 * W) >= nvec) break;
        float e[VN];
        LpVec<T>::get(r[b], e);
#pragma unroll
        for (int i = 0; i < VN; ++i) f(e[i], head + (v + b * (32 * W)) * VN + i);
      }
    }
    const int tail = head + nvec * VN;
    if (t < n - tail) f(LpVec<T>::one(x + tail + t), tail + t);
  }
  // Sums of the thread's logits.  The warp's chunks pass through its LP_STAGES
  // places of shared memory, a barrier each; lane 0 keeps the copies of the
  // next ones on their way.  best: first vector of the step with the largest
  // logit (nvec: none); no other step has one above m2.  False: a copy did
  // not land in time.
  __device__ __forceinline__ bool sums(LpSums& a, int& best, float& m2, uint4* ring, uint64_t* landed) const {
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int cnt = warp < chunks() ? (chunks() - warp + W - 1) / W : 0;
    const int tail = head + nvec * VN;
    auto copy = [&](int i) {
      const int v0 = (warp + i * W) << chunk_log;
      const uint32_t bytes = static_cast<uint32_t>(min(1 << chunk_log, nvec - v0)) * 16u;
      uint64_t* bar = landed + i % LP_STAGES;
      mbar_arrive_expect_tx(bar, bytes);
      bulk_load(ring + i % LP_STAGES * LP_CHUNK_VECS, vecs() + v0, bytes, bar);
    };
    if (lane == 0)
      for (int i = 0; i < LP_STAGES && i < cnt; ++i) copy(i);
    bool low = false;  // a logit far below the others, or a NaN, has been met
    if (t < head) a.take(LpVec<T>::one(x + t));
    if (t < n - tail) a.take(LpVec<T>::one(x + tail + t));
    auto wait = [&](int i) {
      const bool in = mbar_wait(landed + i % LP_STAGES, i / LP_STAGES & 1, nullptr, PF_DEV_TIMEOUT_PRODUCER);
      return __all_sync(0xffffffffu, in) != 0;
    };
#pragma unroll 1
    for (int i = 0; i < cnt; ++i) {
      if (!wait(i)) {
        for (int j = i + 1; j < min(i + LP_STAGES, cnt); ++j) wait(j);  // copies on their way
        return false;
      }
      const int v0 = (warp + i * W) << chunk_log;
      const uint4* c = ring + i % LP_STAGES * LP_CHUNK_VECS + lane;
      auto raise = [&](float mx, int v) {
        if (mx > a.m) {
          m2 = a.m;
          a.rebase(mx);
          best = v;
        } else {
          m2 = fmaxf(m2, mx);
        }
      };
      if (chunk_log == LP_CHUNK_LOG && v0 + LP_CHUNK_VECS <= nvec) {
        static_assert(LP_CHUNK_VECS % (32 * TAKE) == 0, "a chunk is a number of whole steps");
#pragma unroll 1
        for (int b = 0; b < LP_CHUNK_VECS / 32; b += TAKE) {
          float e[16];
#pragma unroll
          for (int k = 0; k < TAKE; ++k) LpVec<T>::get(c[32 * (b + k)], e + k * VN);
          float mx = fmaxf(e[0], e[1]);
#pragma unroll
          for (int k = 2; k < 16; k += 2) mx = lp_max3(mx, e[k], e[k + 1]);
          raise(mx, v0 + 32 * b + lane);
          if (low || !a.template add<16, false>(e)) {
            low = true;
            a.template add<16, true>(e);
          }
        }
      } else {
#pragma unroll 1
        for (int b = 0; b < 1 << (chunk_log - 5) && v0 + 32 * b + lane < nvec; ++b) {
          float e[VN];
          LpVec<T>::get(c[32 * b], e);
          float mx = fmaxf(e[0], e[1]);
#pragma unroll
          for (int k = 2; k < VN; k += 2) mx = lp_max3(mx, e[k], e[k + 1]);
          raise(mx, v0 + 32 * (b >> step_log() << step_log()) + lane);
          a.template add<VN, true>(e);
        }
      }
      __syncwarp();  // the place has been read
      if (lane == 0 && i + LP_STAGES < cnt) copy(i + LP_STAGES);
    }
    return true;
  }
};

template <int W>
struct LpShared {
  unsigned long long top[LP_TOP_MAX];  // the CTA's best, in order
  union {
    unsigned long long cand[LP_CAND];
    int hist[256];
  };
  float m[W], s[W], h[W];
  alignas(16) float group[LP_GROUPS];
  float tau;
  int queue[(32 * W)];  // steps that reach tau from its start, threads from its end
  int n_few, n_many, count, prefix, left, warp_count[W];
  uint64_t landed[W * LP_STAGES];  // barriers of the copies
};
// rank 0 of a cluster: what the CTAs bring, behind the ring
struct LpCluster {
  unsigned long long top[LP_CLUSTER_MAX * LP_TOP_MAX];
  float4 sums[LP_CLUSTER_MAX];  // m, s, h
};

// The n best of sh.cand[0 .. cnt) (all different) into dst, in order: a
// candidate's rank is the number of larger ones.
template <int W>
__device__ __forceinline__ void lp_rank(const unsigned long long* cand, int cnt, int n, unsigned long long* dst) {
  for (int i = threadIdx.x; i < cnt; i += (32 * W)) {
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
template <class T, int W>
__device__ __noinline__ void lp_select(const LpSlice<T, W>& sl, int id0, int n, LpShared<W>& sh) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t prefix = 0;
  int left = n;  // of the values with this prefix
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = tid; i < 256; i += (32 * W)) sh.hist[i] = 0;
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
  for (int base = 0; base < sl.n && found < left; base += (32 * W)) {
    const int i = base + tid;
    const bool eq = i < sl.n && lp_order(LpVec<T>::one(sl.x + i)) == prefix;
    const unsigned b = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) sh.warp_count[warp] = __popc(b);
    __syncthreads();
    int at = found, total = found;
    for (int w = 0; w < W; ++w) {
      if (w < warp) at += sh.warp_count[w];
      total += sh.warp_count[w];
    }
    at += __popc(b & ((1u << lane) - 1u));
    if (eq && at < left) sh.cand[larger + at] = lp_key(prefix, id0 + i);
    found = total;
    __syncthreads();
  }
  lp_rank<W>(sh.cand, n, n, sh.top);
}

template <class T, int W>
__global__ void __launch_bounds__(32 * W, lp_ctas_per_sm(W)) logprobs_kernel(const LogprobArgs a, int cluster_log) {
  __shared__ LpShared<W> sh;
  extern __shared__ __align__(16) uint4 lp_ring[];
  LpCluster& all = *reinterpret_cast<LpCluster*>(lp_ring + lp_ring_bytes(W) / 16);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cluster = 1 << cluster_log;
  const int r = static_cast<int>(blockIdx.x >> cluster_log), rank = static_cast<int>(blockIdx.x) & (cluster - 1);
  const T* x = static_cast<const T*>(a.logits) + static_cast<int64_t>(r) * a.ld;
  const int id0 = rank * a.slice;
  const LpSlice<T, W> sl(x + id0, min(a.vocab - id0, a.slice));
  // no CTA writes into another before that one runs: arrive now, wait there
  if (cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  if (tid == 0) sh.count = sh.n_few = sh.n_many = 0;
  uint64_t* landed = &sh.landed[warp * LP_STAGES];
  if (lane == 0) {
    for (int i = 0; i < LP_STAGES; ++i) mbar_init(&landed[i], 1);
    fence_mbar_init();
  }
  __syncwarp();
  pdl_wait();

  // the asked token's logit, well before it is needed
  int tok = -1;
  float x_tok = 0.f;
  if (tid == 0 && rank == 0 && a.logp) {
    tok = a.tok[r];
    if (tok >= 0 && tok < a.vocab) x_tok = LpVec<T>::one(x + tok);
  }
  LpSums q;
  int best = sl.nvec;
  float m2 = -INFINITY;
  // a copy that never lands makes the row one without a distribution
  if (!sl.sums(q, best, m2, lp_ring + warp * (LP_STAGES * LP_CHUNK_VECS), landed)) q.s = __int_as_float(0x7fc00000);
  // (earlier, the next call's CTAs would fill the SMs unevenly: 512 rows 15.4 us instead of 14.8)
  pdl_launch();
  const float own = q.m;
  constexpr int GROUP = 32 * W / LP_GROUPS;  // threads of a group
  // the warp's sums, and the maxima of the groups of threads
  {
    float g = own;
#pragma unroll
    for (int o = 1; o < GROUP; o <<= 1) g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, o));
    if (tid % GROUP == 0) sh.group[tid / GROUP] = g;
    q.join();
    if (lane == 0) sh.m[warp] = q.m, sh.s[warp] = q.s, sh.h[warp] = q.h;
  }
  __syncthreads();
  const int n = a.n_top;
  if (n > 0) {
    // the n-th largest of the maxima, of pairs of groups or of the groups
    if (n > LP_PAIRS_MAX) {
      if (tid < LP_GROUPS) {
        const float g = sh.group[tid];
        int rk = 0;
#pragma unroll 4
        for (int i = 0; i < LP_GROUPS; i += 4) {
          const float4 o = *reinterpret_cast<const float4*>(sh.group + i);
          rk += (o.x > g || (o.x == g && i < tid)) + (o.y > g || (o.y == g && i + 1 < tid)) +
                (o.z > g || (o.z == g && i + 2 < tid)) + (o.w > g || (o.w == g && i + 3 < tid));
        }
        if (rk == n - 1) sh.tau = g;
      }
    } else if (warp == 0) {
      const float g = fmaxf(sh.group[2 * lane], sh.group[2 * lane + 1]);
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
    if (own >= tau) {
      // (both lists fit: a thread is in one)
      if (m2 < tau)
        sh.queue[atomicAdd(&sh.n_few, 1)] = best;
      else
        sh.queue[(32 * W) - 1 - atomicAdd(&sh.n_many, 1)] = tid;
    }
    __syncthreads();
    const int n_many = sh.n_many;
    sl.from(sh.queue, sh.n_few, sh.queue + (32 * W) - n_many, n_many, tau, [&](float v, int at_id) {
      const int at = atomicAdd(&sh.count, 1);
      if (at < LP_CAND) sh.cand[at] = lp_key(lp_order(v), id0 + at_id);
    });
    __syncthreads();
    const int cnt = sh.count;
    if (cnt <= LP_CAND) {
      lp_rank<W>(sh.cand, cnt, n, sh.top);
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
    if (lane < W) z.m = sh.m[lane], z.s = sh.s[lane], z.h = sh.h[lane];
    z.join();
  }
  if (cluster > 1) {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (warp == 0) {
      if (lane == 0) {
        const uint32_t at = map_to_rank(smem_u32(&all.sums[rank]), 0);
        asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(z.m), "f"(z.s), "f"(z.h), "f"(0.f)
                     : "memory");
      }
      if (lane < n) {
        const uint32_t at = map_to_rank(smem_u32(&all.top[rank * n + lane]), 0);
        asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(at), "l"(sh.top[lane]) : "memory");
      }
    }
    cluster_sync_all();
    if (rank != 0) return;
    if (n > 0) {
      lp_rank<W>(all.top, cluster * n, n, sh.cand);
      top = sh.cand;
      __syncthreads();
    }
    if (warp != 0) return;
    z = LpSums();
    if (lane < cluster) z.m = all.sums[lane].x, z.s = all.sums[lane].y, z.h = all.sums[lane].z;
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

// For few rows a cluster: as many CTAs a row as leave a slice of LP_SLICE_MIN
// logits and no more than two CTAs to an SM (32768 fp32 logits, 1 row: 4.5 us
// in 8 slices, 6.5 in one; 64 rows: 7.8 in 4, 8.4 in one, 9.3 in 8; 300 rows:
// 10.5 in one, 11.2 in 2).
constexpr int LP_SLICE_MIN = 2048;

template <class T, int W>
static cudaError_t launch_logprobs(const LogprobArgs& a, int cluster, cudaStream_t s) {
  constexpr int smem = lp_ring_bytes(W) + static_cast<int>(sizeof(LpCluster));
  static_assert(smem + sizeof(LpShared<W>) <= 48 * 1024, "more shared memory has to be asked for");
  return launch_k(logprobs_kernel<T, W>, dim3(static_cast<unsigned>(a.rows) * cluster), dim3(32 * W),
                  cluster > 1 ? smem : lp_ring_bytes(W), s, cluster, a, __builtin_ctz(cluster));
}

template <class T>
static cudaError_t logprobs_of(LogprobArgs a, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  int cluster = 1;
  while (cluster < LP_CLUSTER_MAX && a.vocab / (2 * cluster) >= LP_SLICE_MIN &&
         static_cast<int64_t>(a.rows) * 2 * cluster <= 2 * sms)
    cluster *= 2;
  a.slice = ((a.vocab + cluster - 1) / cluster + 7) / 8 * 8;
  // Many short rows: CTAs of 4 warps, 8 to an SM, so that more rows are being
  // begun or finished while others stream (4096 x 32768 bf16: 58 us, 68 with 8
  // warps; 2000 x 32768 fp32 47, 49).  Longer rows want fewer at once (3000 x
  // 50257 fp32: 108 us with 8 warps, 124 with 4), fewer rows more threads each
  // (300 x 32768 fp32: 10.5, 12.9).
  const bool four = a.rows >= 4 * sms && static_cast<int64_t>(a.vocab) * sizeof(T) <= 131072;
  return four ? launch_logprobs<T, 4>(a, cluster, s) : launch_logprobs<T, 8>(a, cluster, s);
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
  const LogprobArgs a{logits_dev, ld, rows, vocab, 0, tok_dev, n_top, logp_dev, entropy_dev, top_id_dev, top_logp_dev};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      ltype == PF_L_F32 ? logprobs_of<float>(a, s) : logprobs_of<__nv_bfloat16>(a, s);
  if (e != cudaSuccess) return fail(PF_E_CUDA, std::string("log probabilities launch: ") + cudaGetErrorString(e));
  return PF_OK;
}
