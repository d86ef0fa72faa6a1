// Drafted tokens accepted or refused against the target's probabilities, from
// given random numbers, and the token that follows (pfop_verify_draft).
//
// With p, q the softmax of a target and of its draft row, d the drafted token
// and u uniform: accepted where u q(d) < p(d).  At the first refusal the next
// token is drawn from max(p - q, 0), after the last draft from p: the v with
// the largest w(v) / E(v), E exponential random numbers (the first arrival of
// independent processes of rates w), so that no running sum over the
// vocabulary decides.
//
// Two kernels.  draft_sums_kernel: maximum and sum of exponentials of each
// row, target rows and draft rows alike.  The rows' chunks of 2 KB lie end to
// end and every warp takes the same number of them, so that no row's end and
// no last wave leaves SMs idle; a warp leaves a (maximum, sum) for each row
// that it has a part of.  draft_pick_kernel: a cluster a sequence; every CTA
// joins the parts of the sequence's rows, finds the first refusal, and looks
// through its share of that row for the largest w / E.  (Sums by CTAs of a slice
// of a row each: 42.6 us for the 256 chains below, 70.6 with short slices.)
//
// Figures: one chain of 4 over 32768 fp32 6.7 us, two launches' latency; 64
// chains of 0 to 5 over 32000 fp32 15.1 us, latency of few chunks a warp; 256
// of 4 over 32768 bf16 without a draft model, 117 MB, 27 us: the sums at 70%
// of a measured copy, then eight batches a thread of one CTA a sequence.
#include "../../include/prefill_ops.h"
#include "common.cuh"
#include "kernels.h"

#include <algorithm>
#include <string>

namespace pf {

constexpr int VD_SUM_WARPS = 4, VD_SUM_CTAS = 8;  // of a CTA, of an SM
constexpr int VD_FLY = 4;                         // 16-byte vectors of a chunk per lane
constexpr int VD_PARTS_MAX = 64;                  // warps that share a row
// draft_pick_kernel, two CTAs to an SM.  (256 threads: 256 sequences of 32768
// 28.2 to 33.0 us in all instead of 27.5, 64 ragged ones 16.6 to 17.9 instead
// of 16.6, one sequence 7.9 instead of 8.1.)
constexpr int VD_THREADS = 512;
constexpr int VD_CLUSTER_MAX = 8;
constexpr int VD_VECS = 2;  // vectors of four tokens that a thread looks at together
constexpr int VD_GROUP = 32;  // rows whose decisions are made together
constexpr float VD_LOG2E = 1.4426950408889634f;

struct VerifyArgs {
  const void *target, *draft;  // draft null: drafted without a distribution
  int64_t t_ld, d_ld;
  int rows, n_seq, vocab;
  const int *tokens, *first;
  const float *u, *noise;
  int *n_accept, *token;
  float* p_accept;
  // [target rows, then draft rows][parts]: maximum and sum.  Row r's chunks are
  // r chunks .. (r + 1) chunks - 1 of all; warp w takes per of them from w per on.
  float2* sums;
  int parts, chunks, per;  // (all rows' chunks are below 2^31)

  // the warp that has chunk j of row
  __device__ __forceinline__ int warp_of(int row, int j) const {
    return static_cast<int>((static_cast<uint32_t>(row) * static_cast<uint32_t>(chunks) + static_cast<uint32_t>(j)) /
                            static_cast<uint32_t>(per));
  }
};

__device__ __forceinline__ float vd_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float vd_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <class T>
struct VdVec;
template <>
struct VdVec<float> {
  static constexpr int N = 4;
  static constexpr uint32_t NONE = 0xff800000u;  // -inf
  // the largest of CNT vectors (NaNs aside)
  template <int CNT>
  static __device__ __forceinline__ float most(const uint4* r) {
    float m[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int k = 0; k < CNT; ++k) {
      m[0] = fmaxf(m[0], fmaxf(__uint_as_float(r[k].x), __uint_as_float(r[k].y)));
      m[1] = fmaxf(m[1], fmaxf(__uint_as_float(r[k].z), __uint_as_float(r[k].w)));
    }
    return fmaxf(m[0], m[1]);
  }
  static __device__ __forceinline__ void get(const uint4& r, float* v) {
    v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y), v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  static __device__ __forceinline__ float one_l2(const float* p) { return __ldcg(p); }
  static __device__ __forceinline__ void four(const float* p, float* v) {
    const float4 f = *reinterpret_cast<const float4*>(p);
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
  }
};
template <>
struct VdVec<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t NONE = 0xff80ff80u;
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  template <int CNT>
  static __device__ __forceinline__ float most(const uint4* r) {
    uint32_t m[2] = {NONE, NONE};
#pragma unroll
    for (int k = 0; k < CNT; ++k) {
      m[0] = max2(m[0], max2(r[k].x, r[k].y));
      m[1] = max2(m[1], max2(r[k].z, r[k].w));
    }
    float v[2];
    two(max2(m[0], m[1]), v);
    return fmaxf(v[0], v[1]);
  }
  static __device__ __forceinline__ void two(uint32_t w, float* v) {
    v[0] = __uint_as_float(w << 16);
    v[1] = __uint_as_float(w & 0xffff0000u);
  }
  static __device__ __forceinline__ void get(const uint4& r, float* v) {
    two(r.x, v), two(r.y, v + 2), two(r.z, v + 4), two(r.w, v + 6);
  }
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ float one_l2(const __nv_bfloat16* p) {
    return __uint_as_float(static_cast<uint32_t>(__ldcg(reinterpret_cast<const unsigned short*>(p))) << 16);
  }
  static __device__ __forceinline__ void four(const __nv_bfloat16* p, float* v) {
    const uint2 f = *reinterpret_cast<const uint2*>(p);
    two(f.x, v), two(f.y, v + 2);
  }
};

__device__ __forceinline__ uint64_t vd_pack(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 vd_unpack(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
// (x - m) log2 e of two.  The difference first: the rounding of m log2 e would
// be a factor of the whole sum.
__device__ __forceinline__ float2 vd_exponents(float a, float b, float minus_m) {
  uint64_t d = vd_pack(a, b);
  asm("add.rn.f32x2 %0, %0, %1;" : "+l"(d) : "l"(vd_pack(minus_m, minus_m)));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(d) : "l"(vd_pack(VD_LOG2E, VD_LOG2E)));
  return vd_unpack(d);
}

// running maximum and sum of 2^((x - m) log2 e).  A NaN makes the sum one, and
// so does +inf (inf - inf).
struct VdSum {
  float m = -INFINITY, z = 0.f;
  __device__ __forceinline__ void raise(float to) {
    if (to > m) {
      z = m == -INFINITY ? (z != z ? z : 0.f) : z * vd_ex2((m - to) * VD_LOG2E);
      m = to;
    }
  }
  __device__ __forceinline__ void one(float x) {
    raise(x);
    z += vd_ex2((x - (m == -INFINITY ? 0.f : m)) * VD_LOG2E);
  }
  // CNT more, a multiple of 4, none above m
  template <int CNT>
  __device__ __forceinline__ void add(const float* x) {
    const float nm = m == -INFINITY ? 0.f : -m;
    uint64_t s[2] = {0ull, 0ull};
#pragma unroll
    for (int i = 0; i < CNT; i += 2) {
      const float2 t = vd_exponents(x[i], x[i + 1], nm);
      asm("add.rn.f32x2 %0, %0, %1;" : "+l"(s[(i >> 1) & 1]) : "l"(vd_pack(vd_ex2(t.x), vd_ex2(t.y))));
    }
    const float2 a = vd_unpack(s[0]), b = vd_unpack(s[1]);
    z += (a.x + a.y) + (b.x + b.y);
  }
  __device__ __forceinline__ void join(float m2, float z2) {
    raise(m2);
    // (m2 -inf: nothing there but perhaps a NaN)
    z += m2 == -INFINITY ? (z2 != z2 ? z2 : 0.f) : z2 * vd_ex2((m2 - m) * VD_LOG2E);
  }
  // over W lanes, the same in each
  template <int W>
  __device__ __forceinline__ void join_lanes() {
    float to = m;
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, o));
    raise(to);
#pragma unroll
    for (int o = W / 2; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
  }
};

template <class T>
__global__ void __launch_bounds__(32 * VD_SUM_WARPS, VD_SUM_CTAS) draft_sums_kernel(const VerifyArgs a) {
  constexpr int N = VdVec<T>::N, CHUNK = 32 * VD_FLY;  // vectors
  const int lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch();  // after the wait: what the next kernel reads ahead of its own is there
  const int w = static_cast<int>(blockIdx.x) * VD_SUM_WARPS + static_cast<int>(threadIdx.x >> 5);
  const int rows = a.rows + (a.draft ? a.rows - a.n_seq : 0);
  const int64_t c0 = static_cast<int64_t>(w) * a.per, c1 = min(c0 + a.per, static_cast<int64_t>(rows) * a.chunks);
  if (c0 >= c1) return;
  int r = static_cast<int>(static_cast<uint32_t>(c0) / static_cast<uint32_t>(a.chunks));  // row and its chunk
  int j = static_cast<int>(c0 - static_cast<int64_t>(r) * a.chunks);
  int left = static_cast<int>(c1 - c0);
  // a row: logits up to 16 bytes' alignment, vectors, the rest
  const T* x;
  int head, nvec;
  auto begin_row = [&](int row) {
    x = row < a.rows ? static_cast<const T*>(a.target) + row * a.t_ld : static_cast<const T*>(a.draft) + (row - a.rows) * a.d_ld;
    const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
    head = min(a.vocab, mis ? N - mis : 0);
    nvec = (a.vocab - head) / N;
  };
  auto fetch = [&](uint4 (&v)[VD_FLY], int chunk) {
    const uint4* p = reinterpret_cast<const uint4*>(x + head) + chunk * CHUNK + lane;
    const int n = nvec - chunk * CHUNK - lane;
    if (32 * (VD_FLY - 1) < n) {
#pragma unroll
      for (int k = 0; k < VD_FLY; ++k) v[k] = p[32 * k];
    } else {
      const uint32_t none = VdVec<T>::NONE;
#pragma unroll
      for (int k = 0; k < VD_FLY; ++k) v[k] = 32 * k < n ? p[32 * k] : make_uint4(none, none, none, none);
    }
  };
  VdSum s;
  // one chunk in `v`, the next one on its way into `next`
  auto chunk = [&](const uint4 (&v)[VD_FLY], uint4 (&next)[VD_FLY]) {
    const bool ends = j == a.chunks - 1 || left == 1;
    // the ragged ends go with the row's first and last chunk
    float first = -INFINITY, last = -INFINITY;
    if (j == 0 && lane < head) first = VdVec<T>::one(x + lane);
    if (j == a.chunks - 1 && lane < a.vocab - head - nvec * N) last = VdVec<T>::one(x + head + nvec * N + lane);
    const int row = r;
    --left;
    if (++j == a.chunks) {
      j = 0, ++r;
      if (left > 0) begin_row(r);
    }
    if (left > 0) fetch(next, j);
    s.raise(VdVec<T>::template most<VD_FLY>(v));
#pragma unroll
    for (int k = 0; k < VD_FLY; k += 16 / N) {
      float e[16];
#pragma unroll
      for (int i = 0; i < 16 / N; ++i) VdVec<T>::get(v[k + i], e + i * N);
      s.add<16>(e);
    }
    if (first != -INFINITY) s.one(first);
    if (ends) {
      if (last != -INFINITY) s.one(last);
      s.join_lanes<32>();
      const int part = w - a.warp_of(row, 0);
      if (lane == 0) a.sums[static_cast<int64_t>(row) * a.parts + part] = make_float2(s.m, s.z);
      s = VdSum();
    }
  };
  uint4 even[VD_FLY], odd[VD_FLY];
  begin_row(r);
  fetch(even, j);
#pragma unroll 1
  for (;;) {
    chunk(even, odd);
    if (left == 0) break;
    chunk(odd, even);
    if (left == 0) break;
  }
}

// a score above 0 and its token as one key: larger scores first, then lower
// tokens (0: none)
__device__ __forceinline__ unsigned long long vd_key(float score, int id) {
  return static_cast<unsigned long long>(__float_as_uint(score)) << 32 | (0xffffffffu - static_cast<uint32_t>(id));
}

// what the next token is drawn from
enum VdKind : int { VD_NONE = -1, VD_P = 0, VD_P_MINUS_Q = 1, VD_P_BUT_DRAFTED = 2 };

// Bound of the fast forms' errors, of p (and of q <= p).  ex2.approx is off by
// 2^-22, its argument by three roundings of at most 126 2^-24 (times ln 2),
// the reciprocal and the products by 2^-22: below 2^-16 each.
constexpr float VD_OFF = 0x1p-15f;

// How far the sums of rows that are alike may be apart: each has terms of
// 2^-22, of an exponent rounded by 2^-24 of itself, and fp32 additions.
constexpr float VD_ALIKE = 0x1p-17f;

// The thread's share of the tokens: vectors of four, VD_VECS of them at once
// (a batch), v0 + i step.  ALIGNED: a vector is one load in each array.
template <class T, bool ALIGNED>
struct VdScan {
  const T *x, *y;  // target and draft row (null: none)
  const float* noise;
  float nm_p, nm_q;  // minus the maxima
  float share;       // (1 / sum of q) / (1 / sum of p): w in units of 1 / sum of p
  float z_p, z_q;    // 1 / sum
  int vocab, d, v0, step;

  __device__ __forceinline__ void logits(const T* row, int v, float* e) const {
    if (ALIGNED) {
      if (4 * v < vocab) {
        VdVec<T>::four(row + 4 * v, e);
      } else {
        e[0] = e[1] = e[2] = e[3] = -INFINITY;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = 4 * v + i < vocab ? VdVec<T>::one(row + 4 * v + i) : -INFINITY;
    }
  }
  // (L2: read from L2, not by what the SM may still hold of it)
  template <bool L2 = false>
  __device__ __forceinline__ void noises(int v, float* e) const {
    if (ALIGNED) {
      if (4 * v < vocab) {
        const float4* p = reinterpret_cast<const float4*>(noise + 4 * v);
        const float4 f = L2 ? __ldcg(p) : *p;
        e[0] = f.x, e[1] = f.y, e[2] = f.z, e[3] = f.w;
      } else {
        e[0] = e[1] = e[2] = e[3] = 1.f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = 4 * v + i < vocab ? (L2 ? __ldcg(noise + 4 * v + i) : noise[4 * v + i]) : 1.f;
    }
  }
  // the same for a whole batch
  template <bool L2 = false>
  __device__ __forceinline__ void noises_of(int v, float (&e)[VD_VECS][4]) const {
#pragma unroll
    for (int g = 0; g < VD_VECS; ++g) noises<L2>(v + g * step, e[g]);
  }

  // Bounds of the largest w / E: hi of the thread's best batch, hi2 of the
  // others, lo of the true value.  e: the first batch's noise.
  template <bool Q>
  __device__ __forceinline__ void bounds(float (&e)[VD_VECS][4], float& hi, float& hi2, float& lo, int& at) const {
    hi = hi2 = lo = 0.f;
    at = v0;
#pragma unroll 1
    for (int v = v0; 4 * v < vocab; v += VD_VECS * step) {
      float px[VD_VECS][4], qx[VD_VECS][4], next[VD_VECS][4];
#pragma unroll
      for (int g = 0; g < VD_VECS; ++g) {
        logits(x, v + g * step, px[g]);
        if (Q) logits(y, v + g * step, qx[g]);
      }
      noises_of(v + VD_VECS * step, next);
      float h = 0.f, l = 0.f;
#pragma unroll
      for (int g = 0; g < VD_VECS; ++g) {
        if (!Q && static_cast<unsigned>(d - 4 * (v + g * step)) < 4u) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (4 * (v + g * step) + i == d) px[g][i] = -INFINITY;
        }
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const float2 tp = vd_exponents(px[g][i], px[g][i + 1], nm_p);
          float p[2] = {vd_ex2(tp.x), vd_ex2(tp.y)};
          const float r[2] = {vd_rcp(e[g][i]), vd_rcp(e[g][i + 1])};
          if (Q) {
            const float2 tq = vd_exponents(qx[g][i], qx[g][i + 1], nm_q);
            const float q[2] = {vd_ex2(tq.x), vd_ex2(tq.y)};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float w = __fmaf_rn(-q[k], share, p[k]);
              h = fmaxf(h, __fmaf_rn(p[k], VD_OFF, w) * r[k]);
              l = fmaxf(l, __fmaf_rn(p[k], -VD_OFF, w) * r[k]);
            }
          } else {
            h = fmaxf(h, fmaxf(p[0] * r[0], p[1] * r[1]));
          }
        }
      }
      hi2 = fmaxf(hi2, fminf(hi, h));
      if (h > hi) hi = h, at = v;
      lo = fmaxf(lo, l);
#pragma unroll
      for (int g = 0; g < VD_VECS; ++g)
#pragma unroll
        for (int i = 0; i < 4; ++i) e[g][i] = next[g][i];
    }
    if (!Q) {
      lo = hi * (1.f - VD_OFF);
      hi *= 1.f + VD_OFF;
      hi2 *= 1.f + VD_OFF;
    }
  }
  // a batch's logits and noise, and its scores with expf and a division
  struct Batch {
    float px[VD_VECS][4], qx[VD_VECS][4], e[VD_VECS][4];
  };
  __device__ __forceinline__ void fetch(int v, bool minus_q, Batch& f) const {
#pragma unroll
    for (int g = 0; g < VD_VECS; ++g) {
      logits(x, v + g * step, f.px[g]);
      if (minus_q) logits(y, v + g * step, f.qx[g]);
      noises(v + g * step, f.e[g]);
    }
  }
  __device__ __forceinline__ void exact(int v, bool minus_q, bool but_d, const Batch& f, unsigned long long& best) const {
#pragma unroll
    for (int g = 0; g < VD_VECS; ++g)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int id = 4 * (v + g * step) + i;
        // (a fused w would leave p's rounding where p and q are alike)
        float w = __fmul_rn(expf(f.px[g][i] + nm_p), z_p);
        if (minus_q) w = __fsub_rn(w, __fmul_rn(expf(f.qx[g][i] + nm_q), z_q));
        const float score = w / f.e[g][i];
        if (w > 0.f && score >= 0.f && !(but_d && id == d)) best = max(best, vd_key(score, id));
      }
  }
};

template <class T, bool ALIGNED>
__global__ void __launch_bounds__(VD_THREADS, 2) draft_pick_kernel(const VerifyArgs a, int cluster_log) {
  constexpr int WARPS = VD_THREADS / 32;
  __shared__ int sh_at, sh_kind;
  __shared__ float2 sh_p, sh_q;
  __shared__ float2 sh_sums[2][VD_GROUP];  // maximum and 1 / sum (0: no distribution) of target and draft rows
  __shared__ float sh_lo[WARPS];
  __shared__ unsigned long long sh_best[2], sh_all[2][VD_CLUSTER_MAX];  // the CTA's, and each CTA's; of both rounds
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cluster = 1 << cluster_log;
  const int s = static_cast<int>(blockIdx.x >> cluster_log), rank = static_cast<int>(blockIdx.x) & (cluster - 1);
  // no CTA writes into another before that one runs: arrive now, wait there
  if (cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_launch();
  const T* target = static_cast<const T*>(a.target);
  const T* draft = static_cast<const T*>(a.draft);
  VdScan<T, ALIGNED> scan;
  scan.noise = a.noise + static_cast<int64_t>(s) * a.vocab;
  scan.vocab = a.vocab;
  scan.v0 = rank * VD_THREADS + tid;
  scan.step = cluster * VD_THREADS;
  // What the sums do not make is fetched while they are still being formed:
  // draft_sums_kernel lets this one start only when the kernels before both are
  // over.  From L2, since this kernel itself has not waited for them.
  float e[VD_VECS][4];
  scan.template noises_of<true>(scan.v0, e);
  const int r0 = __ldcg(a.first + s), r1 = __ldcg(a.first + s + 1);
  // in the target's rows, and its drafts' rows r - s in the draft's
  const bool fits = r0 >= 0 && r1 > r0 && r1 <= a.rows &&
                    (!a.draft || r1 - r0 == 1 || (r0 >= s && r1 - s - 1 <= a.rows - a.n_seq));
  bool waited = false;
  // of the first rows the outputs are written at the end: a cluster's barriers
  // wait for what a thread has written (2000 clocks)
  float first_share = 0.f;
  if (tid == 0) sh_at = -1, sh_kind = VD_NONE, sh_p = sh_q = make_float2(0.f, 0.f), sh_best[0] = sh_best[1] = 0ull;
  // VD_GROUP rows at a time; rank 0 also writes the shares of those behind the stop
  for (int base = r0; fits && base < r1; base += VD_GROUP) {
    const int r = base + lane, dr = r - s;
    const bool judges = warp == 0 && r < r1 - 1;
    const int d = judges ? __ldcg(a.tokens + r + 1) : -1;
    const float u = judges ? __ldcg(a.u + r) : 0.f;
    const bool known = d >= 0 && d < a.vocab;
    const float xd = known ? VdVec<T>::one_l2(target + r * a.t_ld + d) : -INFINITY;
    const float yd = known && draft ? VdVec<T>::one_l2(draft + dr * a.d_ld + d) : -INFINITY;
    if (!waited) pdl_wait();
    waited = true;
    // the parts of a row in 16 lanes
    const int count = min(VD_GROUP, r1 - base), items = draft ? 2 * count : count;
    for (int it0 = 2 * warp; it0 < items; it0 += 2 * WARPS) {
      const int it = it0 + (lane >> 4), of_draft = it >= count ? 1 : 0, i = it - (of_draft ? count : 0);
      const bool is = it < items && (!of_draft || base + i < r1 - 1);
      VdSum z;
      if (is) {
        const int row = of_draft ? a.rows + base + i - s : base + i;
        const int n = a.warp_of(row, a.chunks - 1) - a.warp_of(row, 0) + 1;
        const float2* sums = a.sums + static_cast<int64_t>(row) * a.parts;
        float2 p[VD_PARTS_MAX / 16];
#pragma unroll
        for (int k = 0; k < VD_PARTS_MAX / 16; ++k) {
          p[k] = make_float2(-INFINITY, 0.f);
          if ((lane & 15) + 16 * k < n) p[k] = __ldcg(sums + (lane & 15) + 16 * k);
        }
#pragma unroll
        for (int k = 0; k < VD_PARTS_MAX / 16; ++k) z.join(p[k].x, p[k].y);
      }
      z.join_lanes<16>();
      if (is && (lane & 15) == 0)
        sh_sums[of_draft][i] = make_float2(z.m, z.z >= 0.5f && z.m < INFINITY ? 1.f / z.z : 0.f);
    }
    __syncthreads();
    if (warp == 0) {
      float2 p = make_float2(0.f, 0.f), q = p;
      float pd = 0.f, qd = 1.f;
      int k = VD_NONE;
      bool stop = false;
      if (r < r1) {
        p = sh_sums[0][lane];
        stop = true;
        if (!judges) {
          if (p.y > 0.f) k = VD_P;
        } else {
          if (draft) q = sh_sums[1][lane];
          // Rows that are alike up to a shift: their sums, formed in other
          // orders, differ by their roundings, and those would be drawn from.
          // Taken as equal, w is 0 throughout, as it is.  (Rows that are alike
          // in sum and drafted token only get a q that is off by that much.)
          if (draft && xd - p.x == yd - q.x && fabsf(q.y - p.y) <= VD_ALIKE * p.y) q.y = p.y;
          if (p.y > 0.f && (!draft || q.y > 0.f)) {
            k = draft ? VD_P_MINUS_Q : VD_P_BUT_DRAFTED;
            pd = known ? expf(xd - p.x) * p.y : 0.f;
            qd = known && draft ? expf(yd - q.x) * q.y : 1.f;
            stop = !(u * qd < pd);
          }
        }
      }
      const unsigned stops = __ballot_sync(0xffffffffu, stop);
      if (stops && sh_at < 0 && lane == __ffs(stops) - 1) {
        sh_kind = k, sh_p = p, sh_q = q;
        sh_at = r;
      }
      if (rank == 0 && a.p_accept && r < r1) {
        const float share = !judges ? 0.f : k == VD_NONE ? __int_as_float(0x7fc00000) : pd >= qd ? (pd > 0.f ? 1.f : 0.f) : pd / qd;
        if (base == r0)
          first_share = share;
        else
          a.p_accept[r] = share;
      }
    }
    __syncthreads();
    if (sh_at >= 0 && (rank != 0 || !a.p_accept)) break;
  }
  if (!waited) pdl_wait();
  __syncthreads();
  const int at = sh_at;
  int kind = sh_kind;
  const float2 zp = sh_p, zq = sh_q;
  scan.d = kind == VD_P_BUT_DRAFTED ? a.tokens[at + 1] : -1;
  scan.x = target + max(at, 0) * a.t_ld;
  scan.y = kind == VD_P_MINUS_Q ? draft + (at - s) * a.d_ld : nullptr;
  scan.nm_p = -zp.x, scan.z_p = zp.y;
  scan.nm_q = -zq.x, scan.z_q = zq.y;
  scan.share = zq.y / zp.y;
  unsigned long long best = 0ull;
  // A second round, of p itself, where nothing is left to draw from (p and q
  // alike, or all of p on the drafted token).
  for (int round = 0; round < 2; ++round) {
    if (kind != VD_NONE) {
      // Batches to be looked at exactly: the thread's best one where it may
      // hold the CTA's answer, all of the warp's where others may too.
      int v = scan.v0;
      bool all = true, mine = true;
      typename VdScan<T, ALIGNED>::Batch f;
      if (round == 0) {
        float hi, hi2, lo;
        int batch;
        if (kind == VD_P_MINUS_Q)
          scan.template bounds<true>(e, hi, hi2, lo, batch);
        else
          scan.template bounds<false>(e, hi, hi2, lo, batch);
        v = batch;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) lo = fmaxf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        if (lane == 0) sh_lo[warp] = lo;
        __syncthreads();
        lo = sh_lo[lane % WARPS];
#pragma unroll
        for (int o = WARPS / 2; o > 0; o >>= 1) lo = fmaxf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        all = __any_sync(0xffffffffu, hi2 > 0.f && hi2 >= lo);
        mine = all || (hi > 0.f && hi >= lo);
      }
      if (!all) {
        if (mine) {
          scan.fetch(v, kind == VD_P_MINUS_Q, f);
          scan.exact(v, kind == VD_P_MINUS_Q, kind == VD_P_BUT_DRAFTED, f, best);
        }
      } else {
        for (v = scan.v0; 4 * v < a.vocab; v += VD_VECS * scan.step) {
          scan.fetch(v, kind == VD_P_MINUS_Q, f);
          scan.exact(v, kind == VD_P_MINUS_Q, kind == VD_P_BUT_DRAFTED, f, best);
        }
      }
      if (best) atomicMax(&sh_best[round], best);
    }
    __syncthreads();
    best = sh_best[round];
    if (cluster > 1) {
      if (round == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      if (tid < cluster) {
        const uint32_t to = map_to_rank(smem_u32(&sh_all[round][rank]), tid);
        asm volatile("st.shared::cluster.b64 [%0], %1;" ::"r"(to), "l"(best) : "memory");
      }
      cluster_sync_all();
      for (int c = 0; c < cluster; ++c) best = max(best, sh_all[round][c]);
    }
    if (best || kind == VD_NONE || kind == VD_P) break;
    kind = VD_P;
  }
  if (rank != 0 || warp != 0) return;
  if (fits && a.p_accept && r0 + lane < r1) a.p_accept[r0 + lane] = first_share;
  if (lane == 0) {
    a.n_accept[s] = fits ? at - r0 : -1;
    a.token[s] = best ? static_cast<int>(0xffffffffu - static_cast<uint32_t>(best)) : -1;
  }
}

// logits of a chunk
template <class T>
constexpr int vd_chunk() {
  return 32 * VD_FLY * VdVec<T>::N;
}

template <class T>
static cudaError_t launch_verify(VerifyArgs a, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t rows = a.rows + (a.draft ? a.rows - a.n_seq : 0);
  a.chunks = (a.vocab + vd_chunk<T>() - 1) / vd_chunk<T>();
  // even shares over the resident warps; a row in at most VD_PARTS_MAX of them
  const int64_t all = rows * a.chunks, warps = int64_t(sms) * VD_SUM_CTAS * VD_SUM_WARPS;
  a.per = static_cast<int>(std::max((all + warps - 1) / warps, (int64_t(a.chunks) + VD_PARTS_MAX - 2) / (VD_PARTS_MAX - 1)));
  a.parts = static_cast<int>(std::min<int64_t>(VD_PARTS_MAX, (a.chunks - 1) / a.per + 2));
  const int64_t used = (all + a.per - 1) / a.per;
  e = launch_k(draft_sums_kernel<T>, dim3(static_cast<unsigned>((used + VD_SUM_WARPS - 1) / VD_SUM_WARPS)),
               dim3(32 * VD_SUM_WARPS), 0, s, 1, a);
  if (e != cudaSuccess) return e;
  auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  const bool aligned = a.vocab % 4 == 0 && a.t_ld % 4 == 0 && (!a.draft || a.d_ld % 4 == 0) &&
                       ((at(a.target) | at(a.draft)) & (4 * sizeof(T) - 1)) == 0 && (at(a.noise) & 15) == 0;
  // more CTAs a sequence while all fit the GPU at once and each thread has a batch
  int cluster = 1;
  while (cluster < VD_CLUSTER_MAX && int64_t(a.n_seq) * cluster * 2 <= 2 * sms &&
         a.vocab > cluster * VD_THREADS * VD_VECS * 4)
    cluster *= 2;
  const dim3 grid(static_cast<unsigned>(a.n_seq) * cluster), block(VD_THREADS);
  return aligned ? launch_k(draft_pick_kernel<T, true>, grid, block, 0, s, cluster, a, __builtin_ctz(cluster))
                 : launch_k(draft_pick_kernel<T, false>, grid, block, 0, s, cluster, a, __builtin_ctz(cluster));
}

}  // namespace pf

extern "C" int64_t pfop_verify_draft_work_bytes(int32_t rows, int32_t n_seq) {
  if (rows < 0 || n_seq < 0 || n_seq > rows || rows > (1 << 20)) {
    pf::set_op_error("rows outside [0, 2^20] or n_seq outside [0, rows]");
    return PF_E_ARG;
  }
  return (2 * int64_t(rows) - n_seq) * pf::VD_PARTS_MAX * static_cast<int64_t>(sizeof(float2)) + 256;
}

extern "C" int pfop_verify_draft(int32_t ltype, const void* target_dev, int64_t target_ld, const void* draft_dev,
                                 int64_t draft_ld, int32_t rows, int32_t n_seq, int32_t vocab,
                                 const int32_t* tokens_dev, const int32_t* first_dev, const float* u_dev,
                                 const float* noise_dev, int32_t* n_accept_dev, int32_t* token_dev,
                                 float* p_accept_dev, void* work_dev, int64_t work_bytes, void* stream) {
  using namespace pf;
  auto fail = [](int code, const std::string& m) {
    set_op_error(m);
    return code;
  };
  if (ltype != PF_L_F32 && ltype != PF_L_BF16) return fail(PF_E_ARG, "ltype");
  if (rows < 0 || rows > (1 << 20) || n_seq < 0 || n_seq > rows) return fail(PF_E_ARG, "rows outside [0, 2^20] or n_seq outside [0, rows]");
  if (vocab < 1 || vocab >= (1 << 30) || target_ld < vocab || (draft_dev && draft_ld < vocab))
    return fail(PF_E_ARG, "vocab, or a row stride below it");
  if (n_seq == 0) return PF_OK;
  // (the kernels count chunks in 32 bits)
  const int chunk = ltype == PF_L_F32 ? vd_chunk<float>() : vd_chunk<__nv_bfloat16>();
  if (((vocab - 1) / chunk + 1) * (rows + (draft_dev ? int64_t(rows) - n_seq : 0)) >= int64_t(1) << 31)
    return fail(PF_E_ARG, "2^31 chunks of logits or more");
  if (!target_dev || !tokens_dev || !first_dev || !u_dev || !noise_dev || !n_accept_dev || !token_dev || !work_dev)
    return fail(PF_E_ARG, "null buffer");
  auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  if (((at(tokens_dev) | at(first_dev) | at(u_dev) | at(noise_dev) | at(n_accept_dev) | at(token_dev) | at(p_accept_dev)) & 3) ||
      ((at(target_dev) | at(draft_dev)) & (ltype == PF_L_F32 ? 3 : 1)) || (at(work_dev) & 255))
    return fail(PF_E_ARG, "misaligned buffer");
  if (work_bytes < pfop_verify_draft_work_bytes(rows, n_seq)) return fail(PF_E_ARG, "the scratch is smaller than these rows need");
  const VerifyArgs a{target_dev, draft_dev, target_ld, draft_ld, rows, n_seq, vocab, tokens_dev, first_dev, u_dev,
                     noise_dev, n_accept_dev, token_dev, p_accept_dev, static_cast<float2*>(work_dev), 1, 1, 1};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = ltype == PF_L_F32 ? launch_verify<float>(a, s) : launch_verify<__nv_bfloat16>(a, s);
  if (e != cudaSuccess) return fail(PF_E_CUDA, std::string("draft verification launch: ") + cudaGetErrorString(e));
  return PF_OK;
}
