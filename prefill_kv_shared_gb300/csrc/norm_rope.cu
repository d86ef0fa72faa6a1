// Queries and keys of a step: RMS norm of each head, rotation by position and
// the fp16 write, keys and values into their cells of the cache, in one pass
// (pfop_qk_norm_rope).
//
//   y = x / sqrt(mean x^2 + eps) (1 + g)            (norm, where a gain is given)
//   (a, b) = (y_i, y_{i + hd/2}):  a cos t - b sin t,  a sin t + b cos t,
//   t = pos base^(-2i/hd)
//
// Angles: a turn's fraction f_i = base^(-2i/hd) / 2 pi is held as a 64-bit
// binary fraction, so that pos f_i modulo a turn is one integer product that
// wraps: exact but for f_i's own rounding (2^-53 relative, 2^-25 of a turn at
// position 2^31), where fp32 would be off by whole radians at 2^24.
//
// A lane holds E = 16 bytes' elements of each half of a head (the pair of a
// rotation lies in one thread), HD / 2 / E lanes a head; the heads that a warp
// holds at once are a step.  All rows' steps lie end to end and every warp
// takes the same number of them, so that its sines serve most of a row.
//
// Bound by HBM from fp32 (8192 rows of 32 heads over 4 of 64: 22.4 us, 5.6 TB/s,
// 84% of a measured copy); from bf16, with twice the elements a byte, by
// instructions and their latency (16384 rows of 8 heads over 1 of 256: 34 us,
// 4.9 TB/s; over 200 instructions a step, 20 warps an SM).  One row: 2 us, 512 rows
// of queries 3.
#include "../../include/prefill_ops.h"
#include "common.cuh"
#include "kernels.h"

#include <cmath>
#include <string>
#include <type_traits>

namespace pf {

struct NormRopeArgs {
  const void *q, *k, *v;
  int64_t q_ld, k_ld, v_ld;  // elements from a row to the next
  const int *pos, *slots;
  __half *q_out, *k_cache, *v_cache;
  int64_t n_cells;
  const float *q_gain, *k_gain;
  int rows, Hq, Hkv;
  float eps;
  int steps, per;  // of a row, of a warp
};
template <int HD>
struct Turns {
  uint64_t f[HD / 2];
};

// E elements of 16 bytes as floats
template <class T>
struct NrVec;
template <>
struct NrVec<float> {
  static constexpr int E = 4, CTAS = 8;  // elements, CTAs that an SM's registers hold
  static __device__ __forceinline__ void get(const uint4& r, float* v) {
    v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y), v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
  }
};
template <>
struct NrVec<__nv_bfloat16> {
  static constexpr int E = 8, CTAS = 5;
  static __device__ __forceinline__ void get(const uint4& r, float* v) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

template <int E>
__device__ __forceinline__ void nr_store(__half* dst, const float* v) {
  uint32_t h[E / 2];
#pragma unroll
  for (int i = 0; i < E / 2; ++i) {
    const __half2 p = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    h[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  if constexpr (E == 8)
    *reinterpret_cast<uint4*>(dst) = make_uint4(h[0], h[1], h[2], h[3]);
  else
    *reinterpret_cast<uint2*>(dst) = make_uint2(h[0], h[1]);
}

// two fp32 operations in one instruction
__device__ __forceinline__ uint64_t nr_pack(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 nr_unpack(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t nr_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t nr_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

constexpr int NR_WARPS = 4;
// steps whose loads are on their way (8192 rows of 32 heads over 4 of 64, fp32:
// 22.3 us with 2, 29.6 with 3, whose registers do not fit)
constexpr int NR_FLY = 2;

template <class T, int HD>
__global__ void __launch_bounds__(32 * NR_WARPS, NrVec<T>::CTAS) qk_norm_rope_kernel(const NormRopeArgs a,
    const __grid_constant__ Turns<HD> turns) {
  constexpr int E = NrVec<T>::E, LANES = HD / 2 / E, HEADS = 32 / LANES;  // heads of a step
  __shared__ uint64_t f[HD / 2];
  __shared__ alignas(16) float gain[2][HD];  // 1 + g of queries and of keys
  for (int i = threadIdx.x; i < HD / 2; i += 32 * NR_WARPS) f[i] = turns.f[i];
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31, i0 = lane % LANES * E, in_step = lane / LANES;
  const int heads = a.Hq + 2 * a.Hkv;
  const int64_t g0 = (static_cast<int64_t>(blockIdx.x) * NR_WARPS + (threadIdx.x >> 5)) * a.per;
  int left = static_cast<int>(min(static_cast<int64_t>(a.per), static_cast<int64_t>(a.rows) * a.steps - g0));
  // a step on its way
  struct Step {
    uint4 lo, hi;
    int pos, slot, row, step;
  };
  const int lane_at = in_step * HD + i0;
  // (a step of queries only, as most are, needs no choice between three tensors)
  auto all_q = [&](int step) { return (step + 1) * HEADS <= a.Hq; };
  int row = static_cast<int>(g0 / a.steps), step = static_cast<int>(g0 - static_cast<int64_t>(row) * a.steps), ahead = left;
  auto fetch = [&](Step& s) {
    if (ahead <= 0) return;
    --ahead;
    const int64_t t = row;
    s.row = row;
    s.step = step;
    s.pos = a.pos[t];
    if (all_q(step)) {
      const T* src = static_cast<const T*>(a.q) + t * a.q_ld + step * (HEADS * HD) + lane_at;
      s.lo = *reinterpret_cast<const uint4*>(src);
      s.hi = *reinterpret_cast<const uint4*>(src + HD / 2);
    } else {
      const int h = step * HEADS + in_step;
      s.slot = a.Hkv > 0 ? a.slots[t] : -1;
      if (h < heads) {
        const T* src = h < a.Hq           ? static_cast<const T*>(a.q) + t * a.q_ld + h * HD
                       : h < a.Hq + a.Hkv ? static_cast<const T*>(a.k) + t * a.k_ld + (h - a.Hq) * HD
                                          : static_cast<const T*>(a.v) + t * a.v_ld + (h - a.Hq - a.Hkv) * HD;
        s.lo = *reinterpret_cast<const uint4*>(src + i0);
        s.hi = *reinterpret_cast<const uint4*>(src + HD / 2 + i0);
      }
    }
    if (++step == a.steps) step = 0, ++row;
  };
  uint64_t cs[E / 2], sn[E / 2], ns[E / 2];  // cosines, sines, minus the sines
  int of_row = -1;                           // whose they are
  auto work = [&](const Step& st, auto only_q) {
    constexpr bool ALL_Q = decltype(only_q)::value;
    if (st.row != of_row) {
      of_row = st.row;
      float c[E], n[E];
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const uint64_t turn = static_cast<uint64_t>(static_cast<int64_t>(st.pos)) * f[i0 + i];
        // the nearest of 2^32 steps of a turn, in [-1/2, 1/2) turns
        const int phase = static_cast<int>(static_cast<uint32_t>((turn + 0x80000000ull) >> 32));
        // (sin.approx and cos.approx: 2^-20.5 there, and 2^-20.8 for the angle's
        // three roundings; a result y of a, b is off by less than 2^-19 (|a| + |b|)
        // so far, which is little beside its rounding to fp16, 2^-11 |y|, unless the
        // two products cancel to 2^-8 and less of the pair.  sincospif instead: 512
        // rows of queries 3.4 us for 2.7, 16384 rows from bf16 35.2 for 33.8.)
        __sincosf(static_cast<float>(phase) * (6.283185307f * 0x1p-32f), &n[i], &c[i]);
      }
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        cs[i] = nr_pack(c[2 * i], c[2 * i + 1]);
        sn[i] = nr_pack(n[2 * i], n[2 * i + 1]);
        ns[i] = nr_pack(-n[2 * i], -n[2 * i + 1]);
      }
    }
    float x[2 * E];
    NrVec<T>::get(st.lo, x);
    NrVec<T>::get(st.hi, x + E);
    uint64_t p[E / 2], q[E / 2], sq[2] = {0ull, 0ull};
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      p[i] = nr_pack(x[2 * i], x[2 * i + 1]);
      q[i] = nr_pack(x[E + 2 * i], x[E + 2 * i + 1]);
      sq[0] = nr_fma(p[i], p[i], sq[0]);
      sq[1] = nr_fma(q[i], q[i], sq[1]);
    }
    const float2 s0 = nr_unpack(sq[0]), s1 = nr_unpack(sq[1]);
    float s = (s0.x + s0.y) + (s1.x + s1.y);
#pragma unroll
    for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const int h = st.step * HEADS + in_step;
    const bool is_q = ALL_Q || h < a.Hq, is_v = !ALL_Q && h >= a.Hq + a.Hkv;
    __half* dst;
    if (is_q) {
      dst = a.q_out + (static_cast<int64_t>(st.row) * a.Hq + st.step * HEADS) * HD + lane_at;
    } else {
      if (h >= heads || st.slot < 0 || st.slot >= a.n_cells) return;
      dst = (is_v ? a.v_cache : a.k_cache) + (static_cast<int64_t>(st.slot) * a.Hkv + (h - a.Hq - (is_v ? a.Hkv : 0))) * HD + i0;
    }
    if (!is_v) {
      if (is_q ? a.q_gain != nullptr : a.k_gain != nullptr) {
        const float r = rsqrtf(s * (1.f / HD) + a.eps);
        const uint64_t r2 = nr_pack(r, r);
        const ulonglong2* g = reinterpret_cast<const ulonglong2*>(gain[is_q ? 0 : 1] + i0);
#pragma unroll
        for (int i = 0; i < E / 4; ++i) {
          const ulonglong2 a0 = g[i], a1 = g[HD / 8 + i];
          p[2 * i] = nr_mul(p[2 * i], nr_mul(r2, a0.x));
          p[2 * i + 1] = nr_mul(p[2 * i + 1], nr_mul(r2, a0.y));
          q[2 * i] = nr_mul(q[2 * i], nr_mul(r2, a1.x));
          q[2 * i + 1] = nr_mul(q[2 * i + 1], nr_mul(r2, a1.y));
        }
      }
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const float2 lo = nr_unpack(nr_fma(q[i], ns[i], nr_mul(p[i], cs[i])));
        const float2 hi = nr_unpack(nr_fma(p[i], sn[i], nr_mul(q[i], cs[i])));
        x[2 * i] = lo.x, x[2 * i + 1] = lo.y, x[E + 2 * i] = hi.x, x[E + 2 * i + 1] = hi.y;
      }
    }
    nr_store<E>(dst, x);
    nr_store<E>(dst + HD / 2, x + E);
  };
  Step st[NR_FLY] = {};
#pragma unroll
  for (int i = 0; i < NR_FLY; ++i) fetch(st[i]);
  for (int i = threadIdx.x; i < HD; i += 32 * NR_WARPS) {
    gain[0][i] = a.q_gain ? 1.f + a.q_gain[i] : 1.f;
    gain[1][i] = a.k_gain ? 1.f + a.k_gain[i] : 1.f;
  }
  __syncthreads();
  while (left > 0) {
#pragma unroll
    for (int i = 0; i < NR_FLY; ++i) {
      if (left <= 0) break;
      --left;
      if (all_q(st[i].step))
        work(st[i], std::true_type());
      else
        work(st[i], std::false_type());
      __syncwarp();
      fetch(st[i]);
    }
  }
}

// the turns of a rotation, made once per thread for a base
template <int HD>
static const Turns<HD>& turns_of(float base) {
  static thread_local Turns<HD> t;
  static thread_local float made = 0.f;
  if (made != base) {
    for (int i = 0; i < HD / 2; ++i) {
      const double turn = std::pow(static_cast<double>(base), -2.0 * i / HD) / 6.283185307179586476925;
      t.f[i] = static_cast<uint64_t>(std::ldexp(turn, 64));
    }
    made = base;
  }
  return t;
}

template <class T, int HD>
static cudaError_t launch_norm_rope(NormRopeArgs a, float base, cudaStream_t s) {
  constexpr int HEADS = 32 / (HD / 2 / NrVec<T>::E);
  a.steps = (a.Hq + 2 * a.Hkv + HEADS - 1) / HEADS;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // even shares of all rows' steps
  const int64_t all = int64_t(a.rows) * a.steps, warps = int64_t(sms) * NrVec<T>::CTAS * NR_WARPS;
  a.per = static_cast<int>((all + warps - 1) / warps);
  const int64_t used = (all + a.per - 1) / a.per;
  return launch_k(qk_norm_rope_kernel<T, HD>, dim3(static_cast<unsigned>((used + NR_WARPS - 1) / NR_WARPS)),
                  dim3(32 * NR_WARPS), 0, s, 1, a, turns_of<HD>(base));
}

}  // namespace pf

extern "C" int pfop_qk_norm_rope(int32_t itype, const void* q_dev, int64_t q_ld, const void* k_dev, int64_t k_ld,
                                 const void* v_dev, int64_t v_ld, int32_t rows, int32_t Hq, int32_t Hkv, int32_t hd,
                                 const int32_t* pos_dev, const int32_t* slots_dev, const float* q_gain_dev,
                                 const float* k_gain_dev, float eps, float rope_base, void* q_out_dev, void* kc_dev,
                                 void* vc_dev, int64_t n_cells, void* stream) {
  using namespace pf;
  auto fail = [](int code, const std::string& m) {
    set_op_error(m);
    return code;
  };
  if (itype != PF_L_F32 && itype != PF_L_BF16) return fail(PF_E_ARG, "itype");
  if (hd != 64 && hd != 256) return fail(PF_E_ARG, "head_dim must be 64 or 256");
  if (rows < 0 || rows > (1 << 24) || Hq < 1 || Hq > 1024 || Hkv < 0 || Hkv > 1024)
    return fail(PF_E_ARG, "rows outside [0, 2^24], n_head outside [1, 1024] or n_head_kv outside [0, 1024]");
  if (!(rope_base >= 1.f) || std::isinf(rope_base) || !(eps >= 0.f) || std::isinf(eps))
    return fail(PF_E_ARG, "rope_base below 1 or eps below 0, or not finite");
  if (n_cells < 0 || n_cells > (int64_t(1) << 31) - 1) return fail(PF_E_ARG, "n_cells outside [0, 2^31)");
  const int64_t unit = itype == PF_L_F32 ? 4 : 8;  // elements of 16 bytes
  if (q_ld < int64_t(Hq) * hd || q_ld % unit || (Hkv > 0 && (k_ld < int64_t(Hkv) * hd || k_ld % unit ||
                                                             v_ld < int64_t(Hkv) * hd || v_ld % unit)))
    return fail(PF_E_ARG, "a row stride below the row's heads, or no multiple of 16 bytes");
  if (rows == 0) return PF_OK;
  if (!q_dev || !pos_dev || !q_out_dev || (Hkv > 0 && (!k_dev || !v_dev || !slots_dev || !kc_dev || !vc_dev)))
    return fail(PF_E_ARG, "null buffer");
  auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  uintptr_t wide = at(q_dev) | at(q_out_dev), words = at(pos_dev) | at(q_gain_dev);
  if (Hkv > 0) wide |= at(k_dev) | at(v_dev) | at(kc_dev) | at(vc_dev), words |= at(slots_dev) | at(k_gain_dev);
  if ((wide & 15) || (words & 3)) return fail(PF_E_ARG, "a buffer that is not 16-byte (pos, slots, gains: 4-byte) aligned");
  const NormRopeArgs a{q_dev, k_dev, v_dev, q_ld, k_ld, v_ld, pos_dev, slots_dev, static_cast<__half*>(q_out_dev),
                       static_cast<__half*>(kc_dev), static_cast<__half*>(vc_dev), n_cells, q_gain_dev,
                       Hkv > 0 ? k_gain_dev : nullptr,  // (the kernel reads what is not null)
                       rows, Hq, Hkv, eps, 1, 1};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      itype == PF_L_F32 ? (hd == 256 ? launch_norm_rope<float, 256>(a, rope_base, s) : launch_norm_rope<float, 64>(a, rope_base, s))
                        : (hd == 256 ? launch_norm_rope<__nv_bfloat16, 256>(a, rope_base, s)
                                     : launch_norm_rope<__nv_bfloat16, 64>(a, rope_base, s));
  if (e != cudaSuccess) return fail(PF_E_CUDA, std::string("norm and rotation launch: ") + cudaGetErrorString(e));
  return PF_OK;
}
