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
// rotation lies in one thread), HD / 2 / E lanes a head.  A warp takes some of
// a row's heads one after another, so its sines serve all of them.
#include "../../include/prefill_ops.h"
#include "common.cuh"
#include "kernels.h"

#include <cmath>
#include <string>

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
  int parts, per;  // warps that share a row, and the steps of each
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
  static constexpr int E = 4;
  static __device__ __forceinline__ void get(const uint4& r, float* v) {
    v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y), v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
  }
};
template <>
struct NrVec<__nv_bfloat16> {
  static constexpr int E = 8;
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

constexpr int NR_WARPS = 4, NR_CTAS = 6;  // of a CTA, of an SM
constexpr int NR_BATCH = 2;  // steps whose loads are on their way together

template <class T, int HD>
__global__ void __launch_bounds__(32 * NR_WARPS, NR_CTAS) qk_norm_rope_kernel(const NormRopeArgs a,
                                                                              const __grid_constant__ Turns<HD> turns) {
  constexpr int E = NrVec<T>::E, LANES = HD / 2 / E, HEADS = 32 / LANES;  // heads of a step
  __shared__ uint64_t f[HD / 2];
  __shared__ alignas(16) float gain[2][HD];  // 1 + g of queries and of keys
  for (int i = threadIdx.x; i < HD / 2; i += 32 * NR_WARPS) f[i] = turns.f[i];
  pdl_launch();
  pdl_wait();
  for (int i = threadIdx.x; i < HD; i += 32 * NR_WARPS) {
    gain[0][i] = a.q_gain ? 1.f + a.q_gain[i] : 1.f;
    gain[1][i] = a.k_gain ? 1.f + a.k_gain[i] : 1.f;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, sub = lane % LANES, in_step = lane / LANES, i0 = sub * E;
  const int heads = a.Hq + 2 * a.Hkv;
  const int64_t units = static_cast<int64_t>(a.rows) * a.parts;
  for (int64_t unit = static_cast<int64_t>(blockIdx.x) * NR_WARPS + (threadIdx.x >> 5); unit < units;
       unit += static_cast<int64_t>(gridDim.x) * NR_WARPS) {
    const int64_t t = a.parts == 1 ? unit : unit / a.parts;
    const int part = static_cast<int>(unit - t * a.parts);
    const int first = part * a.per * HEADS, end = min(heads, first + a.per * HEADS);
    const int64_t pos = a.pos[t];
    const int slot = a.Hkv > 0 ? a.slots[t] : -1;
    const bool has_cell = slot >= 0 && slot < a.n_cells;
    float cs[E], sn[E];
    for (int h0 = first; h0 < end; h0 += NR_BATCH * HEADS) {
      uint4 lo[NR_BATCH], hi[NR_BATCH];
#pragma unroll
      for (int b = 0; b < NR_BATCH; ++b) {
        const int h = h0 + b * HEADS + in_step;
        lo[b] = hi[b] = make_uint4(0u, 0u, 0u, 0u);
        if (h < end) {
          const T* src = h < a.Hq           ? static_cast<const T*>(a.q) + t * a.q_ld + h * HD
                         : h < a.Hq + a.Hkv ? static_cast<const T*>(a.k) + t * a.k_ld + (h - a.Hq) * HD
                                            : static_cast<const T*>(a.v) + t * a.v_ld + (h - a.Hq - a.Hkv) * HD;
          lo[b] = *reinterpret_cast<const uint4*>(src + i0);
          hi[b] = *reinterpret_cast<const uint4*>(src + HD / 2 + i0);
        }
      }
      if (h0 == first) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const uint64_t turn = static_cast<uint64_t>(pos) * f[i0 + i];
          // the nearest of 2^32 steps of a turn, in [-1/2, 1/2) turns
          const int phase = static_cast<int>(static_cast<uint32_t>((turn + 0x80000000ull) >> 32));
          // (sin.approx and cos.approx are off by 2^-20.9 there, 2^-9 of an fp16 step)
          __sincosf(static_cast<float>(phase) * (6.283185307f * 0x1p-32f), &sn[i], &cs[i]);
        }
      }
#pragma unroll
      for (int b = 0; b < NR_BATCH; ++b) {
        const int h = h0 + b * HEADS + in_step;
        if (h0 + b * HEADS >= end) break;
        float x[2 * E];
        NrVec<T>::get(lo[b], x);
        NrVec<T>::get(hi[b], x + E);
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < 2 * E; ++i) s = __fmaf_rn(x[i], x[i], s);
#pragma unroll
        for (int o = LANES / 2; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        const bool is_q = h < a.Hq, is_v = h >= a.Hq + a.Hkv;
        __half* dst = nullptr;
        if (h < end) {
          if (is_q)
            dst = a.q_out + (t * a.Hq + h) * HD;
          else if (has_cell)
            dst = (is_v ? a.v_cache : a.k_cache) + (static_cast<int64_t>(slot) * a.Hkv + (h - a.Hq - (is_v ? a.Hkv : 0))) * HD;
        }
        if (!is_v) {
          if (is_q ? a.q_gain != nullptr : a.k_gain != nullptr) {
            const float r = rsqrtf(s * (1.f / HD) + a.eps);
            const float* g = gain[is_q ? 0 : 1];
#pragma unroll
            for (int i = 0; i < E; i += 4) {
              const float4 g0 = *reinterpret_cast<const float4*>(g + i0 + i);
              const float4 g1 = *reinterpret_cast<const float4*>(g + HD / 2 + i0 + i);
              x[i] *= r * g0.x, x[i + 1] *= r * g0.y, x[i + 2] *= r * g0.z, x[i + 3] *= r * g0.w;
              x[E + i] *= r * g1.x, x[E + i + 1] *= r * g1.y, x[E + i + 2] *= r * g1.z, x[E + i + 3] *= r * g1.w;
            }
          }
#pragma unroll
          for (int i = 0; i < E; ++i) {
            const float p = x[i], q = x[E + i];
            x[i] = p * cs[i] - q * sn[i];
            x[E + i] = p * sn[i] + q * cs[i];
          }
        }
        if (dst) {
          nr_store<E>(dst + i0, x);
          nr_store<E>(dst + HD / 2 + i0, x + E);
        }
      }
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
  const int steps = (a.Hq + 2 * a.Hkv + HEADS - 1) / HEADS;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // a warp a row where that fills the GPU, else a row's heads over more warps
  int64_t parts = (int64_t(sms) * 16 + a.rows - 1) / a.rows;
  if (parts > steps) parts = steps;
  if (parts < 1) parts = 1;
  a.per = static_cast<int>((steps + parts - 1) / parts);
  a.parts = (steps + a.per - 1) / a.per;
  const int64_t ctas = (int64_t(a.rows) * a.parts + NR_WARPS - 1) / NR_WARPS, fit = int64_t(sms) * NR_CTAS;
  return launch_k(qk_norm_rope_kernel<T, HD>, dim3(static_cast<unsigned>(ctas < fit ? ctas : fit)), dim3(32 * NR_WARPS), 0,
                  s, 1, a, turns_of<HD>(base));
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
                       static_cast<__half*>(kc_dev), static_cast<__half*>(vc_dev), n_cells, q_gain_dev, k_gain_dev,
                       rows, Hq, Hkv, eps, 1, 1};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      itype == PF_L_F32 ? (hd == 256 ? launch_norm_rope<float, 256>(a, rope_base, s) : launch_norm_rope<float, 64>(a, rope_base, s))
                        : (hd == 256 ? launch_norm_rope<__nv_bfloat16, 256>(a, rope_base, s)
                                     : launch_norm_rope<__nv_bfloat16, 64>(a, rope_base, s));
  if (e != cudaSuccess) return fail(PF_E_CUDA, std::string("norm and rotation launch: ") + cudaGetErrorString(e));
  return PF_OK;
}
