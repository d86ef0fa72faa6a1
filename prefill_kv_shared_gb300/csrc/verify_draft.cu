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
// row, target rows and draft rows alike, a row cut into slices where rows are
// few.  draft_pick_kernel: a cluster a sequence; every CTA joins the slices'
// sums of the sequence's rows, finds the first refusal, and looks through its
// part of that row for the largest w / E.
#include "../../include/prefill_ops.h"
#include "common.cuh"
#include "kernels.h"

#include <string>

namespace pf {

constexpr int VD_THREADS = 256;
constexpr int VD_SLICES_MAX = 8;
constexpr int VD_CLUSTER_MAX = 8;
constexpr float VD_LOG2E = 1.4426950408889634f;

struct VerifyArgs {
  const void *target, *draft;  // draft null: drafted without a distribution
  int64_t t_ld, d_ld;
  int rows, n_seq, vocab;
  const int *tokens, *first;
  const float *u, *noise;
  int *n_accept, *token;
  float* p_accept;
  float2* sums;  // [target rows, then draft rows][slices]: maximum, sum
  int slices, slice;
};

__device__ __forceinline__ float vd_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
template <class T>
struct VdVec;
template <>
struct VdVec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void get(const uint4& r, float* v) {
    v[0] = __uint_as_float(r.x), v[1] = __uint_as_float(r.y), v[2] = __uint_as_float(r.z), v[3] = __uint_as_float(r.w);
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
};
template <>
struct VdVec<__nv_bfloat16> {
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
  template <int CNT>
  __device__ __forceinline__ void add(const float* x) {
    float mx = x[0];
#pragma unroll
    for (int i = 1; i < CNT; ++i) mx = fmaxf(mx, x[i]);
    raise(mx);
    const float at = m == -INFINITY ? 0.f : m;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < CNT; ++i) s += vd_ex2((x[i] - at) * VD_LOG2E);
    z += s;
  }
  __device__ __forceinline__ void join(float m2, float z2) {
    raise(m2);
    // (m2 -inf: nothing there but perhaps a NaN)
    z += m2 == -INFINITY ? (z2 != z2 ? z2 : 0.f) : z2 * vd_ex2((m2 - m) * VD_LOG2E);
  }
};

template <class T>
__global__ void __launch_bounds__(VD_THREADS) draft_sums_kernel(const VerifyArgs a) {
  constexpr int N = VdVec<T>::N;
  __shared__ float2 warps[VD_THREADS / 32];
  const int tid = threadIdx.x;
  pdl_launch();
  pdl_wait();
  const int r = static_cast<int>(blockIdx.x) / a.slices, sl = static_cast<int>(blockIdx.x) % a.slices;
  const T* row = r < a.rows ? static_cast<const T*>(a.target) + r * a.t_ld
                            : static_cast<const T*>(a.draft) + (r - a.rows) * a.d_ld;
  const T* x = row + static_cast<int64_t>(sl) * a.slice;
  const int n = max(0, min(a.slice, a.vocab - sl * a.slice));
  const int mis = static_cast<int>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  const int head = min(n, mis ? N - mis : 0), nvec = (n - head) / N, tail = head + nvec * N;
  VdSum s;
  if (tid < head) {
    const float v = VdVec<T>::one(x + tid);
    s.add<1>(&v);
  }
  if (tid < n - tail) {
    const float v = VdVec<T>::one(x + tail + tid);
    s.add<1>(&v);
  }
  const uint4* vec = reinterpret_cast<const uint4*>(x + head);
  constexpr int FLY = 32 / N;
  for (int i = tid; i < nvec; i += FLY * VD_THREADS) {
    uint4 v[FLY];
#pragma unroll
    for (int k = 0; k < FLY; ++k)
      if (i + k * VD_THREADS < nvec) v[k] = vec[i + k * VD_THREADS];
#pragma unroll
    for (int k = 0; k < FLY; ++k)
      if (i + k * VD_THREADS < nvec) {
        float e[N];
        VdVec<T>::get(v[k], e);
        s.add<N>(e);
      }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s.join(__shfl_xor_sync(0xffffffffu, s.m, o), __shfl_xor_sync(0xffffffffu, s.z, o));
  if ((tid & 31) == 0) warps[tid >> 5] = make_float2(s.m, s.z);
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < VD_THREADS / 32; ++w) s.join(warps[w].x, warps[w].y);
    a.sums[static_cast<int64_t>(r) * a.slices + sl] = make_float2(s.m, s.z);
  }
}

// a candidate: the largest w / E and the lowest id at it (id -1: none)
struct VdBest {
  float v = 0.f;
  int id = -1;
  __device__ __forceinline__ void take(float v2, int id2) {
    if (v2 > v || (v2 == v && id2 >= 0 && id2 < id)) v = v2, id = id2;
  }
};

// what the next token is drawn from
enum VdKind : int { VD_NONE = -1, VD_P = 0, VD_P_MINUS_Q = 1, VD_P_BUT_DRAFTED = 2 };

template <class T>
__global__ void __launch_bounds__(VD_THREADS) draft_pick_kernel(const VerifyArgs a, int cluster_log) {
  __shared__ int sh_at, sh_kind;
  __shared__ float2 sh_p, sh_q;
  __shared__ VdBest sh_warp[VD_THREADS / 32];
  __shared__ float2 sh_all[2][VD_CLUSTER_MAX];  // each CTA's candidate, of both rounds
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cluster = 1 << cluster_log;
  const int s = static_cast<int>(blockIdx.x >> cluster_log), rank = static_cast<int>(blockIdx.x) & (cluster - 1);
  // no CTA writes into another before that one runs: arrive now, wait there
  if (cluster > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  pdl_launch();
  pdl_wait();
  const int r0 = a.first[s], r1 = a.first[s + 1];
  const bool fits = r0 >= 0 && r1 > r0 && r1 <= a.rows && r1 - s - 1 <= a.rows - a.n_seq && r0 >= s;
  const T* target = static_cast<const T*>(a.target);
  const T* draft = static_cast<const T*>(a.draft);
  if (warp == 0) {
    // maximum and 1 / sum of row r of the sums; y 0: no distribution
    auto joined = [&](int r) {
      VdSum z;
      for (int i = 0; i < a.slices; ++i) {
        const float2 p = __ldcg(a.sums + static_cast<int64_t>(r) * a.slices + i);
        z.join(p.x, p.y);
      }
      return make_float2(z.m, z.z >= 0.5f && z.m < INFINITY ? 1.f / z.z : 0.f);
    };
    int at = -1, kind = VD_NONE;
    float2 zp = make_float2(0.f, 0.f), zq = zp;
    // 32 rows at a time; rank 0 also writes the shares of those behind the stop
    for (int base = r0; fits && base < r1 && (at < 0 || rank == 0); base += 32) {
      const int r = base + lane;
      float2 p = make_float2(0.f, 0.f), q = p;
      int k = VD_NONE;
      bool stop = false;
      if (r < r1) {
        p = joined(r);
        float share = 0.f;
        if (r == r1 - 1) {
          stop = true;
          if (p.y > 0.f) k = VD_P;
        } else {
          const int d = a.tokens[r + 1], dr = r - s;
          const bool known = d >= 0 && d < a.vocab;
          if (draft) q = joined(a.rows + dr);
          if (p.y > 0.f && (!draft || q.y > 0.f)) {
            k = draft ? VD_P_MINUS_Q : VD_P_BUT_DRAFTED;
            const float pd = known ? expf(VdVec<T>::one(target + r * a.t_ld + d) - p.x) * p.y : 0.f;
            const float qd = known && draft ? expf(VdVec<T>::one(draft + dr * a.d_ld + d) - q.x) * q.y : 1.f;
            share = pd >= qd ? (pd > 0.f ? 1.f : 0.f) : pd / qd;
            stop = !(a.u[r] * qd < pd);
          } else {
            share = __int_as_float(0x7fc00000);
            stop = true;
          }
        }
        if (rank == 0 && a.p_accept) a.p_accept[r] = share;
      }
      const unsigned stops = __ballot_sync(0xffffffffu, stop);
      if (at < 0 && stops) {
        const int src = __ffs(stops) - 1;
        at = base + src;
        kind = __shfl_sync(0xffffffffu, k, src);
        zp = make_float2(__shfl_sync(0xffffffffu, p.x, src), __shfl_sync(0xffffffffu, p.y, src));
        zq = make_float2(__shfl_sync(0xffffffffu, q.x, src), __shfl_sync(0xffffffffu, q.y, src));
      }
    }
    if (lane == 0) {
      sh_at = at, sh_kind = kind, sh_p = zp, sh_q = zq;
      if (rank == 0) a.n_accept[s] = fits ? at - r0 : -1;
    }
  }
  __syncthreads();
  const int at = sh_at;
  int kind = sh_kind;
  const float2 zp = sh_p, zq = sh_q;
  const int d = kind == VD_P_BUT_DRAFTED ? a.tokens[at + 1] : -1;
  VdBest best;
  if (cluster > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  // Where nothing is left to draw from (p and q alike, or all of p on the
  // drafted token), p itself, in a second round.
  for (int round = 0; round < 2; ++round) {
    if (kind != VD_NONE) {
      const T* x = target + at * a.t_ld;
      const T* y = kind == VD_P_MINUS_Q ? draft + (at - s) * a.d_ld : nullptr;
      const float* noise = a.noise + static_cast<int64_t>(s) * a.vocab;
      for (int v = rank * VD_THREADS + tid; v < a.vocab; v += cluster * VD_THREADS) {
        // (a fused w would leave p's rounding where p and q are alike)
        float w = __fmul_rn(expf(VdVec<T>::one(x + v) - zp.x), zp.y);
        if (y) w = __fsub_rn(w, __fmul_rn(expf(VdVec<T>::one(y + v) - zq.x), zq.y));
        if (kind == VD_P_BUT_DRAFTED && v == d) w = 0.f;
        if (w > 0.f) best.take(w / noise[v], v);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) best.take(__shfl_xor_sync(0xffffffffu, best.v, o), __shfl_xor_sync(0xffffffffu, best.id, o));
    if (lane == 0) sh_warp[warp] = best;
    __syncthreads();
    best = sh_warp[0];
    for (int w = 1; w < VD_THREADS / 32; ++w) best.take(sh_warp[w].v, sh_warp[w].id);
    if (cluster > 1) {
      if (tid < cluster) {
        const uint32_t to = map_to_rank(smem_u32(&sh_all[round][rank]), tid);
        asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(to), "r"(__float_as_int(best.v)), "r"(best.id) : "memory");
      }
      cluster_sync_all();
      for (int c = 0; c < cluster; ++c) best.take(sh_all[round][c].x, __float_as_int(sh_all[round][c].y));
    }
    if (best.id >= 0 || kind == VD_NONE || kind == VD_P) break;
    kind = VD_P;
    __syncthreads();
  }
  if (rank == 0 && tid == 0) a.token[s] = best.id;
}

template <class T>
static cudaError_t launch_verify(VerifyArgs a, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t rows = a.rows + (a.draft ? a.rows - a.n_seq : 0);
  int slices = 1;
  while (slices < VD_SLICES_MAX && rows * slices * 2 <= 4 * sms && a.vocab / (2 * slices) >= 2048) slices *= 2;
  a.slices = slices;
  a.slice = ((a.vocab + slices - 1) / slices + 7) / 8 * 8;
  e = launch_k(draft_sums_kernel<T>, dim3(static_cast<unsigned>(rows * slices)), dim3(VD_THREADS), 0, s, 1, a);
  if (e != cudaSuccess) return e;
  int cluster = 1;
  while (cluster < VD_CLUSTER_MAX && int64_t(a.n_seq) * cluster * 2 <= 4 * sms) cluster *= 2;
  return launch_k(draft_pick_kernel<T>, dim3(static_cast<unsigned>(a.n_seq) * cluster), dim3(VD_THREADS), 0, s, cluster, a,
                  __builtin_ctz(cluster));
}

}  // namespace pf

extern "C" int64_t pfop_verify_draft_work_bytes(int32_t rows, int32_t n_seq) {
  if (rows < 0 || n_seq < 0 || n_seq > rows || rows > (1 << 20)) {
    pf::set_op_error("rows outside [0, 2^20] or n_seq outside [0, rows]");
    return PF_E_ARG;
  }
  return (2 * int64_t(rows) - n_seq) * pf::VD_SLICES_MAX * static_cast<int64_t>(sizeof(float2)) + 256;
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
  if (!target_dev || !tokens_dev || !first_dev || !u_dev || !noise_dev || !n_accept_dev || !token_dev || !work_dev)
    return fail(PF_E_ARG, "null buffer");
  auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  if (((at(tokens_dev) | at(first_dev) | at(u_dev) | at(noise_dev) | at(n_accept_dev) | at(token_dev) | at(p_accept_dev)) & 3) ||
      ((at(target_dev) | at(draft_dev)) & (ltype == PF_L_F32 ? 3 : 1)) || (at(work_dev) & 255))
    return fail(PF_E_ARG, "misaligned buffer");
  if (work_bytes < pfop_verify_draft_work_bytes(rows, n_seq)) return fail(PF_E_ARG, "the scratch is smaller than these rows need");
  const VerifyArgs a{target_dev, draft_dev, target_ld, draft_ld, rows, n_seq, vocab, tokens_dev, first_dev, u_dev,
                     noise_dev, n_accept_dev, token_dev, p_accept_dev, static_cast<float2*>(work_dev), 1, 0};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = ltype == PF_L_F32 ? launch_verify<float>(a, s) : launch_verify<__nv_bfloat16>(a, s);
  if (e != cudaSuccess) return fail(PF_E_CUDA, std::string("draft verification launch: ") + cudaGetErrorString(e));
  return PF_OK;
}
