// Attention of several sequences' rows in one call (pfop_attention_packed,
// pfop_attention_tree): causal over each sequence's own keys, or over a
// context and a tree of drafted tokens, on the 5th-generation tensor cores.
//
// MMA rows are (row, head-in-group) pairs of a run: row R = t*G + g is the
// run's row t and query head kvh*G + g, so the G heads of a KV head share its
// K/V.  A pair of CTAs (a 2-CTA cluster, tcgen05 .cta_group::2) takes 256
// rows of one run and KV head and a group of gc consecutive 128-key chunks
// of the run's positions, and runs one online softmax over the group:
//     S = Q K^T, m' = max(m, max_k s_k), p_k = 2^((s_k - m') c),
//     l' = l 2^((m - m') c) + sum_k p_k, O' = O 2^((m - m') c) + fp16(P) V
// with c = log2(e)/sqrt(hd), S, O, m, l in fp32.  A row whose keys lie in one
// group writes O/l; otherwise each group leaves (O, m, l) in the scratch and
// attn_runs_merge_kernel joins them in group order.
//
// Why pairs: 128 rows against a chunk need 64 bytes of K/V per SM clock at
// the full tensor rate, more than L2 delivers to all SMs at once; 256 rows
// over a pair, each CTA holding half of every K chunk (64 keys) and half of
// every V chunk (hd/2 dims), need 32, and the halves leave room for 2.5
// chunks in flight beside Q at hd 256.
//
// Roles of a CTA: warp 1 copies Q and the K/V halves by TMA (one ring of
// stages, in the order in which the MMAs use them; the copies of both CTAs
// complete on the even CTA's barriers); warp 0 of the even CTA issues the
// MMAs of the pair; the others own the CTA's 128 rows (thread = TMEM lane =
// row): softmax, P (fp16, over the columns of S that it came from), the
// rescale of O, the output.  Two S buffers let S of the next chunk be formed
// while P of this one is.  At hd 256 one warpgroup (warps 2..5) keeps up
// with the MMAs; at hd 64, where a chunk has a quarter of the MMA work for
// the same exponentials, two warpgroups take one half of every chunk's keys
// each, with their own m, l and O (TMEM has room for two), and join them at
// the end.  All waits are bounded (PF_WAIT_CYCLES): one that gives up flags
// the scratch's error word and the pair unwinds.
#include "../../include/prefill_ops.h"
#include "attn.cuh"
#include "common.cuh"
#include "kernels.h"

#include <algorithm>
#include <string>

namespace pf {

constexpr int RUNS_MAX = 128;
constexpr int RCH = 128;    // keys of a chunk
constexpr int RROWS = 256;  // MMA rows of a pair

// the call's runs, passed in the kernel's parameters
struct RunTable {
  int n_runs = 0;
  int row0[RUNS_MAX];  // first packed row
  int n[RUNS_MAX], pos0[RUNS_MAX], cell0[RUNS_MAX];
  int item0[RUNS_MAX];  // first work item; a run has (row blocks) x (groups) of them
  int groups[RUNS_MAX];
};

struct RunsShape {
  int Hq, Hkv, log_g;  // G = 1 << log_g query heads per KV head
  int gc;              // chunks per group
  int slot_rows;       // rows of a state slot in the scratch
  int items;           // work items per KV head
};

template <int HD>
struct RunsCfg {
  static constexpr int Q_BYTES = 128 * HD * 2;  // [64-dim box][128 rows][128 B]
  static constexpr int STAGE = 64 * HD * 2;     // half a chunk: K [box][64 keys][128 B], V [box][128 keys][hd/2 dims]
  static constexpr int NST = HD == 256 ? 5 : 8;
  static constexpr int NH = HD == 256 ? 1 : 2;  // parts of a chunk's keys, a warpgroup each
  static constexpr int KPT = RCH / NH;          // keys per thread and chunk
  static constexpr int OFF_ST = Q_BYTES;
  static constexpr int OFF_BAR = OFF_ST + NST * STAGE;
  static constexpr int OFF_ML = OFF_BAR + 256;        // (m, l) of each part's rows
  static constexpr int SMEM = OFF_ML + (NH > 1 ? NH * 128 * 8 : 0) + 1024;  // + alignment slack
  static constexpr int TMEM_S = 0;          // two S buffers
  static constexpr int TMEM_O = 2 * RCH;    // one O per part
  static constexpr int TMEM_COLS = 512;
  static_assert(TMEM_O + NH * HD <= TMEM_COLS, "TMEM");
  static constexpr int THREADS = 64 + 128 * NH;
  static_assert(SMEM <= 232448, "shared memory");
};

// floats of one row's state: o[HD], m, l, 2 pad
__host__ __device__ constexpr int runs_state_stride(int hd) { return hd + 4; }

// 64-byte-swizzled MN-major operand descriptor: rows (K) of 64 bytes, 8-row
// groups of 512 bytes, one 32-element atom along MN
__device__ __forceinline__ uint64_t sdesc_sw64_mn(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(512 >> 4) << 16;
  d |= static_cast<uint64_t>(512 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(4) << 61;
  return d;
}

// A pair's D (+)= A[tmem] * B[smem]: each CTA's 128 rows of A lie in its own TMEM
__device__ __forceinline__ void tc_mma_f16_ts_pair(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                                   uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// TMA copies of a pair: into this CTA's shared memory, completing on the
// barrier at a shared::cluster address (here always the even CTA's)
__device__ __forceinline__ void tma_load_3d_pair(void* smem_dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                                                 int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 "
      "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d_pair(void* smem_dst, const CUtensorMap* map, uint32_t bar, int c0, int c1,
                                                 int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2 "
      "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// Arrive on a barrier of the pair without ordering other memory: what is
// handed over lies in TMEM and is ordered by the tcgen05 fences around the
// arrive and the wait.  (A release at cluster scope waits for all of the
// thread's outstanding accesses: it was the kernel's first stall.)
__device__ __forceinline__ void mbar_arrive_pair_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// two fp32 operations in one instruction
__device__ __forceinline__ uint64_t pack_f32x2(float a, float b) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float2 unpack_f32x2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// bounded wait for a barrier on an error path (about 0.2 s)
__device__ __forceinline__ void runs_drain(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  const long long t0 = clock64();
  while (!mbar_try_wait(a, parity)) {
    if (clock64() - t0 > 400000000ll) return;
  }
}

// The run of work item (or row) `it`: the last one whose first is not above it.
__device__ __forceinline__ int find_run(const int* first, int n_runs, int it) {
  int lo = 0, hi = n_runs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= it)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// bits of the keys kk .. kk+31 (positions) that the row sees: the context
// [0, pos0), then its mask's bits for the drafted tokens [0, n)
__device__ __forceinline__ uint32_t tree_bits(const uint64_t* row_mask, int words, int pos0, int n, int kk) {
  const int d = kk - pos0;  // drafted token of the word's first bit
  if (d <= -32) return 0xffffffffu;
  if (d >= n) return 0u;
  uint64_t w;
  if (d < 0) {
    w = (__ldg(row_mask) << -d) | ((1ull << -d) - 1ull);
  } else {
    w = __ldg(row_mask + (d >> 6)) >> (d & 63);
    if ((d & 63) > 32 && (d >> 6) + 1 < words) w |= __ldg(row_mask + (d >> 6) + 1) << (64 - (d & 63));
  }
  if (n - d < 32) w &= (1ull << (n - d)) - 1ull;
  return static_cast<uint32_t>(w);
}

// scores of 32 keys of this thread's row: the ones it does not see to -inf
__device__ __forceinline__ void mask_scores(uint32_t (&x)[32], uint32_t bits) {
#pragma unroll
  for (int k = 0; k < 32; ++k)
    if (!(bits >> k & 1u)) x[k] = 0xff800000u;
}
__device__ __forceinline__ void max_scores(const uint32_t (&x)[32], float (&mx)[4]) {
#pragma unroll
  for (int k = 0; k < 32; k += 8) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      mx[q] = fmaxf(mx[q], fmaxf(__uint_as_float(x[k + 2 * q]), __uint_as_float(x[k + 2 * q + 1])));
  }
}
// p = 2^(s c - mc) of 32 keys, as 16 fp16 pairs, and their sum
__device__ __forceinline__ void exp_scores(const uint32_t (&x)[32], uint64_t c2, uint64_t nmc2, uint32_t* pw,
                                           uint64_t (&ls)[4]) {
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float2 e = unpack_f32x2(
        fma_f32x2(pack_f32x2(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), c2, nmc2));
    const float p0 = ex2_approx(e.x), p1 = ex2_approx(e.y);
    const __half2 h = __floats2half2_rn(p0, p1);
    pw[k] = *reinterpret_cast<const uint32_t*>(&h);
    ls[k & 3] = add_f32x2(ls[k & 3], pack_f32x2(p0, p1));
  }
}

template <int HD, bool TREE>
__global__ void __launch_bounds__(RunsCfg<HD>::THREADS, 1)
    attn_runs_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ RunTable rt, const RunsShape sh,
                     const uint64_t* __restrict__ mask, int words, __nv_bfloat16* __restrict__ out,
                     float* __restrict__ part, int* err) {
  using C = RunsCfg<HD>;
  constexpr float cexp = attn_c<HD>();
  extern __shared__ uint8_t smem_raw[];
  // The two CTAs' buffers lie at the same shared-memory offset (one
  // descriptor addresses both): same kernel, same alignment rounding.
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* q_full = bars;        // in the even CTA: Q of both has landed
  uint64_t* full = bars + 1;      // NST, in the even CTA: a stage has landed in both
  uint64_t* empty = bars + 9;     // NST: the MMAs have read it
  uint64_t* s_full = bars + 17;   // by S buffer (chunk parity)
  uint64_t* p_full = bars + 19;   // [part][S buffer], the even CTA's count the warps of both
  uint64_t* pv_done = bars + 23;  // by chunk parity
  uint64_t* tail = bars + 25;     // odd CTA: V of the last chunk has landed; even CTA: it is cleared there
  uint64_t* drain = bars + 26;    // error path only
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 27);
  static_assert(C::NST <= 8 && C::NH <= 2, "barrier layout");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  pdl_launch();

  // ---- the pair's work item
  const int idx = static_cast<int>(blockIdx.x >> 1);
  const int kvh = idx % sh.Hkv, it = idx / sh.Hkv;
  const int run = find_run(rt.item0, rt.n_runs, it);
  const int n_rows = rt.n[run], pos0 = rt.pos0[run], row0 = rt.row0[run];
  const int total_rows = n_rows << sh.log_g;
  const int nb = (total_rows + RROWS - 1) / RROWS;
  const int local = it - rt.item0[run];
  const int grp = local / nb;
  const int R0 = (nb - 1 - local % nb) * RROWS;  // blocks with the most keys first
  const int t_last = min(n_rows - 1, (R0 + RROWS - 1) >> sh.log_g);
  const int keys = TREE ? pos0 + n_rows : pos0 + t_last + 1;
  const int ch_first = grp * sh.gc;
  const int n = min((keys + RCH - 1) / RCH, ch_first + sh.gc) - ch_first;  // chunks
  if (n <= 0) {  // no keys of this group reach the block's rows
    pdl_wait();
    return;
  }
  const int run_keys = pos0 + n_rows;
  const int RC = R0 + rank * 128;  // this CTA's first row
  // warps of rows, here and in the other CTA
  auto row_warps = [&](int r) { return min(4, max(0, (total_rows - R0 - r * 128 + 31) >> 5)); };

  if (threadIdx.x == 0) {
    mbar_init(q_full, 1);
    for (int b = 0; b < C::NST; ++b) {
      mbar_init(&full[b], 1);
      mbar_init(&empty[b], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&s_full[b], 1);
      mbar_init(&pv_done[b], 1);
    }
    for (int b = 0; b < 2 * C::NH; ++b) mbar_init(&p_full[b], row_warps(0) + row_warps(1));
    mbar_init(tail, 1);
    mbar_init(drain, 1);
    fence_mbar_init();
  }
  if (warp == 1 && lane == 0) {
    prefetch_tensormap(&tmQ);
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  if (warp == 0) tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();

  // K(i) and V(i) in the order of their use: S(i+1) is formed before P(i) V(i)
  const int n_seq = 2 * n;
  auto seq_is_k = [&](int u) { return u == 0 || (u < n_seq - 1 && (u & 1)); };
  auto seq_chunk = [&](int u) { return u == 0 ? 0 : u == n_seq - 1 ? n - 1 : (u & 1) ? (u + 1) / 2 : u / 2 - 1; };
  // The V rows of keys past the run (only in the run's last chunk) are
  // cleared in shared memory before the MMAs read them: P is 0 there, but
  // what lies in those cells may be an infinity or NaN.
  const int tail_keys = run_keys - (ch_first + n - 1) * RCH;  // of the item's last chunk
  const bool has_tail = tail_keys < RCH;
  auto clear_tail = [&]() {
    constexpr int VB = HD == 256 ? 128 : 64;  // bytes of a key's row in a box
    uint8_t* v = smem + C::OFF_ST + ((n_seq - 1) % C::NST) * C::STAGE;
    for (int box = 0; box < C::STAGE / (RCH * VB); ++box)
      for (int o = tail_keys * VB + lane * 16; o < RCH * VB; o += 512)
        *reinterpret_cast<uint4*>(v + box * RCH * VB + o) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    __syncwarp();
  };

  if (warp == 1) {
    // ---------------- TMA producer (each CTA its own rows and halves)
    if (lane == 0) {
      if (rank == 0) mbar_arrive_expect_tx(q_full, 2 * C::Q_BYTES);
      tma_load_4d_pair(smem, &tmQ, map_to_rank(smem_u32(q_full), 0), 0, kvh << sh.log_g, row0 + (RC >> sh.log_g), 0);
      bool ok = true;
      int u = 0;
      for (; u < n_seq && ok; ++u) {
        const int s = u % C::NST;
        if (u >= C::NST) ok = mbar_wait(&empty[s], ((u - C::NST) / C::NST) & 1, err, PF_DEV_TIMEOUT_PRODUCER);
        if (!ok) break;
        uint8_t* dst = smem + C::OFF_ST + s * C::STAGE;
        const int cell = rt.cell0[run] + (ch_first + seq_chunk(u)) * RCH;
        const bool last = has_tail && u == n_seq - 1;
        const uint32_t bar = map_to_rank(smem_u32(&full[s]), 0);
        if (rank == 0) mbar_arrive_expect_tx(&full[s], last ? C::STAGE : 2 * C::STAGE);
        if (seq_is_k(u)) {
          tma_load_3d_pair(dst, &tmK, bar, kvh * HD, cell + rank * 64, 0);
        } else if (last && rank == 1) {
          mbar_arrive_expect_tx(tail, C::STAGE);
          tma_load_3d(dst, &tmV, tail, kvh * HD + HD / 2, cell, 0);
        } else {
          tma_load_3d_pair(dst, &tmV, bar, kvh * HD + rank * (HD / 2), cell, 0);
        }
      }
      // On an error the copies in flight land before the pair may leave (the
      // even CTA's barriers count those of both).
      if (!ok || read_error(err) != 0) {
        if (rank == 0) {
          runs_drain(q_full, 0);
          for (int x = max(0, u - C::NST); x < u; ++x) runs_drain(&full[x % C::NST], (x / C::NST) & 1);
        } else if (has_tail && u == n_seq) {
          runs_drain(tail, 0);
        }
      }
    }
    __syncwarp();
  } else if (warp == 0 && rank == 1) {
    if (has_tail) {
      bool ok = mbar_wait(tail, 0, err, PF_DEV_TIMEOUT_MMA);
      ok = __all_sync(0xffffffffu, ok);
      if (ok) {
        clear_tail();
        if (lane == 0) mbar_arrive_cluster(map_to_rank(smem_u32(tail), 0));
      }
    }
    __syncwarp();
  } else if (warp == 0) {
    // ---------------- MMA issue for the pair: the warp runs the loop in
    // step, one elected lane issues
    const bool leader = elect_one();
    constexpr uint32_t id_qk = idesc_f16_f32(256, RCH, false);
    constexpr uint32_t id_pv = idesc_f16_f32(256, HD, true);
    const uint64_t qd0 = sdesc_sw128(smem_u32(smem));
    bool ok = mbar_wait_spin(q_full, 0, err, PF_DEV_TIMEOUT_MMA);
    ok = __all_sync(0xffffffffu, ok);
    bool issued = false;
    for (int u = 0; u < n_seq && ok; ++u) {
      const int s = u % C::NST, j = seq_chunk(u);
      const int b = j & 1;
      const uint32_t st = smem_u32(smem + C::OFF_ST + s * C::STAGE);
      ok = mbar_wait_spin(&full[s], (u / C::NST) & 1, err, PF_DEV_TIMEOUT_MMA);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      if (seq_is_k(u)) {
        // S(j): P(j-2), which lay in this buffer, was read by MMAs issued before
        tc_fence_after();
        if (leader) {
          const uint64_t kd0 = sdesc_sw128(st);
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {
            const int bx = kk >> 2, w = kk & 3;  // 64-dim box, 16-dim step within it
            tc_mma_f16_pair(tmem + C::TMEM_S + b * RCH, qd0 + ((bx * (128 * 128) + w * 32) >> 4),
                            kd0 + ((bx * (64 * 128) + w * 32) >> 4), id_qk, kk > 0 ? 1u : 0u);
          }
          tc_commit_pair(map_to_rank(smem_u32(&s_full[b]), 0));
          tc_commit_pair(map_to_rank(smem_u32(&s_full[b]), 1));
        }
      } else {
        if (has_tail && u == n_seq - 1) {
          ok = mbar_wait<true>(tail, 0, err, PF_DEV_TIMEOUT_MMA);
          clear_tail();
        }
        const uint64_t vd0 = HD == 256 ? sdesc_sw128_lbo_sbo(st, RCH * 128, 1024) : sdesc_sw64_mn(st);
        constexpr int KSTEP = 16 * (HD == 256 ? 128 : 64);  // bytes of 16 keys
#pragma unroll
        for (int h = 0; h < C::NH; ++h) {
          if (ok) ok = mbar_wait_spin(&p_full[2 * h + b], (j >> 1) & 1, err, PF_DEV_TIMEOUT_MMA);
          ok = __all_sync(0xffffffffu, ok);
          tc_fence_after();
          if (ok && leader) {
#pragma unroll
            for (int kk = 0; kk < C::KPT / 16; ++kk)
              tc_mma_f16_ts_pair(tmem + C::TMEM_O + h * HD, tmem + C::TMEM_S + b * RCH + h * C::KPT + kk * 8,
                                 vd0 + (((h * (C::KPT / 16) + kk) * KSTEP) >> 4), id_pv, (j > 0 || kk > 0) ? 1u : 0u);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (leader) {
          tc_commit_pair(map_to_rank(smem_u32(&pv_done[b]), 0));
          tc_commit_pair(map_to_rank(smem_u32(&pv_done[b]), 1));
        }
      }
      if (leader) {
        tc_commit_pair(map_to_rank(smem_u32(&empty[s]), 0));
        tc_commit_pair(map_to_rank(smem_u32(&empty[s]), 1));
      }
      __syncwarp();
      issued = true;
    }
    if (!ok && issued && leader) {
      // the MMAs already issued finish before TMEM is freed
      tc_commit_pair(map_to_rank(smem_u32(drain), 0));
      runs_drain(drain, 0);
    }
    __syncwarp();
  } else if ((warp & 3) < row_warps(rank)) {
    // ---------------- rows (warps 2..: TMEM lane quarter warp % 4, part h of each chunk)
    const int qw = warp & 3, h = (warp - 2) >> 2;
    const int R = RC + 32 * qw + lane;
    const int t = R >> sh.log_g, head = (kvh << sh.log_g) + (R & ((1 << sh.log_g) - 1));
    const bool row = R < total_rows;
    const int pos = row ? pos0 + t : -1;
    const uint64_t* row_mask = TREE && row ? mask + static_cast<size_t>(row0 + t) * words : nullptr;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * qw) << 16);
    constexpr int NB = C::KPT / 32;
    const uint64_t c2 = pack_f32x2(cexp, cexp);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n && ok; ++j) {
      const int b = j & 1;
      const int key0 = (ch_first + j) * RCH + h * C::KPT;
      const uint32_t ts = lanes + C::TMEM_S + b * RCH + h * C::KPT;
      if (lane == 0) ok = mbar_wait_spin(&s_full[b], (j >> 1) & 1, err, PF_DEV_TIMEOUT_EPILOGUE);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      uint32_t x[NB][32];
#pragma unroll
      for (int w = 0; w < NB; ++w) tmem_ld32(ts + 32 * w, x[w]);
      // the row's view of its keys, skipped where every row of the warp sees all of them
      const bool all = TREE ? key0 + C::KPT <= pos0 : __all_sync(0xffffffffu, pos >= key0 + C::KPT - 1);
#pragma unroll
      for (int w = 0; w < NB; ++w) tmem_ld_wait32(x[w]);
      if (!all) {
#pragma unroll
        for (int w = 0; w < NB; ++w) {
          uint32_t bits;
          if (TREE) {
            bits = row ? tree_bits(row_mask, words, pos0, n_rows, key0 + 32 * w) : 0u;
          } else {
            const int nv = pos - key0 - 32 * w + 1;
            bits = nv >= 32 ? 0xffffffffu : nv <= 0 ? 0u : (1u << nv) - 1u;
          }
          mask_scores(x[w], bits);
        }
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int w = 0; w < NB; ++w) max_scores(x[w], mx);
      const float mj = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      // The reference moves only when this chunk's maximum passes it by more
      // than 2^8 (or on the row's first visible keys); until then P is taken
      // against the old one (p <= 2^8, well inside fp16) and O needs no touch.
      const bool grow = mj != -INFINITY && (m == -INFINITY || (mj - m) * cexp > 8.f);
      const float mn = grow ? mj : m;
      const bool resc = grow && m != -INFINITY;
      const float scale = resc ? ex2_approx((m - mn) * cexp) : 1.f;
      const float nmc = mn == -INFINITY ? 0.f : -mn * cexp;
      const uint64_t nmc2 = pack_f32x2(nmc, nmc);
      uint64_t ls[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
      for (int w = 0; w < NB; w += 2) {
        uint32_t pw[32];  // 64 fp16 probabilities
        exp_scores(x[w], c2, nmc2, pw, ls);
        exp_scores(x[w + 1], c2, nmc2, pw + 16, ls);
        tmem_st32(ts + 16 * w, pw);  // over scores that have been read
      }
      const float2 l01 = unpack_f32x2(add_f32x2(add_f32x2(ls[0], ls[1]), add_f32x2(ls[2], ls[3])));
      l = __fmaf_rn(l, scale, l01.x + l01.y);
      m = mn;
      tmem_st_wait();
      // O *= scale once P V(j-1) has landed, only in the warps where a row
      // moved its reference.  (S(j) was issued after P V(j-2), so each of the
      // two barriers has at most the awaited phase outstanding.)
      if (j >= 1 && __any_sync(0xffffffffu, resc)) {
        if (lane == 0) ok = mbar_wait(&pv_done[(j - 1) & 1], ((j - 1) >> 1) & 1, err, PF_DEV_TIMEOUT_EPILOGUE);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < HD / 32; ++c) {
          uint32_t y[32];
          tmem_ld32(lanes + C::TMEM_O + h * HD + 32 * c, y);
          tmem_ld_wait32(y);
#pragma unroll
          for (int q = 0; q < 32; ++q) y[q] = __float_as_uint(__uint_as_float(y[q]) * scale);
          tmem_st32(lanes + C::TMEM_O + h * HD + 32 * c, y);
        }
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_pair_relaxed(map_to_rank(smem_u32(&p_full[2 * h + b]), 0));
    }
    if (ok) {
      if (lane == 0) ok = mbar_wait_spin(&pv_done[(n - 1) & 1], ((n - 1) >> 1) & 1, err, PF_DEV_TIMEOUT_EPILOGUE);
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    // the parts' weights: w_h = 2^((m_h - m) c); each of a row's two warps
    // writes half of the dims
    float w0 = 1.f, w1 = 0.f;
    if constexpr (C::NH > 1) {
      float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
      ml[h * 128 + 32 * qw + lane] = make_float2(ok ? m : __int_as_float(0x7fc00000), l);
      asm volatile("bar.sync %0, 64;" ::"r"(1 + qw) : "memory");
      const float2 a = ml[32 * qw + lane], c = ml[128 + 32 * qw + lane];
      m = fmaxf(a.x, c.x);
      w0 = a.x == -INFINITY ? 0.f : ex2_approx((a.x - m) * cexp);
      w1 = c.x == -INFINITY ? 0.f : ex2_approx((c.x - m) * cexp);
      l = w0 * a.y + w1 * c.y;
    }
    if (ok) {
      // Every MMA of the pair and every copy is done.  Each 32 x 32 block of O
      // goes through a warp-private buffer in the idle ring, so that global
      // stores cover whole row segments.
      tc_fence_after();
      // groups with keys of this row; 0: nothing to write
      const int n_g = !row ? 0 : TREE ? rt.groups[run] : (pos / RCH) / sh.gc + 1;
      const int kind = grp >= n_g ? 0 : n_g == 1 ? 1 : 2;  // 1: output row, 2: group state
      const float inv = kind != 1 ? 1.f : l == 0.f ? 0.f : __frcp_rn(l);  // a row that sees nothing: zeros
      w0 *= inv;
      w1 *= inv;
      const size_t own = kind == 1 ? (static_cast<size_t>(row0 + t) * sh.Hq + head) * HD
                                   : (static_cast<size_t>(idx) * sh.slot_rows + (R - R0)) * runs_state_stride(HD);
      const int rs = lane >> 3, pc = lane & 7;
      size_t dst[8];
      int dk[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dk[i] = __shfl_sync(0xffffffffu, kind, 4 * i + rs);
        dst[i] = __shfl_sync(0xffffffffu, static_cast<unsigned long long>(own), 4 * i + rs);
      }
      uint8_t* stg = smem + C::OFF_ST + (h * 4 + qw) * 4096;
#pragma unroll 1
      for (int c = h * (HD / 32 / C::NH); c < (h + 1) * (HD / 32 / C::NH); ++c) {
        uint32_t y[32];
        tmem_ld32(lanes + C::TMEM_O + 32 * c, y);
        tmem_ld_wait32(y);
        if constexpr (C::NH > 1) {
          uint32_t z[32];
          tmem_ld32(lanes + C::TMEM_O + HD + 32 * c, z);
          tmem_ld_wait32(z);
#pragma unroll
          for (int q = 0; q < 32; ++q)
            y[q] = __float_as_uint(__fmaf_rn(w0, __uint_as_float(y[q]), w1 * __uint_as_float(z[q])));
        } else {
#pragma unroll
          for (int q = 0; q < 32; ++q) y[q] = __float_as_uint(w0 * __uint_as_float(y[q]));
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
          *reinterpret_cast<uint4*>(stg + lane * 128 + ((q ^ (lane & 7)) << 4)) =
              make_uint4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int rr = 4 * i + rs;
          if (dk[i] == 0) continue;
          const float4 v = *reinterpret_cast<const float4*>(stg + rr * 128 + ((pc ^ (rr & 7)) << 4));
          if (dk[i] == 1) {
            const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
            *reinterpret_cast<uint2*>(out + dst[i] + 32 * c + 4 * pc) =
                make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
          } else {
            *reinterpret_cast<float4*>(part + dst[i] + 32 * c + 4 * pc) = v;
          }
        }
        __syncwarp();
      }
      if (kind == 2 && h == 0) *reinterpret_cast<float2*>(part + own + HD) = make_float2(m, l);
    }
  }
  tc_fence_before();
  __syncthreads();
  // neither CTA leaves (or frees TMEM) while the pair's MMAs may still use it
  cluster_sync_all();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, C::TMEM_COLS);
  }
}

// Rows with several groups: m = max m_g, w_g = 2^((m_g - m) c), out =
// (sum w_g o_g) / (sum w_g l_g), sums in group order.  A warp per row R of a
// row block, lane owning HD/32 consecutive dims; bound by the states' bytes
// (L2: they were just written).
template <int HD, bool TREE>
__global__ void __launch_bounds__(256) attn_runs_merge_kernel(const __grid_constant__ RunTable rt, const RunsShape sh,
                                                              const float* __restrict__ part,
                                                              __nv_bfloat16* __restrict__ out) {
  constexpr int PER = HD / 32;
  constexpr float c = attn_c<HD>();
  pdl_launch();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int kvh = blockIdx.y;
  // blockIdx.x: (row block of any run) x (8-row slice); a run's blocks start
  // at item0 / groups blocks of its own items
  const int slices = sh.slot_rows / 8;
  int blk = static_cast<int>(blockIdx.x) / slices;
  const int R_in = (static_cast<int>(blockIdx.x) % slices) * 8 + (threadIdx.x >> 5);
  int run = 0, nb = 0;
  for (;; ++run) {
    nb = ((rt.n[run] << sh.log_g) + RROWS - 1) / RROWS;
    if (blk < nb || run == rt.n_runs - 1) break;
    blk -= nb;
  }
  const int R = blk * RROWS + R_in;
  if (R >= rt.n[run] << sh.log_g) return;
  const int t = R >> sh.log_g;
  const int n_g = TREE ? rt.groups[run] : ((rt.pos0[run] + t) / RCH) / sh.gc + 1;
  if (n_g < 2) return;
  // group g's slot of this block
  const size_t step = static_cast<size_t>(nb) * sh.Hkv * sh.slot_rows * runs_state_stride(HD);
  const float* base =
      part + ((static_cast<size_t>(rt.item0[run] + (nb - 1 - blk)) * sh.Hkv + kvh) * sh.slot_rows + R_in) *
                 runs_state_stride(HD);
  float m = -INFINITY;
  for (int g = lane; g < n_g; g += 32) m = fmaxf(m, base[g * step + HD]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float acc[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) acc[i] = 0.f;
  float l = 0.f;
  for (int g0 = 0; g0 < n_g; g0 += 4) {  // four groups' loads in flight
    float o[4][PER];
    float2 ml[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int g = min(g0 + k, n_g - 1);
      const float* p = base + g * step;
      ml[k] = *reinterpret_cast<const float2*>(p + HD);
      if constexpr (PER >= 4) {
#pragma unroll
        for (int i = 0; i < PER; i += 4) {
          const float4 v = *reinterpret_cast<const float4*>(p + lane * PER + i);
          o[k][i] = v.x, o[k][i + 1] = v.y, o[k][i + 2] = v.z, o[k][i + 3] = v.w;
        }
      } else {
        const float2 v = *reinterpret_cast<const float2*>(p + lane * PER);
        o[k][0] = v.x, o[k][1] = v.y;
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (g0 + k >= n_g || ml[k].x == -INFINITY) continue;
      const float w = ex2_approx((ml[k].x - m) * c);
      l = __fmaf_rn(w, ml[k].y, l);
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] = __fmaf_rn(w, o[k][i], acc[i]);
    }
  }
  const float inv = l == 0.f ? 0.f : __frcp_rn(l);
  __nv_bfloat16* d = out + (static_cast<size_t>(rt.row0[run] + t) * sh.Hq + (kvh << sh.log_g) +
                            (R & ((1 << sh.log_g) - 1))) * HD + lane * PER;
#pragma unroll
  for (int i = 0; i < PER; i += 2)
    *reinterpret_cast<__nv_bfloat162*>(d + i) = __floats2bfloat162_rn(acc[i] * inv, acc[i + 1] * inv);
}

// ---------------------------------------------------------------------------
// host: the cut of a call into work items

struct RunsPlan {
  RunTable rt;
  RunsShape sh;
  int blocks = 0;      // row blocks of all runs
  bool split = false;  // some run has several groups
  int64_t state_bytes = 0;
};

static int sm_count() {
  static const int n = [] {
    int dev = 0, v = 0;
    if (cudaGetDevice(&dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return 152;
    }
    return v > 0 ? v : 152;
  }();
  return n;
}

// The chunks per group: as many groups as shorten the call, by a count of
// chunk times.  An item costs its chunks and `fixed` chunk times (prologue,
// Q, output); the call ends no earlier than its longest item and its total
// work over the pairs that fit at once, and splitting adds the states'
// traffic and the merge launch (`fixed` again).  State slots are bounded by
// four per resident pair.
static void make_plan(RunsPlan& p, const pfop_attn_run* runs, int n_runs, int Hq, int Hkv, int hd, bool tree) {
  const int G = Hq / Hkv;
  int order[RUNS_MAX], row0[RUNS_MAX], cnt = 0, row = 0;
  for (int r = 0; r < n_runs; ++r) {
    if (runs[r].n_rows > 0) {
      order[cnt++] = r;
      row0[r] = row;
    }
    row += runs[r].n_rows;
  }
  // runs with the most keys first: their blocks are the longest items
  std::stable_sort(order, order + cnt, [&](int a, int b) {
    return runs[a].pos0 + runs[a].n_rows > runs[b].pos0 + runs[b].n_rows;
  });
  const int units = sm_count() / 2;
  const int fixed = hd == 256 ? 3 : 4;
  int max_ch = 0, max_rows = 0;
  double work = 0;  // chunks over all row blocks
  p.blocks = 0;
  for (int i = 0; i < cnt; ++i) {
    const pfop_attn_run& r = runs[order[i]];
    const int nb = (r.n_rows * G + RROWS - 1) / RROWS, ch = (r.pos0 + r.n_rows + RCH - 1) / RCH;
    max_ch = std::max(max_ch, ch);
    max_rows = std::max(max_rows, std::min(RROWS, r.n_rows * G));
    p.blocks += nb;
    work += tree ? double(nb) * ch : nb * (r.pos0 + 0.5 * (r.n_rows + RROWS / G)) / RCH + 0.5 * nb;
  }
  auto items_of = [&](int gc) {
    int64_t n = 0;
    for (int i = 0; i < cnt; ++i) {
      const pfop_attn_run& r = runs[order[i]];
      n += int64_t((r.n_rows * G + RROWS - 1) / RROWS) * (((r.pos0 + r.n_rows + RCH - 1) / RCH + gc - 1) / gc);
    }
    return n;
  };
  int best_gc = max_ch;
  double best = 1e30;
  for (int gc = max_ch, s = 1; gc >= 1;) {
    const int64_t items = items_of(gc);
    if (gc < max_ch && items * Hkv > 4 * int64_t(units)) break;
    const double live = std::max<double>(p.blocks, tree ? double(items) : work / gc + 0.5 * p.blocks);
    const double t = std::max(double(gc + fixed), (work + fixed * live) * Hkv / units) + (gc < max_ch ? fixed : 0);
    if (t < best) best = t, best_gc = gc;
    // the next smaller group that makes another number of groups
    int next = gc;
    while (next >= gc && s <= max_ch) next = (max_ch + s) / (s + 1), ++s;
    if (next >= gc) break;
    gc = next;
  }
  p.sh.Hq = Hq;
  p.sh.Hkv = Hkv;
  p.sh.log_g = 0;
  while ((1 << p.sh.log_g) < G) ++p.sh.log_g;
  p.sh.gc = best_gc;
  p.sh.slot_rows = (max_rows + 31) / 32 * 32;
  p.split = false;
  int items = 0;
  p.rt.n_runs = cnt;
  for (int i = 0; i < cnt; ++i) {
    const pfop_attn_run& r = runs[order[i]];
    const int nb = (r.n_rows * G + RROWS - 1) / RROWS, ch = (r.pos0 + r.n_rows + RCH - 1) / RCH;
    p.rt.row0[i] = row0[order[i]];
    p.rt.n[i] = r.n_rows;
    p.rt.pos0[i] = r.pos0;
    p.rt.cell0[i] = r.cell0;
    p.rt.item0[i] = items;
    p.rt.groups[i] = (ch + best_gc - 1) / best_gc;
    if (p.rt.groups[i] > 1) p.split = true;
    items += nb * p.rt.groups[i];
  }
  p.sh.items = items;
  p.state_bytes =
      p.split ? int64_t(items) * Hkv * p.sh.slot_rows * runs_state_stride(hd) * int64_t(sizeof(float)) : 0;
}

template <int HD, bool TREE>
static cudaError_t launch_runs(const RunsPlan& p, const __half* q, const __half* k, const __half* v, int64_t n_cells,
                               int total, const uint64_t* mask, int words, __nv_bfloat16* out, float* part, int* err,
                               cudaStream_t s) {
  using C = RunsCfg<HD>;
  cudaError_t e = smem_opt_in<attn_runs_kernel<HD, TREE>>(C::SMEM);
  if (e != cudaSuccess) return e;
  const int Hq = p.sh.Hq, Hkv = p.sh.Hkv, G = Hq / Hkv;
  // Q as [64-dim box][row][head][64 dims], K as [64-dim box][cell][64 dims],
  // V as [box][cell][dims of one box]: hd/2 dims a CTA, in 64-dim boxes
  // (128-byte swizzle) at hd 256, one 32-dim box (64-byte swizzle) at hd 64
  CUtensorMap tq, tk, tv;
  std::string why;
  {
    const uint64_t dims[4] = {64, static_cast<uint64_t>(Hq), static_cast<uint64_t>(total), HD / 64};
    const uint64_t st[3] = {HD * 2, static_cast<uint64_t>(Hq) * HD * 2, 128};
    const uint32_t box[4] = {64, static_cast<uint32_t>(G), static_cast<uint32_t>(128 / G), HD / 64};
    if (!encode_fp16_sw128(&tq, q, 4, dims, st, box, &why)) return cudaErrorInvalidValue;
  }
  {
    const uint64_t dims[3] = {static_cast<uint64_t>(Hkv) * HD, static_cast<uint64_t>(n_cells), HD / 64};
    const uint64_t st[2] = {static_cast<uint64_t>(Hkv) * HD * 2, 128};
    const uint32_t box[3] = {64, 64, HD / 64};
    if (!encode_fp16_sw128(&tk, k, 3, dims, st, box, &why)) return cudaErrorInvalidValue;
    const uint32_t vbox[3] = {HD == 256 ? 64u : 32u, RCH, HD == 256 ? 2u : 1u};
    if (!(HD == 256 ? encode_fp16_sw128(&tv, v, 3, dims, st, vbox, &why)
                    : encode_fp16_sw64(&tv, v, 3, dims, st, vbox, &why)))
      return cudaErrorInvalidValue;
  }
  e = launch_k(attn_runs_kernel<HD, TREE>, dim3(2u * p.sh.items * Hkv), dim3(C::THREADS), C::SMEM, s, 2, tq, tk, tv,
               p.rt, p.sh, mask, words, out, part, err);
  if (e != cudaSuccess || !p.split) return e;
  return launch_k(attn_runs_merge_kernel<HD, TREE>, dim3(p.blocks * (p.sh.slot_rows / 8), Hkv), dim3(256), 0, s, 1,
                  p.rt, p.sh, static_cast<const float*>(part), out);
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
  RunsPlan p;
  make_plan(p, runs, n_runs, Hq, Hkv, hd, tree);
  if (work_bytes < WORK_HEADER + p.state_bytes) return fail(PF_E_ARG, "the scratch is smaller than these runs need");
  int* err = static_cast<int*>(work);
  float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(work) + WORK_HEADER);
  auto go = [&](auto launch) {
    return launch(p, static_cast<const __half*>(q), static_cast<const __half*>(k), static_cast<const __half*>(v),
                  n_cells, static_cast<int>(total), mask, words, static_cast<__nv_bfloat16*>(out), part, err, s);
  };
  const cudaError_t e = hd == 256 ? (tree ? go(launch_runs<256, true>) : go(launch_runs<256, false>))
                                  : (tree ? go(launch_runs<64, true>) : go(launch_runs<64, false>));
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
  if (rc != PF_OK) return rc;
  if (total == 0) return WORK_HEADER;
  RunsPlan a, b;
  make_plan(a, runs, n_runs, Hq, Hkv, hd, false);
  make_plan(b, runs, n_runs, Hq, Hkv, hd, true);
  return WORK_HEADER + std::max(a.state_bytes, b.state_bytes);
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
