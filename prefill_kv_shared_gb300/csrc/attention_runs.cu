// Attention of several sequences' rows in one call (pfop_attention_packed,
// pfop_attention_tree): causal over each sequence's own keys, or over a
// context and a tree of drafted tokens, on the 5th-generation tensor cores.
//
// MMA rows are (row, head-in-group) pairs of a run: row R = t*G + g is the
// run's row t and query head kvh*G + g, so the G heads of a KV head share its
// K/V.  256 consecutive rows of a run and KV head are an item, worked on by a
// pair of CTAs (a 2-CTA cluster, tcgen05 .cta_group::2); at hd 64, where rows
// or items are few, 128 and one CTA (below a pair too).  A pair works through
// segments, a segment being an item and a range of its 128-key chunks, with
// one online softmax:
//     S = Q K^T, m' = max(m, max_k s_k), p_k = 2^((s_k - m') c),
//     l' = l 2^((m - m') c) + sum_k p_k, O' = O 2^((m - m') c) + fp16(P) V
// with c = log2(e)/sqrt(hd), S, O, m, l in fp32.
//
// The cut: either a pair per item, or all items laid end to end (each
// weighing its chunks and a fixed cost) and every resident pair given the
// same share of that line, so that long and short sequences, many rows and
// few, load the SMs evenly (make_plan).  A segment that holds all chunks of
// its item writes O/l.  Of an item cut in two, the first part (in pair p)
// leaves its state (O, m, l) in the scratch and the second (in pair p+1)
// joins it with its own: a pair takes its segments from the line's end, so
// the state is the first thing pair p makes and the last that pair p+1
// needs, and pair p+1 waits only for a pair of a lower index, which never
// waits before that.  (A merge kernel for these took 24 us of a 250 us call.)
// Where an item may be cut in three or more, all cut items leave their states
// to attn_runs_merge_kernel.
//
// Why pairs: 128 rows against a chunk need 64 bytes of K/V per SM clock at
// the full tensor rate, more than L2 delivers to all SMs at once; 256 rows
// over a pair, each CTA holding half of every K chunk (64 keys) and half of
// every V chunk (hd/2 dims), need 32, and the halves leave room for 2.5
// chunks in flight beside Q at hd 256.
//
// Roles of a CTA: warp 1 copies the K/V halves by TMA (one ring of
// stages, in the order in which the MMAs use them; the copies of both CTAs
// complete on the even CTA's barriers), warp 2 Q; warp 0 of the even CTA
// issues the pair's MMAs, at hd 64 with warp 3 for O += P V (waiting and
// issuing for both took one warp about 1400 clocks a chunk, twice the MMAs of
// a chunk at hd 64; at hd 256 one warp is better, since S(j+2) then needs no
// wait for P(j) V(j)); warps 4 and up own the CTA's 128 rows (thread = TMEM lane =
// row): softmax, P (fp16, over the columns of S that it came from), the
// rescale of O, the output.  At hd 256 one warpgroup keeps up with the MMAs
// (2048 clocks a chunk against about 1600) and two S buffers let S of the
// next chunk be formed while P of this one is.  At hd 64 a chunk has a
// quarter of the MMA work for the same exponentials: two warpgroups take the
// chunks in turn, each with its own m, l and O (joined at the segment's
// end), so that one's exponentials run while the other loads, looks for the
// maximum or hands over, and three S buffers keep both supplied.  All waits
// are bounded (PF_WAIT_CYCLES, and more where a wait lasts as long as a number
// of chunks): one that gives up flags the scratch's error word and the pair
// unwinds.
//
// Bounds and figures (one call, GB300): long prompts at hd 256 are bound by
// the MMAs (2058 clocks a chunk, 2048 at the full rate; six prompts, 15845
// rows in all, 8 heads over 2: 223 to 235 us with the power limit, 206 without
// it, 1560 to 1780 TFLOP/s); at hd 64 by the chain of a chunk's softmax and
// hand-overs (about 1100 clocks, of which the exponential unit is busy for
// 512; prompts of 4096 and 2048, 32 heads over 4: 108.6 us, 790 TFLOP/s).
// Drafted trees read each context once: 12 trees of 1 to 64 rows, 159 MB, 40.6
// us, 3.9 TB/s; 64 trees of 16 rows, 69 MB, 25.0 us, 2.8 TB/s, where a segment's
// first scores and output (4000 to 5000 clocks) count as much as its chunks;
// 64 sequences of one row over 4096 keys, 8 heads over 1, 268 MB, 45.8 us, 5.9
// TB/s.  Small calls are bound by latency: 25 rows 5.1 us, 512 rows of 8 heads
// 10.8 us.
#include "../../include/prefill_ops.h"
#include "attn.cuh"
#include "common.cuh"
#include "kernels.h"

#include <algorithm>
#include <string>

namespace pf {

constexpr int RUNS_MAX = 128;
constexpr int RCH = 128;  // keys of a chunk

// the call's runs, passed in the kernel's parameters; a run's items are its
// row blocks, last (longest) first, once per KV head
struct RunTable {
  int n_runs = 0;
  int row0[RUNS_MAX];  // first packed row
  int n[RUNS_MAX], pos0[RUNS_MAX], cell0[RUNS_MAX];
  int item0[RUNS_MAX + 1];  // items before the run
  int w0[RUNS_MAX + 1];     // their weight
};

struct RunsShape {
  int Hq, Hkv, log_g;  // G = 1 << log_g query heads per KV head
  int bs_log;          // 1 << bs_log of a run's rows are an item's
  int fixed;           // item_fixed
  int per;             // weight of a pair's share; 0: a pair per item
  int pairs;
  int merge;  // an item may be cut in three or more: the merge kernel joins all that are cut
  int desc_by_item;  // the merge kernel's table has an entry per item, not per pair (the smaller of the two)
  int slot_rows;  // rows of a state slot in the scratch
};

// weight of an item besides its chunks: its Q copy, first scores and output,
// in chunk times.  (hd 256: 15845 rows of 6 prompts 250, 228 and 238 us with 2,
// 3 and 4; hd 64: prompts of 4096 and 2048 124, 114, 109, 108 and 116 with 2,
// 3, 4, 5 and 8, 64 trees of 16 rows 25.7, 25.5, 24.8, 25.6 and 25.9.)
constexpr int item_fixed(int hd) { return hd == 256 ? 3 : 4; }

// CL: CTAs of an item
template <int HD, int CL>
struct RunsCfg {
  static constexpr int Q_BYTES = 128 * HD * 2;  // [64-dim box][128 rows][128 B]
  static constexpr int KEYS = RCH / CL;                // keys of a chunk in a CTA
  static constexpr int STAGE = KEYS * HD * 2;          // K [box][KEYS][128 B] or V [box][128 keys][VB], hd/CL dims
  static constexpr int VB = HD / CL >= 64 ? 128 : 64;  // bytes of a key's row in a box of V
  static constexpr int V_BOXES = HD / CL * 2 / VB;
  // as many stages as fit beside Q (at hd 256 four, with the output staged
  // through the room of the fifth, took 354 us for 254)
  static constexpr int NST = HD == 256 ? 5 : CL == 2 ? 16 : 12;
  static constexpr int NG = HD == 256 ? 1 : 2;  // row warpgroups, taking chunks in turn
  static constexpr int NSB = NG + 1;            // S buffers
  static constexpr int LA = NSB - 1;            // chunks that S is formed ahead of P V
  static constexpr int OFF_ST = Q_BYTES;
  static constexpr int OFF_BAR = OFF_ST + NST * STAGE;
  static constexpr int OFF_ML = OFF_BAR + 512;        // (m, l) of each warpgroup's rows
  static constexpr int SMEM = OFF_ML + (NG > 1 ? NG * 128 * 8 : 0) + 1024;  // + alignment slack
  static constexpr int TMEM_S = 0;
  static constexpr int TMEM_O = NSB * RCH;  // an O per warpgroup
  static constexpr int TMEM_COLS = 512;
  static_assert(TMEM_O + NG * HD <= TMEM_COLS, "TMEM");
  static constexpr int THREADS = 128 + 128 * NG;
  // Row (in the pair's 256) of row i of CTA `rank`.  At hd 64 the CTAs take
  // 32-row groups in turn, so that an item of few rows loads the exponential
  // units of both SMs.
  static constexpr int Q_ROWS = HD == 256 || CL == 1 ? 128 : 32;  // rows of a copy of Q
  static __device__ __forceinline__ int row_of(int rank, int i) {
    return Q_ROWS == 128 ? rank * 128 + i : ((i >> 5) * 2 + rank) * 32 + (i & 31);
  }
  // Registers (setmaxnreg, hd 64): a row thread holds its 128 scores.
  // 128 * 88 + 256 * 208 of the 384 * 168 that the block is launched with.
  static constexpr int LEAN_REGS = 88, ROW_REGS = 208;
  static_assert(SMEM <= 232448, "shared memory");
};

// A state slot, per 32 rows (a warp's): o as [4 dims][row][4], so that lanes
// that hold a row each access 512 contiguous bytes, then (m, l) per row.
// (Rows stored one after another took a segment's end 2 us, a second part
// 10 us: every lane in another line.)
__host__ __device__ constexpr int runs_state_floats(int hd) { return 32 * hd + 64; }

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

// a whole 32-byte sector from one thread
__device__ __forceinline__ void st_global_v8(void* p, const uint32_t* r) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
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

// Bound of a wait that lasts while the pair works through that many chunks:
// four times what the slowest kind takes (2058 clocks), beside the usual bound.
__device__ __forceinline__ long long runs_wait_limit(uint32_t chunks) {
  return PF_WAIT_CYCLES + static_cast<long long>(chunks) * 8192;
}

// bounded wait for a barrier on an error path (about 0.2 s)
__device__ __forceinline__ void runs_drain(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  const long long t0 = clock64();
  while (!mbar_try_wait(a, parity)) {
    if (clock64() - t0 > 400000000ll) return;
  }
}

// Wait (bounded like the barriers' waits) until a flag in global memory has
// counted to n, and make what was written before visible.
__device__ __forceinline__ bool wait_flag(const int* flag, int n, int* err) {
  long long t0 = 0;
  for (uint32_t i = 1;; ++i) {
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
    if (v >= n) return true;
    if ((i & 255u) == 0u) {
      const long long now = clock64();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > PF_WAIT_CYCLES) {
        set_error(err, PF_DEV_TIMEOUT_EPILOGUE);
        return false;
      }
      if (read_error(err) != 0) return false;
    }
  }
}

// the last entry of first[0 .. n-1] not above x
__host__ __device__ __forceinline__ int find_last(const int* first, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (first[mid] <= x)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// A run's row blocks and their chunks.  Block i (counted from the run's
// end) has block b = nb-1-i of 1 << bs_log rows; causal, it needs the
// chunks up to its last row.
template <bool TREE>
struct RunBlocks {
  int n, pos0, bs_log, fixed, nb, last;  // last: chunks of the whole run
  __host__ __device__ RunBlocks(int n_rows, int p0, const RunsShape& sh)
      : n(n_rows), pos0(p0), bs_log(sh.bs_log), fixed(sh.fixed), nb((n_rows + (1 << bs_log) - 1) >> bs_log),
        last(static_cast<int>((static_cast<unsigned>(p0) + n_rows + RCH - 1) / RCH)) {}
  // sum over x' < x of floor(x' / (128 / bs)); modulo 2^32 (differences of it are exact)
  __host__ __device__ unsigned floors(unsigned x) const {
    const int sl = 7 - bs_log;
    const unsigned k = x >> sl;
    const unsigned tri = k & 1 ? k * ((k - 1) >> 1) : (k >> 1) * (k - 1);
    return (tri << sl) + k * (x - (k << sl));
  }
  // chunks of blocks 0 .. B-1 from the run's start, none of them the last
  __host__ __device__ int from_start(int B) const {
    const unsigned c = static_cast<unsigned>(pos0) + (1u << bs_log) + RCH - 1;
    if (bs_log == 8) return static_cast<int>(B * (c / RCH) + static_cast<unsigned>(B) * (B - 1));
    return static_cast<int>(floors((c >> bs_log) + B) - floors(c >> bs_log));
  }
  __host__ __device__ int chunks(int i) const {
    if (TREE || i == 0) return last;
    return static_cast<int>((static_cast<unsigned>(pos0) + (static_cast<unsigned>(nb - i) << bs_log) + RCH - 1) / RCH);
  }
  // weight of items 0 .. i-1
  __host__ __device__ int weight(int i) const {
    if (TREE || i == 0) return i * (last + fixed);
    return i * fixed + last + from_start(nb - 1) - from_start(nb - i);
  }
  // weight(nb), where 32 bits may not hold it: block b of a prompt's, the last
  // one aside, has floor((c + b bs) / 128) chunks
  __host__ int64_t whole() const {
    const int64_t f = int64_t(nb) * fixed;
    if (TREE) return f + int64_t(nb) * last;
    const int64_t B = nb - 1, c = int64_t(pos0) + (1 << bs_log) + RCH - 1;
    if (bs_log == 8) return f + last + B * (c / RCH) + B * (B - 1);
    // sum over x' < x of x' >> sl, sl = 7 - bs_log
    auto floors = [&](int64_t x) {
      const int sl = 7 - bs_log;
      const int64_t k = x >> sl;
      return (k * (k - 1) / 2 << sl) + k * (x - (k << sl));
    };
    return f + last + floors((c >> bs_log) + B) - floors(c >> bs_log);
  }
};

// an item: run, KV head, row block and its place on the line of weights
template <bool TREE>
struct ItemAt {
  int run, kvh, i, w;  // w: weight of all items before
  // by its number
  __host__ __device__ static ItemAt number(const RunTable& rt, const RunsShape& sh, int idx) {
    ItemAt a;
    a.run = find_last(rt.item0, rt.n_runs, idx);
    const RunBlocks<TREE> rb(rt.n[a.run], rt.pos0[a.run], sh);
    const int loc = idx - rt.item0[a.run];
    a.kvh = loc / rb.nb;
    a.i = loc % rb.nb;
    a.w = rt.w0[a.run] + a.kvh * rb.weight(rb.nb) + rb.weight(a.i);
    return a;
  }
  // the one whose weight covers x
  __host__ __device__ static ItemAt weight(const RunTable& rt, const RunsShape& sh, int x) {
    ItemAt a;
    a.run = find_last(rt.w0, rt.n_runs, x);
    const RunBlocks<TREE> rb(rt.n[a.run], rt.pos0[a.run], sh);
    const int head = rb.weight(rb.nb);
    int rem = x - rt.w0[a.run];
    a.kvh = rem / head;
    rem -= a.kvh * head;
    int lo = 0, hi = rb.nb - 1;
    if (TREE) {
      lo = rem / (rb.last + sh.fixed);
    } else {
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (rb.weight(mid) <= rem)
          lo = mid;
        else
          hi = mid - 1;
      }
    }
    a.i = lo;
    a.w = x - rem + rb.weight(lo);
    return a;
  }
};

// The segments of a pair, from the end of its share.  The share is a range of
// the line of weights; the chunk k of an item lies at w + fixed + k.
enum SegKind : int {
  SEG_WHOLE = 0,  // all of its item
  SEG_FIRST = 1,  // first of two: leaves its state to the next pair
  SEG_SECOND = 2,  // second of two: joins the pair before's
  SEG_PART = 3,   // the merge kernel joins it
};
template <bool TREE>
struct Segments {
  const RunTable& rt;
  const RunsShape& sh;
  ItemAt<TREE> at;
  int pair, lo, hi;
  bool left;
  // the segment
  int run, kvh, R0, ch0, n, kind;
  int slot;  // its state's slot: an item's first segment 2 pair + 1, others 2 pair
  __host__ __device__ Segments(const RunTable& t, const RunsShape& s, int p) : rt(t), sh(s), pair(p), left(true) {
    if (sh.per == 0) {
      at = ItemAt<TREE>::number(rt, sh, pair);
      lo = hi = 0;  // not used
    } else {
      lo = pair * sh.per;
      hi = lo + sh.per < rt.w0[rt.n_runs] ? lo + sh.per : rt.w0[rt.n_runs];
      left = lo < hi;
      if (left) at = ItemAt<TREE>::weight(rt, sh, hi - 1);
    }
  }
  __host__ __device__ bool next() {
    while (left) {
      const RunBlocks<TREE> rb(rt.n[at.run], rt.pos0[at.run], sh);
      const int ch = rb.chunks(at.i), w = at.w + sh.fixed;
      const bool all = sh.per == 0;
      const int k0 = all || lo < w ? 0 : lo - w, k1 = all || hi - w > ch ? ch : hi - w;
      run = at.run;
      kvh = at.kvh;
      R0 = (rb.nb - 1 - at.i) << (sh.bs_log + sh.log_g);
      ch0 = k0;
      n = k1 - k0;
      slot = 2 * pair + (k0 == 0 ? 1 : 0);
      kind = SEG_WHOLE;
      if (n < ch) {
        // the item's chunks outside lie before this share, behind it, or both
        if (sh.merge)
          kind = SEG_PART;
        else if (k0 == 0)
          kind = ch - k1 <= sh.per ? SEG_FIRST : SEG_PART;
        else
          kind = k1 == ch && w >= lo - sh.per ? SEG_SECOND : SEG_PART;
      }
      // on to the item before
      if (all || at.w <= lo) {
        left = false;
      } else {
        if (--at.i < 0) {
          if (--at.kvh < 0) {
            at.kvh = sh.Hkv - 1;
            --at.run;
          }
          at.i = RunBlocks<TREE>(rt.n[at.run], rt.pos0[at.run], sh).nb - 1;
        }
        at.w -= sh.fixed + RunBlocks<TREE>(rt.n[at.run], rt.pos0[at.run], sh).chunks(at.i);
      }
      if (n > 0) return true;
    }
    return false;
  }
};

// bits of the keys kk .. kk+31 (positions) that the row sees: the context
// [0, pos0), then its mask's bits for the drafted tokens [0, n)
__device__ __forceinline__ uint32_t tree_bits(const uint64_t* row_mask, int words, int pos0, int n, int kk) {
  const int d = kk - pos0;  // drafted token of the word's first bit
  if (d <= -32) return 0xffffffffu;
  if (d >= n) return 0u;
  // (volatile: loaded where it stands in the program, not where it is used)
  auto word = [&](int i) {
    uint64_t v;
    asm volatile("ld.global.nc.b64 %0, [%1];" : "=l"(v) : "l"(row_mask + i));
    return v;
  };
  uint64_t w;
  if (d < 0) {
    w = (word(0) << -d) | ((1ull << -d) - 1ull);
  } else {
    w = word(d >> 6) >> (d & 63);
    if ((d & 63) > 32 && (d >> 6) + 1 < words) w |= word((d >> 6) + 1) << (64 - (d & 63));
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

template <int HD, int CL, bool TREE>
__global__ void __launch_bounds__(RunsCfg<HD, CL>::THREADS, 1)
    attn_runs_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                     const __grid_constant__ CUtensorMap tmV, const __grid_constant__ RunTable rt, const RunsShape sh,
                     const uint64_t* __restrict__ mask, int words, __nv_bfloat16* __restrict__ out,
                     float* part, int* __restrict__ desc, int* err, int* flags) {
  using C = RunsCfg<HD, CL>;
  constexpr float cexp = attn_c<HD>();
  extern __shared__ uint8_t smem_raw[];
  // The two CTAs' buffers lie at the same shared-memory offset (one
  // descriptor addresses both): same kernel, same alignment rounding.
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* full = bars;            // NST, in the even CTA: a stage has landed in both; in the odd CTA: a
                                    // V to be cleared has landed there (one CTA: the even one)
  uint64_t* empty = bars + C::NST;  // NST: the MMAs that read the stage are done (its S or P V too)
  uint64_t* cleared = bars + 2 * C::NST;  // NST, in the even CTA: the odd CTA's V is cleared
  uint64_t* q_full = bars + 3 * C::NST;   // in the even CTA: Q of both has landed
  uint64_t* q_empty = q_full + 1;         // the segment's last S is formed
  uint64_t* o_free = q_full + 2;          // in the even CTA: the row warps of both have read O
  uint64_t* drain = q_full + 3;           // 2, error path only
  uint64_t* p_full = q_full + 5;          // by S buffer, in the even CTA: a warpgroup of both CTAs
  uint64_t* state_out = p_full + C::NSB;  // this CTA's rows of a first part's state are written
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(state_out + 1);
  volatile int* left_early = reinterpret_cast<volatile int*>(tmem_slot + 1);  // a warp of the pair gave up a wait
  static_assert((3 * C::NST + 7 + C::NSB) * 8 <= 512 && C::NG <= 2, "barrier layout");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CL == 2 ? static_cast<int>(cluster_ctarank()) : 0;
  const int pair = static_cast<int>(blockIdx.x) / CL;
  auto in_even = [](const void* p) { return CL == 2 ? map_to_rank(smem_u32(p), 0) : smem_u32(p); };
  pdl_launch();

  if (threadIdx.x == 0) {
    for (int b = 0; b < C::NST; ++b) {
      mbar_init(&full[b], 1);
      mbar_init(&empty[b], 1);
      mbar_init(&cleared[b], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int b = 0; b < C::NSB; ++b) mbar_init(&p_full[b], 4 * CL);
    mbar_init(o_free, 4 * CL * C::NG);
    mbar_init(state_out, 4 * C::NG);
    mbar_init(&drain[0], 1);
    mbar_init(&drain[1], 1);
    // (a plain store costs the row threads 16 more spilled bytes at hd 64: prompts of 4096 and 2048 109 us for 107)
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(smem_u32(tmem_slot + 1)), "r"(0) : "memory");
    fence_mbar_init();
  }
  if (warp == 1 && lane == 0) {
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  if (warp == 2 && lane == 0) prefetch_tensormap(&tmQ);
  if (warp == 0) {
    if constexpr (CL == 2)
      tmem_alloc_pair(tmem_slot, C::TMEM_COLS);
    else
      tmem_alloc(tmem_slot, C::TMEM_COLS);
  }
  Segments<TREE> sg(rt, sh, pair);
  tc_fence_before();
  __syncthreads();
  if constexpr (CL == 2) cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();

  // What every role does on giving up: note it in both CTAs.
  auto give_up = [&]() {
    if (lane == 0) {
      *left_early = 1;
      if constexpr (CL == 2) {
        const uint32_t at = map_to_rank(smem_u32(const_cast<const int*>(left_early)), static_cast<uint32_t>(rank ^ 1));
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(1) : "memory");
      }
    }
    __syncwarp();
  };

  // Counters that run on over the pair's segments, the same in every role:
  // ring fills (fill f uses stage f % NST, in its use number f / NST), chunks
  // (chunk j uses S buffer j % NSB and warpgroup j % NG) and segments.  A
  // segment's fills: K(0) .. K(LA-1), then K(LA), V(0), K(LA+1), V(1), ..,
  // V(n-1), so that S(j+LA) is formed before P(j) V(j).  The MMAs of a fill
  // arrive on its stage's `empty`, which serves all who wait for them in
  // order: the K/V producer, the row warps for S and for P V, and the S
  // issuer for P V.  (A wait by parity must not come a phase early or late.
  // Not early: who waits for a fill knows that the copies of fewer than NST
  // fills before it were issued and that S and P V up to NSB chunks back are
  // done, so the stage's last use is over.  Not late: the stage's next use is
  // over only after a later P V, which needs the waiting warp's P, its S or
  // its o_free.)
  auto k_fill = [](int jl) { return jl < C::LA ? jl : 2 * jl - C::LA; };
  auto v_fill = [](int jl, int n) { return jl + C::LA < n ? 2 * jl + C::LA + 1 : n + jl; };
  // The V rows of keys past the run (only in the run's last chunk) are
  // cleared in shared memory before the MMAs read them: P is 0 there, but
  // what lies in those cells may be an infinity or NaN.  In the odd CTA that
  // copy completes on the stage's own barrier and its clearing on `cleared`;
  // a bit per stage holds the parity of the next such fill.
  auto tail_keys = [&]() { return rt.pos0[sg.run] + rt.n[sg.run] - (sg.ch0 + sg.n - 1) * RCH; };
  auto clear_tail = [&](uint32_t fill) {
    uint8_t* v = smem + C::OFF_ST + (fill % C::NST) * C::STAGE;
    for (int box = 0; box < C::V_BOXES; ++box)
      for (int o = tail_keys() * C::VB + lane * 16; o < RCH * C::VB; o += 512)
        *reinterpret_cast<uint4*>(v + box * RCH * C::VB + o) = make_uint4(0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
    __syncwarp();
  };

  // what the merge kernel has to know of this pair
  auto leave_table = [&]() {
    if (sh.per == 0) return;
    int4* d = reinterpret_cast<int4*>(desc);
    if (!sh.desc_by_item) d[2 * pair] = make_int4(0, 0, 0, 0);
    Segments<TREE> all(rt, sh, pair);
    while (all.next()) {
      if (all.ch0 > 0 || (all.kind != SEG_PART && !sh.desc_by_item)) continue;
      // the item's first segment: its pairs (0: nothing to join), rows, first packed row, KV head; first row
      const RunBlocks<TREE> rb(rt.n[all.run], rt.pos0[all.run], sh);
      const int rows_log = sh.bs_log + sh.log_g;
      const int i = rb.nb - 1 - (all.R0 >> rows_log);
      const int left = rb.chunks(i) - all.n;  // chunks in the pairs after this one
      const int at = sh.desc_by_item ? rt.item0[all.run] + all.kvh * rb.nb + i : pair;
      d[2 * at] = make_int4(all.kind == SEG_PART ? 1 + (left + sh.per - 1) / sh.per : 0,
                            min(1 << rows_log, (rt.n[all.run] << sh.log_g) - all.R0), rt.row0[all.run], all.kvh);
      d[2 * at + 1] = make_int4(all.R0, pair, 0, 0);
    }
  };

  if (warp >= 4) {
    if constexpr (C::NG > 1) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::ROW_REGS));
    // ---------------- rows (warps 4..: TMEM lane quarter warp % 4, warpgroup h)
    const int qw = warp & 3, h = (warp - 4) >> 2;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * qw) << 16);
    const uint32_t o_at = lanes + C::TMEM_O + h * HD;
    constexpr int NB = RCH / 32;
    const uint64_t c2 = pack_f32x2(cexp, cexp);
    const uint32_t o_free_at = in_even(o_free);
    const uint32_t p_full_at = in_even(p_full);
    bool ok = true;
    uint32_t j0 = 0, f0 = 0;
    // the MMAs of fill f are done
    auto done = [&](uint32_t f) {
      ok = mbar_wait_spin(&empty[f % C::NST], (f / C::NST) & 1, err, PF_DEV_TIMEOUT_EPILOGUE);
      ok = __all_sync(0xffffffffu, ok);
      return ok;
    };
    for (bool more = sg.next(); ok && more;) {
      const int n_rows = rt.n[sg.run], pos0 = rt.pos0[sg.run], row0 = rt.row0[sg.run];
      const int total_rows = n_rows << sh.log_g;
      const int Rw = sg.R0 + C::row_of(rank, 32 * qw);  // the warp's first row
      const bool active = Rw < total_rows;          // warps without rows only keep step
      const int R = Rw + lane;
      const int t = R >> sh.log_g, head = (sg.kvh << sh.log_g) + (R & ((1 << sh.log_g) - 1));
      const bool row = R < total_rows;
      const int pos = row ? pos0 + t : -1;
      const uint64_t* row_mask = TREE && row ? mask + static_cast<size_t>(row0 + t) * words : nullptr;
      float m = -INFINITY, l = 0.f;
      const int first = C::NG == 1 ? 0 : static_cast<int>((j0 + h) & 1);  // of the warpgroup's chunks
      for (int jl = first; jl < sg.n; jl += C::NG) {
        const int b = (j0 + jl) % C::NSB;
        const int key0 = (sg.ch0 + jl) * RCH;
        // the row's view of its keys, skipped where every row of the warp sees
        // all of them; a tree's comes from memory, which the wait for S hides
        const bool all = TREE ? key0 + RCH <= pos0 : __all_sync(0xffffffffu, pos >= key0 + RCH - 1);
        uint32_t bits[NB];
        if (TREE && !all) {
#pragma unroll
          for (int w = 0; w < NB; ++w) bits[w] = row ? tree_bits(row_mask, words, pos0, n_rows, key0 + 32 * w) : 0u;
        }
        if (!done(f0 + k_fill(jl))) break;
        if (active) {
          const uint32_t ts = lanes + C::TMEM_S + b * RCH;
          tc_fence_after();
          uint32_t x[NB][32];
#pragma unroll
          for (int w = 0; w < NB; ++w) tmem_ld32(ts + 32 * w, x[w]);
#pragma unroll
          for (int w = 0; w < NB; ++w) tmem_ld_wait32(x[w]);
          if (!all) {
#pragma unroll
            for (int w = 0; w < NB; ++w) {
              if (!TREE) {
                const int nv = pos - key0 - 32 * w + 1;
                bits[w] = nv >= 32 ? 0xffffffffu : nv <= 0 ? 0u : (1u << nv) - 1u;
              }
              mask_scores(x[w], bits[w]);
            }
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int w = 0; w < NB; ++w) max_scores(x[w], mx);
          const float mj = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
          // The reference moves only when this chunk's maximum passes it by
          // more than 2^8 (or on the row's first visible keys); until then P is
          // taken against the old one (p <= 2^8, well inside fp16) and O needs
          // no touch.
          const bool grow = mj != -INFINITY && (m == -INFINITY || (mj - m) * cexp > 8.f);
          const float mn = grow ? mj : m;
          const bool resc = grow && m != -INFINITY;
          const float scale = resc ? ex2_approx((m - mn) * cexp) : 1.f;
          float nmc = mn == -INFINITY ? 0.f : -mn * cexp;
          // s c - round(m c) is as good as (s - m) c while m c is small: its
          // rounding is 2^-13 at 2^12, and hundreds where q and k are as large
          // as fp16 goes.  Rows beyond 2^12 take the difference first, through
          // TMEM 32 columns at a time: little code beside the path that is
          // always taken (64 x 32 rows at hd 64 28.5 us; 29.3 with the 128
          // subtractions written out, 28.0 without the check).
          if (__any_sync(0xffffffffu, fabsf(nmc) > 4096.f)) {
            const float off = fabsf(nmc) > 4096.f ? mn : 0.f;
            nmc = off != 0.f ? 0.f : nmc;
            const uint64_t off2 = pack_f32x2(-off, -off);
#pragma unroll
            for (int w = 0; w < NB; ++w) tmem_st32(ts + 32 * w, x[w]);
            tmem_st_wait();
#pragma unroll 1
            for (int w = 0; w < NB; ++w) {
              uint32_t y[32];
              tmem_ld32(ts + 32 * w, y);
              tmem_ld_wait32(y);
#pragma unroll
              for (int k = 0; k < 32; k += 2) {
                const float2 d =
                    unpack_f32x2(add_f32x2(pack_f32x2(__uint_as_float(y[k]), __uint_as_float(y[k + 1])), off2));
                y[k] = __float_as_uint(d.x);
                y[k + 1] = __float_as_uint(d.y);
              }
              tmem_st32(ts + 32 * w, y);
            }
            tmem_st_wait();
#pragma unroll
            for (int w = 0; w < NB; ++w) tmem_ld32(ts + 32 * w, x[w]);
#pragma unroll
            for (int w = 0; w < NB; ++w) tmem_ld_wait32(x[w]);
          }
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
          // O *= scale once the last P V of it has landed, only in the warps where a row
          // moved its reference
          if (jl >= C::NG && __any_sync(0xffffffffu, resc)) {
            if (!done(f0 + v_fill(jl - C::NG, sg.n))) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < HD / 32; ++c) {
              uint32_t y[32];
              tmem_ld32(o_at + 32 * c, y);
              tmem_ld_wait32(y);
#pragma unroll
              for (int q = 0; q < 32; ++q) y[q] = __float_as_uint(__uint_as_float(y[q]) * scale);
              tmem_st32(o_at + 32 * c, y);
            }
            tmem_st_wait();
          }
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_pair_relaxed(p_full_at + b * 8);
      }
      // the next segment is looked up while the last P V is formed
      const int n = sg.n, R0 = sg.R0, kind = sg.kind, slot = sg.slot;
      more = sg.next();
      if (ok) done(f0 + v_fill(n - 1, n));
      // the warpgroups' weights: w_h = 2^((m_h - m) c); each of a row's two
      // warps writes half of the 64 dims
      float w0 = 1.f, w1 = 0.f;
      if constexpr (C::NG > 1) {
        float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
        ml[h * 128 + 32 * qw + lane] = make_float2(m, ok ? l : -1.f);  // -1: this warp gave up (l is a sum of p >= 0)
        asm volatile("bar.sync %0, 64;" ::"r"(1 + qw) : "memory");
        const float2 a = ml[32 * qw + lane], c = ml[128 + 32 * qw + lane];
        // Both have read before either writes again.  (A warp that gives up in
        // the next segment gets there without waiting for the other; its -1
        // read here would leave it alone at the next barrier for good.)
        asm volatile("bar.sync %0, 64;" ::"r"(1 + qw) : "memory");
        ok = __all_sync(0xffffffffu, a.y != -1.f && c.y != -1.f);
        m = fmaxf(a.x, c.x);
        w0 = a.x == -INFINITY ? 0.f : ex2_approx((a.x - m) * cexp);
        w1 = c.x == -INFINITY ? 0.f : ex2_approx((c.x - m) * cexp);
        l = w0 * a.y + w1 * c.y;
      }
      if (!ok) {
        *left_early = 1;  // (this CTA's: MMAs that need the other's rows or copies make the MMA warp give up too)
        break;
      }
      if (active) {
        // a thread writes its row, 32-byte sectors at a time
        tc_fence_after();
        const bool whole = kind == SEG_WHOLE || kind == SEG_SECOND;
        // the warp's rows in a state slot
        auto state_at = [&](int slot) {
          return (static_cast<size_t>(slot) * (sh.slot_rows / 32) + ((Rw - R0) >> 5)) * runs_state_floats(HD);
        };
        // the first part's state of this row, and its weight
        const float* other_part = nullptr;
        float w_other = 0.f;
        int* flag = nullptr;
        if (kind == SEG_SECOND) {
          flag = flags + (sg.pair - 1) * (4 * CL) + rank * 4 + qw;
          if (!wait_flag(flag, C::NG, err)) ok = false;
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          other_part = part + state_at(2 * sg.pair - 1);
          const float2 ml = __ldcg(reinterpret_cast<const float2*>(other_part + 32 * HD) + lane);
          const float mm = fmaxf(m, ml.x);
          const float a = m == -INFINITY ? 0.f : ex2_approx((m - mm) * cexp);
          w_other = ml.x == -INFINITY ? 0.f : ex2_approx((ml.x - mm) * cexp);
          l = a * l + w_other * ml.y;
          w0 *= a;
          w1 *= a;
        }
        const float inv = !whole ? 1.f : l == 0.f ? 0.f : __frcp_rn(l);  // a row that sees nothing: zeros
        w0 *= inv;
        w1 *= inv;
        w_other *= inv;
        __nv_bfloat16* own_out = out + (static_cast<size_t>(row0 + t) * sh.Hq + head) * HD;
        float* own_state = part + state_at(slot);
        auto store = [&](int c, const uint32_t (&y)[32]) {
          if (row && whole) {
            uint32_t hb[16];
            float f[32];
#pragma unroll
            for (int q = 0; q < 32; ++q) f[q] = __uint_as_float(y[q]);
            if (kind == SEG_SECOND) {
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                const float4 o = __ldcg(reinterpret_cast<const float4*>(other_part) + (8 * c + q) * 32 + lane);
                f[4 * q] = __fmaf_rn(w_other, o.x, f[4 * q]);
                f[4 * q + 1] = __fmaf_rn(w_other, o.y, f[4 * q + 1]);
                f[4 * q + 2] = __fmaf_rn(w_other, o.z, f[4 * q + 2]);
                f[4 * q + 3] = __fmaf_rn(w_other, o.w, f[4 * q + 3]);
              }
            }
#pragma unroll
            for (int q = 0; q < 16; ++q) {
              const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * q], f[2 * q + 1]);
              hb[q] = *reinterpret_cast<const uint32_t*>(&v);
            }
            st_global_v8(own_out + 32 * c, hb);
            st_global_v8(own_out + 32 * c + 16, hb + 8);
          } else if (!whole) {  // rows past the run's as well: their lanes' places are there
#pragma unroll
            for (int q = 0; q < 8; ++q)
              *(reinterpret_cast<uint4*>(own_state) + (8 * c + q) * 32 + lane) =
                  make_uint4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
          }
          __syncwarp();
        };
        // two loads of 32 columns in flight
        uint32_t y[32], z[32];
        if constexpr (C::NG == 1) {
#pragma unroll 1
          for (int c = 0; c < HD / 32; c += 2) {
            tmem_ld32(lanes + C::TMEM_O + 32 * c, y);
            tmem_ld32(lanes + C::TMEM_O + 32 * c + 32, z);
            tmem_ld_wait32(y);
            tmem_ld_wait32(z);
#pragma unroll
            for (int q = 0; q < 32; ++q) {
              y[q] = __float_as_uint(w0 * __uint_as_float(y[q]));
              z[q] = __float_as_uint(w0 * __uint_as_float(z[q]));
            }
            store(c, y);
            store(c + 1, z);
          }
        } else {
          // columns h * 32 .. + 31 of both O; after one chunk the other
          // warpgroup's holds nothing
          const int own_g = static_cast<int>(j0 & 1), other = n > 1 ? own_g ^ 1 : own_g;
          const float wa = own_g ? w1 : w0, wb = n > 1 ? (own_g ? w0 : w1) : 0.f;
          tmem_ld32(lanes + C::TMEM_O + own_g * HD + 32 * h, y);
          tmem_ld32(lanes + C::TMEM_O + other * HD + 32 * h, z);
          tmem_ld_wait32(y);
          tmem_ld_wait32(z);
#pragma unroll
          for (int q = 0; q < 32; ++q)
            y[q] = __float_as_uint(__fmaf_rn(wa, __uint_as_float(y[q]), wb * __uint_as_float(z[q])));
          store(h, y);
        }
        if (!whole && h == 0) reinterpret_cast<float2*>(own_state + 32 * HD)[lane] = make_float2(m, l);
        __syncwarp();
        // the warp's rows of the first part's state are read: the flag as it was
        if (lane == 0 && kind == SEG_SECOND && atomicAdd(flag, 1) == 2 * C::NG - 1) atomicExch(flag, 0);
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_pair_relaxed(o_free_at);
        if (kind == SEG_FIRST) mbar_arrive(state_out);
      }
      j0 += n;
      f0 += 2 * n;
    }
  } else {
    if constexpr (C::NG > 1) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::LEAN_REGS));
    if (warp == 1) {
      // ---------------- K/V producer (each CTA its own halves).  A stage comes
      // as one copy per 64-dim box, a lane each: copies of one thread are
      // served one after another, those of several overlap.
      bool ok = true;
      uint32_t f = 0, tails = 0;
      while (ok && sg.next()) {
        const bool has_tail = tail_keys() < RCH;
        auto load = [&](bool is_k, int jl) {
          const int s = f % C::NST;
          if (f >= C::NST) ok = mbar_wait(&empty[s], (f / C::NST + 1) & 1, err, PF_DEV_TIMEOUT_PRODUCER);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) return;
          uint8_t* dst = smem + C::OFF_ST + s * C::STAGE;
          const int cell = rt.cell0[sg.run] + (sg.ch0 + jl) * RCH;
          const bool last = !is_k && has_tail && jl == sg.n - 1;
          if (lane == 0) {
            if (rank == 0) mbar_arrive_expect_tx(&full[s], last ? C::STAGE : CL * C::STAGE);
            if (rank == 1 && last) mbar_arrive_expect_tx(&full[s], C::STAGE);
          }
          __syncwarp();
          if (lane < (is_k ? HD / 64 : C::V_BOXES)) {
            const CUtensorMap* map = is_k ? &tmK : &tmV;
            uint8_t* box = dst + lane * (is_k ? C::KEYS * 128 : RCH * C::VB);
            const int c0 = sg.kvh * HD + (is_k ? 0 : rank * (HD / 2)), c1 = cell + (is_k ? rank * C::KEYS : 0);
            if (CL == 1 || (last && rank == 1))
              tma_load_3d(box, map, &full[s], c0, c1, lane);
            else
              tma_load_3d_pair(box, map, in_even(&full[s]), c0, c1, lane);
          }
          if (last) tails ^= 1u << s;
          ++f;
        };
        for (int jl = -C::LA; jl < sg.n && ok; ++jl) {
          if (jl + C::LA < sg.n) load(true, jl + C::LA);
          if (jl >= 0 && ok) load(false, jl);
        }
      }
      // On an error the copies in flight land before the pair may leave (the
      // even CTA's barriers count those of both).
      if (lane == 0 && (!ok || read_error(err) != 0)) {
        if (rank == 0) {
          for (uint32_t x = f > C::NST ? f - C::NST : 0; x < f; ++x) runs_drain(&full[x % C::NST], (x / C::NST) & 1);
        } else {
          // a stage that never held such a copy is in phase 0, whose waiting
          // for parity 1 ends at once
          for (int x = 0; x < C::NST; ++x) runs_drain(&full[x], (tails >> x & 1u) ^ 1u);
        }
      }
      __syncwarp();
      if (!ok) give_up();
    } else if (warp == 2) {
      // ---------------- Q producer: a copy per 64-dim box, or per 32 rows
      bool ok = true, first = false;
      int active = 0;  // row warps of a first part that have rows
      int first_n = 0, last_n = 0;  // chunks of the first and of the last segment copied for
      // A first part (only a pair's first segment is one): its state is passed
      // on from here, so that the row warps need not wait until their stores
      // have reached L2.
      auto pass_on = [&]() {
        ok = mbar_wait(state_out, 0, err, PF_DEV_TIMEOUT_EPILOGUE, runs_wait_limit(first_n));
        ok = __all_sync(0xffffffffu, ok);
        if (ok && lane < active) {
          __threadfence();
          atomicAdd(flags + pair * (4 * CL) + rank * 4 + lane, C::NG);
        }
        __syncwarp();
        first = false;
      };
      uint32_t seg = 0;
      for (; ok && sg.next(); ++seg) {
        if (seg == 0) {
          first = sg.kind == SEG_FIRST;
          first_n = sg.n;
          for (int qw = 0; qw < 4; ++qw)
            if (sg.R0 + C::row_of(rank, 32 * qw) < rt.n[sg.run] << sh.log_g) active = qw + 1;
        }
        if (seg == 2 && first) pass_on();
        if (!ok) break;
        if (seg > 0) ok = mbar_wait(q_empty, (seg - 1) & 1, err, PF_DEV_TIMEOUT_PRODUCER, runs_wait_limit(last_n));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        last_n = sg.n;
        if (lane == 0 && rank == 0) mbar_arrive_expect_tx(q_full, CL * C::Q_BYTES);
        __syncwarp();
        constexpr int GROUPS = 128 / C::Q_ROWS;
        if (lane < GROUPS * (HD / 64)) {
          const int box = lane / GROUPS, g = lane % GROUPS;
          uint8_t* dst = smem + box * (128 * 128) + g * C::Q_ROWS * 128;
          const int head = sg.kvh << sh.log_g;
          const int row = rt.row0[sg.run] + ((sg.R0 + C::row_of(rank, g * C::Q_ROWS)) >> sh.log_g);
          if constexpr (CL == 2)
            tma_load_4d_pair(dst, &tmQ, in_even(q_full), 0, head, row, box);
          else
            tma_load_4d(dst, &tmQ, q_full, 0, head, row, box);
        }
      }
      if (lane == 0 && (!ok || read_error(err) != 0) && rank == 0 && seg > 0) runs_drain(q_full, (seg - 1) & 1);
      if (ok && first) pass_on();
      if (CL == 1 && lane == 0) leave_table();
      __syncwarp();
      if (!ok) give_up();
    } else if (warp == 0 && rank == 1) {
      // ---------------- the odd CTA's half of the run's last V
      bool ok = true;
      uint32_t f = 0, f_seen = 0, tails = 0;
      while (ok && sg.next()) {
        f += 2 * sg.n;
        if (tail_keys() >= RCH) continue;
        const int s = (f - 1) % C::NST;
        ok = mbar_wait(&full[s], tails >> s & 1u, err, PF_DEV_TIMEOUT_MMA, runs_wait_limit((f - f_seen) / 2));
        f_seen = f;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tails ^= 1u << s;
        clear_tail(f - 1);
        if (lane == 0) mbar_arrive_cluster(in_even(&cleared[s]));
      }
      __syncwarp();
      if (!ok) give_up();
    } else if (rank == 1) {
      // ---------------- warp 3 of the odd CTA
      if (lane == 0) leave_table();
      __syncwarp();
    } else {
      // ---------------- MMA issue for the pair: a warp runs its loop in step,
      // one elected lane issues.  Every lane waits; only the elected lane's
      // success lets MMAs go.
      const bool leader = elect_one();
      const uint32_t ring = smem_u32(smem + C::OFF_ST);
      // arrives on a barrier of every CTA of the item once the MMAs issued so far are done
      auto commit = [&](uint64_t* bar) {
        if constexpr (CL == 2) {
          tc_commit_pair(map_to_rank(smem_u32(bar), 0));
          tc_commit_pair(map_to_rank(smem_u32(bar), 1));
        } else {
          tc_commit(bar);
        }
      };
      bool ok = true, issued = false;
      uint32_t f0 = 0, j0 = 0, seg = 0, tails = 0;
      constexpr bool TWO = C::NG > 1;  // S and P V have a warp each
      constexpr uint32_t id_qk = idesc_f16_f32(128 * CL, RCH, false);
      constexpr uint32_t id_pv = idesc_f16_f32(128 * CL, HD, true);
      const uint64_t qd0 = sdesc_sw128(smem_u32(smem));
      uint32_t v_of[C::NSB];  // fills of V of the last NSB chunks, oldest first
#pragma unroll
      for (int i = 0; i < C::NSB; ++i) v_of[i] = 0;
      // S(j) = Q K^T
      auto issue_s = [&](int jl) {
        const uint32_t f = f0 + k_fill(jl), s = f % C::NST, j = j0 + jl, b = j % C::NSB;
        ok = ok && mbar_wait_spin(&full[s], (f / C::NST) & 1, err, PF_DEV_TIMEOUT_MMA);
        if (TWO) {
          // the buffer's last P has been used (one warp: by MMAs issued before)
          if (j >= C::NSB)
            ok = ok && mbar_wait_spin(&empty[v_of[0] % C::NST], (v_of[0] / C::NST) & 1, err, PF_DEV_TIMEOUT_MMA);
          tc_fence_after();
#pragma unroll
          for (int i = 0; i + 1 < C::NSB; ++i) v_of[i] = v_of[i + 1];
          v_of[C::NSB - 1] = f0 + v_fill(jl, sg.n);
        }
        if (leader && ok) {
          const uint64_t kd0 = sdesc_sw128(ring + s * C::STAGE);
#pragma unroll
          for (int kk = 0; kk < HD / 16; ++kk) {
            const int bx = kk >> 2, w = kk & 3;  // 64-dim box, 16-dim step within it
            const uint64_t qd = qd0 + ((bx * (128 * 128) + w * 32) >> 4), kd = kd0 + ((bx * (C::KEYS * 128) + w * 32) >> 4);
            if constexpr (CL == 2)
              tc_mma_f16_pair(tmem + C::TMEM_S + b * RCH, qd, kd, id_qk, kk > 0 ? 1u : 0u);
            else
              tc_mma_f16(tmem + C::TMEM_S + b * RCH, qd, kd, id_qk, kk > 0 ? 1u : 0u);
          }
          commit(&empty[s]);
          if (jl == sg.n - 1) commit(q_empty);
          issued = true;
        }
        __syncwarp();
      };
      // O += P(j) V(j)
      auto issue_pv = [&](int jl) {
        const uint32_t f = f0 + v_fill(jl, sg.n), s = f % C::NST, j = j0 + jl, b = j % C::NSB;
        ok = ok && mbar_wait_spin(&full[s], (f / C::NST) & 1, err, PF_DEV_TIMEOUT_MMA);
        if (jl == sg.n - 1 && tail_keys() < RCH) {
          if constexpr (CL == 2) {
            ok = ok && mbar_wait<true>(&cleared[s], tails >> s & 1u, err, PF_DEV_TIMEOUT_MMA);
            tails ^= 1u << s;
          }
          ok = __all_sync(0xffffffffu, ok);
          if (ok) clear_tail(f);
        }
        // the last segment's O is read out before this one's replaces it
        if (jl == 0 && seg > 0) ok = ok && mbar_wait(o_free, (seg - 1) & 1, err, PF_DEV_TIMEOUT_MMA);
        ok = ok && mbar_wait_spin(&p_full[b], (j / C::NSB) & 1, err, PF_DEV_TIMEOUT_MMA);
        tc_fence_after();
        if (leader && ok) {
          const uint32_t st = ring + s * C::STAGE;
          const uint64_t vd0 = C::VB == 128 ? sdesc_sw128_lbo_sbo(st, RCH * 128, 1024) : sdesc_sw64_mn(st);
          const uint32_t a = tmem + C::TMEM_S + b * RCH, d = tmem + C::TMEM_O + (j % C::NG) * HD;
#pragma unroll
          for (int kk = 0; kk < RCH / 16; ++kk) {
            const uint64_t vd = vd0 + ((kk * 16 * C::VB) >> 4);
            if constexpr (CL == 2)
              tc_mma_f16_ts_pair(d, a + kk * 8, vd, id_pv, (jl >= C::NG || kk > 0) ? 1u : 0u);
            else
              tc_mma_f16_ts(d, a + kk * 8, vd, id_pv, (jl >= C::NG || kk > 0) ? 1u : 0u);
          }
          commit(&empty[s]);
          issued = true;
        }
      };
      for (; (TWO || warp == 0) && sg.next(); j0 += sg.n, f0 += 2 * sg.n, ++seg) {
        if (warp == 0) {
          ok = ok && mbar_wait_spin(q_full, seg & 1, err, PF_DEV_TIMEOUT_MMA);
          for (int jl = 0; jl < (TWO ? sg.n : C::LA) && jl < sg.n; ++jl) {
            issue_s(jl);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
        }
        if (!TWO || warp == 3)
          for (int jl = 0; jl < sg.n; ++jl) {
            if (!TWO && jl + C::LA < sg.n) issue_s(jl + C::LA);
            issue_pv(jl);
            // every lane knows of one that gave up: the leader then drains,
            // whether or not its own waits ended
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
        if (!ok) break;
      }
      if (!ok && issued && leader) {
        // the MMAs already issued finish before TMEM is freed
        uint64_t* bar = &drain[warp == 0 ? 0 : 1];
        if constexpr (CL == 2)
          tc_commit_pair(map_to_rank(smem_u32(bar), 0));
        else
          tc_commit(bar);
        runs_drain(bar, 0);
      }
      __syncwarp();
      if (!ok) give_up();
    }
  }
  tc_fence_before();
  __syncthreads();
  // neither CTA leaves (or frees TMEM) while the pair's MMAs may still use it
  if constexpr (CL == 2) cluster_sync_all();
  if (warp == 0) {
    // The roles' drains miss copies that one CTA's producer issued after the
    // other's had given up (the even CTA's barriers count both), and those that
    // were in flight when another role gave up.  Nothing is issued any more, a
    // copy takes microseconds, and neither CTA's shared memory is given away
    // before some milliseconds have passed.
    if (*left_early) {
      const long long t0 = clock64();
      while (clock64() - t0 < 10000000ll) __nanosleep(1000);
    }
    __syncwarp();
    tc_fence_after();
    if constexpr (CL == 2)
      tmem_dealloc_pair(tmem, C::TMEM_COLS);
    else
      tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

// Cut items: m = max m_p, w_p = 2^((m_p - m) c), out =
// (sum w_p o_p) / (sum w_p l_p) over the item's pairs p, p+1, .. in order.
// blockIdx.x counts items, or pairs with the item that starts in a pair's
// first segment (desc: 8 ints each); blockIdx.y 32-row groups; `ways` warps
// take four dims of the group's rows (lane = row), the states dealt out among
// them and their sums joined in warp order.  Bound by the latency of reading
// the states from L2: eight are in flight, and many states want many warps
// (25 rows over 32768 keys, 65 states: 20.0 us with 8 ways, 30.8 with one; few
// states do not: 4 trees, 15 states over 4 items, 14.3 with one, 19.6 with 8).
template <int HD>
__global__ void __launch_bounds__(256) attn_runs_merge_kernel(const RunsShape sh, int ways, const int* desc,
                                                              const float* part, __nv_bfloat16* out) {
  constexpr float c = attn_c<HD>();
  constexpr int FLY = 8;
  __shared__ float4 sum[8][32];
  __shared__ float2 sum_ml[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp % ways;
  const int quad = static_cast<int>(blockIdx.z) * (8 / ways) + warp / ways;
  pdl_launch();
  pdl_wait();
  const int4 d = __ldcg(reinterpret_cast<const int4*>(desc) + 2 * blockIdx.x);  // pairs, rows, first packed row, KV head
  const int2 e = __ldcg(reinterpret_cast<const int2*>(desc) + 4 * blockIdx.x + 2);
  const int R0 = e.x, p0 = e.y, np = d.x;
  const int R_in = static_cast<int>(blockIdx.y) * 32 + lane;
  if (np == 0 || static_cast<int>(blockIdx.y) * 32 >= d.y) return;  // nothing to join, or none of the rows
  float m = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int q = sub; q < np; q += FLY * ways) {
    float4 o[FLY];
    float2 ml[FLY];
#pragma unroll
    for (int k = 0; k < FLY; ++k) {
      const int p = q + k * ways;
      // the first pair's slot is its second
      const float* s = part + (static_cast<size_t>(p == 0 ? 2 * p0 + 1 : 2 * (p0 + p)) * (sh.slot_rows / 32) + blockIdx.y) *
                                  runs_state_floats(HD);
      ml[k] = make_float2(-INFINITY, 0.f);
      o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p < np) {
        ml[k] = __ldcg(reinterpret_cast<const float2*>(s + 32 * HD) + lane);
        o[k] = __ldcg(reinterpret_cast<const float4*>(s) + quad * 32 + lane);
      }
    }
    float mn = m;
#pragma unroll
    for (int k = 0; k < FLY; ++k) mn = fmaxf(mn, ml[k].x);
    if (mn == -INFINITY) continue;
    const float w = m == -INFINITY ? 0.f : ex2_approx((m - mn) * c);
    l *= w;
    acc.x *= w, acc.y *= w, acc.z *= w, acc.w *= w;
    m = mn;
#pragma unroll
    for (int k = 0; k < FLY; ++k) {
      if (ml[k].x == -INFINITY) continue;
      const float wk = ex2_approx((ml[k].x - m) * c);
      l = __fmaf_rn(wk, ml[k].y, l);
      acc.x = __fmaf_rn(wk, o[k].x, acc.x);
      acc.y = __fmaf_rn(wk, o[k].y, acc.y);
      acc.z = __fmaf_rn(wk, o[k].z, acc.z);
      acc.w = __fmaf_rn(wk, o[k].w, acc.w);
    }
  }
  if (ways > 1) {
    sum[warp][lane] = acc;
    sum_ml[warp][lane] = make_float2(m, l);
    __syncthreads();
    if (sub != 0) return;
    float mn = m;
    for (int k = 1; k < ways; ++k) mn = fmaxf(mn, sum_ml[warp + k][lane].x);
    const float w = m == -INFINITY ? 0.f : ex2_approx((m - mn) * c);
    l *= w;
    acc.x *= w, acc.y *= w, acc.z *= w, acc.w *= w;
    for (int k = 1; k < ways; ++k) {
      const float2 ml = sum_ml[warp + k][lane];
      const float4 o = sum[warp + k][lane];
      const float wk = ml.x == -INFINITY ? 0.f : ex2_approx((ml.x - mn) * c);
      l = __fmaf_rn(wk, ml.y, l);
      acc.x = __fmaf_rn(wk, o.x, acc.x);
      acc.y = __fmaf_rn(wk, o.y, acc.y);
      acc.z = __fmaf_rn(wk, o.z, acc.z);
      acc.w = __fmaf_rn(wk, o.w, acc.w);
    }
  }
  if (R_in >= d.y) return;
  const float inv = l == 0.f ? 0.f : __frcp_rn(l);
  const int R = R0 + R_in;
  __nv_bfloat16* dst = out + (static_cast<size_t>(d.z + (R >> sh.log_g)) * sh.Hq + (d.w << sh.log_g) +
                              (R & ((1 << sh.log_g) - 1))) * HD + 4 * quad;
  const __nv_bfloat162 v0 = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
  const __nv_bfloat162 v1 = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(dst) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&v0), *reinterpret_cast<const uint32_t*>(&v1));
}

// ---------------------------------------------------------------------------
// host: the cut of a call into work items

struct RunsPlan {
  RunTable rt;
  RunsShape sh;
  int cl;  // CTAs of an item
  int items = 0;
  int64_t desc_bytes = 0;   // the merge kernel's table, ahead of the states
  int64_t state_bytes = 0;  // both
};

// of the current device; without one, a GB300's
static int sm_count() {
  int dev = 0, v = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    cudaGetLastError();
    return 152;
  }
  return v > 0 ? v : 152;
}

// Which cut: a pair per item where the items fit the GPU at once and the
// longest takes no longer than an even share would with what joining costs;
// else even shares over the resident pairs, but none below MIN_SHARE.
// Joining costs merge_cost chunk times and one for every merge_bytes of
// states written and read.  (hd 256: a 2048-row prompt of 8 heads 24.8 us
// with a pair per item, 34.2 in shares; 4 trees of 16 rows of 8 heads over
// 1300 keys 18.5 and 13.7; hd 64: 256 rows over 2000 keys 15.2 and 16.2, a
// tree of 5 rows over 3000 17.2 and 8.8.)  Where no item covers a whole share,
// a pair per item is better throughout (512 rows: 10.8 and 15.4 us).
// False: more work than the line of weights can count.
constexpr int merge_cost(int hd) { return hd == 256 ? 6 : 8; }
constexpr int64_t merge_bytes(int hd) { return (hd == 256 ? 4 : 2) << 20; }
constexpr int MAX_PAIRS = 120;  // twice as many of one CTA: flags of 4 words a CTA in the scratch's header
constexpr int MIN_SHARE = 4;
constexpr int64_t MAX_WEIGHT = int64_t(1) << 30;

template <bool TREE>
static bool make_plan(RunsPlan& p, const pfop_attn_run* runs, int n_runs, int Hq, int Hkv, int hd) {
  p.sh.Hq = Hq;
  p.sh.Hkv = Hkv;
  p.sh.log_g = 0;
  while ((1 << p.sh.log_g) < Hq / Hkv) ++p.sh.log_g;
  int64_t ones = 0, twos = 0;  // items of 128 rows, and of 256
  for (int r = 0; r < n_runs; ++r) {
    const int64_t rows = int64_t(runs[r].n_rows) << p.sh.log_g;
    ones += (rows + 127) / 128 * Hkv;
    twos += (rows + 255) / 256 * Hkv;
  }
  // At hd 64 a CTA works alone where there is not an item of 128 rows for
  // every SM (25 rows of 8 heads: 5.1 us, with pairs 5.7) or where pairs would
  // hold 15% more rows that are none (64 trees of 16 rows: 25.1 us, 32.4; 20
  // runs of 40 rows over 900 keys 20.8, 23.2); else the pair's half as many K/V
  // copies count (64 x 32 rows: 28.5 us with pairs, 32.5 without; prompts of
  // 4096 and 2048: 108, 123).
  const int sms = sm_count();
  const int cl = p.cl = hd == 64 && (ones <= sms || 200 * twos > 115 * ones) ? 1 : 2, item_rows = 128 * cl;
  p.sh.bs_log = (cl == 2 ? 8 : 7) - p.sh.log_g;
  p.sh.fixed = item_fixed(hd);
  int row = 0, n = 0, longest = 0, max_rows = 0;
  int64_t items = 0, weight = 0;
  for (int r = 0; r < n_runs; ++r) {
    if (runs[r].n_rows > 0) {
      const RunBlocks<TREE> rb(runs[r].n_rows, runs[r].pos0, p.sh);
      // the weights below are 32-bit
      if (weight + rb.whole() * Hkv >= MAX_WEIGHT) return false;
      p.rt.row0[n] = row;
      p.rt.n[n] = runs[r].n_rows;
      p.rt.pos0[n] = runs[r].pos0;
      p.rt.cell0[n] = runs[r].cell0;
      p.rt.item0[n] = static_cast<int>(items);
      p.rt.w0[n] = static_cast<int>(weight);
      ++n;
      items += int64_t(rb.nb) * Hkv;
      weight += rb.whole() * Hkv;
      longest = std::max(longest, rb.last);
      max_rows = std::max(max_rows, std::min(item_rows, runs[r].n_rows << p.sh.log_g));
    }
    row += runs[r].n_rows;
  }
  p.rt.n_runs = n;
  p.rt.item0[n] = static_cast<int>(items);
  p.rt.w0[n] = static_cast<int>(weight);
  p.items = static_cast<int>(items);
  p.sh.slot_rows = (max_rows + 31) / 32 * 32;
  const int units = std::min(MAX_PAIRS * 2 / cl, std::max(1, sms / cl));
  const int share = std::max<int>(MIN_SHARE, static_cast<int>((weight + units - 1) / units));
  const int pairs = static_cast<int>((weight + share - 1) / share);
  const int64_t states = (pairs + items) * p.sh.slot_rows * hd * 4 * 2;
  if (items <= units &&
      (longest <= share + 1 || longest + p.sh.fixed <= share + merge_cost(hd) + states / merge_bytes(hd))) {
    p.sh.per = p.sh.desc_by_item = 0;
    p.sh.pairs = p.items;
    p.desc_bytes = p.state_bytes = 0;
    p.sh.merge = 0;
  } else {
    p.sh.per = share;
    p.sh.pairs = pairs;
    p.sh.merge = longest > share + 1 ? 1 : 0;  // else no item covers a whole share
    p.sh.desc_by_item = p.items < p.sh.pairs ? 1 : 0;
    p.desc_bytes = (int64_t(std::min(p.sh.pairs, p.items)) * 32 + 255) / 256 * 256;
    p.state_bytes =
        p.desc_bytes + int64_t(2) * p.sh.pairs * (p.sh.slot_rows / 32) * runs_state_floats(hd) * static_cast<int64_t>(sizeof(float));
  }
  return true;
}

template <int HD, int CL, bool TREE>
static cudaError_t launch_runs(const RunsPlan& p, const __half* q, const __half* k, const __half* v, int64_t n_cells,
                               int total, const uint64_t* mask, int words, __nv_bfloat16* out, uint8_t* states,
                               int* err, int* flags, cudaStream_t s) {
  using C = RunsCfg<HD, CL>;
  cudaError_t e = smem_opt_in<attn_runs_kernel<HD, CL, TREE>>(C::SMEM);
  if (e != cudaSuccess) return e;
  const int Hq = p.sh.Hq, Hkv = p.sh.Hkv, G = Hq / Hkv;
  // Q as [64-dim box][row][head][64 dims], K as [64-dim box][cell][64 dims],
  // V as [box][cell][dims of one box]: 64 (128-byte swizzle) or, of a pair at
  // hd 64, 32 (64-byte swizzle)
  CUtensorMap tq, tk, tv;
  std::string why;
  {
    const uint64_t dims[4] = {64, static_cast<uint64_t>(Hq), static_cast<uint64_t>(total), HD / 64};
    const uint64_t st[3] = {HD * 2, static_cast<uint64_t>(Hq) * HD * 2, 128};
    const uint32_t box[4] = {64, static_cast<uint32_t>(G), static_cast<uint32_t>(C::Q_ROWS / G), 1};
    if (!encode_fp16_sw128(&tq, q, 4, dims, st, box, &why)) return cudaErrorInvalidValue;
  }
  {
    const uint64_t dims[3] = {static_cast<uint64_t>(Hkv) * HD, static_cast<uint64_t>(n_cells), HD / 64};
    const uint64_t st[2] = {static_cast<uint64_t>(Hkv) * HD * 2, 128};
    const uint32_t box[3] = {64, C::KEYS, 1};
    if (!encode_fp16_sw128(&tk, k, 3, dims, st, box, &why)) return cudaErrorInvalidValue;
    const uint32_t vbox[3] = {C::VB / 2, RCH, 1};
    if (!(C::VB == 128 ? encode_fp16_sw128(&tv, v, 3, dims, st, vbox, &why)
                       : encode_fp16_sw64(&tv, v, 3, dims, st, vbox, &why)))
      return cudaErrorInvalidValue;
  }
  int* desc = reinterpret_cast<int*>(states);
  float* part = reinterpret_cast<float*>(states + p.desc_bytes);
  e = launch_k(attn_runs_kernel<HD, CL, TREE>, dim3(CL * p.sh.pairs), dim3(C::THREADS), C::SMEM, s, CL, tq, tk, tv, p.rt,
               p.sh, mask, words, out, part, desc, err, flags);
  if (e != cudaSuccess || !p.sh.merge) return e;
  // an item lies in about pairs / items pairs: one round of loads each
  const int spread = p.sh.pairs / p.items;
  const int ways = spread <= 8 ? 1 : spread <= 16 ? 2 : spread <= 32 ? 4 : 8;
  return launch_k(attn_runs_merge_kernel<HD>,
                  dim3(std::min(p.sh.pairs, p.items), p.sh.slot_rows / 32, HD / 32 * ways), dim3(256), 0, s, 1, p.sh,
                  ways, static_cast<const int*>(desc), static_cast<const float*>(part), out);
}

}  // namespace pf

namespace {

using namespace pf;

constexpr int64_t WORK_HEADER = 4096;  // the error word; from word FLAGS_AT the pairs' flags
constexpr int FLAGS_AT = 64;
constexpr int MASK_WORDS_MAX = 4;
constexpr const char* TOO_MUCH = "more work than one call takes: 2^30 chunks of 128 keys over all blocks of MMA rows";
static_assert((FLAGS_AT + 8 * MAX_PAIRS) * 4 <= WORK_HEADER, "scratch header");

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
    if (words < 1 || words > MASK_WORDS_MAX) return fail(PF_E_ARG, "mask_words outside [1, 4]");
    for (int r = 0; r < n_runs; ++r)
      if (runs[r].n_rows > 64 * words) return fail(PF_E_ARG, "a run has more rows than its mask has bits");
  }
  if (total == 0) return PF_OK;
  if (!q || !k || !v || !out || !work || (tree && !mask)) return fail(PF_E_ARG, "null buffer");
  if (((reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15) ||
      (reinterpret_cast<uintptr_t>(out) & 31))
    return fail(PF_E_ARG, "q, k and v must be 16-byte aligned, out 32-byte aligned");
  if (tree && (reinterpret_cast<uintptr_t>(mask) & 7)) return fail(PF_E_ARG, "mask must be 8-byte aligned");
  if (reinterpret_cast<uintptr_t>(work) & 255) return fail(PF_E_ARG, "the scratch must be 256-byte aligned");
  RunsPlan p;
  if (!(tree ? make_plan<true>(p, runs, n_runs, Hq, Hkv, hd) : make_plan<false>(p, runs, n_runs, Hq, Hkv, hd)))
    return fail(PF_E_ARG, TOO_MUCH);
  if (work_bytes < WORK_HEADER + p.state_bytes) return fail(PF_E_ARG, "the scratch is smaller than these runs need");
  int* err = static_cast<int*>(work);
  uint8_t* states = static_cast<uint8_t*>(work) + WORK_HEADER;
  auto go = [&](auto launch) {
    return launch(p, static_cast<const __half*>(q), static_cast<const __half*>(k), static_cast<const __half*>(v),
                  n_cells, static_cast<int>(total), mask, words, static_cast<__nv_bfloat16*>(out), states, err, err + FLAGS_AT, s);
  };
  const cudaError_t e = hd == 256   ? (tree ? go(launch_runs<256, 2, true>) : go(launch_runs<256, 2, false>))
                        : p.cl == 2 ? (tree ? go(launch_runs<64, 2, true>) : go(launch_runs<64, 2, false>))
                                    : (tree ? go(launch_runs<64, 1, true>) : go(launch_runs<64, 1, false>));
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
  if (!make_plan<false>(a, runs, n_runs, Hq, Hkv, hd)) return fail(PF_E_ARG, TOO_MUCH);
  // a tree's rows all see the whole context: runs that no tree has are not
  // counted as one, and what only the tree call refuses it refuses itself
  bool tree = true;
  for (int r = 0; r < n_runs; ++r) tree = tree && runs[r].n_rows <= 64 * MASK_WORDS_MAX;
  const bool both = tree && make_plan<true>(b, runs, n_runs, Hq, Hkv, hd);
  return WORK_HEADER + std::max(a.state_bytes, both ? b.state_bytes : 0);
}

extern "C" int pfop_attention_status(void* work_dev, void* stream) {
  if (!work_dev) return fail(PF_E_ARG, "null scratch");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int h = 0;
  cudaError_t e = cudaMemcpyAsync(&h, work_dev, 4, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && h) {
    // flags of a call that gave up too; over before this returns, since the next call may come on any stream
    e = cudaMemsetAsync(work_dev, 0, WORK_HEADER, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  if (e != cudaSuccess) return fail(PF_E_CUDA, std::string("attention status: ") + cudaGetErrorString(e));
  if (h) return fail(PF_E_DEVICE_TIMEOUT, "attention gave up a bounded wait, code " + std::to_string(h));
  return PF_OK;
}
