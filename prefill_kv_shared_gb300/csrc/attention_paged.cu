// Attention over a paged cache (pfop_attention_paged).
//
// Chunks of prompts and drafted trees run on the kernel of attention_runs.cuh
// with its copies going through the page table.  Where no run has more MMA rows
// (rows times the heads of a KV head) than the 8 to 24 columns of a few small
// matrix products, as in plain decoding, attn_few_kernel takes the call: there
// the keys and values are the work, and 128 or 256 rows of tcgen05 would be
// mostly padding with a TMEM round trip and four hand-overs per chunk (64 rows
// over 4096 keys: 56.5 us for 45 at 8 heads over 1 of 256, 66.5 for 44 at 32
// over 4 of 64).
#include "attention_runs.cuh"

namespace pf {

// CTAs of 8 warps, of an SM.  (hd 256 with two of 4 warps: 64 tokens over 1024
// keys, 8 heads over 2, 28.2 us instead of 23.5, one over 32768 14.5 instead of
// 13.6.)
constexpr int few_ctas(int hd, int cols) { return hd == 64 && cols <= 16 ? 2 : 1; }
// Least tiles of a CTA, and how many more tiles than an even share an item may
// have for a CTA of its own (beside an eighth of the share), which saves the
// merge kernel.  `little`: work for less than half of the CTAs.  (hd 64, 32 heads
// over 4, cost of 64 and of 32: 64 tokens over 100 to 1300 keys at random 12.1 and
// 15.4 us, 32 over 1000 9.2 and 10.9, 8 over 800 5.5 and 6.1, one over 1000 5.8 and
// 6.1; one long among short ones, 1200 keys and 63 of 300 8.9 and 9.2, 32 of 400
// 7.1 and 7.9, but 1500 and 63 of 500 10.8 and 10.6; 48 is between them.
// hd 256: 16 over 1024 keys, 8 heads over 2, 11.0 with 16 tiles and 24, 12.5
// with 8; one over 500, 8 heads over 1, 5.5 with 8 and 12, 7.7 with 16 and 24.)
constexpr int few_min(bool little) { return little ? 8 : 16; }
constexpr int few_cost(int hd, bool little) { return hd == 64 ? 64 : little ? 12 : 24; }
// Most columns of a run (as many as O's registers allow at hd 256).  (hd 64, 8
// heads a KV head: 64 runs of 3 rows over 900 keys 23.7 us, 24.8 with the other
// kernel, over 4096 56.3 and 68.9; with 40 columns 64 of 5 rows over 900 30.2
// and 26.8, 16 over 2000 18.1 and 22.5.  hd 256, 8 heads over 2: 16 runs of 4
// rows over 2000 keys 19.9 and 23.4, 64 over 4096 85.7 and 105.9.)
constexpr int few_cols(int hd) { return hd == 64 ? 24 : 16; }
constexpr int FEW_ROWS = 16;  // bits that are looked at of a row's mask
constexpr int few_nt(int cols) { return (cols + 7) / 8; }
static_assert(few_cols(64) <= 24 && few_cols(256) <= 16, "the kernels that are launched");

// attn_few_kernel.  With C columns (row, head) of a run and KV head:
//     S^T = K Q^T       (m16n8k16: 16 keys by 8 columns, hd deep)
//     O^T += V^T P^T    (16 dims by 8 columns, 16 keys deep)
// The order of the contraction's dims and of the outputs' dims is free, so a
// lane takes 16 bytes at a time: of K dims 8t .. 8t+7 of every 32 for the keys
// g and g + 8 (lane = 4g + t), of V dims 8g .. 8g+7 of every 64 for the keys
// 2t, 2t+1, 2t+8, 2t+9, whose pairs two byte permutations put together.  P^T
// is S^T's layout transposed: one movmatrix for 8 keys.  K and V come by
// cp.async into the warp's own places in shared memory, whole 128-byte lines
// at a time for 8 lanes (where 8 lanes took 32 bytes of four rows, each was
// fetched twice), so no warp waits for another before the end of its keys.  (In
// registers instead, 61 us: 16 KB a warp do not fit.)
//
// The online softmax keeps a reference per column that follows the maximum by
// steps of more than 2^8 (P within fp16), so that most tiles need a vote and no
// shuffles.  Sums and O are fp32.  P is fp16, what the matrix instruction takes
// beside V: 2^-11 of a p of 2^-14 and more, 2^-25 in all below, where a key counts
// in the sum but at the end no more in O (to be seen only where one key outweighs
// all others, its v is small, and there are more than some 2^16 of them).
//
// Work: the items (run, KV head), counted in tiles of 16 keys, lie end to end
// and every CTA takes the same number of tiles; or a CTA takes an item where
// that is about as even.  A CTA's warps share a segment (its tiles of an item)
// and join their states in shared memory; the states of cut items are joined
// by attn_few_merge_kernel.
//
// Bound by HBM for long contexts (64 sequences over 16384 keys: 6.8 TB/s for 8
// heads over 1 of 256, 6.4 for 32 over 4 of 64; over 4096 45 and 44 us, 6.0
// and 6.1 TB/s), by the chain launch, page ids, first keys, states for short
// ones (64 sequences over 500 to 1319 keys, 32 heads over 4 of 64, 60 MB: 13.1
// us; one over 32768, 8 heads over 1 of 256: 12.3; one over 532: 4.3).
struct FewRun {
  int row0, n, pos0, entry0;
};
struct FewTable {
  FewRun run[RUNS_MAX];
  int at[RUNS_MAX + 1];  // tiles before the run's items
  int n_runs = 0;
};
struct FewShape {
  int Hq, Hkv, log_g;
  int share;  // tiles of a CTA; 0: an item each
};

template <int HD, int NT>
struct FewCfg {
  static constexpr int WARPS = 8, CTAS = few_ctas(HD, 8 * NT);
  static constexpr int COLS = 8 * NT;
  static constexpr int UNIT = HD * 32;                 // bytes of a tile's K or V
  static constexpr int SLOTS = 196608 / CTAS / (WARPS * UNIT);  // units that a warp has place for
  static constexpr int STATE_SLOTS = COLS * HD * 4 / UNIT;  // the last ones hold its O at a segment's end
  static constexpr int OFF_Q = WARPS * SLOTS * UNIT;
  static constexpr int OFF_ML = OFF_Q + HD / 32 * NT * 512;
  static constexpr int SMEM = OFF_ML + WARPS * COLS * 8;
  // a state in the scratch: (m, l) of every column, then O
  static constexpr int STATE = COLS * (HD + 2);
  static_assert(STATE_SLOTS < SLOTS && SMEM <= 232448 / CTAS - 1024, "shared memory");
};

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 16 bytes from global to shared memory; is false: zeros, and p is not read
__device__ __forceinline__ void copy_16(uint32_t dst, const void* p, bool is) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(p), "r"(is ? 16 : 0) : "memory");
}
__device__ __forceinline__ uint32_t transposed_8x8(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

// an item: run, KV head, and its place on the line of tiles
struct FewItem {
  FewRun run;
  int at, tiles;
  __device__ FewItem(const FewTable& ft, int i, int kvh) : run(ft.run[i]) {
    tiles = (run.pos0 + run.n + 15) >> 4;
    at = ft.at[i] + kvh * tiles;
  }
};

template <int HD, int NT>
__global__ void __launch_bounds__(32 * FewCfg<HD, NT>::WARPS, FewCfg<HD, NT>::CTAS)
    attn_few_kernel(const __grid_constant__ FewTable ft, const FewShape sh, const __half* __restrict__ q,
                    const __half* __restrict__ k, const __half* __restrict__ v, const RunPages pg,
                    const uint64_t* __restrict__ mask, int words, __nv_bfloat16* __restrict__ out, float* __restrict__ part) {
  using C = FewCfg<HD, NT>;
  constexpr float cexp = attn_c<HD>();
  constexpr int KC = HD / 32, VC = HD / 64;  // 16-byte pieces of a K row per lane, of a V row
  extern __shared__ __align__(16) uint8_t smem[];
  uint4(*sq)[NT][32] = reinterpret_cast<uint4(*)[NT][32]>(smem + C::OFF_Q);  // Q as the B operand of two steps of 16 dims
  float2(*sml)[C::COLS] = reinterpret_cast<float2(*)[C::COLS]>(smem + C::OFF_ML);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * (C::SLOTS * C::UNIT);
  const uint32_t ring_at = smem_u32(ring);
  // O of warp w: column by column, the pairs of every 8 dims in an order of the column's
  auto state_of = [&](int w, int col, int pair) {
    float* o = reinterpret_cast<float*>(smem + (w + 1) * (C::SLOTS * C::UNIT) - C::STATE_SLOTS * C::UNIT);
    return reinterpret_cast<float2*>(o + col * HD + 2 * (pair ^ (col >> 1 & 3)));
  };
  pdl_launch();
  // the CTA's share of the line, and its first item
  int pos, end, run, kvh;
  if (sh.share == 0) {
    int item = static_cast<int>(blockIdx.x);
    run = item / sh.Hkv;
    kvh = item - run * sh.Hkv;
    const FewItem it(ft, run, kvh);
    pos = it.at, end = it.at + it.tiles;
  } else {
    pos = static_cast<int>(blockIdx.x) * sh.share;
    end = min(pos + sh.share, ft.at[ft.n_runs]);
    run = find_last(ft.at, ft.n_runs, pos);
    kvh = (pos - ft.at[run]) / FewItem(ft, run, 0).tiles;
  }
  pdl_wait();

  while (pos < end) {
    const FewItem it(ft, run, kvh);
    const int n_rows = it.run.n, pos0 = it.run.pos0, row0 = it.run.row0, keys = pos0 + n_rows;
    const int tile0 = pos - it.at, tile1 = min(it.tiles, end - it.at);
    const int cols = n_rows << sh.log_g;
    // the warp's tiles
    const int per = (tile1 - tile0 + C::WARPS - 1) / C::WARPS;
    const int w0 = tile0 + warp * per, w1 = min(tile1, w0 + per);

    // Cells of groups of 8 keys: lane i holds that of the i-th from the
    // group's first tile on; -1: no keys, or no page.
    auto fetch_id = [&](int tile) {
      const int key = (tile << 4) + (lane << 3);
      return key < keys && key < w1 << 4 ? __ldcg(pg.table + it.run.entry0 + (key >> pg.page_log)) : -1;
    };
    auto cells_of = [&](int id, int tile) {
      const int key = (tile << 4) + (lane << 3);
      if (!(key < keys && key < w1 << 4)) return -1;
      if (static_cast<unsigned>(id) >= static_cast<unsigned>(pg.n_pages)) {
        atomicAdd(pg.bad, 1);
        return -1;
      }
      return (id << pg.page_log) + (key & ((1 << pg.page_log) - 1));
    };
    const int64_t ld = static_cast<int64_t>(sh.Hkv) * HD;
    const __half* kh = k + kvh * HD + 8 * (lane & 7) + (lane >> 3) * ld;
    const __half* vh = v + kvh * HD + 8 * (lane & 7) + (lane >> 3) * ld;
    int cells = -1, next_id = -1;
    // unit u: K (even) or V of tile w0 + u / 2, into place u % SLOTS; one group of copies each
    const int units = 2 * max(0, w1 - w0);
    int sent = 0, to = 0;  // units sent, the next one's place
    auto send = [&]() {
      if (sent < units) {
        const int rel = sent >> 1, tile = w0 + rel;
        if (sent == 0) {
          cells = cells_of(fetch_id(w0), w0);
          next_id = fetch_id(w0 + 16);
        } else if ((sent & 31) == 0) {
          cells = cells_of(next_id, tile);
          next_id = fetch_id(tile + 16);
        }
        const uint32_t dst = ring_at + to * C::UNIT;
        const int c0 = __shfl_sync(0xffffffffu, cells, (2 * rel) & 31), c1 = __shfl_sync(0xffffffffu, cells, (2 * rel + 1) & 31);
        // 16-byte pieces of a row, exchanged within every 128 bytes so that the reads meet no bank conflicts
        const bool is_v = sent & 1;
        const __half* kv = is_v ? vh : kh;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int cell = i & 2 ? c1 : c0, row = 4 * i + (lane >> 3);
          const __half* p = kv + (max(cell, 0) + 4 * (i & 1)) * ld;
          const uint32_t to_row = dst + row * (HD * 2) + ((lane & 7) ^ (is_v ? row & 6 : (row & 1) << 2)) * 16;
          // (V behind the run's end: what lies there may be no number)
          const bool is = cell >= 0 && (!is_v || (tile << 4) + row < keys);
#pragma unroll
          for (int c = 0; c < HD / 64; ++c) copy_16(to_row + c * 128, p + 64 * c, is);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      ++sent;
      to = to + 1 == C::SLOTS ? 0 : to + 1;
    };
    // the oldest unit on its way has landed
    auto landed = [&]() {
      asm volatile("cp.async.wait_group %0;" ::"n"(C::SLOTS - 1) : "memory");
      __syncwarp();
    };
    // Q, asked for before the page ids and the first keys
    constexpr int QV = (KC * NT + C::WARPS - 1) / C::WARPS;
    uint4 qv[QV];
#pragma unroll
    for (int j = 0; j < QV; ++j) {
      const int i = tid + j * 32 * C::WARPS, l = i & 31, col = 8 * ((i >> 5) % NT) + (l >> 2), c = i / (32 * NT);
      qv[j] = make_uint4(0u, 0u, 0u, 0u);
      if (i < KC * NT * 32 && col < cols)
        qv[j] = __ldcg(reinterpret_cast<const uint4*>(
            q + (static_cast<int64_t>(row0 + (col >> sh.log_g)) * sh.Hq + (kvh << sh.log_g) + (col & ((1 << sh.log_g) - 1))) * HD +
            32 * c + 8 * (l & 3)));
    }
    for (int i = 0; i < C::SLOTS; ++i) send();
#pragma unroll
    for (int j = 0; j < QV; ++j) {
      const int i = tid + j * 32 * C::WARPS;
      if (i < KC * NT * 32) sq[i / (32 * NT)][(i >> 5) % NT][i & 31] = qv[j];
    }
    // which of the run's own tokens the lane's columns see
    uint32_t seen[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = (8 * nt + 2 * t + e) >> sh.log_g;
        seen[nt][e] = 0u;
        if (row < n_rows) {
          const uint32_t all = (1u << n_rows) - 1u;  // (at most 16 rows)
          seen[nt][e] = mask ? static_cast<uint32_t>(mask[static_cast<int64_t>(row0 + row) * words]) & all : (2u << row) - 1u;
        }
      }
    __syncthreads();
    float o[VC][4][NT][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) m[nt][e] = -INFINITY, l[nt][e] = 0.f;
#pragma unroll
      for (int c = 0; c < VC; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[c][j][nt][e] = 0.f;
    }
    int from = 0;  // the next unit's place
#pragma unroll 1
    for (int tile = w0; tile < w1; ++tile) {
      float s[2][NT][4];  // two sums, over half of the dims each
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[i][nt][e] = 0.f;
      landed();
      const uint8_t* kr = ring + from * C::UNIT + g * (HD * 2);
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const int at = ((4 * c + t) ^ ((g & 1) << 2)) * 16;
        const uint4 k0 = *reinterpret_cast<const uint4*>(kr + at), k1 = *reinterpret_cast<const uint4*>(kr + 8 * HD * 2 + at);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint4 b = sq[c][nt][lane];
          mma_16816(s[0][nt], k0.x, k1.x, k0.y, k1.y, b.x, b.y);
          mma_16816(s[1][nt], k0.z, k1.z, k0.w, k1.w, b.z, b.w);
        }
      }
      from = from + 1 == C::SLOTS ? 0 : from + 1;
      __syncwarp();
      send();
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[0][nt][e] += s[1][nt][e];
      if (((tile + 1) << 4) > pos0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int d = (tile << 4) + g + 8 * (e >> 1) - pos0;
            if (d >= 0 && (d >= 32 || !(seen[nt][e & 1] >> d & 1u))) s[0][nt][e] = -INFINITY;
          }
      }
      bool grow = false;
      float mx[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mx[nt][e] = fmaxf(s[0][nt][e], s[0][nt][e + 2]);
          grow = grow || (mx[nt][e] - m[nt][e]) * cexp > 8.f;
        }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float scale[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float x = mx[nt][e];
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, w));
            scale[e] = 1.f;
            if ((x - m[nt][e]) * cexp > 8.f) {
              scale[e] = ex2_approx((m[nt][e] - x) * cexp);  // (from -inf: 0)
              m[nt][e] = x;
            }
            l[nt][e] *= scale[e];
          }
#pragma unroll
          for (int c = 0; c < VC; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
              for (int e = 0; e < 4; ++e) o[c][j][nt][e] *= scale[e & 1];
        }
      }
      uint32_t b[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float r[2] = {m[nt][0] == -INFINITY ? 0.f : m[nt][0], m[nt][1] == -INFINITY ? 0.f : m[nt][1]};
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] = ex2_approx((s[0][nt][e] - r[e & 1]) * cexp);
          l[nt][e & 1] += p[e];
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const __half2 x = __floats2half2_rn(p[2 * h], p[2 * h + 1]);
          b[nt][h] = transposed_8x8(*reinterpret_cast<const uint32_t*>(&x));
        }
      }
      landed();
      const uint8_t* vr = ring + from * C::UNIT + 2 * t * (HD * 2) + (g ^ 2 * t) * 16;  // (6 of a row's number: 2t)
#pragma unroll
      for (int c = 0; c < VC; ++c) {
        uint32_t x[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 y = *reinterpret_cast<const uint4*>(vr + ((i & 1) + (i & 2) * 4) * (HD * 2) + c * 128);
          x[i][0] = y.x, x[i][1] = y.y, x[i][2] = y.z, x[i][3] = y.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a0 = __byte_perm(x[0][j], x[1][j], 0x5410), a1 = __byte_perm(x[0][j], x[1][j], 0x7632);
          const uint32_t a2 = __byte_perm(x[2][j], x[3][j], 0x5410), a3 = __byte_perm(x[2][j], x[3][j], 0x7632);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) mma_16816(o[c][j][nt], a0, a1, a2, a3, b[nt][0], b[nt][1]);
        }
      }
      from = from + 1 == C::SLOTS ? 0 : from + 1;
      __syncwarp();
      send();
    }
    // the warp's state, where its last units were
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], w);
        const int col = 8 * nt + 2 * t + e;
        if (g == 0) sml[warp][col] = make_float2(m[nt][e], l[nt][e]);
#pragma unroll
        for (int c = 0; c < VC; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *state_of(warp, col, 32 * c + 4 * g + j) = make_float2(o[c][j][nt][e], o[c][j][nt][e + 2]);
      }
    __syncthreads();
    // the CTA's: a warp a column
    const bool whole = tile1 - tile0 == it.tiles;
    float* state = part + static_cast<int64_t>(2 * blockIdx.x + (tile0 == 0 ? 1 : 0)) * C::STATE;
    for (int col = warp; col < cols; col += C::WARPS) {
      float mm = -INFINITY, ll = 0.f, w[C::WARPS];
#pragma unroll
      for (int i = 0; i < C::WARPS; ++i) mm = fmaxf(mm, sml[i][col].x);
#pragma unroll
      for (int i = 0; i < C::WARPS; ++i) {
        const float2 x = sml[i][col];
        w[i] = x.x == -INFINITY ? 0.f : ex2_approx((x.x - mm) * cexp);
        ll = __fmaf_rn(w[i], x.y, ll);
      }
      // the lane's dims: pairs, 64 apart
      float2 acc[VC];
#pragma unroll
      for (int c = 0; c < VC; ++c) acc[c] = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < C::WARPS; ++i)
#pragma unroll
        for (int c = 0; c < VC; ++c) {
          const float2 x = *state_of(i, col, 32 * c + lane);
          acc[c].x = __fmaf_rn(w[i], x.x, acc[c].x);
          acc[c].y = __fmaf_rn(w[i], x.y, acc[c].y);
        }
      if (whole) {
        const float inv = ll == 0.f ? 0.f : __frcp_rn(ll);  // a row that sees nothing: zeros
        __nv_bfloat162* dst = reinterpret_cast<__nv_bfloat162*>(
            out + (static_cast<int64_t>(row0 + (col >> sh.log_g)) * sh.Hq + (kvh << sh.log_g) + (col & ((1 << sh.log_g) - 1))) * HD);
#pragma unroll
        for (int c = 0; c < VC; ++c) dst[32 * c + lane] = __floats2bfloat162_rn(acc[c].x * inv, acc[c].y * inv);
      } else {
        if (lane == 0) reinterpret_cast<float2*>(state)[col] = make_float2(mm, ll);
        float2* dst = reinterpret_cast<float2*>(state + 2 * C::COLS + col * HD);
#pragma unroll
        for (int c = 0; c < VC; ++c) dst[32 * c + lane] = acc[c];
      }
    }
    // on to the next item
    pos = it.at + tile1;
    if (tile1 == it.tiles && ++kvh == sh.Hkv) kvh = 0, ++run;
    __syncthreads();
  }
}

// Cut items: blockIdx.x counts items; `ways` warps take 64 dims of a column, the
// states of the CTAs that the item lies in dealt out among them, in order, and
// their sums joined in warp order.  Bound by the latency of the states' reads
// from L2, a round of FLY a warp.
constexpr int FEW_MERGE_WARPS = 16;
template <int HD, int NT>
__global__ void __launch_bounds__(32 * FEW_MERGE_WARPS)
    attn_few_merge_kernel(const __grid_constant__ FewTable ft, const FewShape sh, int ways, const float* __restrict__ part,
                          __nv_bfloat16* __restrict__ out) {
  using C = FewCfg<HD, NT>;
  constexpr float c = attn_c<HD>();
  constexpr int FLY = 8, PARTS = HD / 64;
  __shared__ float2 sml[FEW_MERGE_WARPS];
  __shared__ float2 so[FEW_MERGE_WARPS][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = warp & (ways - 1);
  const int unit = (static_cast<int>(blockIdx.y) * FEW_MERGE_WARPS + warp) / ways, col = unit / PARTS, dims = unit % PARTS * 64;
  const int run = static_cast<int>(blockIdx.x) / sh.Hkv, kvh = static_cast<int>(blockIdx.x) - run * sh.Hkv;
  const FewItem it(ft, run, kvh);
  const int p0 = it.at / sh.share, p1 = (it.at + it.tiles - 1) / sh.share;
  pdl_launch();
  pdl_wait();
  if (p0 == p1) return;
  const bool real = col < it.run.n << sh.log_g;
  float m = -INFINITY, l = 0.f;
  float2 acc = make_float2(0.f, 0.f);
  for (int p = p0 + sub; real && p <= p1; p += ways * FLY) {
    float2 ml[FLY], x[FLY];
#pragma unroll
    for (int i = 0; i < FLY; ++i) {
      const int pp = p + ways * i;
      ml[i] = make_float2(-INFINITY, 0.f);
      x[i] = make_float2(0.f, 0.f);
      if (pp <= p1) {
        const float* s = part + static_cast<int64_t>(2 * pp + (pp == p0 ? 1 : 0)) * C::STATE;
        ml[i] = __ldcg(reinterpret_cast<const float2*>(s) + col);
        x[i] = __ldcg(reinterpret_cast<const float2*>(s + 2 * C::COLS + col * HD + dims) + lane);
      }
    }
    float mn = m;
#pragma unroll
    for (int i = 0; i < FLY; ++i) mn = fmaxf(mn, ml[i].x);
    if (mn == -INFINITY) {  // nothing seen, or no numbers: their sum is NaN and stays it
#pragma unroll
      for (int i = 0; i < FLY; ++i) l += ml[i].y;
      continue;
    }
    const float w = m == -INFINITY ? 0.f : ex2_approx((m - mn) * c);
    l *= w;
    acc.x *= w, acc.y *= w;
    m = mn;
#pragma unroll
    for (int i = 0; i < FLY; ++i) {
      const float wi = ml[i].x == -INFINITY ? 0.f : ex2_approx((ml[i].x - m) * c);
      l = __fmaf_rn(wi, ml[i].y, l);
      acc.x = __fmaf_rn(wi, x[i].x, acc.x);
      acc.y = __fmaf_rn(wi, x[i].y, acc.y);
    }
  }
  if (ways > 1) {
    if (lane == 0) sml[warp] = make_float2(m, l);
    so[warp][lane] = acc;
    __syncthreads();
    if (sub != 0) return;
    float mm = m;
    for (int i = 1; i < ways; ++i) mm = fmaxf(mm, sml[warp + i].x);
    const float w = m == -INFINITY ? 0.f : ex2_approx((m - mm) * c);
    l *= w;
    acc.x *= w, acc.y *= w;
    for (int i = 1; i < ways; ++i) {
      const float2 ml = sml[warp + i], x = so[warp + i][lane];
      const float wi = ml.x == -INFINITY ? 0.f : ex2_approx((ml.x - mm) * c);
      l = __fmaf_rn(wi, ml.y, l);
      acc.x = __fmaf_rn(wi, x.x, acc.x);
      acc.y = __fmaf_rn(wi, x.y, acc.y);
    }
  }
  if (!real) return;
  const float inv = l == 0.f ? 0.f : __frcp_rn(l);
  __nv_bfloat16* dst = out + (static_cast<int64_t>(it.run.row0 + (col >> sh.log_g)) * sh.Hq + (kvh << sh.log_g) +
                              (col & ((1 << sh.log_g) - 1))) * HD + dims;
  reinterpret_cast<__nv_bfloat162*>(dst)[lane] = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
}

// ---------------------------------------------------------------------------
// host: the cut of a call of few rows a run

struct FewPlan {
  FewTable ft;
  FewShape sh;
  int ctas = 0, cols = 0;  // cols: of the longest run
  int ways = 1;            // of the merge kernel
  bool merge = false;
  int64_t state_bytes = 0;
};

// Which calls: no run of more columns than the kernel takes, and so few tiles
// that they can be counted.  One longer run takes the whole call to the other
// kernel: the two kernels one after the other leave SMs idle twice, which costs
// more unless the tokens are most of the work.  (Together and apart, us: 8 heads
// over 2 of 256, 512 rows behind 3584 with 13 tokens over 1000 keys 33.9 and
// 40.1, 64 behind 500 with 16 over 1000 19.4 and 27.1, 2048 with 63 over 2000 72.9
// and 76.1, but 64 rows with 64 tokens over 4096 105.3 and 92.8; 32 heads over 4 of
// 64, 64 behind 500 with 16 over 1000 12.0 and 17.2, but 2048 with 63 over 2000 81.0
// and 70.8, 64 with 64 over 4096 69.0 and 50.5.  A program with such a batch makes
// two calls.)
static bool few_plan(FewPlan& p, const pfop_attn_run* runs, int n_runs, int Hq, int Hkv, int hd) {
  const int group = Hq / Hkv, most = std::min(FEW_ROWS, few_cols(hd) / group);
  p.sh.Hq = Hq, p.sh.Hkv = Hkv, p.sh.log_g = 0;
  while ((1 << p.sh.log_g) < group) ++p.sh.log_g;
  int64_t tiles = 0, longest = 0;
  int row = 0, n = 0;
  for (int r = 0; r < n_runs; ++r) {
    if (runs[r].n_rows > 0) {
      if (runs[r].n_rows > most) return false;
      const int64_t t = (static_cast<int64_t>(runs[r].pos0) + runs[r].n_rows + 15) / 16;
      p.ft.run[n] = FewRun{row, runs[r].n_rows, runs[r].pos0, runs[r].cell0};
      p.ft.at[n] = static_cast<int>(tiles);
      p.cols = std::max(p.cols, runs[r].n_rows * group);
      ++n;
      tiles += t * Hkv;
      longest = std::max(longest, t);
      if (tiles >= int64_t(1) << 30) return false;
    }
    row += runs[r].n_rows;
  }
  if (n == 0) return false;
  p.ft.n_runs = n;
  p.ft.at[n] = static_cast<int>(tiles);
  const int nt = few_nt(p.cols);
  const int64_t slots = int64_t(sm_count()) * few_ctas(hd, p.cols), items = int64_t(n) * Hkv;
  const bool little = 2 * tiles < few_min(false) * slots;
  const int64_t share = std::max<int64_t>(few_min(little), (tiles + slots - 1) / slots);
  if (longest <= share + share / 8 + few_cost(hd, little) && items <= slots) {
    p.sh.share = 0;
    p.ctas = static_cast<int>(items);
  } else {
    p.sh.share = static_cast<int>(share);
    p.ctas = static_cast<int>((tiles + share - 1) / share);
    p.merge = true;
    // a warp for every eight states of the longest item
    while (p.ways < FEW_MERGE_WARPS && longest / share + 2 > 8 * p.ways) p.ways *= 2;
    p.state_bytes = int64_t(2) * p.ctas * (8 * nt) * (hd + 2) * static_cast<int64_t>(sizeof(float));
  }
  return true;
}

template <int HD, int NT>
static cudaError_t launch_few(const FewPlan& p, const __half* q, const __half* k, const __half* v, const RunPages& pages,
                              const uint64_t* mask, int words, __nv_bfloat16* out, float* part, cudaStream_t s) {
  using C = FewCfg<HD, NT>;
  cudaError_t e = smem_opt_in<attn_few_kernel<HD, NT>>(C::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_k(attn_few_kernel<HD, NT>, dim3(p.ctas), dim3(32 * C::WARPS), C::SMEM, s, 1, p.ft, p.sh, q, k, v, pages,
                           mask, words, out, part);
  if (e != cudaSuccess || !p.merge) return e;
  const int units = FEW_MERGE_WARPS / p.ways;
  return launch_k(attn_few_merge_kernel<HD, NT>, dim3(p.ft.n_runs * p.sh.Hkv, (p.cols * (HD / 64) + units - 1) / units),
                  dim3(32 * FEW_MERGE_WARPS), 0, s, 1, p.ft, p.sh, p.ways, static_cast<const float*>(part), out);
}

}  // namespace pf

namespace {

using namespace pf;

int pages_log(int page_size) {
  int l = 0;
  while ((1 << l) < page_size && l < 30) ++l;
  return l;
}

// What the call and the size query share.  (page ids are device data: the
// kernel looks at them)
int check_paged(int Hq, int Hkv, int hd, const pfop_attn_run* runs, int n_runs, bool tree, int words, int64_t* total) {
  const int rc = check_runs(Hq, Hkv, hd, runs, n_runs, -1, total);
  if (rc != PF_OK) return rc;
  if (tree) {
    if (words < 1 || words > MASK_WORDS_MAX) return runs_fail(PF_E_ARG, "mask_words outside [1, 4]");
    for (int r = 0; r < n_runs; ++r)
      if (runs[r].n_rows > 64 * words) return runs_fail(PF_E_ARG, "a run has more rows than its mask has bits");
  }
  return PF_OK;
}

}  // namespace

extern "C" int pfop_attention_paged(const void* q_dev, const void* k_dev, const void* v_dev, int32_t n_pages,
                                    int32_t page_size, int32_t Hq, int32_t Hkv, int32_t hd, const pfop_attn_run* runs,
                                    int32_t n_runs, const int32_t* table_dev, int64_t n_entries,
                                    const uint64_t* mask_dev, int32_t mask_words, void* out_dev, void* work_dev,
                                    int64_t work_bytes, void* stream) {
  if (page_size < 8 || (page_size & (page_size - 1)) != 0)
    return runs_fail(PF_E_ARG, "page_size must be a power of two, at least 8");
  if (n_pages < 0 || int64_t(n_pages) * page_size > (int64_t(1) << 31) - 1024)
    return runs_fail(PF_E_ARG, "n_pages negative or more than 2^31 - 1024 cells");
  const bool tree = mask_dev != nullptr;
  int64_t total = 0;
  const int rc = check_paged(Hq, Hkv, hd, runs, n_runs, tree, mask_words, &total);
  if (rc != PF_OK) return rc;
  const int page_log = pages_log(page_size);
  for (int r = 0; r < n_runs; ++r) {
    const int64_t end = static_cast<int64_t>(runs[r].pos0) + runs[r].n_rows;
    // (the kernels count entries in 32 bits)
    if (runs[r].n_rows > 0 && runs[r].cell0 + ((end + page_size - 1) >> page_log) > std::min<int64_t>(n_entries, INT32_MAX))
      return runs_fail(PF_E_ARG, "a run past the table's entries");
  }
  if (total == 0) return PF_OK;
  if (!q_dev || !k_dev || !v_dev || !table_dev || !out_dev || !work_dev || n_pages == 0)
    return runs_fail(PF_E_ARG, "null buffer, or no pages");
  if (((reinterpret_cast<uintptr_t>(q_dev) | reinterpret_cast<uintptr_t>(k_dev) | reinterpret_cast<uintptr_t>(v_dev)) & 15) ||
      (reinterpret_cast<uintptr_t>(out_dev) & 31))
    return runs_fail(PF_E_ARG, "q, k and v must be 16-byte aligned, out 32-byte aligned");
  if ((reinterpret_cast<uintptr_t>(mask_dev) & 7) || (reinterpret_cast<uintptr_t>(table_dev) & 3))
    return runs_fail(PF_E_ARG, "mask must be 8-byte aligned, the table 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(work_dev) & 255) return runs_fail(PF_E_ARG, "the scratch must be 256-byte aligned");
  int* err = static_cast<int*>(work_dev);
  const int64_t n_cells = int64_t(n_pages) << page_log;
  const RunPages pages{table_dev, n_pages, page_log, static_cast<int>(n_cells), err + BAD_PAGE_AT};
  FewPlan few;
  if (few_plan(few, runs, n_runs, Hq, Hkv, hd)) {
    if (work_bytes < WORK_HEADER + few.state_bytes) return runs_fail(PF_E_ARG, "the scratch is smaller than these runs need");
    auto go = [&](auto launch) {
      return launch(few, static_cast<const __half*>(q_dev), static_cast<const __half*>(k_dev),
                    static_cast<const __half*>(v_dev), pages, mask_dev, mask_words, static_cast<__nv_bfloat16*>(out_dev),
                    reinterpret_cast<float*>(static_cast<uint8_t*>(work_dev) + WORK_HEADER), static_cast<cudaStream_t>(stream));
    };
    const int nt = few_nt(few.cols);
    const cudaError_t e = hd == 256 ? (nt == 2 ? go(launch_few<256, 2>) : go(launch_few<256, 1>))
                          : nt == 1 ? go(launch_few<64, 1>)
                          : nt == 2 ? go(launch_few<64, 2>)
                                    : go(launch_few<64, 3>);
    if (e != cudaSuccess) return runs_fail(PF_E_CUDA, std::string("paged attention launch: ") + cudaGetErrorString(e));
    return PF_OK;
  }
  RunsPlan p;
  if (!(tree ? make_plan<true>(p, runs, n_runs, Hq, Hkv, hd) : make_plan<false>(p, runs, n_runs, Hq, Hkv, hd)))
    return runs_fail(PF_E_ARG, TOO_MUCH);
  if (work_bytes < WORK_HEADER + p.state_bytes) return runs_fail(PF_E_ARG, "the scratch is smaller than these runs need");
  auto go = [&](auto launch) {
    return launch(p, static_cast<const __half*>(q_dev), static_cast<const __half*>(k_dev),
                  static_cast<const __half*>(v_dev), n_cells, static_cast<int>(total), mask_dev, mask_words,
                  static_cast<__nv_bfloat16*>(out_dev), static_cast<uint8_t*>(work_dev) + WORK_HEADER, err,
                  err + FLAGS_AT, pages, static_cast<cudaStream_t>(stream));
  };
  const cudaError_t e = hd == 256 ? (tree ? go(launch_runs<256, 2, true, RunPages>) : go(launch_runs<256, 2, false, RunPages>))
                        : p.cl == 2 ? (tree ? go(launch_runs<64, 2, true, RunPages>) : go(launch_runs<64, 2, false, RunPages>))
                                    : (tree ? go(launch_runs<64, 1, true, RunPages>) : go(launch_runs<64, 1, false, RunPages>));
  if (e != cudaSuccess) return runs_fail(PF_E_CUDA, std::string("paged attention launch: ") + cudaGetErrorString(e));
  return PF_OK;
}

extern "C" int64_t pfop_attention_paged_work_bytes(int32_t Hq, int32_t Hkv, int32_t hd, const pfop_attn_run* runs,
                                                   int32_t n_runs) {
  const int64_t need = pfop_attention_work_bytes(Hq, Hkv, hd, runs, n_runs);
  FewPlan few;
  if (need < 0 || !few_plan(few, runs, n_runs, Hq, Hkv, hd)) return need;
  return std::max(need, WORK_HEADER + few.state_bytes);
}

extern "C" int pfop_attention_paged_status(void* work_dev, void* stream) {
  if (!work_dev) return runs_fail(PF_E_ARG, "null scratch");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int h[2] = {0, 0};
  static_assert(BAD_PAGE_AT == 1, "one copy brings both words");
  cudaError_t e = cudaMemcpyAsync(h, work_dev, sizeof(h), cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  if (e == cudaSuccess && (h[0] || h[1])) {
    // over before this returns, since the next call may come on any stream
    e = cudaMemsetAsync(work_dev, 0, WORK_HEADER, s);
    if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  }
  if (e != cudaSuccess) return runs_fail(PF_E_CUDA, std::string("attention status: ") + cudaGetErrorString(e));
  if (h[0]) return runs_fail(PF_E_DEVICE_TIMEOUT, "attention gave up a bounded wait, code " + std::to_string(h[0]));
  if (h[1]) return runs_fail(PF_E_ARG, "a page id outside the cache");
  return PF_OK;
}
