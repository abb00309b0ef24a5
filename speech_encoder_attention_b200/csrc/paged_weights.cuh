// paged_weights.cuh -- the attention weight that a chunk's query rows put on
// each slot of a paged cache, summed over rows and query heads:
//
//   w_out[b, j] = w_in[b, j] + sum_{i, h : j in A_i} e^{s_ij - lse_ih}.
//
// With few query rows bound by reading K; with many, by one exponential per
// (row, head, slot). A CTA owns 128 slots of one sequence and computes
// S^T = K Q^T on tcgen05 tiles: 128 slots x N rows, N = 16 or 32 for a step or
// a drafted block, 128 for a longer chunk (20 heads, us: a step over 1500 slots of
// five sequences 8.2 with 16, 8.6 with 32; 24 rows of those 8.9 with 32, 18.3 with
// 128). A slot is a tensor-memory lane, so its
// weights are summed by one thread, in a fixed order, with no shuffles; the
// normaliser of a row is a column's constant that every thread reads from
// shared memory.
//   warps 0-3  one thread per slot: e^{s - lse} and the sums. N = 128 has two such
//              groups, 64 columns each: four warps per scheduler keep the
//              exponential unit busier than two.
//   then       a producer warp: K tiles (one TMA copy per page, the table is read once
//              per key tile), Q tiles and their normalisers.
//   last       a tcgen05.mma issuer, into two S buffers in turn.
// An item is one S^T tile: (key tile, K/V head, query tile). The items of all
// key tiles that some row sees lie in one line, in that order, cut into equal
// shares, one per resident CTA, so prompts (whose first slots more rows see) and
// ragged batches come out even. A key tile whose items fall into several shares
// leaves partial sums in the workspace, which paged_weights_merge_kernel adds in
// the order of the line. Where there are few key tiles with few items each, a
// cluster of up to 8 CTAs takes one key tile, rank 0 adds the sums through
// distributed shared memory, and there is no second launch and no workspace.
//
// Measured on a B200, 20 heads: one token of each of 16 sequences of 3.1 to 8.2
// thousand slots 52 us = 4.6 TB/s (the loads run at 6.5 TB/s; 10 us are launch,
// the first tile's latency and the merge), 4 causal prompts of 1500 tokens 52 us
// at 55 % of the exponential rate (64 scores per thread, of which 216 bytes are
// spilled at 96 registers).
#pragma once

#include <cfloat>

#include "flash_attn.cuh"
#include "paged_common.cuh"

namespace sea {
namespace pg {

struct WeightParams {
  Geo g;               // tok_per_tile: tokens of a query tile of at most N rows
  const float* lse;    // [batch * t_q, n_heads]
  const float* w_in;   // [batch, cap] or null (zeros)
  float* w_out;        // [batch, cap]
  float scale_log2;
  fa::DivC dv_group;
  int tiles;           // key tiles per sequence, by the table's size
  int cluster;         // 0: shares of the line; else so many CTAs, a cluster, per key tile
  float* ws_sum;       // [CTAs][2][128] sums of cut key tiles: one begun earlier, one that goes on
  int* ws_state;       // [CTAs][2]: the entry of the one that goes on (-1: none), and in how many
                       // more shares
  uint32_t* err;
  uint64_t limit_ns;
};

template <int N_>
struct WeightCfg {
  static constexpr int N = N_;
  static constexpr int SPLIT = N == 128 ? 2 : 1;  // column halves, each with its own four warps
  static constexpr int NC = N / SPLIT;            // columns of a thread
  static constexpr int WARPS = 4 * SPLIT;
  static constexpr int THREADS = 32 * (WARPS + 2);
  // Four CTAs per SM hide each other's waits; a third K stage fits them beside 16
  // rows only (32 rows of 16 x 8000 slots, us: three CTAs of three stages 68, of
  // four stages 66, four of two 65).
  static constexpr int K_STAGES = N == 16 ? 3 : 2;
  static constexpr int Q_STAGES = 3;
  static constexpr int CTAS_PER_SM = N == 128 ? 2 : 4;
  static constexpr int Q_BYTES = N * DH * 2;
  static constexpr uint32_t TMEM_COLS = 2 * N;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_Q = OFF_K + K_STAGES * TILE_BYTES;
  static constexpr int OFF_LSE = OFF_Q + Q_STAGES * Q_BYTES;  // [Q_STAGES][N] -normaliser, log2 units
  static constexpr int OFF_BARS = OFF_LSE + Q_STAGES * N * 4;
  // k_full[K], k_empty[K], q_full[Q], q_empty[Q], s_full[2], s_free[2], drain, half_full, half_empty
  static constexpr int NUM_BARS = 2 * K_STAGES + 2 * Q_STAGES + 7;
  static constexpr int OFF_SCAN = OFF_BARS + 8 * NUM_BARS;  // long long [10], then what locate() found
  static constexpr int OFF_HALF = OFF_SCAN + 8 * 10 + 32;   // [128] the second half's sums
  static constexpr int OFF_MISC = OFF_HALF + (SPLIT == 2 ? BKV * 4 : 0);
  static constexpr int SMEM_BYTES = 1024 + OFF_MISC + 16;
  static_assert(CTAS_PER_SM * (SMEM_BYTES + 1024) <= 228 * 1024, "the CTAs of an SM do not fit it together");
};

template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 64) {
    tmem_ld64(taddr, r);
  } else if constexpr (N == 32) {
    tmem_ld32(taddr, r);
  } else {
    static_assert(N == 16, "");
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32"
        " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
  }
}

// Tokens [lo, hi) of the chunk that see slots of [a, z) -- all of them when z = a + 1.
struct Tokens {
  int lo, hi;
};

__device__ __forceinline__ Tokens tokens_seeing(const Geo& g, const Seq& s, int a, int z) {
  Tokens t{0, s.q};
  z = min(z, s.kv);
  if (a >= z) return Tokens{0, 0};
  if (g.causal) t.lo = max(t.lo, a - s.off);
  if (g.window && a >= g.first) {
    t.lo = max(t.lo, a - g.window + 1 - s.off);
    t.hi = min(t.hi, z - 1 + g.window - s.off);
  }
  if (t.hi < t.lo) t.hi = t.lo;
  return t;
}

// A key tile's place in the line: entry b * tiles + tile, and its items.
struct Entry {
  int b, tile;
  Seq s;
  Tokens seen;
  int chunks, items;   // query tiles that see it, times K/V heads
};

__device__ __forceinline__ void entry_at(const WeightParams& p, Entry& e, int b, int tile) {
  const Geo& g = p.g;
  if (b != e.b) {
    e.b = b;
    e.s = seq_of(g, b);
  }
  e.tile = tile;
  e.seen = tokens_seeing(g, e.s, tile * BKV, (tile + 1) * BKV);
  e.chunks = (e.seen.hi - e.seen.lo + g.tok_per_tile - 1) / g.tok_per_tile;
  e.items = e.chunks * g.kv_heads;
}

// Whether a row that sees the slot, of tokens `mine` of sequence b, has a NaN for its
// normaliser. Asked only of infinite sums.
__device__ __forceinline__ bool nan_among(const WeightParams& p, int b, const Tokens& mine) {
  const float* row = p.lse + (static_cast<int64_t>(b) * p.g.t_q + mine.lo) * p.g.n_heads;
  const float* end = row + static_cast<int64_t>(mine.hi - mine.lo) * p.g.n_heads;
  bool any = false;
#pragma unroll 1
  for (; row < end; ++row) any |= *row != *row;
  return any;
}

// The next entry with items. Sequences end at their last slot, and no row sees
// what lies between the first slots and the window of row 0.
__device__ __forceinline__ bool entry_next(const WeightParams& p, Entry& e) {
  const Geo& g = p.g;
  int b = e.b, tile = e.tile;
  do {
    ++tile;
    if (g.window && tile * BKV >= g.first) tile = max(tile, max(0, e.s.off - g.window + 1) / BKV);
    if (tile >= p.tiles || tile * BKV >= e.s.kv) {
      if (++b >= g.batch) return false;
      tile = 0;
    }
    entry_at(p, e, b, tile);
  } while (e.items == 0);
  return true;
}

// A CTA's share of the line, entry by entry: items [i0, i1) of entry e.
struct Share {
  Entry e;
  long long left;      // items of the share from i0 on
  int i0, i1;
  __device__ __forceinline__ void cut() {
    i1 = static_cast<int>(min(static_cast<long long>(e.items), i0 + left));
  }
  __device__ __forceinline__ bool next(const WeightParams& p) {
    left -= i1 - i0;
    if (left <= 0 || !entry_next(p, e)) return false;
    i0 = 0;
    cut();
    return true;
  }
};

// The whole CTA: where share `cta` of `ctas` begins. Each thread adds up the items of a
// run of entries; the thread whose run holds the share's first item finds it.
struct Located {
  long long per, left;
  int b, tile, i0;
};

__device__ __forceinline__ void locate(const WeightParams& p, int cta, int ctas, int threads, long long* scan,
                                       Located* found) {
  const Geo& g = p.g;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  if (g.q_tiles == 1) {
    // One query tile: the key tiles of a sequence are those of its span, with
    // as many items each as there are K/V heads. One warp places the share.
    if (warp == 0) {
      const long long total = tiles_before(g, g.batch) * g.kv_heads;
      const long long per = (total + ctas - 1) / ctas;
      const long long pos = per * cta;
      if (lane == 0) {
        found->per = per;
        found->left = max(0ll, min(per, total - pos));
      }
      long long base = 0;
      for (int b0 = 0; b0 < g.batch && base <= pos && pos < total; b0 += 32) {
        Span u{};
        if (b0 + lane < g.batch) u = span_of(g, seq_of(g, b0 + lane), 0);
        const long long mine = static_cast<long long>(u.n) * g.kv_heads;
        long long incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const long long v = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += v;
        }
        const long long before = base + incl - mine;
        if (pos >= before && pos < before + mine) {
          const int k = static_cast<int>((pos - before) / g.kv_heads);
          found->b = b0 + lane;
          found->tile = u.tile(k);
          found->i0 = static_cast<int>(pos - before - static_cast<long long>(k) * g.kv_heads);
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    __syncthreads();
    return;
  }
  const int entries = g.batch * p.tiles;
  const int run = (entries + threads - 1) / threads;
  const int a = min(entries, t * run), z = min(entries, a + run);
  Entry e;
  e.b = -1;
  long long mine = 0;
  auto skip = [&](int x) {  // entries behind the end of a sequence hold nothing
    const int b = x / p.tiles, tile = x - b * p.tiles;
    entry_at(p, e, b, tile);
    return tile * BKV >= e.s.kv ? (b + 1) * p.tiles : x + 1;
  };
  for (int x = a; x < z;) {
    const int nx = skip(x);
    mine += e.items;
    x = nx;
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) scan[warp] = incl;
  __syncthreads();
  long long before = incl - mine, total = 0;
  for (int i = 0; i < threads / 32; ++i) {
    if (i < warp) before += scan[i];
    total += scan[i];
  }
  const long long per = (total + ctas - 1) / ctas;
  const long long pos = per * cta;
  if (t == 0) {
    found->per = per;
    found->left = max(0ll, min(per, total - pos));
  }
  if (pos < total && pos >= before && pos < before + mine) {
    for (int x = a; x < z;) {
      const int nx = skip(x);
      if (before + e.items > pos) break;
      before += e.items;
      x = nx;
    }
    found->b = e.b;
    found->tile = e.tile;
    found->i0 = static_cast<int>(pos - before);
  }
  __syncthreads();
}

template <int N>
__global__ void __launch_bounds__(WeightCfg<N>::THREADS, WeightCfg<N>::CTAS_PER_SM)
    paged_weights_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                         const WeightParams p) {
  using C = WeightCfg<N>;
  constexpr int KS = C::K_STAGES, QS = C::Q_STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::OFF_BARS;
  auto k_full = [&](int s) { return bar0 + 8u * s; };
  auto k_empty = [&](int s) { return bar0 + 8u * (KS + s); };
  auto q_full = [&](int s) { return bar0 + 8u * (2 * KS + s); };
  auto q_empty = [&](int s) { return bar0 + 8u * (2 * KS + QS + s); };
  auto s_full = [&](int s) { return bar0 + 8u * (2 * KS + 2 * QS + s); };
  auto s_free = [&](int s) { return bar0 + 8u * (2 * KS + 2 * QS + 2 + s); };
  const uint32_t drain_bar = bar0 + 8u * (2 * KS + 2 * QS + 4);
  const uint32_t half_full = drain_bar + 8u, half_empty = drain_bar + 16u;
  float* lse_ring = reinterpret_cast<float*>(smem + C::OFF_LSE);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC + 4);
  const Geo& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < KS; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 1);
    }
    for (int s = 0; s < QS; ++s) {
      mbar_init(q_full(s), 1);
      mbar_init(q_empty(s), 1 + C::WARPS);  // the MMA and the warps that read the normalisers
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_full(s), 1);
      mbar_init(s_free(s), C::WARPS);
    }
    mbar_init(drain_bar, 1);
    mbar_init(half_full, 4);
    mbar_init(half_empty, 4);
    *abort_flag = 0u;
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
  }
  if (warp == C::WARPS + 1) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();
  const WaitCtl wc{abort_flag, p.err, p.limit_ns};

  Located* found = reinterpret_cast<Located*>(smem + C::OFF_SCAN + 80);
  Share w;
  w.e.b = -1;
  long long per = 1;
  int rank = 0;
  if (p.cluster > 0) {
    const int entry = blockIdx.x / p.cluster;
    rank = blockIdx.x - entry * p.cluster;
    const int b = entry / p.tiles;
    entry_at(p, w.e, b, entry - b * p.tiles);
    w.i0 = static_cast<int>(static_cast<long long>(w.e.items) * rank / p.cluster);
    w.left = static_cast<int>(static_cast<long long>(w.e.items) * (rank + 1) / p.cluster) - w.i0;
    w.cut();
  } else {
    locate(p, blockIdx.x, gridDim.x, C::THREADS, reinterpret_cast<long long*>(smem + C::OFF_SCAN), found);
    w.left = found->left;
    per = found->per;
    if (w.left > 0) {
      entry_at(p, w.e, found->b, found->tile);
      w.i0 = found->i0;
      w.cut();
    }
  }

  if (warp == C::WARPS && w.left > 0) {
    // ---------------- producer ----------------
    const int n_pages = pages_per_tile(g);
    const uint32_t page_bytes = TILE_BYTES / n_pages;
    const uint32_t q_bytes = static_cast<uint32_t>(g.tok_per_tile * g.group) * DH * 2;
    // Normalisers of an item's rows, negated, read an item ahead: each costs a
    // round trip to L2. -inf takes a row's weight to zero. A NaN is handed over as
    // the largest number, which makes infinities of the slots that the row sees and
    // leaves the others, whose scores are -inf by then, alone.
    constexpr int LANE_ROWS = (N + 31) / 32;
    const int q_rows = g.tok_per_tile * g.group;
    int row_tok[LANE_ROWS], row_head[LANE_ROWS];  // this lane's rows of a query tile
#pragma unroll
    for (int x = 0; x < LANE_ROWS; ++x) {
      const int r = 32 * x + lane;
      row_tok[x] = r < q_rows ? fa::div_c(r, p.dv_group) : g.t_q;
      row_head[x] = r - row_tok[x] * g.group;
    }
    float norm[LANE_ROWS];
    auto read_norms = [&](int i) {
      const int h = i / w.e.chunks;
      const int tok0 = w.e.seen.lo + (i - h * w.e.chunks) * g.tok_per_tile;
#pragma unroll
      for (int x = 0; x < LANE_ROWS; ++x) {
        const int tok = tok0 + row_tok[x];
        norm[x] = -INFINITY;
        if (i < w.i1 && tok < w.e.seen.hi)
          norm[x] = __ldg(p.lse + (static_cast<int64_t>(w.e.b) * g.t_q + tok) * g.n_heads + h * g.group + row_head[x]);
      }
    };
    int kn = 0, qn = 0;
    bool ok = true;
    do {
    PageLoad l{false, 0};
    if (lane < n_pages) {
      Span all{};
      all.hi = w.e.s.kv;
      l = page_of_tile(g, w.e.b, all, w.e.tile, lane);
    }
    read_norms(w.i0);
    const uint32_t k_bytes = __popc(__ballot_sync(0xffffffffu, l.load)) * page_bytes;
    for (int i = w.i0; i < w.i1; ++i) {
      const int h = i / w.e.chunks, ch = i - h * w.e.chunks;
      const int tok0 = w.e.seen.lo + ch * g.tok_per_tile;
      if (i == w.i0 || ch == 0) {  // the next head's K
        const int st = kn % KS;
        ok = __all_sync(0xffffffffu, mbar_wait(k_empty(st), ((kn / KS) & 1) ^ 1u, wc));
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(k_full(st), k_bytes);
        __syncwarp();
        if (l.load) tma_load_2d(sbase + C::OFF_K + st * TILE_BYTES + lane * page_bytes, &tm_k, k_full(st), h * DH, l.row);
        ++kn;
      }
      const int st = qn % QS;
      ok = __all_sync(0xffffffffu, mbar_wait(q_empty(st), ((qn / QS) & 1) ^ 1u, wc));
      if (!ok) break;
#pragma unroll
      for (int x = 0; x < LANE_ROWS; ++x)
        if (32 * x + lane < N)
          lse_ring[st * N + 32 * x + lane] =
              norm[x] != norm[x] ? FLT_MAX : norm[x] == -INFINITY ? -INFINITY : -norm[x] * kLog2e;
      read_norms(i + 1);
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_expect_tx(q_full(st), q_bytes);
        tma_load_4d(sbase + C::OFF_Q + st * C::Q_BYTES, &tm_q, q_full(st), 0, h * g.group, tok0, w.e.b);
      }
      ++qn;
    }
    } while (ok && w.next(p));
    // Let the last copies land before the CTA may exit.
    for (int i = max(0, kn - KS); i < kn; ++i) mbar_wait_drain(k_full(i % KS), (i / KS) & 1, p.limit_ns);
    for (int i = max(0, qn - QS); i < qn; ++i) mbar_wait_drain(q_full(i % QS), (i / QS) & 1, p.limit_ns);
  } else if (warp == C::WARPS + 1 && w.left > 0) {
    if (lane == 0) {
      // ---------------- MMA issuer ----------------
      constexpr uint32_t idesc = idesc_f16_f32(BKV, N, 0, 0);  // K and Q both K-major
      int kn = 0, n = 0;
      bool ok = true;
      do {
        int ch = w.i0 % w.e.chunks;
        for (int i = w.i0; i < w.i1 && ok; ++i, ++n) {
          if (i == w.i0 || ch == 0) {
            ok = mbar_wait(k_full(kn % KS), (kn / KS) & 1, wc);
            ++kn;
          }
          const int ks = (kn - 1) % KS, qs = n % QS, buf = n & 1;
          ok = ok && mbar_wait(q_full(qs), (n / QS) & 1, wc) && mbar_wait(s_free(buf), ((n >> 1) & 1) ^ 1u, wc);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < DH / 16; ++kk)
            mma_f16_ss(tmem_base + buf * N, smem_desc_sw128(sbase + C::OFF_K + ks * TILE_BYTES + kk * 32, 16, 1024),
                       smem_desc_sw128(sbase + C::OFF_Q + qs * C::Q_BYTES + kk * 32, 16, 1024), idesc, kk > 0 ? 1u : 0u);
          mma_commit(s_full(buf));
          mma_commit(q_empty(qs));
          if (++ch == w.e.chunks) ch = 0;
          if (ch == 0 || i + 1 == w.i1) mma_commit(k_empty(ks));
        }
      } while (ok && w.next(p));
      mma_commit(drain_bar);
      mbar_wait_drain(drain_bar, 0, p.limit_ns);
    }
  } else if (warp < C::WARPS) {
    // ---------------- weights: thread = slot ----------------
    constexpr int NC = C::NC;
    const int half = warp >> 2;  // columns [half * NC, half * NC + NC)
    const uint32_t s_tmem = tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16) + half * NC;
    const int t = threadIdx.x & (BKV - 1);
    float* half_sum = reinterpret_cast<float*>(smem + C::OFF_HALF);
    int n = 0, entry_n = 0;
    int on = -1, more = 0;  // for the merge: see ws_state
    // For rank 0, where the last query tile was: its products are done by then.
    float* total = reinterpret_cast<float*>(smem + C::OFF_Q);
    if (p.cluster > 1 && half == 0 && w.left <= 0) total[t] = 0.f;
    bool ok = true;
    if (w.left > 0) do {
    const int j = w.e.tile * BKV + t;
    const Tokens mine = tokens_seeing(g, w.e.s, j, j + 1);
    // A slot in a hole, or behind the end, has none (its K may be anything).
    int page = -1;
    if (j < w.e.s.kv) page = __ldg(g.table + static_cast<int64_t>(w.e.b) * g.pages_per_seq + (j >> g.page_shift));
    const int64_t at = static_cast<int64_t>(w.e.b) * g.cap + j;
    const bool whole = w.i0 == 0 && w.i1 == w.e.items;
    const float w_old = whole && half == 0 && j < g.cap && p.w_in != nullptr ? p.w_in[at] : 0.f;
    float sum = 0.f;
    int ch = w.i0 % w.e.chunks;
    for (int i = w.i0; i < w.i1; ++i, ++n) {
      const int qs = n % QS, buf = n & 1;
      ok = mbar_wait(q_full(qs), (n / QS) & 1, wc) && mbar_wait(s_full(buf), (n >> 1) & 1, wc);  // normalisers, scores
      if (!ok) break;
      tc_fence_after();
      float x[NC];
      {
        uint32_t r[NC];
        tmem_ld_cols<NC>(s_tmem + buf * N, r);
#pragma unroll
        for (int e = 0; e < NC; ++e) x[e] = __uint_as_float(r[e]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_free(buf));
      // Columns [c_lo, c_hi) are rows that see this slot.
      const int tok0 = w.e.seen.lo + ch * g.tok_per_tile;
      if (++ch == w.e.chunks) ch = 0;
      const int c_lo = (mine.lo - tok0) * g.group - half * NC;
      const int c_hi = min(mine.hi - tok0, g.tok_per_tile) * g.group - half * NC;
      if (c_lo > 0) {
#pragma unroll
        for (int e = 0; e < NC; ++e)
          if (e < c_lo) x[e] = -INFINITY;
      }
      if (c_hi < NC) {
#pragma unroll
        for (int e = 0; e < NC; ++e)
          if (e >= c_hi) x[e] = -INFINITY;
      }
      const float4* norm = reinterpret_cast<const float4*>(lse_ring + qs * N + half * NC);
      const uint64_t sl2x2 = f2_pack(p.scale_log2, p.scale_log2);
      uint64_t acc2[2] = {0ull, 0ull};
#pragma unroll
      for (int e = 0; e < NC; e += 4) {
        const float4 v = norm[e / 4];
        float y0, y1, y2, y3;
        f2_unpack(f2_fma(f2_pack(x[e], x[e + 1]), sl2x2, f2_pack(v.x, v.y)), y0, y1);
        f2_unpack(f2_fma(f2_pack(x[e + 2], x[e + 3]), sl2x2, f2_pack(v.z, v.w)), y2, y3);
        acc2[0] = f2_add(acc2[0], f2_pack(ex2_approx(y0), ex2_approx(y1)));
        acc2[1] = f2_add(acc2[1], f2_pack(ex2_approx(y2), ex2_approx(y3)));
      }
      float a, c;
      f2_unpack(f2_add(acc2[0], acc2[1]), a, c);
      sum += a + c;  // one tile's weights, then the running sum: fp32 in two levels
      __syncwarp();
      if (lane == 0) mbar_arrive(q_empty(qs));
    }
    if (page < 0 || page >= g.num_pages)
      sum = 0.f;
    else if (sum == INFINITY && nan_among(p, w.e.b, mine))
      sum = NAN;
    if constexpr (C::SPLIT == 2) {
      if (!ok) break;
      if (half == 1) {
        ok = mbar_wait(half_empty, (entry_n & 1) ^ 1u, wc);
        half_sum[t] = sum;
        __syncwarp();
        if (lane == 0) mbar_arrive(half_full);
      } else {
        ok = mbar_wait(half_full, entry_n & 1, wc);
        sum += half_sum[t];
        __syncwarp();
        if (lane == 0) mbar_arrive(half_empty);
      }
      ++entry_n;
      if (half == 1) continue;
    }
    if (p.cluster > 1) {
      total[t] = sum;
    } else if (whole) {
      if (j < g.cap) p.w_out[at] = w_old + sum;
    } else {
      const bool starts = w.i0 == 0;
      p.ws_sum[(2 * static_cast<int64_t>(blockIdx.x) + (starts ? 1 : 0)) * BKV + t] = sum;
      if (starts) {
        on = w.e.b * p.tiles + w.e.tile;
        more = static_cast<int>((w.e.items - w.i1 + per - 1) / per);
      }
    }
    } while (ok && w.next(p));
    if (threadIdx.x == 0 && p.cluster == 0) {
      p.ws_state[2 * blockIdx.x] = on;
      p.ws_state[2 * blockIdx.x + 1] = more;
    }
    // Slots of key tiles that no row sees keep their weights.
    if (p.w_in != p.w_out && half == 0) {
      Entry e;
      e.b = -1;
      for (int x = blockIdx.x; x < g.batch * p.tiles; x += gridDim.x) {
        entry_at(p, e, x / p.tiles, x % p.tiles);
        const int j = e.tile * BKV + t;
        if (e.items > 0 || j >= g.cap) continue;
        const int64_t at = static_cast<int64_t>(e.b) * g.cap + j;
        p.w_out[at] = p.w_in != nullptr ? p.w_in[at] : 0.f;
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == C::WARPS + 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
  if (p.cluster <= 1) return;
  cluster_sync();
  const int j = w.e.tile * BKV + static_cast<int>(threadIdx.x);
  if (rank == 0 && threadIdx.x < BKV && w.e.items > 0 && j < g.cap) {
    const uint32_t mine = sbase + C::OFF_Q + 4 * threadIdx.x;
    const int64_t at = static_cast<int64_t>(w.e.b) * g.cap + j;
    float part[8], v = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      part[i] = 0.f;
      if (i < p.cluster)
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(part[i]) : "r"(mapa_shared(mine, i)) : "memory");
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v += part[i];
    p.w_out[at] = (p.w_in != nullptr ? p.w_in[at] : 0.f) + v;
  }
  cluster_sync();  // no CTA leaves while rank 0 still reads its sums
}

// Adds up the key tiles that were cut: block c the one that begins in share c.
__global__ void __launch_bounds__(BKV) paged_weights_merge_kernel(const WeightParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int c = blockIdx.x, t = threadIdx.x;
  const int entry = p.ws_state[2 * c];
  if (entry < 0) return;
  const int more = p.ws_state[2 * c + 1];
  const int b = entry / p.tiles, j = (entry - b * p.tiles) * BKV + t;
  float v = p.ws_sum[(2 * static_cast<int64_t>(c) + 1) * BKV + t];
#pragma unroll 4
  for (int i = 1; i <= more; ++i) v += p.ws_sum[2 * static_cast<int64_t>(c + i) * BKV + t];
  if (j >= p.g.cap) return;
  const int64_t at = static_cast<int64_t>(b) * p.g.cap + j;
  p.w_out[at] = (p.w_in != nullptr ? p.w_in[at] : 0.f) + v;
}

}  // namespace pg
}  // namespace sea
