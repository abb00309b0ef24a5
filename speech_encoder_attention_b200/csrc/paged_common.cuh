// paged_common.cuh -- what the kernels on a paged K/V cache share: the cache's
// addressing, which slots a query row sees, and the split of the work.
//
// Slot j of sequence b lives in pool row table[b][j / page] * page + j % page;
// a table entry outside [0, num_pages) is a hole, and the slots of a hole hold
// nothing. KV = lens[b] counts the new tokens too: query row i of Q sits at
// position p = i + KV - Q and sees
//   j < KV, not in a hole, j <= p if causal, and with a window
//   |p - j| < window or j < first.
// Both ends of the window part and the end of the first part do not decrease
// in i, so the slots that any row of a query tile sees are [lo, hi) and
// [0, f), and the tile walks the 128-slot key tiles that meet them.
#pragma once

#include "sm100_ptx.cuh"

namespace sea {
namespace pg {

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}

// Warp-collective load of 64 consecutive columns, waiting once.
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
#define SEA_R8(i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), \
                  "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32"
      " {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15,"
      " %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31,"
      " %32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47,"
      " %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : SEA_R8(0), SEA_R8(8), SEA_R8(16), SEA_R8(24), SEA_R8(32), SEA_R8(40), SEA_R8(48), SEA_R8(56)
      : "r"(taddr)
      : "memory");
#undef SEA_R8
}

constexpr int DH = 64;
constexpr int BKV = 128;                      // slots per key tile
constexpr int TILE_BYTES = BKV * DH * 2;      // one 128-slot x 64-column fp16 tile
constexpr int GRANULE = 16;                   // smallest page: one bit of a tile's hole mask
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

struct Geo {
  int batch, t_q, n_heads, kv_heads, group;  // group = n_heads / kv_heads query heads share a K/V head
  int tok_per_tile, q_tiles;                 // query tile: tok_per_tile tokens x group heads
  int page_shift, pages_per_seq, num_pages;
  int cap;                                   // slots the table can address
  const int* table;
  const int* kv_lens;
  const int* q_lens;                         // may be null: every row is valid
  int window, first, causal;                 // window 0: none
};

struct Seq {
  int q, kv, off;
};

__device__ __forceinline__ Seq seq_of(const Geo& g, int b) {
  Seq s;
  s.kv = min(max(__ldg(g.kv_lens + b), 0), g.cap);
  s.q = g.q_lens != nullptr ? min(max(__ldg(g.q_lens + b), 0), g.t_q) : g.t_q;
  s.off = s.kv - s.q;
  return s;
}

// What the row at position p sees: [lo, hi) and [0, f).
struct RowSpan {
  int lo, hi, f;
};

__device__ __forceinline__ RowSpan row_span(const Geo& g, const Seq& s, int p) {
  const int end = max(0, g.causal ? min(s.kv, p + 1) : s.kv);
  RowSpan r{0, end, 0};
  if (g.window) {
    r.lo = max(0, p - g.window + 1);
    r.hi = max(0, min(end, p + g.window));
    r.f = min(g.first, end);
  }
  return r;
}

// The key tiles of a query tile: k = 0 .. n-1 stands for tile k (k < n_first)
// or t_lo + k - n_first.
struct Span {
  int tok0, ntok;       // valid tokens [tok0, tok0 + ntok) of the sequence's chunk
  int lo, hi, f;        // union over the tile's rows
  int n_first, t_lo, n;
  __device__ __forceinline__ int tile(int k) const { return k < n_first ? k : t_lo + k - n_first; }
};

__device__ __forceinline__ Span span_of(const Geo& g, const Seq& s, int qt) {
  Span u;
  u.tok0 = qt * g.tok_per_tile;
  u.ntok = min(g.tok_per_tile, s.q - u.tok0);
  u.lo = u.hi = u.f = u.n_first = u.t_lo = u.n = 0;
  if (u.ntok <= 0) {
    u.ntok = 0;
    return u;
  }
  const RowSpan a = row_span(g, s, u.tok0 + s.off);
  const RowSpan z = row_span(g, s, u.tok0 + u.ntok - 1 + s.off);
  u.lo = a.lo;
  u.hi = z.hi;
  u.f = z.f;
  int t_hi = (u.hi + BKV - 1) / BKV;
  u.t_lo = u.lo / BKV;
  if (u.hi <= u.lo) {
    u.lo = u.hi = 0;
    t_hi = u.t_lo = 0;
  }
  // Unless causal, the first part may reach past the window part: the tiles behind
  // the window part that hold first slots are walked with it.
  u.n_first = (u.f + BKV - 1) / BKV;
  if (t_hi > u.t_lo) {
    t_hi = max(t_hi, u.n_first);
    u.n_first = min(u.n_first, u.t_lo);
  }
  u.n = u.n_first + t_hi - u.t_lo;
  return u;
}

// The end of a row's softmax: what its unnormalised output is multiplied by, and
// the log of its denominator, from the sum l with exponent reference m (log2
// units) and the sink (-inf: none), whichever is larger being the common
// reference. l = 0, a row that saw nothing, gives 0 and -inf.
struct RowEnd {
  float inv, lse;
};

__device__ __forceinline__ RowEnd row_end(float l, float m, float sink) {
  if (l == 0.f) return RowEnd{0.f, -INFINITY};
  const float s2 = sink * kLog2e;
  if (s2 > m) {
    const float down = ex2_approx(m - s2);
    const float total = fmaf(l, down, 1.f);
    return RowEnd{down / total, s2 * kLn2 + logf(total)};
  }
  const float total = l + ex2_approx(s2 - m);
  return RowEnd{1.f / total, m * kLn2 + logf(total)};
}

// ---------------------------------------------------------------------------
// work split: the key tiles of all (sequence, query tile) units in one line,
// cut into equal parts; CTA part * kv_heads + h walks its part for K/V head h.
// The heads of a part run side by side over the same slots, whose rows lie next
// to each other in memory. A unit whose tiles fall into several parts leaves
// unnormalised partials in the workspace.
// ---------------------------------------------------------------------------

__device__ __forceinline__ int tiles_of_seq(const Geo& g, int b) {
  const Seq s = seq_of(g, b);
  int n = 0;
  for (int qt = 0; qt < g.q_tiles; ++qt) n += span_of(g, s, qt).n;
  return n;
}

// One warp: the tiles of all sequences before b (b == batch: of all). Lanes
// take sequences; with many query tiles per sequence they take query tiles.
__device__ __forceinline__ long long tiles_before(const Geo& g, int b) {
  const int lane = threadIdx.x & 31;
  long long sum = 0;
  if (g.q_tiles <= 4) {
    for (int i = lane; i < b; i += 32) sum += tiles_of_seq(g, i);
  } else {
    for (int i = 0; i < b; ++i) {
      const Seq s = seq_of(g, i);
      for (int qt = lane; qt < g.q_tiles; qt += 32) sum += span_of(g, s, qt).n;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// Tiles of query tiles [0, qt) of one sequence (one warp).
__device__ __forceinline__ int tiles_before_q(const Geo& g, const Seq& s, int qt) {
  int sum = 0;
  for (int i = threadIdx.x & 31; i < qt; i += 32) sum += span_of(g, s, i).n;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return sum;
}

// Tiles per part: an equal share, and one of an empty line, which others divide by.
__device__ __forceinline__ long long share_of(long long total, int parts) {
  return max(1ll, (total + parts - 1) / parts);
}

// One part, unit by unit. Every warp of the CTA walks the same steps.
struct Walk {
  long long pos, end;   // tiles left: [pos, end)
  long long begin;
  int b, qt;
  Seq s;
  Span u;
  int k0, k1;           // key tiles [k0, k1) of the unit u
  bool whole;           // the unit's tiles are all here
  int slot;             // partial slot of this part (0: its first unit, 1: a later one)
};

__device__ __forceinline__ void walk_cut(const Geo& g, Walk& w, int k0) {
  w.k0 = k0;
  const long long left = w.end - w.pos;
  w.k1 = static_cast<int>(min(static_cast<long long>(w.u.n), k0 + left));
  w.whole = k0 == 0 && w.k1 == w.u.n;
  w.slot = w.pos == w.begin ? 0 : 1;
}

// One warp; returns false if the part is empty.
__device__ __forceinline__ bool walk_start(const Geo& g, Walk& w, int part, int parts) {
  const int lane = threadIdx.x & 31;
  // Up to 32 sequences: a lane each, looked at once.
  const bool once = g.q_tiles <= 4 && g.batch <= 32;
  const int lane_tiles = once && lane < g.batch ? tiles_of_seq(g, lane) : 0;
  const long long total = once ? __reduce_add_sync(0xffffffffu, lane_tiles) : tiles_before(g, g.batch);
  const long long per = share_of(total, parts);
  w.begin = w.pos = per * part;
  w.end = min(total, w.pos + per);
  if (w.pos >= w.end) return false;
  // the sequence that holds tile `pos`
  long long base = 0;
  int b = 0;
  if (g.q_tiles <= 4) {
    for (int b0 = 0; b0 < g.batch; b0 += 32) {
      const int n = once ? lane_tiles : b0 + lane < g.batch ? tiles_of_seq(g, b0 + lane) : 0;
      long long incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      const unsigned past = __ballot_sync(0xffffffffu, base + incl > w.pos);
      if (past) {
        const int i = __ffs(past) - 1;
        b = b0 + i;
        base += __shfl_sync(0xffffffffu, incl - n, i);
        break;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
  } else {
    for (b = 0; b < g.batch; ++b) {
      const int n = tiles_before_q(g, seq_of(g, b), g.q_tiles);
      if (base + n > w.pos) break;
      base += n;
    }
  }
  w.b = b;
  w.s = seq_of(g, b);
  int rest = static_cast<int>(w.pos - base);
  // the query tile that holds it
  int qt = 0;
  for (int q0 = 0; q0 < g.q_tiles; q0 += 32) {
    const int n = q0 + lane < g.q_tiles ? span_of(g, w.s, q0 + lane).n : 0;
    int incl = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    const unsigned past = __ballot_sync(0xffffffffu, incl > rest);
    if (past) {
      const int i = __ffs(past) - 1;
      qt = q0 + i;
      rest -= __shfl_sync(0xffffffffu, incl - n, i);
      break;
    }
    rest -= __shfl_sync(0xffffffffu, incl, 31);
  }
  w.qt = qt;
  w.u = span_of(g, w.s, qt);
  walk_cut(g, w, rest);
  return true;
}

// The next unit of the part; false when the part is done. Any thread.
__device__ __forceinline__ bool walk_next(const Geo& g, Walk& w) {
  w.pos += w.k1 - w.k0;
  if (w.pos >= w.end) return false;
  do {
    if (++w.qt == g.q_tiles) {
      w.qt = 0;
      ++w.b;
      w.s = seq_of(g, w.b);
    }
    w.u = span_of(g, w.s, w.qt);
  } while (w.u.n == 0);
  walk_cut(g, w, 0);
  return true;
}

// ---------------------------------------------------------------------------
// loads of one key tile (the producer warp)
// ---------------------------------------------------------------------------

// Lane i's page of key tile t: whether any row of the query tile may see it,
// its pool row, and the granules it covers.
struct PageLoad {
  bool load;
  int row;
};

__device__ __forceinline__ int pages_per_tile(const Geo& g) { return g.page_shift >= 7 ? 1 : BKV >> g.page_shift; }

__device__ __forceinline__ PageLoad page_of_tile(const Geo& g, int b, const Span& u, int t, int i) {
  PageLoad l{false, 0};
  const int rows = g.page_shift >= 7 ? BKV : 1 << g.page_shift;
  const int j = t * BKV + i * rows;  // first slot
  const bool seen = (j < u.hi && j + rows > u.lo) || j < u.f;
  if (!seen) return l;
  const int page = __ldg(g.table + static_cast<long long>(b) * g.pages_per_seq + (j >> g.page_shift));
  if (page < 0 || page >= g.num_pages) return l;
  l.load = true;
  l.row = (page << g.page_shift) + (j & ((1 << g.page_shift) - 1));
  return l;
}

// The whole warp: pages of the 32 / n_pages key tiles of a unit from tile k on, in one
// read of the table; tile k + x's page i is in lane x * n_pages + i. A producer that
// reads the table tile by tile waits for it before each of its first copies.
__device__ __forceinline__ PageLoad pages_ahead(const Geo& g, int b, const Span& u, int k, int k1, int n_pages) {
  const int lane = threadIdx.x & 31;
  const int kk = k + lane / n_pages;
  return kk < k1 ? page_of_tile(g, b, u, u.tile(kk), lane & (n_pages - 1)) : PageLoad{false, 0};
}

// The whole warp: lane i < n_pages gets page i of the x-th of those tiles.
__device__ __forceinline__ PageLoad page_from(const PageLoad& ahead, int x, int n_pages) {
  const int lane = threadIdx.x & 31;
  const int row = __shfl_sync(0xffffffffu, ahead.load ? ahead.row : -1, (x * n_pages + lane) & 31);
  return PageLoad{lane < n_pages && row >= 0, row};
}

// Granule bits of the slots the tile's loads leave out, from the ballot of the
// lanes that load.
__device__ __forceinline__ uint32_t hole_bits(const Geo& g, uint32_t loaded) {
  if (g.page_shift >= 7) return loaded & 1u ? 0u : 0xFFu;
  const int per = (1 << g.page_shift) / GRANULE;  // granules per page: 1, 2 or 4
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < BKV / GRANULE; ++i)
    if (!((loaded >> (i / per)) & 1u)) bits |= 1u << i;
  return bits;
}

// Whether no row of the query tile sees slot j.
__device__ __forceinline__ bool unseen(const Span& u, int j) { return !((j >= u.lo && j < u.hi) || j < u.f); }

}  // namespace pg
}  // namespace sea
