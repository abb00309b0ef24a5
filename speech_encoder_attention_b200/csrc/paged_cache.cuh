// paged_cache.cuh -- writing to and shrinking a paged K/V cache.
//
// Append: row i of a chunk goes to slot i + KV - Q. A copy, bound by its
// bytes; one thread per 16 bytes.
//
// Evict: of the slots that hold something, keep the `first` first, the
// `recent` last and the heaviest of the rest up to `budget`, ties to the
// lowest slot, and move what is kept, in order, to the front.
//   select  the weights as 32-bit keys that order like them, a radix selection
//           of the budget-th largest key (up to four passes of 8 bits), then a
//           scan that numbers the kept slots.
//   move    bound by the bytes moved. Kept slot n comes from slot kept[n] >= n,
//           so a CTA that owns some columns of a sequence and walks the rows
//           upwards, loading a step before it stores it, may work in place.
//
// Measured on a B200, 20 K/V heads: appending 8 x 1500 rows 21.4 us = 5.7 TB/s;
// evicting eight caches of 7 to 16 thousand slots down to 4096 into other pools
// 69 us, 14 of them the selection, the move at 6.1 TB/s; in place 97 us, and one
// such cache alone 67 us: its 40 CTAs leave most SMs idle.
#pragma once

#include "flash_attn.cuh"
#include "paged_common.cuh"

namespace sea {
namespace pg {

struct AppendParams {
  Geo g;
  const __half *k_new, *v_new;
  int64_t k_new_stride, v_new_stride;
  __half *k, *v;
  int64_t k_stride, v_stride;
  int vecs;            // 16-byte pieces per row
  int rows_per_cta;
  fa::DivC dv_vecs, dv_t;
};

__global__ void __launch_bounds__(256) paged_append_kernel(const AppendParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const Geo& g = p.g;
  const int row0 = blockIdx.x * p.rows_per_cta;
  const int pieces = min(p.rows_per_cta, g.batch * g.t_q - row0) * p.vecs;
  for (int x = threadIdx.x; x < pieces; x += 256) {
    const int local = fa::div_c(x, p.dv_vecs);
    const int v = x - local * p.vecs;
    const int row = row0 + local;
    const int b = fa::div_c(row, p.dv_t);
    const int i = row - b * g.t_q;
    const Seq s = seq_of(g, b);
    const int slot = i + s.off;
    if (i >= s.q || slot < 0) continue;
    const int page = __ldg(g.table + static_cast<int64_t>(b) * g.pages_per_seq + (slot >> g.page_shift));
    if (page < 0 || page >= g.num_pages) continue;
    const int64_t dst = (static_cast<int64_t>(page) << g.page_shift) + (slot & ((1 << g.page_shift) - 1));
    const uint4 a = *(reinterpret_cast<const uint4*>(p.k_new + row * p.k_new_stride) + v);
    const uint4 c = *(reinterpret_cast<const uint4*>(p.v_new + row * p.v_new_stride) + v);
    *(reinterpret_cast<uint4*>(p.k + dst * p.k_stride) + v) = a;
    *(reinterpret_cast<uint4*>(p.v + dst * p.v_stride) + v) = c;
  }
}

struct EvictParams {
  Geo g;                  // the source cache (t_q, heads and window unused)
  int budget, first, recent;
  const float* w_in;      // [batch, cap]
  int out_pages_per_seq, out_num_pages, out_cap;
  const int* out_table;
  int* out_lens;
  float* w_out;           // [batch, out_cap] or null
  int* kept;              // [batch, budget]
  const __half *k, *v;
  int64_t k_stride, v_stride;
  __half *k_out, *v_out;
  int64_t k_out_stride, v_out_stride;
  int rows_per_cta;       // move: rows of a CTA (budget when in place)
  int move_vecs;          // and 16-byte pieces of a row
  fa::DivC dv_vecs;
};

// Keys that order like the weights: 0 for a slot that holds nothing, all ones
// for one that is always kept; NaN counts as -inf, -0 as 0.
__device__ __forceinline__ uint32_t evict_key(const EvictParams& p, const Seq& s, int b, int j, const float* w) {
  const int page = __ldg(p.g.table + static_cast<int64_t>(b) * p.g.pages_per_seq + (j >> p.g.page_shift));
  if (page < 0 || page >= p.g.num_pages) return 0u;
  if (j < p.first || j >= s.kv - p.recent) return 0xFFFFFFFFu;
  float x = w[j] + 0.f;
  if (x != x) x = -INFINITY;
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Select: a cluster of up to 8 CTAs per sequence, each with an equal run of its
// slots. Bound by latency: a pass costs a histogram in shared memory, a cluster
// barrier and 8 remote reads per digit, so the keys are computed once (8192 of
// a CTA's stay in shared memory; longer runs recompute the rest). One CTA alone
// (up to 1024 slots) is quicker with 512 threads, whose barriers are cheaper
// (five caches of up to 448 slots: 9.6 against 11.0 us with the move).
constexpr int SELECT_CACHED = 8192;

__device__ __forceinline__ uint32_t ld_shared_cluster_u32(const uint32_t* mine, uint32_t rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa_shared(smem_u32(mine), rank)) : "memory");
  return v;
}

template <int SELECT_THREADS>
__global__ void __launch_bounds__(SELECT_THREADS, 1) paged_select_kernel(const EvictParams p) {
  __shared__ uint32_t keys[SELECT_CACHED];
  __shared__ uint32_t hist[2][256];          // by pass, so one cluster barrier per pass is enough
  __shared__ uint32_t warp_sum[32], warp_eq[32];
  __shared__ uint32_t found[3];              // digit, how many of it are wanted, how many there are
  __shared__ uint32_t counts[2];             // this CTA's larger and equal keys
  __shared__ uint32_t bases[4];              // both in the CTAs before this one, and in all
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int rank = blockIdx.x, ranks = gridDim.x, b = blockIdx.y;
  if (t < 512) hist[t >> 8][t & 255] = 0u;
  if (t < 32) warp_sum[t] = warp_eq[t] = 0u;
  griddep_wait();
  griddep_launch_dependents();
  const Seq s = seq_of(p.g, b);
  const float* w = p.w_in + static_cast<int64_t>(b) * p.g.cap;
  const int run = (s.kv + ranks - 1) / ranks;
  const int ja = min(s.kv, rank * run), jz = min(s.kv, ja + run);
  auto key_at = [&](int j) { return j - ja < SELECT_CACHED ? keys[j - ja] : evict_key(p, s, b, j, w); };
  __syncthreads();

  // The budget-th largest key, digit by digit from the top: kept are the keys
  // of at least `limit` (and then no equal ones), or those above it and the
  // first `want` equal ones.
  uint32_t prefix = 0, limit = 1, want = static_cast<uint32_t>(p.budget);
  bool equal = false;  // `limit` is one key's value and only `want` of it stay
  uint32_t n_gt = 0, n_eq = 0;  // this CTA's larger and equal keys, summed over threads
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    uint32_t* h = hist[pass & 1];
    for (int j0 = ja; j0 < jz; j0 += SELECT_THREADS) {
      const int j = j0 + t;
      uint32_t key = 0u;
      if (j < jz) {
        key = pass == 0 ? evict_key(p, s, b, j, w) : key_at(j);
        if (pass == 0 && j - ja < SELECT_CACHED) keys[j - ja] = key;
      }
      const bool in = key != 0u && (pass == 0 || (key >> (shift + 8)) == prefix);
      const uint32_t digit = in ? (key >> shift) & 255u : 256u;
      const uint32_t same = __match_any_sync(0xffffffffu, digit);  // equal digits of a warp count once
      if (in && lane == __ffs(same) - 1) atomicAdd(&h[digit], __popc(same));
    }
    cluster_sync();
    uint32_t mine = 0, own = 0, above = 0;
    if (t < 256) {
      own = h[255 - t];
      for (int r = 0; r < ranks; ++r) mine += ld_shared_cluster_u32(&h[255 - t], r);  // thread t: digit 255 - t
      uint32_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) warp_sum[warp] = incl;
      above = incl - mine;
    }
    if (t == 0) found[2] = 0u;
    __syncthreads();
    if (t < 256) {
      for (int i = 0; i < warp; ++i) above += warp_sum[i];
      if (above < want && above + mine >= want) {
        found[0] = 255 - t;
        found[1] = want - above;
        found[2] = mine;
      }
      hist[(pass + 1) & 1][t] = 0u;  // read by others before the last barrier
    }
    __syncthreads();
    const bool some = found[2] != 0u;  // else fewer slots than the budget: all stay
    if (t < 256) {
      const uint32_t digit = 255 - t;
      if (!some || digit > found[0])
        n_gt += own;
      else if (digit == found[0] && found[2] == found[1])
        n_gt += own;  // every key of this digit stays
      else if (digit == found[0] && pass == 3)
        n_eq += own;
    }
    if (!some) break;
    prefix = prefix << 8 | found[0];
    want = found[1];
    limit = prefix << shift;
    if (found[2] == want) break;  // every key of this digit stays
    equal = pass == 3;
  }
  auto larger = [&](uint32_t key) { return key != 0u && (equal ? key > limit : key >= limit); };

  // Number what stays, in order. Earlier CTAs' counts first.
  n_gt = __reduce_add_sync(0xffffffffu, n_gt);
  n_eq = __reduce_add_sync(0xffffffffu, n_eq);
  if (lane == 0) {
    warp_sum[warp] = n_gt;
    warp_eq[warp] = n_eq;
  }
  __syncthreads();
  if (warp == 0) {
    counts[0] = __reduce_add_sync(0xffffffffu, warp_sum[lane]);
    counts[1] = __reduce_add_sync(0xffffffffu, warp_eq[lane]);
  }
  cluster_sync();
  if (warp == 0) {  // lane r: CTA r's counts
    const uint32_t x = lane < ranks ? ld_shared_cluster_u32(&counts[0], lane) : 0u;
    const uint32_t y = lane < ranks ? ld_shared_cluster_u32(&counts[1], lane) : 0u;
    bases[0] = __reduce_add_sync(0xffffffffu, lane < rank ? x : 0u);
    bases[1] = __reduce_add_sync(0xffffffffu, lane < rank ? y : 0u);
    bases[2] = __reduce_add_sync(0xffffffffu, x);
    bases[3] = __reduce_add_sync(0xffffffffu, y);
  }
  __syncthreads();
  uint32_t base_gt = bases[0], base_eq = bases[1];
  const uint32_t total = bases[2], total_eq = bases[3];
  const int count = static_cast<int>(total + min(total_eq, equal ? want : 0u));
  int* kept = p.kept + static_cast<int64_t>(b) * p.budget;
  const bool w_apart = p.w_out != nullptr && p.w_out != p.w_in;
  for (int j0 = ja; j0 < jz; j0 += SELECT_THREADS) {
    const int j = j0 + t;
    const uint32_t key = j < jz ? key_at(j) : 0u;
    const bool gt = larger(key), eq = equal && key == limit;
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    __syncthreads();
    if (lane == 0) {
      warp_sum[warp] = __popc(bg);
      warp_eq[warp] = __popc(be);
    }
    __syncthreads();
    const uint32_t xg = warp_sum[lane], xe = warp_eq[lane], below = (1u << lane) - 1u;
    const uint32_t g_before = base_gt + __reduce_add_sync(0xffffffffu, lane < warp ? xg : 0u) + __popc(bg & below);
    const uint32_t e_before = base_eq + __reduce_add_sync(0xffffffffu, lane < warp ? xe : 0u) + __popc(be & below);
    if (gt || (eq && e_before < want)) {
      const uint32_t n = g_before + min(e_before, want);
      kept[n] = j;
      if (w_apart) p.w_out[static_cast<int64_t>(b) * p.out_cap + n] = w[j];
    }
    base_gt += __reduce_add_sync(0xffffffffu, xg);
    base_eq += __reduce_add_sync(0xffffffffu, xe);
  }
  for (int n = count + rank * SELECT_THREADS + t; n < p.budget; n += ranks * SELECT_THREADS) kept[n] = -1;

  // Weights in place move like the rows: n <= kept[n], so a barrier between the
  // reads and the writes of a step is enough.
  if (p.w_out != nullptr) {
    float* w_out = p.w_out + static_cast<int64_t>(b) * p.out_cap;
    if (!w_apart) {
      __threadfence();  // kept, for the other CTAs
      cluster_sync();
      for (int n0 = 0; n0 < count; n0 += ranks * SELECT_THREADS) {
        const int n = n0 + rank * SELECT_THREADS + t;
        float x = 0.f;
        if (n < count) x = w[*const_cast<const volatile int*>(kept + n)];
        cluster_sync();
        if (n < count) w_out[n] = x;
      }
    }
    for (int n = count + rank * SELECT_THREADS + t; n < p.out_cap; n += ranks * SELECT_THREADS) w_out[n] = 0.f;
  }
  cluster_sync();  // every CTA has read the lengths, and the counts of this one
  if (rank == 0 && t == 0) p.out_lens[b] = count;
}

// Moves the rows of the kept slots: CTA (row range, columns of K or of V,
// sequence), MOVE_STEPS 16-byte pieces per thread and step, row by row.
constexpr int MOVE_THREADS = 256;
constexpr int MOVE_STEPS = 4;

template <bool SAME_POOL>
__global__ void __launch_bounds__(MOVE_THREADS) paged_move_kernel(const EvictParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.z;
  const int halves = gridDim.y / 2;  // column ranges of K, then of V
  const bool is_v = static_cast<int>(blockIdx.y) >= halves;
  const int col0 = (is_v ? blockIdx.y - halves : blockIdx.y) * p.move_vecs;
  const uint4* src = reinterpret_cast<const uint4*>(is_v ? p.v : p.k) + col0;
  uint4* dst = reinterpret_cast<uint4*>(is_v ? p.v_out : p.k_out) + col0;
  const int64_t ss = (is_v ? p.v_stride : p.k_stride) / 8, ds = (is_v ? p.v_out_stride : p.k_out_stride) / 8;
  const int mask = (1 << p.g.page_shift) - 1;
  const int n_begin = blockIdx.x * p.rows_per_cta;
  const int n_end = min(p.budget, n_begin + p.rows_per_cta);
  const int* kept = p.kept + static_cast<int64_t>(b) * p.budget;
  const int* t_in = p.g.table + static_cast<int64_t>(b) * p.g.pages_per_seq;
  const int* t_out = p.out_table + static_cast<int64_t>(b) * p.out_pages_per_seq;
  const int pieces = (n_end - n_begin) * p.move_vecs;  // below 2^23 * 8, or a few rows
  constexpr int STEP = MOVE_THREADS * MOVE_STEPS;
  if constexpr (!SAME_POOL) {
    for (int x0 = 0; x0 < pieces; x0 += STEP) {
      uint4 x[MOVE_STEPS];
      int64_t to[MOVE_STEPS];
#pragma unroll
      for (int i = 0; i < MOVE_STEPS; ++i) {
        const int at = x0 + i * MOVE_THREADS + static_cast<int>(threadIdx.x);
        to[i] = -1;
        if (at >= pieces) continue;
        const int row = fa::div_c(at, p.dv_vecs);
        const int vec = at - row * p.move_vecs;
        const int n = n_begin + row;
        const int j = kept[n];
        if (j < 0) continue;
        const int pi = t_in[j >> p.g.page_shift], po = t_out[n >> p.g.page_shift];
        if (po < 0 || po >= p.out_num_pages) continue;
        to[i] = ((static_cast<int64_t>(po) << p.g.page_shift) + (n & mask)) * ds + vec;
        x[i] = src[((static_cast<int64_t>(pi) << p.g.page_shift) + (j & mask)) * ss + vec];
      }
#pragma unroll
      for (int i = 0; i < MOVE_STEPS; ++i)
        if (to[i] >= 0) dst[to[i]] = x[i];
    }
    return;
  }
  struct Step {
    uint4 x[MOVE_STEPS];
    int64_t to[MOVE_STEPS];
  };
  auto slots = [&](int x0, int (&j)[MOVE_STEPS]) {
#pragma unroll
    for (int i = 0; i < MOVE_STEPS; ++i) {
      const int at = x0 + i * MOVE_THREADS + static_cast<int>(threadIdx.x);
      j[i] = at < pieces ? kept[n_begin + fa::div_c(at, p.dv_vecs)] : -1;
    }
  };
  auto load = [&](int x0, const int (&j)[MOVE_STEPS], Step& s) {
#pragma unroll
    for (int i = 0; i < MOVE_STEPS; ++i) {
      const int at = x0 + i * MOVE_THREADS + static_cast<int>(threadIdx.x);
      s.to[i] = -1;
      if (j[i] < 0) continue;
      const int row = fa::div_c(at, p.dv_vecs);
      const int vec = at - row * p.move_vecs;
      const int n = n_begin + row;
      const int pi = t_in[j[i] >> p.g.page_shift], po = t_out[n >> p.g.page_shift];
      if (po < 0 || po >= p.out_num_pages) continue;
      s.to[i] = ((static_cast<int64_t>(po) << p.g.page_shift) + (n & mask)) * ds + vec;
      s.x[i] = src[((static_cast<int64_t>(pi) << p.g.page_shift) + (j[i] & mask)) * ss + vec];
    }
  };
  auto store = [&](const Step& s) {
    __syncthreads();  // this step's rows are read before any is overwritten
#pragma unroll
    for (int i = 0; i < MOVE_STEPS; ++i)
      if (s.to[i] >= 0) dst[s.to[i]] = s.x[i];
  };
  // Two steps are on their way at a time, and the slots of the third are known:
  // what a step loads lies at or behind its own destinations, so the step before
  // cannot overwrite it. Eight 16000-slot caches to 4096 in place: 96 us against
  // 135 us one step at a time.
  int j[MOVE_STEPS];
  Step a, c;
  slots(0, j);
  load(0, j, a);
  slots(STEP, j);
  for (int x0 = 0; x0 < pieces; x0 += 2 * STEP) {
    load(x0 + STEP, j, c);
    slots(x0 + 2 * STEP, j);
    store(a);
    load(x0 + 2 * STEP, j, a);
    slots(x0 + 3 * STEP, j);
    store(c);
  }
}

}  // namespace pg
}  // namespace sea
