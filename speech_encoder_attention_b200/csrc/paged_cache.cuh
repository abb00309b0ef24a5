// paged_cache.cuh -- writing to and shrinking a paged K/V cache.
//
// Append: row i of a chunk goes to slot i + KV - Q. A copy, bound by its
// bytes; one thread per 16 bytes.
//
// Evict: of the slots that hold something, keep the `first` first, the
// `recent` last and the heaviest of the rest up to `budget`, ties to the
// lowest slot, and move what is kept, in order, to the front.
//   select  one CTA per sequence: the weights as 32-bit keys that order like
//           them, a radix selection of the budget-th largest key (four passes
//           of 8 bits over the keys), then a scan that numbers the kept slots.
//   move    bound by the bytes moved. Kept slot n comes from slot kept[n] >= n,
//           so a CTA that owns some columns of a sequence and walks the rows
//           upwards, loading a step before it stores it, may work in place.
#pragma once

#include "paged_common.cuh"

namespace sea {
namespace pg {

struct AppendParams {
  Geo g;
  const __half *k_new, *v_new;
  int64_t k_new_stride, v_new_stride;
  __half *k, *v;
  int64_t k_stride, v_stride;
  int vecs;  // 16-byte pieces per row
};

__global__ void __launch_bounds__(256) paged_append_kernel(const AppendParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const Geo& g = p.g;
  const int64_t total = static_cast<int64_t>(g.batch) * g.t_q * p.vecs;
  for (int64_t x = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; x < total;
       x += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = x / p.vecs;
    const int v = static_cast<int>(x - row * p.vecs);
    const int b = static_cast<int>(row / g.t_q);
    const int i = static_cast<int>(row - static_cast<int64_t>(b) * g.t_q);
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

constexpr int SELECT_THREADS = 1024;

__global__ void __launch_bounds__(SELECT_THREADS, 1) paged_select_kernel(const EvictParams p) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t found[2];              // digit, how many are still wanted
  __shared__ uint32_t warp_gt[32], warp_eq[32];
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const Seq s = seq_of(p.g, b);
  const float* w = p.w_in + static_cast<int64_t>(b) * p.g.cap;
  // The budget-th largest key: prefix, digit by digit from the top.
  uint32_t prefix = 0, want = static_cast<uint32_t>(p.budget);
  bool all = false;  // fewer slots than the budget
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (t < 256) hist[t] = 0u;
    __syncthreads();
    for (int j0 = 0; j0 < s.kv; j0 += SELECT_THREADS) {
      const int j = j0 + t;
      const uint32_t key = j < s.kv ? evict_key(p, s, b, j, w) : 0u;
      const bool in = key != 0u && (shift == 24 || (key >> (shift + 8)) == prefix);
      // equal digits of a warp count once
      const uint32_t digit = in ? (key >> shift) & 255u : 256u;
      const uint32_t same = __match_any_sync(0xffffffffu, digit);
      if (in && lane == __ffs(same) - 1) atomicAdd(&hist[digit], __popc(same));
    }
    __syncthreads();
    if (warp == 0) {
      // lane i holds digits [8i, 8i + 8); digits above come first
      uint32_t mine = 0;
      for (int i = 0; i < 8; ++i) mine += hist[8 * lane + i];
      uint32_t above = 0;  // keys in higher lanes
      for (int o = 31; o > 0; --o) {
        const uint32_t x = __shfl_sync(0xffffffffu, mine, o);
        if (lane < o) above += x;
      }
      if (shift == 24 && lane == 0) found[1] = 0xFFFFFFFFu;
      __syncwarp();
      if (above < want && above + mine >= want) {
        uint32_t left = want - above;
        int d = 8 * lane + 7;
        while (hist[d] < left) left -= hist[d--];
        found[0] = d;
        found[1] = left;
      }
    }
    __syncthreads();
    if (shift == 24 && found[1] == 0xFFFFFFFFu) {
      all = true;
      break;
    }
    prefix = prefix << 8 | found[0];
    want = found[1];
    __syncthreads();
  }
  // Number the kept slots in order: larger keys, and the first `want` equal ones.
  uint32_t base_gt = 0, base_eq = 0;
  int* kept = p.kept + static_cast<int64_t>(b) * p.budget;
  float* w_out = p.w_out != nullptr ? p.w_out + static_cast<int64_t>(b) * p.out_cap : nullptr;
  for (int j0 = 0; j0 < s.kv; j0 += SELECT_THREADS) {
    const int j = j0 + t;
    const uint32_t key = j < s.kv ? evict_key(p, s, b, j, w) : 0u;
    const float wj = j < s.kv ? w[j] : 0.f;
    const bool gt = all ? key != 0u : key > prefix;
    const bool eq = !all && key == prefix && key != 0u;
    const uint32_t bg = __ballot_sync(0xffffffffu, gt), be = __ballot_sync(0xffffffffu, eq);
    if (lane == 0) {
      warp_gt[warp] = __popc(bg);
      warp_eq[warp] = __popc(be);
    }
    __syncthreads();
    uint32_t g_before = base_gt, e_before = base_eq, g_all = 0, e_all = 0;
    {
      const uint32_t xg = warp_gt[lane], xe = warp_eq[lane];
      g_all = __reduce_add_sync(0xffffffffu, xg);
      e_all = __reduce_add_sync(0xffffffffu, xe);
      g_before += __reduce_add_sync(0xffffffffu, lane < warp ? xg : 0u);
      e_before += __reduce_add_sync(0xffffffffu, lane < warp ? xe : 0u);
    }
    const uint32_t below = (1u << lane) - 1u;
    g_before += __popc(bg & below);
    e_before += __popc(be & below);
    if (gt || (eq && e_before < want)) {
      const uint32_t n = g_before + min(e_before, want);
      kept[n] = j;
      if (w_out != nullptr) w_out[n] = wj;  // n <= j: these weights have been read
    }
    base_gt += g_all;
    base_eq += e_all;
    __syncthreads();
  }
  const int count = static_cast<int>(all ? base_gt : p.budget);
  for (int n = count + t; n < p.budget; n += SELECT_THREADS) kept[n] = -1;
  if (w_out != nullptr)
    for (int n = count + t; n < p.out_cap; n += SELECT_THREADS) w_out[n] = 0.f;
  if (t == 0) p.out_lens[b] = count;
}

// Rows of the kept slots: CTA (row range, K or V head, sequence), 8 threads
// per 128-byte head row.
constexpr int MOVE_THREADS = 256;
constexpr int MOVE_STEPS = 4;

__global__ void __launch_bounds__(MOVE_THREADS) paged_move_kernel(const EvictParams p) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.z;
  const int heads = gridDim.y / 2;
  const bool is_v = static_cast<int>(blockIdx.y) >= heads;
  const int col = (is_v ? blockIdx.y - heads : blockIdx.y) * DH + (threadIdx.x & 7) * 8;
  const __half* src = (is_v ? p.v : p.k) + col;
  __half* dst = (is_v ? p.v_out : p.k_out) + col;
  const int64_t ss = is_v ? p.v_stride : p.k_stride, ds = is_v ? p.v_out_stride : p.k_out_stride;
  const int mask = (1 << p.g.page_shift) - 1;
  const int n_end = min(p.budget, static_cast<int>(blockIdx.x + 1) * p.rows_per_cta);
  const int* kept = p.kept + static_cast<int64_t>(b) * p.budget;
  const int* t_in = p.g.table + static_cast<int64_t>(b) * p.g.pages_per_seq;
  const int* t_out = p.out_table + static_cast<int64_t>(b) * p.out_pages_per_seq;
  constexpr int ROWS = MOVE_THREADS / 8;
  for (int n0 = blockIdx.x * p.rows_per_cta; n0 < n_end; n0 += ROWS * MOVE_STEPS) {
    uint4 x[MOVE_STEPS];
    int64_t to[MOVE_STEPS];
#pragma unroll
    for (int i = 0; i < MOVE_STEPS; ++i) {
      const int n = n0 + i * ROWS + static_cast<int>(threadIdx.x >> 3);
      to[i] = -1;
      if (n >= n_end) continue;
      const int j = kept[n];
      if (j < 0) continue;
      const int pi = t_in[j >> p.g.page_shift], po = t_out[n >> p.g.page_shift];
      if (po < 0 || po >= p.out_num_pages) continue;
      const int64_t from = (static_cast<int64_t>(pi) << p.g.page_shift) + (j & mask);
      to[i] = (static_cast<int64_t>(po) << p.g.page_shift) + (n & mask);
      x[i] = *reinterpret_cast<const uint4*>(src + from * ss);
    }
    __syncthreads();  // this step's rows are read before any is overwritten
#pragma unroll
    for (int i = 0; i < MOVE_STEPS; ++i)
      if (to[i] >= 0) *reinterpret_cast<uint4*>(dst + to[i] * ds) = x[i];
  }
}

}  // namespace pg
}  // namespace sea
