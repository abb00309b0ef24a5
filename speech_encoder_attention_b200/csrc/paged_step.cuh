// paged_step.cuh -- attention of a few new tokens over a paged K/V cache.
//
//   o_i = sum_{j in A_i} e^{s_ij} v_j / (sum_{j in A_i} e^{s_ij} [+ e^{sink_h}]),
//   s_ij = scale <q_i, k_j>,  lse_i = ln of the denominator,
// for query tiles of at most 16 * MT rows (the tokens of a chunk times the
// query heads that share a K/V head). Bound by reading K and V once.
//
// A 128-row tcgen05 tile would leave at least 96 rows idle and costs a chain
// of tensor-memory round trips per key tile; with so few rows each warp works
// on its own instead: 16-row mma.sync products straight from shared memory,
// P kept in registers, no step of one warp waiting for another inside a unit.
//   warp 4      producer: one TMA copy per page into a ring of key tiles
//               (128 slots of K and V, 128-byte swizzle); the warp reads 32
//               table entries at once (one tile's before each tile: 8.1 us
//               instead of 7.4 at 448 slots in 16-slot pages).
//   warps 0-3   warp w takes slots [32w, 32w + 32) of every key tile with a
//               running max, sum and output of its own; warp 0 merges the
//               four at the end of a unit.
// Two ways to deal out the work. Either the key tiles of all units are cut
// into equal parts, a CTA for each part and K/V head, two CTAs per SM; units that
// are cut leave partials that paged_combine_kernel merges. Or a unit has a cluster
// of 1 to 8 CTAs, each with an equal run of its tiles, merged through distributed
// shared memory, with no second launch and no workspace.
//
// Measured on a B200, 20 heads, one token each: 16 sequences of 3.1 to 8.2
// thousand slots 80 us = 5.9 TB/s of K and V, 0.90 of the copy rate (its TMA
// loads alone take 78 us); 48 sequences with a 1024-slot window and 5 K/V heads
// 16 us = 3.9 TB/s; one sequence in 64-slot pages 5.9 us at 448 slots, 8.0 us at
// 3000 (in 16-slot pages, with eight copies for K and for V per tile, 7.1 and 8.6).
// Registers: 16 rows fit without spills; 32 rows spill 232 bytes a thread where the
// line is cut and 36 bytes where it is not.
#pragma once

#include "paged_common.cuh"

namespace sea {
namespace pg {

// The exponent reference of a row moves only when its max grows by more than
// this (log2 units): p <= 2^15 fits fp16.
constexpr float RESCALE_LIMIT = 15.0f;

struct StepParams {
  Geo g;
  const __half* q;
  int64_t q_stride;
  float scale_log2;
  const float* sinks;
  __half* out;
  int64_t out_stride;
  float* lse;        // [batch * t_q, n_heads] or null
  float* ws_o;       // [2 * CTAs][rows_cap][64] unnormalised partial O
  float2* ws_ml;     // [2 * CTAs][rows_cap] (m in log2 units, l)
  int rows_cap;
  int parts;         // the line of key tiles is cut into this many; 0: a cluster per unit
  int cluster;       // CTAs of that cluster, at most 8
  uint32_t* err;
  uint64_t limit_ns;
};

template <int MT>
struct StepCfg {
  static constexpr int ROWS = 16 * MT;
  static constexpr int STAGES = MT == 1 ? 3 : 2;
  static constexpr int WARPS = 4;
  static constexpr int THREADS = 32 * (WARPS + 1);
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = STAGES * TILE_BYTES;
  static constexpr int MERGE_WARP = MT * (32 * 32 + 4 * 32);  // floats: O fragments, then m, l of two rows
  static constexpr int OFF_MERGE = 2 * STAGES * TILE_BYTES;
  static constexpr int OFF_BARS = OFF_MERGE + 3 * MERGE_WARP * 4;
  static constexpr int NUM_BARS = 2 * STAGES + 2;  // full, empty, merge_full, merge_empty
  static constexpr int OFF_HOLES = OFF_BARS + 8 * NUM_BARS;
  static constexpr int OFF_MISC = OFF_HOLES + 4 * STAGES;
  static constexpr int SMEM_BYTES = 1024 + OFF_MISC + 8;
};

// volatile keeps these between the waits on the tile's barriers; without a
// memory clobber the arithmetic may move around them.
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

// D (16 x 8, fp32) += A (16 x 16, fp16) B (16 x 8, fp16)
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// One warp: the rows of tokens [tok_a, tok_z) of one K/V head see nothing.
__device__ __forceinline__ void zero_rows(const StepParams& p, int b, int h, int tok_a, int tok_z) {
  const Geo& g = p.g;
  for (int x = threadIdx.x & 31; x < (tok_z - tok_a) * g.group * 8; x += 32) {
    const int r = x >> 3;
    const int64_t row = static_cast<int64_t>(b) * g.t_q + tok_a + r / g.group;
    const int head = h * g.group + r % g.group;
    reinterpret_cast<uint4*>(p.out + row * p.out_stride + head * DH)[x & 7] = make_uint4(0u, 0u, 0u, 0u);
    if (p.lse != nullptr && (x & 7) == 0) p.lse[row * g.n_heads + head] = -INFINITY;
  }
}

template <int MT, bool CUT>
__global__ void __launch_bounds__(StepCfg<MT>::THREADS, 2)
    paged_step_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const StepParams p) {
  using C = StepCfg<MT>;
  constexpr int ST = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::OFF_BARS;
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (ST + s); };
  const uint32_t merge_full = bar0 + 8u * (2 * ST), merge_empty = merge_full + 8u;
  volatile uint32_t* holes = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_HOLES);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC);
  const Geo& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < ST; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), C::WARPS);
    }
    mbar_init(merge_full, C::WARPS - 1);
    mbar_init(merge_empty, 1);
    *abort_flag = 0u;
    fence_barrier_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  const WaitCtl wc{abort_flag, p.err, p.limit_ns};

  const int h = (CUT ? blockIdx.x : blockIdx.x / p.cluster) % g.kv_heads;
  // This CTA's partial for its cluster, in the place of warp 1's for warp 0.
  float* part_of_cta = reinterpret_cast<float*>(smem + C::OFF_MERGE);
  Walk w;
  bool any;
  if constexpr (CUT) {
    any = walk_start(g, w, blockIdx.x / g.kv_heads, p.parts);
  } else {
    const int unit = blockIdx.x / p.cluster, rank = blockIdx.x - unit * p.cluster;
    w.b = unit / g.kv_heads;
    w.qt = 0;
    w.s = seq_of(g, w.b);
    w.u = span_of(g, w.s, 0);
    w.k0 = static_cast<int>(static_cast<long long>(w.u.n) * rank / p.cluster);
    w.k1 = static_cast<int>(static_cast<long long>(w.u.n) * (rank + 1) / p.cluster);
    w.whole = p.cluster == 1;
    any = w.k1 > w.k0;
    // rows that see nothing: all of them, or the padding behind the valid ones
    if (warp == 0 && rank == 0) zero_rows(p, w.b, h, w.u.tok0 + (w.u.n > 0 ? w.u.ntok : 0), g.t_q);
    if (warp == 0 && !any) {  // an empty partial
#pragma unroll
      for (int i = 0; i < MT * 4; ++i) part_of_cta[MT * 1024 + i * 32 + lane] = (i & 2) ? 0.f : -INFINITY;
    }
  }
  // the next unit of this CTA
  auto next_unit = [&]() { return CUT && walk_next(g, w); };
  if (any && warp == C::WARPS) {
    // ---------------- producer ----------------
    const int n_pages = pages_per_tile(g);
    const uint32_t page_bytes = TILE_BYTES / n_pages;
    PageLoad ahead{false, 0};
    int it = 0;
    bool ok = true;
    do {
      for (int k = w.k0; k < w.k1 && ok; ++k, ++it) {
        const int st = it % ST;
        const int x = (k - w.k0) & (32 / n_pages - 1);
        if (x == 0) ahead = pages_ahead(g, w.b, w.u, k, w.k1, n_pages);
        const PageLoad l = page_from(ahead, x, n_pages);
        const uint32_t loaded = __ballot_sync(0xffffffffu, l.load);
        ok = mbar_wait(empty(st), ((it / ST) & 1) ^ 1u, wc);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        if (lane == 0) {
          holes[st] = hole_bits(g, loaded);
          mbar_arrive_expect_tx(full(st), 2u * __popc(loaded) * page_bytes);
        }
        __syncwarp();
        if (l.load) {
          tma_load_2d(sbase + C::OFF_K + st * TILE_BYTES + lane * page_bytes, &tm_k, full(st), h * DH, l.row);
          tma_load_2d(sbase + C::OFF_V + st * TILE_BYTES + lane * page_bytes, &tm_v, full(st), h * DH, l.row);
        }
      }
    } while (ok && next_unit());
    // Let the last copies land before the CTA may exit.
    for (int i = max(0, it - ST); i < it; ++i) mbar_wait_drain(full(i % ST), (i / ST) & 1, p.limit_ns);
  } else if (any) {
    // ---------------- consumers ----------------
    const int r4 = lane >> 2, c2 = (lane & 3) * 2;
    const float sl2 = p.scale_log2;
    float* merge_buf = reinterpret_cast<float*>(smem + C::OFF_MERGE);
    int it = 0, unit = 0;
    bool ok = true;
    do {
      const int rows = w.u.ntok * g.group;
      // Q fragments straight from memory (2 KB per unit), and what each row sees.
      uint32_t qf[MT][4][4];
      RowSpan rs[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r = 16 * m + 8 * e + r4;
          const bool valid = r < rows;
          const int tok = w.u.tok0 + r / g.group;
          const int head = h * g.group + r % g.group;
          rs[m][e] = valid ? row_span(g, w.s, tok + w.s.off) : RowSpan{0, 0, 0};
          const __half* src = p.q + (static_cast<int64_t>(w.b) * g.t_q + tok) * p.q_stride + head * DH + c2;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            qf[m][kk][e] = valid ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * kk)) : 0u;
            qf[m][kk][2 + e] = valid ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * kk + 8)) : 0u;
          }
        }
      }
      // Slots that every valid row sees need no mask.
      const RowSpan r_first = row_span(g, w.s, w.u.tok0 + w.s.off);
      const RowSpan r_last = row_span(g, w.s, w.u.tok0 + w.u.ntok - 1 + w.s.off);
      const int all_lo = r_last.lo, all_hi = r_first.hi, all_f = r_first.f;
      float o[MT][8][4];
      float m_run[MT][2], l_run[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int d = 0; d < 8; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[m][d][e] = 0.f;
        m_run[m][0] = m_run[m][1] = -INFINITY;
        l_run[m][0] = l_run[m][1] = 0.f;
      }
      for (int k = w.k0; k < w.k1; ++k, ++it) {
        const int st = it % ST;
        if (!mbar_wait(full(st), (it / ST) & 1, wc)) {
          ok = false;
          break;
        }
        const uint32_t sk = sbase + C::OFF_K + st * TILE_BYTES + warp * 32 * 128;
        const uint32_t sv = sbase + C::OFF_V + st * TILE_BYTES + warp * 32 * 128;
        const int j0 = w.u.tile(k) * BKV + warp * 32;  // this warp's first slot
        const uint32_t hole = (holes[st] >> (2 * warp)) & 3u;
        // S = Q K^T, 32 slots in four groups of 8
        float s[MT][4][4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
          uint32_t b[2][4];
          const int row = 8 * n + (lane & 7);
          const int ch = lane >> 3;
          ldmatrix_x4(sk + row * 128 + ((ch ^ (row & 7)) << 4), b[0]);
          ldmatrix_x4(sk + row * 128 + (((ch + 4) ^ (row & 7)) << 4), b[1]);
#pragma unroll
          for (int m = 0; m < MT; ++m) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[m][n][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_16816(s[m][n], qf[m][kk], b[kk >> 1][2 * (kk & 1)], b[kk >> 1][2 * (kk & 1) + 1]);
          }
        }
        const bool edge = hole != 0 || !((j0 >= all_lo && j0 + 32 <= all_hi) || j0 + 32 <= all_f);
        // Values of slots no row sees (behind the end, outside the window, in
        // a page that was not loaded) may be anything: they are cleared.
        uint32_t keep[2][2] = {{~0u, ~0u}, {~0u, ~0u}};
        if (edge) {
#pragma unroll
          for (int n = 0; n < 4; ++n) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int j = j0 + 8 * n + c2 + x;
              const bool gone = (hole >> (n >> 1)) & 1u;
              if (gone || unseen(w.u, j)) keep[n >> 1][n & 1] &= x ? 0x0000FFFFu : 0xFFFF0000u;
#pragma unroll
              for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const RowSpan& r = rs[m][e];
                  if (gone || !((j >= r.lo && j < r.hi) || j < r.f)) s[m][n][2 * e + x] = -INFINITY;
                }
            }
          }
        }
        // A row's reference moves only when one of its scores would pass 2^15;
        // whether any does takes one vote, and the row's max (two shuffles) only
        // then.
        float top[MT][2];
        bool passes = false;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float a = fmax3(s[m][0][2 * e], s[m][0][2 * e + 1], s[m][1][2 * e]);
            const float c = fmax3(s[m][1][2 * e + 1], s[m][2][2 * e], s[m][2][2 * e + 1]);
            top[m][e] = fmaxf(fmax3(a, c, s[m][3][2 * e]), s[m][3][2 * e + 1]) * sl2;
            passes |= top[m][e] > m_run[m][e] + RESCALE_LIMIT;
          }
        if (__any_sync(0xffffffffu, passes)) {
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mx = fmaxf(top[m][e], __shfl_xor_sync(0xffffffffu, top[m][e], 1));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
              if (mx > m_run[m][e] + RESCALE_LIMIT) {  // the same in the row's four threads
                const float alpha = ex2_approx(m_run[m][e] - mx);
                l_run[m][e] *= alpha;
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                  o[m][d][2 * e] *= alpha;
                  o[m][d][2 * e + 1] *= alpha;
                }
                m_run[m][e] = mx;
              }
            }
        }
        uint32_t pf[MT][2][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float ref = m_run[m][e] == -INFINITY ? 0.f : m_run[m][e];
            float sum[2] = {0.f, 0.f};
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              const float p0 = ex2_approx(fmaf(s[m][n][2 * e], sl2, -ref));
              const float p1 = ex2_approx(fmaf(s[m][n][2 * e + 1], sl2, -ref));
              sum[n & 1] += p0 + p1;
              // P is rounded to fp16 for the tensor cores; the sum is not
              pf[m][n >> 1][(n & 1) * 2 + e] = pack_half2(p0, p1);
            }
            l_run[m][e] += sum[0] + sum[1];
          }
        }
        // O += P V
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
#pragma unroll
          for (int dp = 0; dp < 4; ++dp) {
            uint32_t b[4];
            const int row = 16 * kk + (lane & 15);
            const int ch = 2 * dp + (lane >> 4);
            ldmatrix_x4_trans(sv + row * 128 + ((ch ^ (row & 7)) << 4), b);
            if (edge) {
              b[0] &= keep[kk][0];
              b[1] &= keep[kk][1];
              b[2] &= keep[kk][0];
              b[3] &= keep[kk][1];
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
              mma_16816(o[m][2 * dp], pf[m][kk], b[0], b[1]);
              mma_16816(o[m][2 * dp + 1], pf[m][kk], b[2], b[3]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(st));
      }
      if (!ok) break;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          l_run[m][e] += __shfl_xor_sync(0xffffffffu, l_run[m][e], 1);
          l_run[m][e] += __shfl_xor_sync(0xffffffffu, l_run[m][e], 2);
        }
      // Warps 1-3 hand their partials to warp 0 in fragment order.
      if (warp != 0) {
        if (unit > 0 && !mbar_wait(merge_empty, (unit - 1) & 1, wc)) break;
        float* dst = merge_buf + (warp - 1) * C::MERGE_WARP;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
          for (int i = 0; i < 32; ++i) dst[(m * 32 + i) * 32 + lane] = o[m][i >> 2][i & 3];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            dst[MT * 1024 + (m * 4 + e) * 32 + lane] = m_run[m][e];
            dst[MT * 1024 + (m * 4 + 2 + e) * 32 + lane] = l_run[m][e];
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(merge_full);
      } else {
        if (!mbar_wait(merge_full, unit & 1, wc)) break;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float mw[3], lw[3];
            float mx = l_run[m][e] != 0.f ? m_run[m][e] : -INFINITY;
#pragma unroll
            for (int i = 0; i < 3; ++i) {
              const float* src = merge_buf + i * C::MERGE_WARP + MT * 1024;
              mw[i] = src[(m * 4 + e) * 32 + lane];
              lw[i] = src[(m * 4 + 2 + e) * 32 + lane];
              if (lw[i] != 0.f) mx = fmaxf(mx, mw[i]);
            }
            const float own = l_run[m][e] != 0.f ? ex2_approx(m_run[m][e] - mx) : 0.f;
            float l = l_run[m][e] * own;
#pragma unroll
            for (int d = 0; d < 8; ++d) {
              o[m][d][2 * e] = own != 0.f ? o[m][d][2 * e] * own : 0.f;
              o[m][d][2 * e + 1] = own != 0.f ? o[m][d][2 * e + 1] * own : 0.f;
            }
#pragma unroll
            for (int i = 0; i < 3; ++i) {
              if (lw[i] != 0.f) {
                const float wgt = ex2_approx(mw[i] - mx);
                l += lw[i] * wgt;
                const float* src = merge_buf + i * C::MERGE_WARP + m * 1024;
#pragma unroll
                for (int d = 0; d < 8; ++d) {
                  o[m][d][2 * e] += src[(d * 4 + 2 * e) * 32 + lane] * wgt;
                  o[m][d][2 * e + 1] += src[(d * 4 + 2 * e + 1) * 32 + lane] * wgt;
                }
              }
            }
            if (!CUT && !w.whole) {
              part_of_cta[MT * 1024 + (m * 4 + e) * 32 + lane] = mx;
              part_of_cta[MT * 1024 + (m * 4 + 2 + e) * 32 + lane] = l;
            }
            const int r = 16 * m + 8 * e + r4;
            if (r < rows) {
              if (w.whole) {
                const int64_t row = static_cast<int64_t>(w.b) * g.t_q + w.u.tok0 + r / g.group;
                const int head = h * g.group + r % g.group;
                const RowEnd end = row_end(l, mx, p.sinks != nullptr ? __ldg(p.sinks + head) : -INFINITY);
                __half* dst = p.out + row * p.out_stride + head * DH + c2;
#pragma unroll
                for (int d = 0; d < 8; ++d)
                  *reinterpret_cast<uint32_t*>(dst + 8 * d) =
                      l != 0.f ? pack_half2(o[m][d][2 * e] * end.inv, o[m][d][2 * e + 1] * end.inv) : 0u;
                if (p.lse != nullptr && c2 == 0) p.lse[row * g.n_heads + head] = end.lse;
              } else if constexpr (CUT) {
                const int64_t part = (2 * static_cast<int64_t>(blockIdx.x) + w.slot) * p.rows_cap + r;
                float2* dst = reinterpret_cast<float2*>(p.ws_o + part * DH + c2);
#pragma unroll
                for (int d = 0; d < 8; ++d) dst[4 * d] = make_float2(o[m][d][2 * e], o[m][d][2 * e + 1]);
                if (c2 == 0) p.ws_ml[part] = make_float2(mx, l);
              }
            }
          }
        }
        if (!CUT && !w.whole) {
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 32; ++i) part_of_cta[(m * 32 + i) * 32 + lane] = o[m][i >> 2][i & 3];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(merge_empty);
      }
      ++unit;
    } while (next_unit());
  }
  __syncthreads();
  if (CUT || p.cluster == 1) return;
  // The cluster's partials of the unit, merged as paged_combine_kernel does;
  // rank r writes every cluster-th group of 8 columns, starting with its own.
  cluster_sync();
  if (warp == 0 && w.u.n > 0) {
    const int rank = static_cast<int>(cluster_ctarank());
    const int r4 = lane >> 2, c2 = (lane & 3) * 2;
    const uint32_t base = smem_u32(part_of_cta) + lane * 4;
    auto load = [&](int i, int at) {
      float v;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(base + at * 128, i)));
      return v;
    };
    const int rows = w.u.ntok * g.group;
#pragma unroll 1
    for (int me = 0; me < 2 * MT && 8 * me < rows; ++me) {  // rows 8 me + lane / 4
      const int m = me >> 1, e = me & 1;
      const int r = 8 * me + r4;
      // all of a row's loads before the first use: one round trip
      float li[8], mi[8], x[8], y[8];
      auto load_o = [&](int d) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] = i < p.cluster ? load(i, m * 32 + d * 4 + 2 * e) : 0.f;
          y[i] = i < p.cluster ? load(i, m * 32 + d * 4 + 2 * e + 1) : 0.f;
        }
      };
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        li[i] = i < p.cluster ? load(i, MT * 32 + m * 4 + 2 + e) : 0.f;
        mi[i] = i < p.cluster ? load(i, MT * 32 + m * 4 + e) : 0.f;
      }
      load_o(rank);
      float mx = -INFINITY, l = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (li[i] != 0.f) mx = fmaxf(mx, mi[i]);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        mi[i] = li[i] != 0.f ? ex2_approx(mi[i] - mx) : 0.f;  // now the part's weight
        if (li[i] != 0.f) l += li[i] * mi[i];
      }
      const int64_t row = static_cast<int64_t>(w.b) * g.t_q + w.u.tok0 + r / g.group;
      const int head = h * g.group + r % g.group;
      const RowEnd end = row_end(l, mx, p.sinks != nullptr && r < rows ? __ldg(p.sinks + head) : -INFINITY);
      for (int d = rank; d < 8; d += p.cluster) {
        if (d != rank) load_o(d);
        float a = 0.f, c = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (mi[i] != 0.f) {
            a += x[i] * mi[i];
            c += y[i] * mi[i];
          }
        }
        if (r < rows)
          *reinterpret_cast<uint32_t*>(p.out + row * p.out_stride + head * DH + c2 + 8 * d) =
              l != 0.f ? pack_half2(a * end.inv, c * end.inv) : 0u;
      }
      if (rank == 0 && c2 == 0 && r < rows && p.lse != nullptr) p.lse[row * g.n_heads + head] = end.lse;
    }
  }
  cluster_sync();  // no CTA leaves while another still reads its partial
}

// Merges the partials of cut units and writes the rows that no CTA holds.
//   M = max_s m_s,  L = sum_s l_s 2^(m_s - M) [+ 2^(sink log2e - M)],
//   o = sum_s O_s 2^(m_s - M) / L.
// Rows without a visible slot (l = 0), and padding rows, are zero with lse = -inf.
// Bound by its latency (the partials lie in L2), so a block of 256 threads takes
// `rows` rows of a unit, 8 threads per row and group of parts, each 8 columns:
// the 32 / rows groups of a row read their parts at the same time and meet in
// shared memory.
constexpr int COMBINE_THREADS = 256;

__global__ void __launch_bounds__(COMBINE_THREADS, 4) paged_combine_kernel(const StepParams p, int rows_log2) {
  __shared__ long long sum_all[8], sum_before[8];
  __shared__ float sh_o[32][68];   // [row x group][64 columns, padded]
  __shared__ float2 sh_ml[32];
  const Geo& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  griddep_wait();
  griddep_launch_dependents();
  const int unit = blockIdx.x;
  const int qt = unit % g.q_tiles;
  const int h = unit / g.q_tiles % g.kv_heads;
  const int b = unit / g.q_tiles / g.kv_heads;
  const Seq s = seq_of(g, b);
  const Span u = span_of(g, s, qt);
  const int rows_out = min(g.tok_per_tile, g.t_q - u.tok0) * g.group;  // valid and padding rows
  const int rows = u.n > 0 ? u.ntok * g.group : 0;
  // Where the unit lies in the line of key tiles: every warp takes a share of
  // the (sequence, query tile) entries.
  long long all = 0, before = 0;
  const int entries = g.batch * g.q_tiles;
  for (int e = threadIdx.x; e < entries; e += COMBINE_THREADS) {
    const int eb = e / g.q_tiles, eq = e - eb * g.q_tiles;
    const int n = span_of(g, seq_of(g, eb), eq).n;
    all += n;
    if (eb < b || (eb == b && eq < qt)) before += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, o);
    before += __shfl_xor_sync(0xffffffffu, before, o);
  }
  if (lane == 0) {
    sum_all[warp] = all;
    sum_before[warp] = before;
  }
  __syncthreads();
  all = before = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    all += sum_all[i];
    before += sum_before[i];
  }
  const long long per = share_of(all, p.parts);
  const int c0 = static_cast<int>(before / per);
  const int c1 = rows > 0 ? static_cast<int>((before + u.n - 1) / per) : c0;
  const bool c0_first = before == per * c0;
  const bool cut = c1 > c0;

  const int block_rows = 1 << rows_log2, groups = 32 >> rows_log2;
  const int x = threadIdx.x >> 3;             // row x group
  const int grp = x >> rows_log2;
  const int r = blockIdx.y * block_rows + (x & (block_rows - 1));
  const int c8 = (threadIdx.x & 7) * 8;
  float m = -INFINITY, l = 0.f;
  float o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = 0.f;
  if (cut && r < rows) {
    for (int c = c0 + grp; c <= c1; c += groups) {
      const int64_t cta = static_cast<int64_t>(c) * g.kv_heads + h;
      const int64_t at = (2 * cta + (c == c0 && !c0_first ? 1 : 0)) * p.rows_cap + r;
      const float2 ml = p.ws_ml[at];
      const float4* src = reinterpret_cast<const float4*>(p.ws_o + at * DH + c8);
      const float4 a = src[0], d = src[1];
      if (ml.y != 0.f) {
        const float m_new = fmaxf(m, ml.x);
        const float keep = ex2_approx(m - m_new), wgt = ex2_approx(ml.x - m_new);
        l = l * keep + ml.y * wgt;
        o[0] = o[0] * keep + a.x * wgt;
        o[1] = o[1] * keep + a.y * wgt;
        o[2] = o[2] * keep + a.z * wgt;
        o[3] = o[3] * keep + a.w * wgt;
        o[4] = o[4] * keep + d.x * wgt;
        o[5] = o[5] * keep + d.y * wgt;
        o[6] = o[6] * keep + d.z * wgt;
        o[7] = o[7] * keep + d.w * wgt;
        m = m_new;
      }
    }
  }
  if (groups > 1) {
    reinterpret_cast<float4*>(&sh_o[x][c8])[0] = make_float4(o[0], o[1], o[2], o[3]);
    reinterpret_cast<float4*>(&sh_o[x][c8])[1] = make_float4(o[4], o[5], o[6], o[7]);
    if (c8 == 0) sh_ml[x] = make_float2(m, l);
    __syncthreads();
    if (grp != 0) return;
    // By l, not by m: a group whose scores were all NaN has m = -inf and l = NaN,
    // and NaN is what comes of it.
    float mx = -INFINITY;
    for (int i = 0; i < groups; ++i) mx = fmaxf(mx, sh_ml[(i << rows_log2) + (x & (block_rows - 1))].x);
    l = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = 0.f;
    const int used = min(groups, c1 - c0 + 1);
    for (int i = 0; i < used; ++i) {
      const int y = (i << rows_log2) + (x & (block_rows - 1));
      const float2 ml = sh_ml[y];
      if (ml.y == 0.f) continue;
      const float wgt = ex2_approx(ml.x - mx);
      l += ml.y * wgt;
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] += sh_o[y][c8 + j] * wgt;
    }
    m = mx;
  }
  if (r >= rows_out || (r < rows && !cut)) return;  // rows of whole units are written already
  const int64_t row = static_cast<int64_t>(b) * g.t_q + u.tok0 + r / g.group;
  const int head = h * g.group + r % g.group;
  const RowEnd end = row_end(l, m, p.sinks != nullptr ? __ldg(p.sinks + head) : -INFINITY);
  const float inv = end.inv;
  *reinterpret_cast<uint4*>(p.out + row * p.out_stride + head * DH + c8) =
      make_uint4(pack_half2(o[0] * inv, o[1] * inv), pack_half2(o[2] * inv, o[3] * inv),
                 pack_half2(o[4] * inv, o[5] * inv), pack_half2(o[6] * inv, o[7] * inv));
  if (p.lse != nullptr && c8 == 0) p.lse[row * g.n_heads + head] = end.lse;
}

}  // namespace pg
}  // namespace sea
