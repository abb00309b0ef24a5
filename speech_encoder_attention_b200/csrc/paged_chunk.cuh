// paged_chunk.cuh -- attention of a chunk of new tokens over a paged K/V cache
// on Blackwell tensor cores (the definitions are in paged_step.cuh).
//
// For query tiles of more than 32 rows (a row is a token and one of the query
// heads that share a K/V head; up to 128 rows). Bound by the exponentials, one
// per (row, slot), as flash_attn_kernel is, whose roles and tensor-memory
// layout this kernel shares: 192 threads, two CTAs per SM.
//   warps 0-3  softmax, one thread per row; they also clear the values of slots
//              that no row of the tile sees and write the output.
//   warp 4     TMA producer: Q through a 4-D map (column, head, token,
//              sequence), K and V one copy per page.
//   warp 5     tcgen05.mma issuer: S = Q K^T, then O += P V.
// Two ways to deal out the work. Where units (sequence, head, query tile) even out
// over the SMs each CTA walks whole units, the ones at the end of the prompts, which
// see most, first, every other round in reverse order of the CTAs. Elsewhere the key
// tiles of all units are cut into equal parts as in paged_step_kernel, and
// paged_combine_kernel merges what was cut.
//
// Measured on a B200, 20 heads: eight causal prompts of 1500 tokens 103 us = 448
// TFLOP/s over the visible pairs (exponential unit busy 49 % of the time, tensor
// pipe 24 %); four ragged chunks of up to 509 tokens over up to 6007 slots, 4
// K/V heads, 80 us = 449 TFLOP/s. The two CTAs of an SM leave two softmax warps per
// scheduler, whose chains (scores, max, exponentials, P) overlap only in part.
// Slower, each tried: two threads per row with 64 columns each (128 and 102 us),
// exponentials on half a tile while the other half's max is taken, part of the
// exponentials as polynomials.
#pragma once

#include "flash_attn.cuh"
#include "paged_common.cuh"
#include "paged_step.cuh"

namespace sea {
namespace pg {

// A unit as the producer hands it to the other roles, in shared memory: that
// keeps the walk's state out of the softmax threads' registers. The entry of
// unit n is free again once the producer may load Q of unit n + 4: Q of unit
// n + 2 has then been used up, so every role has left unit n.
struct ChunkUnit {
  int b, h, tok0, ntok;
  int kv, off;             // slots in use, position of the chunk's row 0
  int lo, hi, f;           // what any row of the tile sees
  int n_first, t_lo;       // key tile k is k (k < n_first) or t_lo + k - n_first
  int k0, k1;              // key tiles of this unit; k1 = 0 ends the walk
  int whole, slot;
};
constexpr int kUnitRing = 4;

// Likewise the hole bits of tile t + 4 replace those of tile t when S of tile t + 2
// is there, whose product waited for the softmax threads to read S of tile t + 1.
constexpr int kHoleRing = 4;

struct ChunkCfg : fa::CfgT<2> {
  static constexpr int OFF_HOLES = OFF_MISC + 8;
  static constexpr int OFF_UNITS = OFF_HOLES + 4 * kHoleRing;
  static constexpr int OFF_K_EMPTY = OFF_UNITS + kUnitRing * static_cast<int>(sizeof(ChunkUnit));
  static_assert(OFF_K_EMPTY % 8 == 0, "");
  static constexpr int SMEM_BYTES = 1024 + OFF_K_EMPTY + 8 * STAGES;
};

struct ChunkParams {
  StepParams s;
  int cut;             // 1: equal parts, 0: whole units
  int units;           // batch * kv_heads * q_tiles
  fa::DivC dv_group, dv_heads, dv_bh;  // by group, kv_heads, batch * kv_heads
};

// The units of a CTA: a Walk over its part, or one unit of each round of
// gridDim.x, with the last query tiles of all sequences and heads first.
struct ChunkWalk : Walk {
  int h, unit, round;
};

__device__ __forceinline__ void chunk_unit(const ChunkParams& p, ChunkWalk& w) {
  const Geo& g = p.s.g;
  const int back = fa::div_c(w.unit, p.dv_bh);
  const int bh = w.unit - back * (g.batch * g.kv_heads);
  w.qt = g.q_tiles - 1 - back;
  w.b = fa::div_c(bh, p.dv_heads);
  w.h = bh - w.b * g.kv_heads;
  w.s = seq_of(g, w.b);
  w.u = span_of(g, w.s, w.qt);
  w.k0 = 0;
  w.k1 = w.u.n;
  w.whole = true;
}

// One warp.
__device__ __forceinline__ bool chunk_start(const ChunkParams& p, ChunkWalk& w) {
  const Geo& g = p.s.g;
  if (p.cut) {
    w.h = blockIdx.x % g.kv_heads;
    return walk_start(g, w, blockIdx.x / g.kv_heads, p.s.parts);
  }
  w.round = 0;
  w.unit = blockIdx.x;
  if (w.unit >= p.units) return false;
  chunk_unit(p, w);
  return true;
}

__device__ __forceinline__ bool chunk_next(const ChunkParams& p, ChunkWalk& w) {
  if (p.cut) return walk_next(p.s.g, w);
  ++w.round;
  w.unit = w.round * gridDim.x + (w.round & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
  if (w.unit >= p.units) return false;  // of the last, incomplete round
  chunk_unit(p, w);
  return true;
}

__global__ void __launch_bounds__(ChunkCfg::THREADS, 2)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const ChunkParams cp) {
  using C = ChunkCfg;
  constexpr int ST = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + C::OFF_BARS;
  auto q_full = [&](int i) { return bar0 + 8u * i; };
  auto q_empty = [&](int i) { return bar0 + 8u * (2 + i); };
  auto k_full = [&](int s) { return bar0 + 8u * (4 + s); };
  auto v_full = [&](int s) { return bar0 + 8u * (4 + ST + s); };
  auto v_empty = [&](int s) { return bar0 + 8u * (4 + 2 * ST + s); };
  auto k_empty = [&](int s) { return sbase + C::OFF_K_EMPTY + 8u * s; };
  const uint32_t s_full = bar0 + 8u * (4 + 3 * ST);
  const uint32_t s_free = s_full + 8u;
  const uint32_t p_full = s_full + 16u;
  const uint32_t o_done = s_full + 24u;
  const uint32_t o_free = s_full + 32u;
  const uint32_t drain_bar = s_full + 40u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC + 4);
  volatile uint32_t* holes = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_HOLES);
  ChunkUnit* units = reinterpret_cast<ChunkUnit*>(smem + C::OFF_UNITS);
  const StepParams& p = cp.s;
  const Geo& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full(i), 1);
      mbar_init(q_empty(i), 1);
    }
    for (int s = 0; s < ST; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(v_full(s), 1);
      mbar_init(v_empty(s), 1);
      mbar_init(k_empty(s), 1);
    }
    mbar_init(s_full, 2);  // S, and what the producer wrote beside K
    mbar_init(s_free, 4);
    mbar_init(p_full, 4);
    mbar_init(o_done, 1);
    mbar_init(o_free, 4);
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (warp == C::MMA_WARP) {
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

  if (warp == C::PRODUCER_WARP) {
    // ---------------- TMA producer (whole warp: lane i loads page i of a tile) ----------------
    // K of a tile goes out before V of the tile before it: its stage is free once S
    // is computed, a softmax earlier than V's.
    const int n_pages = pages_per_tile(g);
    const uint32_t page_bytes = TILE_BYTES / n_pages;
    const uint32_t q_bytes = static_cast<uint32_t>(g.tok_per_tile * g.group) * DH * 2;
    int qn = 0, it = 0;
    ChunkWalk w;
    PageLoad lv{false, 0};  // of the V tile that is due, its head's column and bytes
    int v_col = 0;
    uint32_t v_bytes = 0;
    auto load_v = [&](int t) {
      const int st = t % ST;
      if (!__all_sync(0xffffffffu, mbar_wait(v_empty(st), ((t / ST) & 1) ^ 1u, wc))) return false;
      if (lane == 0) mbar_arrive_expect_tx(v_full(st), v_bytes);
      __syncwarp();
      if (lv.load) tma_load_2d(sbase + C::OFF_V + st * TILE_BYTES + lane * page_bytes, &tm_v, v_full(st), v_col, lv.row);
      return true;
    };
    int vn = 0;  // V tiles loaded
    bool more = chunk_start(cp, w), ok = true;
    for (; more; more = ok && chunk_next(cp, w)) {
      if (w.k1 <= w.k0) {  // no row sees anything (whole units only)
        zero_rows(p, w.b, w.h, w.u.tok0, min(w.u.tok0 + g.tok_per_tile, g.t_q));
        continue;
      }
      const int qb = qn & 1;
      ok = __all_sync(0xffffffffu, mbar_wait(q_empty(qb), ((qn >> 1) & 1) ^ 1u, wc));
      if (!ok) break;
      if (lane == 0) {
        ChunkUnit& u = units[qn % kUnitRing];
        u.b = w.b;
        u.h = w.h;
        u.tok0 = w.u.tok0;
        u.ntok = w.u.ntok;
        u.kv = w.s.kv;
        u.off = w.s.off;
        u.lo = w.u.lo;
        u.hi = w.u.hi;
        u.f = w.u.f;
        u.n_first = w.u.n_first;
        u.t_lo = w.u.t_lo;
        u.k0 = w.k0;
        u.k1 = w.k1;
        u.whole = w.whole;
        u.slot = w.slot;
        mbar_arrive_expect_tx(q_full(qb), q_bytes);
        tma_load_4d(sbase + C::OFF_Q + qb * TILE_BYTES, &tm_q, q_full(qb), 0, w.h * g.group, w.u.tok0, w.b);
      }
      ++qn;
      for (int k = w.k0; k < w.k1; ++k, ++it) {
        const int st = it % ST;
        PageLoad l{false, 0};
        if (lane < n_pages) l = page_of_tile(g, w.b, w.u, w.u.tile(k), lane);
        const uint32_t loaded = __ballot_sync(0xffffffffu, l.load);
        ok = __all_sync(0xffffffffu, mbar_wait(k_empty(st), ((it / ST) & 1) ^ 1u, wc));
        if (!ok) break;
        const uint32_t bytes = __popc(loaded) * page_bytes;
        if (lane == 0) {
          holes[it % kHoleRing] = hole_bits(g, loaded);
          mbar_arrive_expect_tx(k_full(st), bytes);
        }
        __syncwarp();
        if (l.load) tma_load_2d(sbase + C::OFF_K + st * TILE_BYTES + lane * page_bytes, &tm_k, k_full(st), w.h * DH, l.row);
        if (it > vn) {
          ok = load_v(vn);
          if (!ok) {
            ++it;
            break;
          }
          ++vn;
        }
        lv = l;
        v_col = w.h * DH;
        v_bytes = bytes;
      }
    }
    if (ok && it > vn) {
      ok = load_v(vn);
      vn += ok ? 1 : 0;
    }
    if (ok && mbar_wait(q_empty(qn & 1), ((qn >> 1) & 1) ^ 1u, wc) && lane == 0) {  // the end of the walk
      units[qn % kUnitRing].k1 = 0;
      mbar_arrive(q_full(qn & 1));
    }
    // Let the last copies land before the CTA may exit.
    if (qn > 0) mbar_wait_drain(q_full((qn - 1) & 1), ((qn - 1) >> 1) & 1, p.limit_ns);
    for (int i = max(0, it - ST); i < it; ++i) mbar_wait_drain(k_full(i % ST), (i / ST) & 1, p.limit_ns);
    for (int i = max(0, vn - ST); i < vn; ++i) mbar_wait_drain(v_full(i % ST), (i / ST) & 1, p.limit_ns);
  } else if (warp == C::MMA_WARP) {
    if (lane == 0) {
      // ---------------- MMA issuer (as in flash_attn_kernel) ----------------
      constexpr uint32_t idesc_s = idesc_f16_f32(fa::BQ, BKV, 0, 0);  // Q, K both K-major
      constexpr uint32_t idesc_o = idesc_f16_f32(fa::BQ, DH, 0, 1);   // P K-major (TMEM), V MN-major
      const uint64_t q_desc0 = smem_desc_sw128(sbase + C::OFF_Q, 16, 1024);
      const uint64_t k_desc0 = smem_desc_sw128(sbase + C::OFF_K, 16, 1024);
      const uint64_t v_desc0 = smem_desc_sw128(sbase + C::OFF_V, TILE_BYTES, 1024);
      constexpr uint64_t kTileUnits = TILE_BYTES >> 4;
      const uint32_t s_t = tmem_base + C::S_COL, o_t = tmem_base + C::O_COL, p_t = tmem_base + C::P_COL;
      int qn = 0, it = 0;
      bool ok = true;
      auto issue_pv = [&](int t, bool first) -> bool {
        const int st = t % ST;
        if (!mbar_wait(v_full(st), (t / ST) & 1, wc)) return false;
        if (first && qn > 1 && !mbar_wait(o_free, (qn - 2) & 1, wc)) return false;
        if (!mbar_wait(p_full, t & 1, wc)) return false;
        tc_fence_after();
        const uint64_t vd = v_desc0 + st * kTileUnits;
#pragma unroll
        for (int kk = 0; kk < BKV / 16; ++kk)
          mma_f16_ts(o_t, p_t + kk * 8, vd + kk * 128, idesc_o, (!first || kk > 0) ? 1u : 0u);
        mma_commit(o_done);
        mma_commit(v_empty(st));
        return true;
      };
      while (ok) {
        const int qb = qn & 1;
        if (!mbar_wait(q_full(qb), (qn >> 1) & 1, wc)) break;
        const int k0 = units[qn % kUnitRing].k0, k1 = units[qn % kUnitRing].k1;
        if (k1 == 0) break;
        ++qn;
        const uint64_t qd = q_desc0 + qb * kTileUnits;
        for (int k = k0; k < k1; ++k, ++it) {
          const int st = it % ST;
          if (!mbar_wait(k_full(st), (it / ST) & 1, wc) || (it > 0 && !mbar_wait(s_free, (it - 1) & 1, wc))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint64_t kd = k_desc0 + st * kTileUnits;
#pragma unroll
          for (int kk = 0; kk < DH / 16; ++kk) mma_f16_ss(s_t, qd + kk * 2, kd + kk * 2, idesc_s, kk > 0 ? 1u : 0u);
          mbar_arrive(s_full);
          mma_commit(s_full);
          mma_commit(k_empty(st));
          if (k > k0 && !issue_pv(it - 1, k == k0 + 1)) {
            ok = false;
            break;
          }
        }
        if (!ok || !issue_pv(it - 1, k1 == k0 + 1)) break;
        mma_commit(q_empty(qb));
      }
      mma_commit(drain_bar);
      mbar_wait_drain(drain_bar, 0, p.limit_ns);
    }
  } else {
    // ---------------- softmax / correction / epilogue ----------------
    const uint32_t lane_field = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t s_tmem = tmem_base + C::S_COL + lane_field;
    const uint32_t o_tmem = tmem_base + C::O_COL + lane_field;
    const uint32_t p_tmem = tmem_base + C::P_COL + lane_field;
    const float sl2 = p.scale_log2;
    const int row = warp * 32 + lane;          // row of the tile == tensor-memory lane
    const int tok_r = fa::div_c(row, cp.dv_group);  // its token within the tile
    const int head_r = row - tok_r * g.group;
    int it = 0;
    bool ok = true;
    for (int n = 0; ok; ++n) {
      if (!mbar_wait(q_full(n & 1), (n >> 1) & 1, wc)) break;
      const ChunkUnit& u = units[n % kUnitRing];
      const int k0 = u.k0, k1 = u.k1;
      if (k1 == 0) break;
      const bool row_ok = tok_r < u.ntok;
      const RowSpan rs = row_ok ? row_span(g, Seq{0, u.kv, 0}, u.tok0 + tok_r + u.off) : RowSpan{0, 0, 0};
      const int n_first = u.n_first, t_lo = u.t_lo;
      float m_run = -INFINITY, l_run = 0.f;
      for (int k = k0; k < k1; ++k) {
        const int st = it % ST;
        if (!mbar_wait(s_full, it & 1, wc)) {
          ok = false;
          break;
        }
        const uint32_t hole = holes[it % kHoleRing];
        tc_fence_after();
        float s[BKV];
        {
          uint32_t r[BKV];
          tmem_ld128(s_tmem, r);
#pragma unroll
          for (int e = 0; e < BKV; ++e) s[e] = __uint_as_float(r[e]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free);

        const int kv0 = (k < n_first ? k : t_lo + k - n_first) * BKV;
        const int a = rs.lo - kv0, bnd = rs.hi - kv0, fb = rs.f - kv0;
        // Hidden: [fb, a) and from max(bnd, fb) on. Three separate loops: one
        // with both conditions spills.
        if (row_ok && !((a <= 0 && bnd >= BKV) || fb >= BKV)) {
          const int top = max(bnd, fb);
          if (a > max(fb, 0)) {
#pragma unroll
            for (int e = 0; e < BKV; ++e)
              if (e >= fb && e < a) s[e] = -INFINITY;
          }
          if (top < BKV / 2) {
#pragma unroll
            for (int e = 0; e < BKV / 2; ++e)
              if (e >= top) s[e] = -INFINITY;
          }
#pragma unroll
          for (int e = BKV / 2; e < BKV; ++e)
            if (e >= top) s[e] = -INFINITY;
        }
        if (hole != 0) {
#pragma unroll
          for (int e = 0; e < BKV; ++e)
            if ((hole >> (e / GRANULE)) & 1u) s[e] = -INFINITY;
        }
        float mx4[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) mx4[i] = fmaxf(s[i], s[BKV - 4 + i]);
#pragma unroll
        for (int e = 4; e < BKV - 4; e += 8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) mx4[i] = fmax3(mx4[i], s[e + i], s[e + 4 + i]);
        }
        const float mx_l2 = fmaxf(fmax3(mx4[0], mx4[1], mx4[2]), mx4[3]) * sl2;
        const bool grow = mx_l2 > m_run + RESCALE_LIMIT;
        const float m_new = grow ? mx_l2 : m_run;
        const float alpha = grow ? ex2_approx(m_run - m_new) : 1.f;
        const bool first = k == k0;
        if (!first) {
          if (!mbar_wait(o_done, (it - 1) & 1, wc)) {
            ok = false;
            break;
          }
          tc_fence_after();
        }
        {
          const float ref = m_new == -INFINITY ? 0.f : m_new;
          const uint64_t sl2x2 = f2_pack(sl2, sl2), negm2 = f2_pack(-ref, -ref);
          uint64_t acc2[2] = {0ull, 0ull};
#pragma unroll
          for (int c = 0; c < BKV / 16; ++c) {
            uint32_t pk[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float x0, x1;
              f2_unpack(f2_fma(f2_pack(s[16 * c + 2 * i], s[16 * c + 2 * i + 1]), sl2x2, negm2), x0, x1);
              const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
              acc2[i & 1] = f2_add(acc2[i & 1], f2_pack(p0, p1));
              pk[i] = pack_half2(p0, p1);  // P in fp16 for the tensor cores; the sum is not rounded
            }
            tmem_st8_async(p_tmem + c * 8, pk);
          }
          tmem_wait_st();
          float sum0, sum1;
          f2_unpack(f2_add(acc2[0], acc2[1]), sum0, sum1);
          l_run = l_run * alpha + (sum0 + sum1);
        }
        if (!first && __any_sync(0xffffffffu, grow)) {
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t r[32];
            tmem_ld32(o_tmem + c * 32, r);
#pragma unroll
            for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
            tmem_st32(o_tmem + c * 32, r);
          }
        }
        // Values of slots that no row of the tile sees may be anything, and a
        // weight of zero does not silence NaN: they are cleared in shared memory.
        if (hole != 0 || !((kv0 >= u.lo && kv0 + BKV <= u.hi) || kv0 + BKV <= u.f)) {
          if (!mbar_wait(v_full(st), (it / ST) & 1, wc)) {
            ok = false;
            break;
          }
          for (int x = row; x < BKV * 8; x += C::SOFTMAX_THREADS) {
            const int j = x >> 3;
            if (((hole >> (j / GRANULE)) & 1u) || !((kv0 + j >= u.lo && kv0 + j < u.hi) || kv0 + j < u.f))
              *reinterpret_cast<uint4*>(smem + C::OFF_V + st * TILE_BYTES + x * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full);
        m_run = m_new;
        ++it;
      }
      if (!ok) break;

      // ---------------- epilogue ----------------
      if (!mbar_wait(o_done, (it - 1) & 1, wc)) break;
      tc_fence_after();
      const bool whole = u.whole != 0;
      const bool row_out = tok_r < g.tok_per_tile && u.tok0 + tok_r < g.t_q;  // valid or padding
      const int64_t out_row = static_cast<int64_t>(u.b) * g.t_q + u.tok0 + tok_r;
      const int head = u.h * g.group + head_r;
      __half* out = p.out + out_row * p.out_stride + head * DH;
      const float l_fin = row_ok ? l_run : 0.f;
      const RowEnd end = row_end(l_fin, m_run, whole && row_ok && p.sinks != nullptr ? __ldg(p.sinks + head) : -INFINITY);
      const float inv = end.inv;
      const int64_t part = (2 * static_cast<int64_t>(blockIdx.x) + u.slot) * p.rows_cap + row;
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t r[32];
        tmem_ld32(o_tmem + c * 32, r);
        if (c == 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(o_free);
        }
        if (whole) {
          if (!row_out) continue;
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint4 x;
            x.x = pack_half2(__uint_as_float(r[8 * v + 0]) * inv, __uint_as_float(r[8 * v + 1]) * inv);
            x.y = pack_half2(__uint_as_float(r[8 * v + 2]) * inv, __uint_as_float(r[8 * v + 3]) * inv);
            x.z = pack_half2(__uint_as_float(r[8 * v + 4]) * inv, __uint_as_float(r[8 * v + 5]) * inv);
            x.w = pack_half2(__uint_as_float(r[8 * v + 6]) * inv, __uint_as_float(r[8 * v + 7]) * inv);
            // a padding row's products may be NaN
            reinterpret_cast<uint4*>(out + c * 32)[v] = l_fin != 0.f ? x : make_uint4(0u, 0u, 0u, 0u);
          }
        } else if (row_ok) {
#pragma unroll
          for (int v = 0; v < 8; ++v)
            reinterpret_cast<float4*>(p.ws_o + part * DH + c * 32)[v] =
                make_float4(__uint_as_float(r[4 * v]), __uint_as_float(r[4 * v + 1]), __uint_as_float(r[4 * v + 2]),
                            __uint_as_float(r[4 * v + 3]));
        }
      }
      if (whole) {
        if (row_out && p.lse != nullptr)
          p.lse[out_row * g.n_heads + head] = end.lse;
      } else if (row_ok) {
        p.ws_ml[part] = make_float2(m_run, l_run);
      }
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == C::MMA_WARP) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

}  // namespace pg
}  // namespace sea
