// paged_weights.cuh -- the attention weight that a chunk's query rows put on
// each slot of a paged cache, summed over rows and query heads:
//
//   w_out[b, j] = w_in[b, j] + sum_{i, h : j in A_i} e^{s_ij - lse_ih}.
//
// With few query rows bound by reading K; with many, by one exponential per
// (row, head, slot). A CTA owns 128 slots of one sequence and computes
// S^T = K Q^T on tcgen05 tiles: 128 slots x N rows, N = 16 or 32 for a step or
// a drafted block, 128 for a longer chunk. A slot is a tensor-memory lane, so its
// weights are summed by one thread, in a fixed order, with no shuffles; the
// normaliser of a row is a column's constant that every thread reads from
// shared memory.
//   warps 0-3  one thread per slot: e^{s - lse} and the sums.
//   warp 4     producer: K tiles of the CTA's K/V heads (one TMA copy per page,
//              the table is read once), Q tiles and their normalisers.
//   warp 5     tcgen05.mma issuer, into two S buffers in turn.
// The (head, query tile) items of a key tile are dealt out to the CTAs of a
// cluster of up to 8 where there are few key tiles; rank 0 adds the sums through
// distributed shared memory.
#pragma once

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
  uint32_t* err;
  uint64_t limit_ns;
};

template <int N_>
struct WeightCfg {
  static constexpr int N = N_;
  static constexpr int THREADS = 192;
  static constexpr int K_STAGES = N == 128 ? 2 : 3;
  static constexpr int Q_STAGES = 3;
  static constexpr int CTAS_PER_SM = N == 128 ? 2 : 4;
  static constexpr int Q_BYTES = N * DH * 2;
  static constexpr uint32_t TMEM_COLS = 2 * N;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_Q = OFF_K + K_STAGES * TILE_BYTES;
  static constexpr int OFF_LSE = OFF_Q + Q_STAGES * Q_BYTES;  // [Q_STAGES][N] normalisers, log2 units
  static constexpr int OFF_TOTAL = OFF_LSE + Q_STAGES * N * 4;  // [128] sums
  static constexpr int OFF_BARS = OFF_TOTAL + BKV * 4;
  // k_full[K], k_empty[K], q_full[Q], q_empty[Q], s_full[2], s_free[2], drain
  static constexpr int NUM_BARS = 2 * K_STAGES + 2 * Q_STAGES + 5;
  static constexpr int OFF_MISC = OFF_BARS + 8 * NUM_BARS;
  static constexpr int SMEM_BYTES = 1024 + OFF_MISC + 16;
};

template <int N>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[N]) {
  if constexpr (N == 128) {
    tmem_ld128(taddr, r);
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
  float* lse_ring = reinterpret_cast<float*>(smem + C::OFF_LSE);
  float* total = reinterpret_cast<float*>(smem + C::OFF_TOTAL);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_MISC);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + C::OFF_MISC + 4);
  const Geo& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Key tiles are the slowest grid dimension: those that most rows see start first.
  const int rank = blockIdx.x, ranks = gridDim.x, b = blockIdx.y, tile = blockIdx.z;

  if (threadIdx.x == 0) {
    for (int s = 0; s < KS; ++s) {
      mbar_init(k_full(s), 1);
      mbar_init(k_empty(s), 1);
    }
    for (int s = 0; s < QS; ++s) {
      mbar_init(q_full(s), 1);
      mbar_init(q_empty(s), 5);  // the MMA and the four warps that read the normalisers
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_full(s), 1);
      mbar_init(s_free(s), 4);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    fence_barrier_init();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
  }
  if (warp == 5) {
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

  const Seq s = seq_of(g, b);
  const Tokens seen = tokens_seeing(g, s, tile * BKV, (tile + 1) * BKV);
  const int chunks = (seen.hi - seen.lo + g.tok_per_tile - 1) / g.tok_per_tile;
  // This rank's items, head by head: item = head * chunks + query tile.
  const int items = g.kv_heads * chunks;
  const int i0 = static_cast<int>(static_cast<long long>(items) * rank / ranks);
  const int i1 = static_cast<int>(static_cast<long long>(items) * (rank + 1) / ranks);

  if (warp == 4) {
    // ---------------- producer ----------------
    const int n_pages = pages_per_tile(g);
    const uint32_t page_bytes = TILE_BYTES / n_pages;
    PageLoad l{false, 0};
    if (i0 < i1 && lane < n_pages) {
      Span all{};
      all.hi = s.kv;
      l = page_of_tile(g, b, all, tile, lane);
    }
    const uint32_t k_bytes = __popc(__ballot_sync(0xffffffffu, l.load)) * page_bytes;
    const uint32_t q_bytes = static_cast<uint32_t>(g.tok_per_tile * g.group) * DH * 2;
    int kn = 0, qn = 0;
    bool ok = true;
    for (int i = i0; i < i1; ++i) {
      const int h = i / chunks, ch = i - h * chunks;
      const int tok0 = seen.lo + ch * g.tok_per_tile;
      // normalisers of the tile's rows; +inf takes a row's weight to zero
      float lse2[(N + 31) / 32];
#pragma unroll
      for (int x = 0; x < (N + 31) / 32; ++x) {
        const int r = 32 * x + lane;
        const int tok = tok0 + r / g.group;
        lse2[x] = INFINITY;
        if (r < N && tok < seen.hi && r < g.tok_per_tile * g.group) {
          const float v =
              __ldg(p.lse + (static_cast<int64_t>(b) * g.t_q + tok) * g.n_heads + h * g.group + r % g.group);
          if (v != -INFINITY) lse2[x] = v * kLog2e;
        }
      }
      if (i == i0 || ch == 0) {  // the next head's K
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
      for (int x = 0; x < (N + 31) / 32; ++x)
        if (32 * x + lane < N) lse_ring[st * N + 32 * x + lane] = lse2[x];
      __syncwarp();
      if (lane == 0) {
        mbar_arrive_expect_tx(q_full(st), q_bytes);
        tma_load_4d(sbase + C::OFF_Q + st * C::Q_BYTES, &tm_q, q_full(st), 0, h * g.group, tok0, b);
      }
      ++qn;
    }
    // Let the last copies land before the CTA may exit.
    for (int i = max(0, kn - KS); i < kn; ++i) mbar_wait_drain(k_full(i % KS), (i / KS) & 1, p.limit_ns);
    for (int i = max(0, qn - QS); i < qn; ++i) mbar_wait_drain(q_full(i % QS), (i / QS) & 1, p.limit_ns);
  } else if (warp == 5) {
    if (lane == 0) {
      // ---------------- MMA issuer ----------------
      constexpr uint32_t idesc = idesc_f16_f32(BKV, N, 0, 0);  // K and Q both K-major
      int kn = 0, n = 0;
      for (int i = i0; i < i1; ++i, ++n) {
        const bool head_starts = i == i0 || i % chunks == 0;
        const bool head_ends = i + 1 == i1 || (i + 1) % chunks == 0;
        if (head_starts) {
          if (!mbar_wait(k_full(kn % KS), (kn / KS) & 1, wc)) break;
          ++kn;
        }
        const int ks = (kn - 1) % KS, qs = n % QS, buf = n & 1;
        if (!mbar_wait(q_full(qs), (n / QS) & 1, wc)) break;
        if (!mbar_wait(s_free(buf), ((n >> 1) & 1) ^ 1u, wc)) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < DH / 16; ++kk)
          mma_f16_ss(tmem_base + buf * N, smem_desc_sw128(sbase + C::OFF_K + ks * TILE_BYTES + kk * 32, 16, 1024),
                     smem_desc_sw128(sbase + C::OFF_Q + qs * C::Q_BYTES + kk * 32, 16, 1024), idesc, kk > 0 ? 1u : 0u);
        mma_commit(s_full(buf));
        mma_commit(q_empty(qs));
        if (head_ends) mma_commit(k_empty(ks));
      }
      mma_commit(drain_bar);
      mbar_wait_drain(drain_bar, 0, p.limit_ns);
    }
  } else {
    // ---------------- weights: thread = slot ----------------
    const int j = tile * BKV + threadIdx.x;
    const Tokens mine = tokens_seeing(g, s, j, j + 1);
    float sum = 0.f;
    const uint32_t s_tmem = tmem_base + (static_cast<uint32_t>(warp * 32) << 16);
    int n = 0;
    for (int i = i0; i < i1; ++i, ++n) {
      const int qs = n % QS, buf = n & 1;
      if (!mbar_wait(q_full(qs), (n / QS) & 1, wc)) break;  // the producer's normalisers
      if (!mbar_wait(s_full(buf), (n >> 1) & 1, wc)) break;
      tc_fence_after();
      float x[N];
      {
        uint32_t r[N];
        tmem_ld_cols<N>(s_tmem + buf * N, r);
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = __uint_as_float(r[e]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(s_free(buf));
      // Columns [c_lo, c_hi) are rows that see this slot.
      const int tok0 = seen.lo + (i % chunks) * g.tok_per_tile;
      const int c_lo = (mine.lo - tok0) * g.group;
      const int c_hi = min(mine.hi - tok0, g.tok_per_tile) * g.group;
      if (c_lo > 0) {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (e < c_lo) x[e] = -INFINITY;
      }
      if (c_hi < N) {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (e >= c_hi) x[e] = -INFINITY;
      }
      const float4* norm = reinterpret_cast<const float4*>(lse_ring + qs * N);
      const uint64_t sl2x2 = f2_pack(p.scale_log2, p.scale_log2);
      uint64_t acc2[2] = {0ull, 0ull};
#pragma unroll
      for (int e = 0; e < N; e += 4) {
        const float4 v = norm[e / 4];
        float y0, y1, y2, y3;
        f2_unpack(f2_fma(f2_pack(x[e], x[e + 1]), sl2x2, f2_pack(-v.x, -v.y)), y0, y1);
        f2_unpack(f2_fma(f2_pack(x[e + 2], x[e + 3]), sl2x2, f2_pack(-v.z, -v.w)), y2, y3);
        acc2[0] = f2_add(acc2[0], f2_pack(ex2_approx(y0), ex2_approx(y1)));
        acc2[1] = f2_add(acc2[1], f2_pack(ex2_approx(y2), ex2_approx(y3)));
      }
      float a, c;
      f2_unpack(f2_add(acc2[0], acc2[1]), a, c);
      sum += a + c;  // one tile's weights, then the running sum: fp32 in two levels
      __syncwarp();
      if (lane == 0) mbar_arrive(q_empty(qs));
    }
    // A slot in a hole, or behind the end, has none (its K may be anything).
    bool held = j < s.kv;
    if (held) {
      const int page = __ldg(g.table + static_cast<int64_t>(b) * g.pages_per_seq + (j >> g.page_shift));
      held = page >= 0 && page < g.num_pages;
    }
    total[threadIdx.x] = held ? sum : 0.f;
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (ranks > 1) cluster_sync();
  const int t = threadIdx.x;
  if (rank == 0 && t < BKV && tile * BKV + t < g.cap) {
    float v = total[t];
    for (int i = 1; i < ranks; ++i) {
      float x;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(x) : "r"(mapa_shared(smem_u32(&total[t]), i)) : "memory");
      v += x;
    }
    const int64_t at = static_cast<int64_t>(b) * g.cap + tile * BKV + t;
    p.w_out[at] = (p.w_in != nullptr ? p.w_in[at] : 0.f) + v;
  }
  if (ranks > 1) cluster_sync();  // no CTA leaves while rank 0 still reads its sums
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::TMEM_COLS);
  }
}

}  // namespace pg
}  // namespace sea
