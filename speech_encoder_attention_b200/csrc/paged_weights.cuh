// paged_weights.cuh -- the attention weight that a chunk's query rows put on
// each slot of a paged cache, summed over rows and query heads:
//
//   w_out[b, j] = w_in[b, j] + sum_{i, h : j in A_i} e^{s_ij - lse_ih}.
//
// One CTA owns 128 slots of one sequence, so every slot has one writer and a
// fixed order of addition; the slots are the 16 rows of mma.sync products
// (S^T = K Q^T), so a slot's sum stays in the four threads that hold its row.
// K and Q fragments are loaded straight from memory, 16 bytes per thread: the
// order of the 64 columns inside the product is free as long as K and Q agree,
// and thread c of a row's four takes columns [8c, 8c+8) and [32+8c, 32+8c+8).
// With few query rows the kernel is bound by reading K; with many, by one
// exponential per (row, head, slot). tcgen05 tiles would not help either
// bound: the product is 64 multiply-adds per exponential.
//   MT = 1  few rows: 8 warps x 16 slots, all K/V heads in turn.
//   MT = 2  many rows: 4 warps x 32 slots (a Q fragment serves 32 slots), two
//           such groups per CTA, and the (head, 128 query rows) items of a
//           key tile dealt out to the groups of a cluster of up to 8 CTAs,
//           whose sums rank 0 adds through distributed shared memory.
#pragma once

#include "paged_common.cuh"
#include "paged_step.cuh"

namespace sea {
namespace pg {

struct WeightParams {
  Geo g;
  const __half* q;
  int64_t q_stride;
  const __half* k;
  int64_t k_stride;
  const float* lse;    // [batch * t_q, n_heads]
  const float* w_in;   // [batch, cap] or null (zeros)
  float* w_out;        // [batch, cap]
  float scale_log2;
  fa::DivC dv_group;
};

constexpr int WEIGHT_WARPS = 8;
constexpr int WEIGHT_ROWS = 128;  // query rows per item

template <int MT>
__global__ void __launch_bounds__(32 * WEIGHT_WARPS, MT == 1 ? 4 : 3) paged_weights_kernel(const WeightParams p) {
  constexpr int GROUPS = MT == 1 ? 1 : 2;  // item groups per CTA
  constexpr int GROUP_WARPS = WEIGHT_WARPS / GROUPS;
  __shared__ float sums[GROUPS][BKV];
  __shared__ float total[BKV];
  griddep_wait();
  griddep_launch_dependents();
  const Geo& g = p.g;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r4 = lane >> 2, c = lane & 3;
  const int b = blockIdx.z, tile = blockIdx.y;
  const int rank = blockIdx.x, ranks = gridDim.x;  // one cluster
  const Seq s = seq_of(g, b);
  const int grp = warp / GROUP_WARPS;
  const int j0 = tile * BKV + (warp % GROUP_WARPS) * 16 * MT;  // this warp's first slot

  // Tokens [t_lo, t_hi) that may see a slot of [a, z).
  auto tokens = [&](int a, int z, int& t_lo, int& t_hi) {
    z = min(z, s.kv);
    t_lo = 0;
    t_hi = s.q;
    if (a >= z) {
      t_hi = 0;
      return;
    }
    const bool firsts = a < g.first;
    if (g.causal) t_lo = max(t_lo, a - s.off);
    if (g.window && !firsts) {
      t_lo = max(t_lo, a - g.window + 1 - s.off);
      t_hi = min(t_hi, z - 1 + g.window - s.off);
    }
  };
  int t_lo, t_hi;
  tokens(tile * BKV, (tile + 1) * BKV, t_lo, t_hi);

  float acc[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = 0.f;
  if (t_hi > t_lo) {
    // This thread's slots (2 * MT rows) and where they lie.
    int64_t krow[MT][2];
    bool held[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = j0 + 16 * m + 8 * e + r4;
        int page = -1;
        if (j < s.kv) page = __ldg(p.g.table + static_cast<int64_t>(b) * g.pages_per_seq + (j >> g.page_shift));
        held[m][e] = page >= 0 && page < g.num_pages;
        krow[m][e] = held[m][e] ? (static_cast<int64_t>(page) << g.page_shift) + (j & ((1 << g.page_shift) - 1)) : 0;
      }
    int w_lo, w_hi;  // tokens that may see this warp's slots
    tokens(j0, j0 + 16 * MT, w_lo, w_hi);
    const int row_lo = t_lo * g.group, row_hi = t_hi * g.group;
    const int chunks = (row_hi - row_lo + WEIGHT_ROWS - 1) / WEIGHT_ROWS;
    const int items = g.kv_heads * chunks;
    for (int item = rank * GROUPS + grp; item < items; item += ranks * GROUPS) {
      const int h = item / chunks, ch = item - h * chunks;
      const int ra = max(row_lo + ch * WEIGHT_ROWS, w_lo * g.group);
      const int rz = min(min(row_lo + (ch + 1) * WEIGHT_ROWS, row_hi), w_hi * g.group);
      if (ra >= rz) continue;
      uint4 kf[MT][2][2];  // [16-slot tile][row half][column half]
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            kf[m][e][x] = held[m][e] ? __ldg(reinterpret_cast<const uint4*>(p.k + krow[m][e] * p.k_stride + h * DH) +
                                             c + 4 * x)
                                     : make_uint4(0u, 0u, 0u, 0u);
      float part[MT][2];
#pragma unroll
      for (int m = 0; m < MT; ++m) part[m][0] = part[m][1] = 0.f;
#pragma unroll 1
      for (int r0 = ra; r0 < rz; r0 += 8) {
        // B fragment: query row r0 + lane / 4
        uint4 qf[2] = {make_uint4(0u, 0u, 0u, 0u), make_uint4(0u, 0u, 0u, 0u)};
        {
          const int r = r0 + r4;
          if (r < rz) {
            const int tok = fa::div_c(r, p.dv_group);
            const uint4* src = reinterpret_cast<const uint4*>(
                p.q + (static_cast<int64_t>(b) * g.t_q + tok) * p.q_stride + (h * g.group + r - tok * g.group) * DH);
            qf[0] = __ldg(src + c);
            qf[1] = __ldg(src + c + 4);
          }
        }
        // the two rows of this thread's score columns
        float lse2[2];
        int pos[2];
        bool rv[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const int r = r0 + 2 * c + x;
          rv[x] = r < rz;
          const int tok = fa::div_c(r, p.dv_group);
          pos[x] = tok + s.off;
          lse2[x] = INFINITY;  // no weight
          if (rv[x]) {
            const float v =
                __ldg(p.lse + (static_cast<int64_t>(b) * g.t_q + tok) * g.n_heads + h * g.group + r - tok * g.group);
            if (v != -INFINITY) lse2[x] = v * kLog2e;
          }
        }
        const int p_min = fa::div_c(r0, p.dv_group) + s.off;
        const int p_max = fa::div_c(min(r0 + 7, rz - 1), p.dv_group) + s.off;
        // whether every row sees every one of this warp's slots
        const bool open = r0 + 8 <= rz && j0 + 16 * MT <= s.kv && (!g.causal || j0 + 16 * MT - 1 <= p_min) &&
                          (!g.window || j0 + 16 * MT <= g.first ||
                           (p_max - j0 < g.window && j0 + 16 * MT - 1 - p_min < g.window));
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const uint32_t a0[4] = {kf[m][0][x].x, kf[m][1][x].x, kf[m][0][x].y, kf[m][1][x].y};
            const uint32_t a1[4] = {kf[m][0][x].z, kf[m][1][x].z, kf[m][0][x].w, kf[m][1][x].w};
            mma_16816(d, a0, qf[x].x, qf[x].y);
            mma_16816(d, a1, qf[x].z, qf[x].w);
          }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float w0 = ex2_approx(fmaf(d[2 * e], p.scale_log2, -lse2[0]));
            float w1 = ex2_approx(fmaf(d[2 * e + 1], p.scale_log2, -lse2[1]));
            if (!open) {
              const int j = j0 + 16 * m + 8 * e + r4;
              auto sees = [&](int x) {
                return rv[x] && (!g.causal || j <= pos[x]) &&
                       (!g.window || j < g.first || (pos[x] - j < g.window && j - pos[x] < g.window));
              };
              if (!sees(0)) w0 = 0.f;
              if (!sees(1)) w1 = 0.f;
            }
            part[m][e] += w0 + w1;
          }
        }
      }
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        acc[m][0] += part[m][0];
        acc[m][1] += part[m][1];
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (!held[m][e]) acc[m][e] = 0.f;
  }
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      acc[m][e] += __shfl_xor_sync(0xffffffffu, acc[m][e], 1);
      acc[m][e] += __shfl_xor_sync(0xffffffffu, acc[m][e], 2);
      if (c == 0) sums[grp][(warp % GROUP_WARPS) * 16 * MT + 16 * m + 8 * e + r4] = acc[m][e];
    }
  __syncthreads();
  const int t = threadIdx.x;
  if (t < BKV) {
    float v = sums[0][t];
    if constexpr (GROUPS == 2) v += sums[1][t];
    total[t] = v;
  }
  if (ranks > 1) cluster_sync();
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
}

}  // namespace pg
}  // namespace sea
