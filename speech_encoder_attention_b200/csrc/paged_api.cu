// paged_api.cu -- the translation unit of libattn.so: attn_api.cu, whose helpers
// serve here too, and the C ABI's paged-cache entry points. Host side of those:
// argument checks (pure arithmetic, before any CUDA call), launch plans and
// launches.
#include "attn_api.cu"

#include "paged_cache.cuh"
#include "paged_chunk.cuh"
#include "paged_common.cuh"
#include "paged_step.cuh"
#include "paged_weights.cuh"

namespace {

bool g_paged_init[kMaxDevices] = {};

template <typename Kernel>
bool set_smem(Kernel* kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) == cudaSuccess;
}

// device_info, and once per device the paged kernels' shared-memory limits.
attn_status paged_device(DeviceInfo** out) {
  if (attn_status st = device_info(out); st != ATTN_OK) return st;
  const auto dev = *out - g_dev;
  std::lock_guard<std::mutex> lock(g_mutex);
  if (g_paged_init[dev]) return ATTN_OK;
  using namespace sea::pg;
  if (!set_smem(paged_step_kernel<1, false>, StepCfg<1>::SMEM_BYTES) ||
      !set_smem(paged_step_kernel<1, true>, StepCfg<1>::SMEM_BYTES) ||
      !set_smem(paged_step_kernel<2, false>, StepCfg<2>::SMEM_BYTES) ||
      !set_smem(paged_step_kernel<2, true>, StepCfg<2>::SMEM_BYTES) ||
      !set_smem(paged_chunk_kernel, ChunkCfg::SMEM_BYTES) ||
      !set_smem(paged_weights_kernel<16>, WeightCfg<16>::SMEM_BYTES) ||
      !set_smem(paged_weights_kernel<32>, WeightCfg<32>::SMEM_BYTES) ||
      !set_smem(paged_weights_kernel<128>, WeightCfg<128>::SMEM_BYTES))
    return ATTN_ERR_CUDA;
  g_paged_init[dev] = true;
  return ATTN_OK;
}

constexpr int kMaxGroup = 128; // query heads per K/V head

bool misaligned4(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 3u) != 0; }

Range byte_range(const void* p, int64_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + static_cast<uintptr_t>(bytes)};
}

bool valid_paged_heads(int32_t batch, int32_t t_q, int32_t n_heads, int32_t n_kv_heads) {
  if (batch <= 0 || batch > 65535 || t_q <= 0 || n_heads <= 0 || n_heads > 32767 || n_kv_heads <= 0) return false;
  if (n_heads % n_kv_heads != 0 || n_heads / n_kv_heads > kMaxGroup) return false;
  return static_cast<int64_t>(batch) * t_q <= INT32_MAX && static_cast<int64_t>(t_q) * (n_heads / n_kv_heads) <= INT32_MAX / 2;
}

int64_t pool_rows(const attn_paged_kv& c) { return static_cast<int64_t>(c.num_pages) * c.page_size; }
int64_t pool_cols(const attn_paged_kv& c) { return static_cast<int64_t>(c.n_kv_heads) * sea::pg::DH; }
Range pool_range(const attn_paged_kv& c, const attn_mat& m) {
  return mat_range(m.ptr, pool_rows(c), pool_cols(c), m.row_stride);
}

bool valid_cache(const attn_paged_kv& c, int32_t batch) {
  if (c.page_size < 16 || c.page_size > 256 || (c.page_size & (c.page_size - 1)) != 0) return false;
  if (c.num_pages <= 0 || c.pages_per_seq <= 0 || c.n_kv_heads <= 0 || c.n_kv_heads > 32767) return false;
  if (pool_rows(c) > INT32_MAX) return false;
  // slots per sequence stay below 2^23: a grid dimension counts their 128-slot tiles
  if (static_cast<int64_t>(c.pages_per_seq) * c.page_size > (int64_t(1) << 23) - 256) return false;
  if (static_cast<int64_t>(batch) * c.pages_per_seq * c.page_size > INT32_MAX) return false;
  if (!valid_mat(c.k, pool_cols(c)) || !valid_mat(c.v, pool_cols(c))) return false;
  return c.table != nullptr && !misaligned4(c.table) && c.kv_lens != nullptr && !misaligned4(c.kv_lens);
}

bool valid_paged_mask(const attn_paged_mask& m) {
  return m.window >= 0 && m.first >= 0 && (m.window > 0 || m.first == 0) && (m.causal == 0 || m.causal == 1) &&
         !misaligned4(m.q_lens);
}

int log2_of(int x) {
  int l = 0;
  while ((1 << l) < x) ++l;
  return l;
}

sea::pg::Geo paged_geo(const attn_paged_kv& c, int32_t batch, int32_t t_q, int32_t n_heads, const attn_paged_mask& m) {
  sea::pg::Geo g{};
  g.batch = batch;
  g.t_q = t_q;
  g.n_heads = n_heads;
  g.kv_heads = c.n_kv_heads;
  g.group = n_heads / c.n_kv_heads;
  g.tok_per_tile = 1;
  g.q_tiles = t_q;
  g.page_shift = log2_of(c.page_size);
  g.pages_per_seq = c.pages_per_seq;
  g.num_pages = c.num_pages;
  g.cap = c.pages_per_seq * c.page_size;
  g.table = c.table;
  g.kv_lens = c.kv_lens;
  g.q_lens = m.q_lens;
  // |p - j| stays below t_q + cap: a wider window changes nothing, and the
  // sums below stay in 32 bits.
  const int64_t reach = static_cast<int64_t>(t_q) + g.cap + 1;
  g.window = static_cast<int>(std::min<int64_t>(m.window, std::min<int64_t>(reach, INT32_MAX / 2)));
  g.first = std::min(m.first, g.cap);
  g.causal = m.causal;
  return g;
}

// One K/V head's 128 bytes of up to 128 pool rows. L2 fetches 128 bytes per
// row, not 256: the next head's half belongs to another CTA, which comes for it
// at another time (16 decode steps over 8k caches: 108 us with 256 bytes, which
// read a third more from memory).
bool encode_pages(CUtensorMap* m, const attn_paged_kv& c, const attn_mat& pool) {
  auto enc = encoder();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(pool_cols(c)), static_cast<cuuint64_t>(pool_rows(c))};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(pool.row_stride) * 2};
  cuuint32_t box[2] = {sea::pg::DH, static_cast<cuuint32_t>(std::min(c.page_size, sea::pg::BKV))};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, pool.ptr, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// (column, head, token, sequence) view of the queries: a tile is `group` heads
// of tok_per_tile tokens, one 128-byte row each.
bool encode_paged_q(CUtensorMap* m, const attn_mat& q, int batch, int t_q, int n_heads, int group, int tok_per_tile) {
  auto enc = encoder();
  if (!enc) return false;
  const cuuint64_t row = static_cast<cuuint64_t>(q.row_stride) * 2;
  cuuint64_t dims[4] = {sea::pg::DH, static_cast<cuuint64_t>(n_heads), static_cast<cuuint64_t>(t_q),
                        static_cast<cuuint64_t>(batch)};
  cuuint64_t strides[3] = {sea::pg::DH * 2, row, row * t_q};
  cuuint32_t box[4] = {sea::pg::DH, static_cast<cuuint32_t>(group), static_cast<cuuint32_t>(tok_per_tile), 1};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, q.ptr, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// A chunk's units are walked whole, not cut into equal parts, where the longest SM
// works at most kCutTiles key tiles and kCutShare of the mean beyond the mean, which
// is what partials, their merging and the parts' uneven unit ends cost. An SM has two
// units at a time; an odd one left alone takes kAloneTile of a pair's time. Longest
// first, causal units of different lengths even out by themselves. 20 heads,
// us: 8 prompts of 1500 tokens 103 whole, 148 cut; one of 6000 143 and 175; 100
// tokens at the end of 1500 slots 22 and 18; 4 chunks of 500 tokens at the end of 6000
// slots, 4 K/V heads, 144 and 110. Over 894 sizes of 40 to 4000 tokens and up to 12000
// slots the choice costs 0.5 % on average against the better of both, at most 18 %.
constexpr float kAloneTile = 0.7f;
constexpr float kCutTiles = 5.5f;
constexpr float kCutShare = 0.1f;

// Units of `run` tiles each go to a CTA each, or to a cluster of 2 to 8 that shares
// the unit's tiles, or all are cut into equal parts, one per resident CTA, and merged:
// whichever the estimate below says is quicker, in tiles of a full device. What it
// leaves out: lengths may be far below the cache's size, or far apart, where equal
// parts are safer; so a CTA gets at most `most` tiles, or the units are cut.
struct SplitCosts {
  float lone;   // time of a tile where few CTAs run
  float setup;  // of a CTA
  float merge;  // of a cluster
  float cut;    // of cut parts: partials and a second kernel
  int most;
};

// CTAs per unit; 0: cut.
int plan_split(int64_t units, int64_t run, int64_t resident, const SplitCosts& costs) {
  float least = costs.cut + costs.setup + static_cast<float>(run) * units / resident;
  int best = 0;
  for (int c = 1; c <= 8 && (c == 1 || units * c <= resident); c *= 2) {
    const int64_t own = (run + c - 1) / c;
    if (own > costs.most) continue;
    const int64_t rest = units * c % resident;
    float waves = static_cast<float>(units * c / resident);
    if (rest != 0) waves += std::max(costs.lone, static_cast<float>(rest) / resident);
    const float cost = (own + costs.setup) * waves + (c > 1 ? costs.merge : 0.f);
    if (cost < least) {
      least = cost;
      best = c;
    }
  }
  return best;
}

// paged_step_kernel, tiles of 128 slots. One token, 20 heads, 64-slot pages, us: a CTA 4.7 at 128
// slots, 6.2 at 448, 7.4 at 700, 10.7 at 1500; a cluster of eight 7.0 at 700, 7.6 at
// 1500, 8.3 at 3000; cut parts 10.9 at 700, 11.6 at 1500, 12.3 at 3000. Over 699 sizes
// of 1 to 64 sequences, 1 to 20 K/V heads and up to 12000 slots the choice costs 1 %
// on average against the best of all, at most 18 %.
constexpr SplitCosts kStepCosts{0.55f, 0.f, 1.75f, 6.f, 24};

struct PagedPlan {
  int rows_cap;       // rows of a query tile
  int tok_per_tile, q_tiles;
  int parts, ctas;    // CTAs: one per part and K/V head; parts 0: nothing is cut, and
  int cluster;        // a step has so many per unit, a chunk walks whole units
  size_t ws_bytes;
};

PagedPlan plan_paged(const sea::pg::Geo& g, int num_sms) {
  const int t_q = g.t_q, kv_heads = g.kv_heads, group = g.group;
  PagedPlan pl{};
  // Up to 32 rows per K/V head: paged_step_kernel with 16 or 32 rows per tile. 20
  // heads, us: a step over 8000 slots of 16 sequences 106 with 16 rows, 125 with 32;
  // 24 tokens there 132, 175 with paged_chunk_kernel; over 448 slots of one sequence
  // 6.2, 9.1 and 9.8, 11.0.
  const int64_t rows = static_cast<int64_t>(t_q) * group;
  pl.rows_cap = rows <= 16 ? 16 : rows <= 32 ? 32 : sea::fa::BQ;
  pl.tok_per_tile = std::max(1, std::min(t_q, pl.rows_cap / group));
  pl.q_tiles = ceil_div(t_q, pl.tok_per_tile);
  pl.parts = std::max(1, 2 * num_sms / kv_heads);
  pl.ctas = pl.parts * kv_heads;
  const int64_t units = int64_t(g.batch) * kv_heads * pl.q_tiles;
  // The cache bounds a unit's key tiles, or the window (its other side too
  // unless causal), whose ends fall inside tiles, and the first tokens.
  const int64_t cap_tiles = ceil_div(g.cap, sea::pg::BKV);
  int64_t tiles = cap_tiles;
  if (g.window > 0) {
    const int64_t reach = int64_t(g.causal ? 1 : 2) * g.window + pl.tok_per_tile;
    tiles = std::min<int64_t>(tiles, reach / sea::pg::BKV + 2 + ceil_div(g.first, sea::pg::BKV));
  }
  if (pl.rows_cap <= 32) {
    const int cluster = plan_split(units, tiles, int64_t(2) * num_sms, kStepCosts);
    if (cluster > 0) {
      pl.parts = 0;
      pl.cluster = cluster;
      pl.ctas = static_cast<int>(units * cluster);
      return pl;
    }
  } else {
    const int64_t sm_units = (units + num_sms - 1) / num_sms;
    const float longest = static_cast<float>(tiles) * (sm_units / 2 + (sm_units % 2 != 0 ? kAloneTile : 0.f));
    const float mean = static_cast<float>(tiles) * units / (2 * num_sms);
    float beyond = longest - mean;
    if (g.causal && tiles == cap_tiles) beyond *= 1.f - std::min(1.f, float(t_q) / g.cap);
    if (beyond <= kCutTiles + kCutShare * mean) {
      pl.parts = 0;
      pl.ctas = static_cast<int>(std::min<int64_t>(units, int64_t(2) * num_sms));
      return pl;
    }
  }
  pl.ws_bytes = size_t(2) * pl.ctas * pl.rows_cap * (sea::pg::DH * sizeof(float) + sizeof(float2));
  return pl;
}

attn_status launch_paged_append(attn_mat k_new, attn_mat v_new, attn_paged_kv cache, int32_t batch, int32_t t_new,
                                const int32_t* q_lens, cudaStream_t stream) {
  if (!valid_paged_heads(batch, t_new, cache.n_kv_heads, cache.n_kv_heads) || !valid_cache(cache, batch))
    return ATTN_ERR_INVALID;
  if (misaligned4(q_lens)) return ATTN_ERR_INVALID;
  const int64_t rows = static_cast<int64_t>(batch) * t_new, cols = pool_cols(cache);
  if (!valid_mat(k_new, cols) || !valid_mat(v_new, cols)) return ATTN_ERR_INVALID;
  for (const attn_mat& m : {k_new, v_new}) {
    const Range r = mat_range(m.ptr, rows, cols, m.row_stride);
    if (overlaps(r, pool_range(cache, cache.k)) || overlaps(r, pool_range(cache, cache.v))) return ATTN_ERR_INVALID;
  }
  DeviceInfo* dev = nullptr;
  if (attn_status st = paged_device(&dev); st != ATTN_OK) return st;
  sea::pg::AppendParams p{};
  attn_paged_mask none{};
  none.q_lens = q_lens;
  p.g = paged_geo(cache, batch, t_new, cache.n_kv_heads, none);
  p.k_new = static_cast<const __half*>(k_new.ptr);
  p.v_new = static_cast<const __half*>(v_new.ptr);
  p.k_new_stride = k_new.row_stride;
  p.v_new_stride = v_new.row_stride;
  p.k = static_cast<__half*>(cache.k.ptr);
  p.v = static_cast<__half*>(cache.v.ptr);
  p.k_stride = cache.k.row_stride;
  p.v_stride = cache.v.row_stride;
  p.vecs = static_cast<int>(cols / 8);
  p.rows_per_cta = std::max(1, 512 / p.vecs);
  p.dv_vecs = make_divc(p.vecs);
  p.dv_t = make_divc(t_new);
  const int grid = ceil_div(rows, p.rows_per_cta);
  if (launch_pdl(sea::pg::paged_append_kernel, dim3(grid), dim3(256), 0, stream, p) != cudaSuccess) return ATTN_ERR_CUDA;
  return ATTN_OK;
}

attn_status launch_paged(attn_mat q, attn_paged_kv cache, int32_t batch, int32_t t_q, int32_t n_heads,
                         attn_paged_mask mask, const float* sinks, float scale, attn_mat out, float* lse,
                         void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!valid_paged_heads(batch, t_q, n_heads, cache.n_kv_heads) || !valid_cache(cache, batch) ||
      !valid_paged_mask(mask))
    return ATTN_ERR_INVALID;
  if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID;
  const int64_t rows = static_cast<int64_t>(batch) * t_q, cols = static_cast<int64_t>(n_heads) * sea::pg::DH;
  if (!valid_mat(q, cols) || !valid_mat(out, cols) || misaligned4(sinks) || misaligned4(lse)) return ATTN_ERR_INVALID;
  const Range ro = mat_range(out.ptr, rows, cols, out.row_stride);
  if (overlaps(ro, mat_range(q.ptr, rows, cols, q.row_stride)) || overlaps(ro, pool_range(cache, cache.k)) ||
      overlaps(ro, pool_range(cache, cache.v)))
    return ATTN_ERR_INVALID;
  if (!aligned16(workspace) || (workspace == nullptr && workspace_bytes != 0)) return ATTN_ERR_INVALID;

  DeviceInfo* dev = nullptr;
  if (attn_status st = paged_device(&dev); st != ATTN_OK) return st;
  sea::pg::StepParams p{};
  p.g = paged_geo(cache, batch, t_q, n_heads, mask);
  const PagedPlan pl = plan_paged(p.g, dev->num_sms);
  if (workspace_bytes < pl.ws_bytes) return ATTN_ERR_INVALID;
  const int64_t units = static_cast<int64_t>(batch) * cache.n_kv_heads * pl.q_tiles;
  if (units > INT32_MAX) return ATTN_ERR_INVALID;

  CUtensorMap tk, tv;
  if (!encode_pages(&tk, cache, cache.k) || !encode_pages(&tv, cache, cache.v)) return ATTN_ERR_CUDA;
  p.g.tok_per_tile = pl.tok_per_tile;
  p.g.q_tiles = pl.q_tiles;
  p.q = static_cast<const __half*>(q.ptr);
  p.q_stride = q.row_stride;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.sinks = sinks;
  p.out = static_cast<__half*>(out.ptr);
  p.out_stride = out.row_stride;
  p.lse = lse;
  p.ws_o = static_cast<float*>(workspace);
  p.ws_ml = reinterpret_cast<float2*>(p.ws_o + size_t(2) * pl.ctas * pl.rows_cap * sea::pg::DH);
  p.rows_cap = pl.rows_cap;
  p.parts = pl.parts;
  p.cluster = pl.cluster;
  p.err = dev->err;
  p.limit_ns = sea::kDefaultTimeoutNs;
  using sea::pg::StepCfg;
  cudaError_t err;
  if (pl.rows_cap == sea::fa::BQ) {
    CUtensorMap tq;
    if (!encode_paged_q(&tq, q, batch, t_q, n_heads, p.g.group, pl.tok_per_tile)) return ATTN_ERR_CUDA;
    sea::pg::ChunkParams cp{};
    cp.s = p;
    cp.units = static_cast<int>(units);
    cp.cut = pl.parts > 0 ? 1 : 0;
    cp.dv_group = make_divc(p.g.group);
    cp.dv_heads = make_divc(cache.n_kv_heads);
    cp.dv_bh = make_divc(batch * cache.n_kv_heads);
    err = launch_pdl(sea::pg::paged_chunk_kernel, dim3(pl.ctas), dim3(sea::pg::ChunkCfg::THREADS),
                     sea::pg::ChunkCfg::SMEM_BYTES, stream, tq, tk, tv, cp);
  } else {
    const unsigned cluster = static_cast<unsigned>(std::max(1, pl.cluster));
    auto launch = [&](auto kernel, int threads, int smem) {
      return launch_pdl_cluster(kernel, dim3(pl.ctas), dim3(threads), smem, stream, cluster, tk, tv, p);
    };
    using One = StepCfg<1>;
    using Two = StepCfg<2>;
    if (pl.rows_cap == 16)
      err = pl.parts > 0 ? launch(sea::pg::paged_step_kernel<1, true>, One::THREADS, One::SMEM_BYTES)
                         : launch(sea::pg::paged_step_kernel<1, false>, One::THREADS, One::SMEM_BYTES);
    else
      err = pl.parts > 0 ? launch(sea::pg::paged_step_kernel<2, true>, Two::THREADS, Two::SMEM_BYTES)
                         : launch(sea::pg::paged_step_kernel<2, false>, Two::THREADS, Two::SMEM_BYTES);
  }
  if (err != cudaSuccess) return ATTN_ERR_CUDA;
  if (pl.parts == 0) return ATTN_OK;
  const int unit_rows = pl.tok_per_tile * p.g.group;
  // Fewer rows per block, and more groups of parts per row, where blocks are few
  // (100 tokens, 20 heads, 1500 slots: 17.3 us, 20.8 us with 32 rows).
  int rows_log2 = log2_of(std::min(unit_rows, 32));
  while (rows_log2 > 0 && units * ceil_div(unit_rows, 1 << rows_log2) < 2 * dev->num_sms) --rows_log2;
  if (launch_pdl(sea::pg::paged_combine_kernel,
                 dim3(static_cast<unsigned>(units), static_cast<unsigned>(ceil_div(unit_rows, 1 << rows_log2))),
                 dim3(sea::pg::COMBINE_THREADS), 0, stream, p, rows_log2) != cudaSuccess)
    return ATTN_ERR_CUDA;
  return ATTN_OK;
}

// paged_weights_kernel: a unit is a key tile, its tiles are the items, of up to 32
// rows or of 128. One token, us: 4 K/V heads at 448 slots 5.3 in a cluster of eight,
// 5.4 of four, 6.2 in a CTA, 7.2 cut; 20 heads 6.5, 7.8, 15.7 and 8.8; 100 tokens of 4 K/V heads, 8 sequences of 1000 slots 20.7,
// 15.0, 28.8 and 17.6. Over 500 sizes the choice costs 0.8 % on average against the
// best of all, at most 20 %.
constexpr SplitCosts kWeightCosts{0.5f, 2.f, 0.5f, 2.5f, 5};
constexpr SplitCosts kWideWeightCosts{0.9f, 2.f, 0.5f, 2.5f, 5};

struct WeightPlan {
  int rows;            // rows of a query tile: as few as hold the chunk, in whole tokens
  int tok_per_tile, q_tiles;
  int tiles;           // key tiles per sequence
  int cluster;         // CTAs per key tile; 0: shares of the line of items
  int ctas;
  size_t ws_bytes;     // sums and states of the CTAs
};

WeightPlan plan_weights(const sea::pg::Geo& g, int num_sms) {
  WeightPlan pl{};
  const int64_t rows = static_cast<int64_t>(g.t_q) * g.group;
  pl.rows = rows <= 16 ? 16 : rows <= 32 ? 32 : 128;
  pl.tok_per_tile = std::min(g.t_q, pl.rows / g.group);
  pl.q_tiles = ceil_div(g.t_q, pl.tok_per_tile);
  pl.tiles = ceil_div(g.cap, sea::pg::BKV);
  pl.ctas = (pl.rows == 128 ? sea::pg::WeightCfg<128>::CTAS_PER_SM : sea::pg::WeightCfg<16>::CTAS_PER_SM) * num_sms;
  const int64_t key_tiles = static_cast<int64_t>(g.batch) * pl.tiles;
  const int64_t items = static_cast<int64_t>(g.kv_heads) * pl.q_tiles;
  if (key_tiles <= pl.ctas)
    pl.cluster = plan_split(key_tiles, items, pl.ctas, pl.rows == 128 ? kWideWeightCosts : kWeightCosts);
  if (pl.cluster > 0) {
    pl.ctas = static_cast<int>(key_tiles * pl.cluster);
  } else {
    pl.ws_bytes = size_t(pl.ctas) * (2 * sea::pg::BKV + 2) * 4;
  }
  return pl;
}

attn_status launch_paged_weights(attn_mat q, attn_paged_kv cache, int32_t batch, int32_t t_q, int32_t n_heads,
                                 attn_paged_mask mask, const float* lse, float scale, const float* w_in, float* w_out,
                                 void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!valid_paged_heads(batch, t_q, n_heads, cache.n_kv_heads) || !valid_cache(cache, batch) ||
      !valid_paged_mask(mask))
    return ATTN_ERR_INVALID;
  if (!(scale > 0.f) || !std::isfinite(scale)) return ATTN_ERR_INVALID;
  const int64_t rows = static_cast<int64_t>(batch) * t_q, cols = static_cast<int64_t>(n_heads) * sea::pg::DH;
  if (!valid_mat(q, cols) || lse == nullptr || misaligned4(lse) || w_out == nullptr || misaligned4(w_out) ||
      misaligned4(w_in))
    return ATTN_ERR_INVALID;
  const Range rw = byte_range(w_out, 4 * static_cast<int64_t>(batch) * cache.pages_per_seq * cache.page_size);
  if (w_in != nullptr && w_in != w_out && overlaps(rw, byte_range(w_in, static_cast<int64_t>(rw.hi - rw.lo))))
    return ATTN_ERR_INVALID;
  if (overlaps(rw, mat_range(q.ptr, rows, cols, q.row_stride)) || overlaps(rw, byte_range(lse, 4 * rows * n_heads)) ||
      overlaps(rw, pool_range(cache, cache.k)))
    return ATTN_ERR_INVALID;
  if (!aligned16(workspace) || (workspace == nullptr && workspace_bytes != 0)) return ATTN_ERR_INVALID;

  DeviceInfo* dev = nullptr;
  if (attn_status st = paged_device(&dev); st != ATTN_OK) return st;
  sea::pg::WeightParams p{};
  p.g = paged_geo(cache, batch, t_q, n_heads, mask);
  const WeightPlan pl = plan_weights(p.g, dev->num_sms);
  if (workspace_bytes < pl.ws_bytes) return ATTN_ERR_INVALID;
  p.g.tok_per_tile = pl.tok_per_tile;
  p.g.q_tiles = pl.q_tiles;
  p.dv_group = make_divc(p.g.group);
  p.tiles = pl.tiles;
  p.cluster = pl.cluster;
  p.ws_sum = static_cast<float*>(workspace);
  p.ws_state = reinterpret_cast<int*>(p.ws_sum + size_t(pl.ctas) * 2 * sea::pg::BKV);
  p.lse = lse;
  p.w_in = w_in;
  p.w_out = w_out;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.err = dev->err;
  p.limit_ns = sea::kDefaultTimeoutNs;
  CUtensorMap tq, tk;
  if (!encode_paged_q(&tq, q, batch, t_q, n_heads, p.g.group, p.g.tok_per_tile) || !encode_pages(&tk, cache, cache.k))
    return ATTN_ERR_CUDA;
  if (static_cast<int64_t>(batch) * p.tiles > INT32_MAX ||
      static_cast<int64_t>(cache.n_kv_heads) * pl.q_tiles > INT32_MAX)
    return ATTN_ERR_INVALID;
  auto launch = [&](auto kernel, auto cfg) {
    using C = decltype(cfg);
    return launch_pdl_cluster(kernel, dim3(pl.ctas), dim3(C::THREADS), C::SMEM_BYTES, stream,
                              static_cast<unsigned>(std::max(1, pl.cluster)), tq, tk, p);
  };
  using sea::pg::WeightCfg;
  const cudaError_t err = pl.rows == 16   ? launch(sea::pg::paged_weights_kernel<16>, WeightCfg<16>{})
                          : pl.rows == 32 ? launch(sea::pg::paged_weights_kernel<32>, WeightCfg<32>{})
                                          : launch(sea::pg::paged_weights_kernel<128>, WeightCfg<128>{});
  if (err != cudaSuccess) return ATTN_ERR_CUDA;
  if (pl.cluster == 0 && launch_pdl(sea::pg::paged_weights_merge_kernel, dim3(pl.ctas), dim3(sea::pg::BKV), 0, stream,
                                    p) != cudaSuccess)
    return ATTN_ERR_CUDA;
  return ATTN_OK;
}

attn_status launch_paged_evict(attn_paged_kv cache, int32_t batch, int32_t budget, int32_t first, int32_t recent,
                               const float* w_in, attn_paged_kv dst, float* w_out, int32_t* kept, cudaStream_t stream) {
  if (batch <= 0 || batch > 65535 || !valid_cache(cache, batch) || !valid_cache(dst, batch)) return ATTN_ERR_INVALID;
  if (dst.page_size != cache.page_size || dst.n_kv_heads != cache.n_kv_heads) return ATTN_ERR_INVALID;
  const int64_t cap = static_cast<int64_t>(cache.pages_per_seq) * cache.page_size;
  const int64_t out_cap = static_cast<int64_t>(dst.pages_per_seq) * dst.page_size;
  if (budget < 1 || budget > out_cap || first < 0 || recent < 0 || static_cast<int64_t>(first) + recent > budget)
    return ATTN_ERR_INVALID;
  if (w_in == nullptr || misaligned4(w_in) || misaligned4(w_out) || kept == nullptr || misaligned4(kept))
    return ATTN_ERR_INVALID;
  const Range r_win = byte_range(w_in, 4 * batch * cap), r_wout = byte_range(w_out, 4 * batch * out_cap);
  const Range r_kept = byte_range(kept, 4 * static_cast<int64_t>(batch) * budget);
  const Range r_lens = byte_range(dst.kv_lens, 4 * static_cast<int64_t>(batch));
  if (w_out != nullptr && overlaps(r_win, r_wout) && !(w_out == w_in && cap == out_cap)) return ATTN_ERR_INVALID;
  if (overlaps(r_kept, r_win) || (w_out != nullptr && (overlaps(r_kept, r_wout) || overlaps(r_lens, r_wout))) ||
      overlaps(r_kept, r_lens) || overlaps(r_lens, r_win))
    return ATTN_ERR_INVALID;
  if (dst.kv_lens != cache.kv_lens && overlaps(r_lens, byte_range(cache.kv_lens, 4 * static_cast<int64_t>(batch))))
    return ATTN_ERR_INVALID;
  const bool same = cache.k.ptr == dst.k.ptr && cache.v.ptr == dst.v.ptr && cache.k.row_stride == dst.k.row_stride &&
                    cache.v.row_stride == dst.v.row_stride && cache.num_pages == dst.num_pages;
  if (!same)
    for (const attn_mat& a : {cache.k, cache.v})
      for (const attn_mat& b : {dst.k, dst.v})
        if (overlaps(pool_range(cache, a), pool_range(dst, b))) return ATTN_ERR_INVALID;

  DeviceInfo* dev = nullptr;
  if (attn_status st = paged_device(&dev); st != ATTN_OK) return st;
  sea::pg::EvictParams p{};
  p.g = paged_geo(cache, batch, 1, cache.n_kv_heads, attn_paged_mask{});
  p.budget = budget;
  p.first = first;
  p.recent = recent;
  p.w_in = w_in;
  p.out_pages_per_seq = dst.pages_per_seq;
  p.out_num_pages = dst.num_pages;
  p.out_cap = static_cast<int>(out_cap);
  p.out_table = dst.table;
  p.out_lens = dst.kv_lens;
  p.w_out = w_out;
  p.kept = kept;
  p.k = static_cast<const __half*>(cache.k.ptr);
  p.v = static_cast<const __half*>(cache.v.ptr);
  p.k_stride = cache.k.row_stride;
  p.v_stride = cache.v.row_stride;
  p.k_out = static_cast<__half*>(dst.k.ptr);
  p.v_out = static_cast<__half*>(dst.v.ptr);
  p.k_out_stride = dst.k.row_stride;
  p.v_out_stride = dst.v.row_stride;
  int ranks = 1;
  while (ranks < 8 && ranks * int64_t(1024) < cap) ranks *= 2;
  const int threads = ranks == 1 ? 512 : 1024;
  if (launch_pdl_cluster(ranks == 1 ? sea::pg::paged_select_kernel<512> : sea::pg::paged_select_kernel<1024>,
                         dim3(ranks, batch), dim3(threads), 0, stream, static_cast<unsigned>(ranks), p) != cudaSuccess)
    return ATTN_ERR_CUDA;
  // Other pools: CTAs of a few whole rows, one step each, in any order, so that
  // a row's bytes are read together. The same pool: a CTA per head's columns,
  // which walks all rows.
  const int row_vecs = cache.n_kv_heads * sea::pg::DH / 8;
  p.rows_per_cta = same ? budget : std::max(1, sea::pg::MOVE_THREADS * sea::pg::MOVE_STEPS / row_vecs);
  p.move_vecs = same ? sea::pg::DH / 8 : row_vecs;
  p.dv_vecs = make_divc(p.move_vecs);
  const dim3 grid(ceil_div(budget, p.rows_per_cta), 2 * (row_vecs / p.move_vecs), batch);
  if (launch_pdl(same ? sea::pg::paged_move_kernel<true> : sea::pg::paged_move_kernel<false>, grid,
                 dim3(sea::pg::MOVE_THREADS), 0, stream, p) != cudaSuccess)
    return ATTN_ERR_CUDA;
  return ATTN_OK;
}

}  // namespace

extern "C" {

attn_status attn_paged_append(attn_mat k_new, attn_mat v_new, attn_paged_kv cache, int32_t batch, int32_t t_new,
                              const int32_t* q_lens, attn_stream_t stream) {
  return launch_paged_append(k_new, v_new, cache, batch, t_new, q_lens, stream);
}

attn_status attn_paged(attn_mat q, attn_paged_kv cache, int32_t batch, int32_t t_q, int32_t n_heads,
                       attn_paged_mask mask, const float* sinks, float scale, attn_mat out, float* lse,
                       void* workspace, size_t workspace_bytes, attn_stream_t stream) {
  return launch_paged(q, cache, batch, t_q, n_heads, mask, sinks, scale, out, lse, workspace, workspace_bytes, stream);
}

size_t attn_paged_workspace_size(attn_paged_kv cache, int32_t batch, int32_t t_q, int32_t n_heads,
                                 attn_paged_mask mask) {
  if (!valid_paged_heads(batch, t_q, n_heads, cache.n_kv_heads) || !valid_cache(cache, batch) ||
      !valid_paged_mask(mask))
    return 0;
  DeviceInfo* dev = nullptr;
  if (paged_device(&dev) != ATTN_OK) return 0;
  return plan_paged(paged_geo(cache, batch, t_q, n_heads, mask), dev->num_sms).ws_bytes;
}

size_t attn_paged_weights_workspace_size(attn_paged_kv cache, int32_t batch, int32_t t_q, int32_t n_heads) {
  if (!valid_paged_heads(batch, t_q, n_heads, cache.n_kv_heads) || !valid_cache(cache, batch)) return 0;
  DeviceInfo* dev = nullptr;
  if (paged_device(&dev) != ATTN_OK) return 0;
  return plan_weights(paged_geo(cache, batch, t_q, n_heads, attn_paged_mask{}), dev->num_sms).ws_bytes;
}

attn_status attn_paged_weights(attn_mat q, attn_paged_kv cache, int32_t batch, int32_t t_q, int32_t n_heads,
                               attn_paged_mask mask, const float* lse, float scale, const float* w_in, float* w_out,
                               void* workspace, size_t workspace_bytes, attn_stream_t stream) {
  return launch_paged_weights(q, cache, batch, t_q, n_heads, mask, lse, scale, w_in, w_out, workspace,
                              workspace_bytes, stream);
}

attn_status attn_paged_evict(attn_paged_kv cache, int32_t batch, int32_t budget, int32_t first, int32_t recent,
                             const float* w_in, attn_paged_kv dst, float* w_out, int32_t* kept, attn_stream_t stream) {
  return launch_paged_evict(cache, batch, budget, first, recent, w_in, dst, w_out, kept, stream);
}

}  // extern "C"
