// bsfa_decode16.cu -- bsfa_decode16: the host side.  The kernels are in
// bsfa_decode16.cuh, instantiated by inst_decode16_*.cu.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "bsfa.h"
#include "bsfa_cache16.h"
#include "bsfa_cache4.h"
#include "bsfa_decode16_wide.cuh"
#include "bsfa_launch.h"

namespace bsfa {

namespace decode16 {
extern template bsfa_status run<64, false>(const DecArgs&, const Plan&, int, int, cudaStream_t);
extern template bsfa_status run<64, true>(const DecArgs&, const Plan&, int, int, cudaStream_t);
extern template bsfa_status run<128, false>(const DecArgs&, const Plan&, int, int, cudaStream_t);
extern template bsfa_status run<128, true>(const DecArgs&, const Plan&, int, int, cudaStream_t);
#define BSFA_WIDE(D, F16)                                                                  \
  extern template bsfa_status run_wide<D, F16>(const CUtensorMap&, const CUtensorMap&,      \
                                               const DecArgs&, const Plan&, int, int, cudaStream_t);
BSFA_WIDE(64, false)
BSFA_WIDE(64, true)
BSFA_WIDE(128, false)
BSFA_WIDE(128, true)
#undef BSFA_WIDE
}  // namespace decode16

namespace {

using namespace decode16;

// Query row tiles of a call: as few tensor-core columns as hold its rows, up
// to 32 to a CTA, and equal shares where one CTA does not hold them.
Plan plan_of(const bsfa_cache16* c, const bsfa_decode4_params* p) {
  Plan pl;
  const long long rows = static_cast<long long>(p->num_heads_q / c->num_heads_kv) * p->q_len;
  const long long eights = rows > 0 ? (rows + 7) / 8 : 1;
  pl.row_tiles = static_cast<int>((rows + 127) / 128);
  pl.segments = static_cast<long long>(p->batch) * c->num_heads_kv * pl.row_tiles;
  pl.wide = rows > WIDE_ROWS && p->max_seqlen >= WIDE_LEAST && pl.segments <= WIDE_SEGMENTS;
  if (pl.wide) {
    pl.nt = 16;
    pl.units = (p->max_seqlen + WIDE_UNIT - 1) / WIDE_UNIT;
    pl.all_units = pl.segments * (pl.units + WIDE_SEGMENT_UNITS);
    pl.max_grid = MAX_SMS;
    pl.warps = WARPS;
    pl.cluster = 1;
    pl.split = true;
    return pl;
  }
  pl.row_tiles = static_cast<int>((eights + 3) / 4);
  pl.nt = static_cast<int>((eights + pl.row_tiles - 1) / pl.row_tiles);
  pl.units = (p->max_seqlen + UNIT - 1) / UNIT;
  if (pl.units < 1) pl.units = 1;
  pl.segments = static_cast<long long>(p->batch) * c->num_heads_kv * pl.row_tiles;
  // (Beyond 2^31 segments, which are refused, the product could overflow.)
  pl.all_units =
      pl.segments >> 31 ? pl.segments : pl.segments * (pl.units + SEGMENT_UNITS);
  constexpr int grids[2][4] = {
      {Shape<64, 1>::MAX_GRID, Shape<64, 2>::MAX_GRID, Shape<64, 3>::MAX_GRID,
       Shape<64, 4>::MAX_GRID},
      {Shape<128, 1>::MAX_GRID, Shape<128, 2>::MAX_GRID, Shape<128, 3>::MAX_GRID,
       Shape<128, 4>::MAX_GRID}};
  pl.max_grid = grids[c->head_dim == 128][pl.nt - 1];
  // A segment gets as many CTAs as keep all resident at once; where one each is too
  // many for that, short ones get CTAs of one warp (256 ragged sequences to 128, 256 and
  // 512 tokens on eight heads: 20.5, 30.7 and 52.1 us, by CTAs of four warps 32.3, 37.4
  // and 51.4).  Clusters of sixteen only where few are met, as each has to find its
  // place within one GPC (1 x 8K on eight heads: 12.3 -> 10.5 us; 2 x 4K would go from
  // 10.3 to 15.2).
  const int resident = pl.max_grid / MAX_SMS * SMS;
  const bool small = pl.segments > resident && pl.nt <= SMALL_NT && pl.units <= SMALL_UNITS;
  pl.warps = small ? SMALL_WARPS : WARPS;
  pl.cluster = 1;
  while (pl.cluster < MAX_CLUSTER && pl.units >= 2 * pl.cluster) {
    const int next = 2 * pl.cluster;
    if (pl.segments * next > (next == MAX_CLUSTER ? GRID_OF_16 : resident)) break;
    pl.cluster = next;
  }
  // Longer segments are cut; those that fill most of the GPU as they are, at twice the
  // length (4 x 16K 46.0 -> 42.7 us, ragged 42.0 -> 38.4; 16 x 4K 47.3 -> 42.9, ragged
  // 31.3 -> 29.2; equal lengths that leave a second wave lose: 40 x 2K 56.7 -> 61.5).
  const bool full = 2 * pl.segments * pl.cluster > resident;
  pl.split = pl.units > (full ? 2 : 1) * CLUSTER_UNITS * pl.cluster;
  if (pl.split) pl.cluster = 1, pl.warps = WARPS;
  return pl;
}

// The tensor map of a pool: copies of `box` tokens of one head and page.
bool map_pool(CUtensorMap* m, const bsfa_cache16* c, const void* pool, const int64_t (&stride)[3],
              int box) {
  // The stride of a dimension of one element may be anything, but not in a map.
  const long long head = c->num_heads_kv > 1 ? stride[1] : c->head_dim;
  const long long page = c->num_pages > 1 ? stride[0] : c->head_dim;
  return make_map(m, pool, c->dtype == BSFA_DTYPE_F16, c->head_dim, c->page_size, c->num_heads_kv,
                  c->num_pages, stride[2], head, page, box);
}

struct Carve {
  size_t part_o, part_ml, joins, anew, kept, bytes;
};

Carve carve(const Plan& pl, const bsfa_cache16* cache, const bsfa_decode4_params* p) {
  Carve c{};
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const int d = cache->head_dim;
  const size_t grid = pl.split ? static_cast<size_t>(pl.max_grid) : 0;
  const size_t rows = 2 * grid * 8 * pl.nt * (pl.wide ? WIDE_PARTS : 1);
  c.part_o = 0;
  c.part_ml = up(c.part_o + rows * d * sizeof(float));
  c.joins = up(c.part_ml + rows * sizeof(float2));
  c.anew = up(c.joins + (pl.wide ? pl.segments : grid) * sizeof(int4));
  c.kept = up(c.anew + (pl.wide ? pl.segments * 4 * sizeof(uint32_t) : 0));
  // (Of every wide call: whether its output is its queries is not known to all who ask.)
  const size_t queries = static_cast<size_t>(p->batch) * p->num_heads_q * p->q_len;
  c.bytes = c.kept + (pl.wide ? up(queries * d * sizeof(uint16_t)) : 0);
  return c;
}

bsfa_status validate_sizes(const bsfa_cache16* c, const bsfa_decode4_params* p) {
  if (c == nullptr || p == nullptr) return BSFA_ERR_INVALID_ARG;
  if (p->batch < 0 || p->q_len < 0 || p->max_seqlen < 0) return BSFA_ERR_INVALID_ARG;
  const bsfa_status v = validate_cache16(c);
  if (v != BSFA_OK) return v;
  if (p->num_heads_q <= 0 || p->num_heads_q % c->num_heads_kv) return BSFA_ERR_INVALID_ARG;
  if (p->dtype != BSFA_DTYPE_BF16 && p->dtype != BSFA_DTYPE_F16) return BSFA_ERR_UNSUPPORTED;
  if (p->dtype != c->dtype) return BSFA_ERR_INVALID_ARG;
  if (p->batch > CACHE4_MAX_BATCH) return BSFA_ERR_UNSUPPORTED;
  if (p->max_seqlen > static_cast<long long>(c->block_table_width) * c->page_size)
    return BSFA_ERR_INVALID_ARG;
  const long long rows = static_cast<long long>(p->num_heads_q / c->num_heads_kv) * p->q_len;
  if (rows > (1 << 24)) return BSFA_ERR_UNSUPPORTED;
  const Plan pl = plan_of(c, p);
  if (pl.all_units > 0x7fffffffLL - 4096 || pl.segments * pl.cluster > 0x7fffffffLL)
    return BSFA_ERR_UNSUPPORTED;
  return BSFA_OK;
}

}  // namespace

}  // namespace bsfa

using namespace bsfa;

extern "C" {

size_t bsfa_decode16_workspace_size(const bsfa_cache16* cache, const bsfa_decode4_params* p) {
  if (validate_sizes(cache, p) != BSFA_OK) return 0;
  return carve(plan_of(cache, p), cache, p).bytes;
}

bsfa_status bsfa_decode16(const bsfa_cache16* cache, const bsfa_decode4_params* p,
                          bsfa_stream_t stream_) {
  bsfa_status v = validate_sizes(cache, p);
  if (v != BSFA_OK) return v;
  if (p->batch == 0 || p->q_len == 0) return BSFA_OK;
  v = validate_cache16_pointers(cache);
  if (v != BSFA_OK) return v;
  if (!p->q || !p->o || !p->seqlens) return BSFA_ERR_INVALID_ARG;
  const int64_t extent[3] = {p->batch, p->num_heads_q, p->q_len};
  if (!rows_aligned(p->q, p->q_stride, extent) || !rows_aligned(p->o, p->o_stride, extent))
    return BSFA_ERR_UNSUPPORTED;
  const Plan pl = plan_of(cache, p);
  const Carve cv = carve(pl, cache, p);
  if (pl.split && (p->workspace == nullptr || (reinterpret_cast<uintptr_t>(p->workspace) & 255u) ||
                   p->workspace_bytes < cv.bytes))
    return BSFA_ERR_WORKSPACE;

  DecArgs a{};
  a.k = static_cast<const uint8_t*>(cache->k);
  a.v = static_cast<const uint8_t*>(cache->v);
  a.k_sp = 2 * cache->k_stride[0];
  a.k_sh = 2 * cache->k_stride[1];
  a.k_st = static_cast<int>(2 * cache->k_stride[2]);
  a.v_sp = 2 * cache->v_stride[0];
  a.v_sh = 2 * cache->v_stride[1];
  a.v_st = static_cast<int>(2 * cache->v_stride[2]);
  for (int i = 0; i < 3; ++i) {
    a.q_s[i] = p->q_stride[i];
    a.o_s[i] = p->o_stride[i];
  }
  a.table = cache->block_table;
  a.table_stride = cache->block_table_stride;
  a.num_pages = cache->num_pages;
  a.tiles_per_page = cache->page_size / TOK;
  a.q = static_cast<const uint16_t*>(p->q);
  a.o = static_cast<uint16_t*>(p->o);
  a.in_place = p->o == p->q;
  a.seqlens = p->seqlens;
  a.batch = p->batch;
  a.heads_kv = cache->num_heads_kv;
  a.group = p->num_heads_q / cache->num_heads_kv;
  a.q_len = p->q_len;
  a.rows = a.group * p->q_len;
  a.row_tiles = pl.row_tiles;
  a.max_len = p->max_seqlen;
  a.causal = p->causal != 0;
  a.f16 = p->dtype == BSFA_DTYPE_F16;
  a.split = pl.split;
  a.cluster = pl.cluster;
  const float sigma =
      p->softmax_scale > 0.f ? p->softmax_scale : 1.0f / std::sqrt((float)cache->head_dim);
  a.sigma_log2 = sigma * 1.4426950408889634f;
  int log2_len = 0;
  while ((1LL << log2_len) < p->max_seqlen) ++log2_len;
  a.shift = -(HEADROOM + static_cast<float>(log2_len));
  a.most = a.shift + HEADROOM;
  a.lse = p->lse;
  a.lse_pitch = static_cast<long long>(p->batch) * p->q_len;
  uint8_t* ws = static_cast<uint8_t*>(p->workspace);
  a.part_o = reinterpret_cast<float*>(ws + cv.part_o);
  a.part_ml = reinterpret_cast<float2*>(ws + cv.part_ml);
  a.joins = reinterpret_cast<int4*>(ws + cv.joins);
  a.anew = reinterpret_cast<uint32_t*>(ws + cv.anew);
  a.kept = reinterpret_cast<uint16_t*>(ws + cv.kept);

  int dev = 0, sms = 0;
  v = status_of(cudaGetDevice(&dev));
  if (v != BSFA_OK) return v;
  v = status_of(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  if (v != BSFA_OK || sms <= 0) return BSFA_ERR_CUDA;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  if (pl.wide) {
    // A copy lies within a page: the largest power of two that divides one.
    a.box = cache->page_size & -cache->page_size;
    if (a.box > WIDE_UNIT) a.box = WIDE_UNIT;
    a.err = device_error_word();
    CUtensorMap k, v;
    if (a.err == nullptr || !map_pool(&k, cache, cache->k, cache->k_stride, a.box) ||
        !map_pool(&v, cache, cache->v, cache->v_stride, a.box))
      return BSFA_ERR_CUDA;
    const auto call = cache->head_dim == 128 ? (a.f16 ? run_wide<128, true> : run_wide<128, false>)
                                             : (a.f16 ? run_wide<64, true> : run_wide<64, false>);
    return call(k, v, a, pl, sms, dev, stream);
  }
  const auto run_call = cache->head_dim == 128 ? (a.f16 ? run<128, true> : run<128, false>)
                                               : (a.f16 ? run<64, true> : run<64, false>);
  return run_call(a, pl, sms, dev, stream);
}

}  // extern "C"
