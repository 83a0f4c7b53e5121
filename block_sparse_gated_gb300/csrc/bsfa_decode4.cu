// bsfa_decode4.cu -- bsfa_decode4: attention of a few new tokens per sequence
// over the 4-bit cache.
//
// Mathematics.  With k_t = code * scale (exact in fp16) and the query row
// scaled by a power of two into fp16's range (elements more than 2^28 below the
// row's largest lose bits there), S^T = K Q^T and O^T = V^T P^T are
// fp16 tensor-core products with fp32 sums.  The softmax is streamed: a
// reference m (log2 units) is subtracted, p = 2^(y - m), and m is raised, with
// O and the sum l rescaled, only when some score passes it by more than
// 2^HEADROOM; p carries a factor 2^SHIFT that cancels in O / l and keeps small
// weights out of fp16's subnormals.
//
// Layout.  Cached tokens are the rows (M) of the products and query rows
// (Hq/Hkv heads times q_len tokens) the columns (N = 8 per tile), so that a
// decode step of up to 8 query heads per KV head wastes no tensor work, and so
// that a lane owns whole scale groups: of a key it needs d/4 consecutive
// elements, of a value d/8.  The codes go from shared memory to fragments with
// one conversion and one product per pair of elements and no transposition:
// keys pair neighbours of one token, values pair two tokens by merging nibbles
// (or, where query rows are four at most, neighbours as well: see there).
//
// Work split.  A segment is one (sequence, KV head, row tile).  Where it is
// short by the caller's bound, a CTA (of two, four or sixteen warps, the fewer the
// more segments there are) takes it, or a cluster of up to eight, which joins its
// sums through distributed shared memory: one launch, no workspace.
// Longer ones are counted in units of 64 tokens; the units of all segments form
// one line, which is cut into equal pieces, one per CTA, from the lengths on the
// device.  Long and short sequences balance without the host knowing them, and a
// captured call stays right as they grow.  A segment that a cut crosses leaves
// partial sums in the workspace, which a second kernel joins in a fixed order.
//
// Bound.  144 bytes per (token, KV head) at d = 128 set the floor: 100 cycles of
// an SM per 16 tokens and head at a copy's rate.  They take 242 issued warp
// instructions (64 conversions, 64 fp16x2 products and 16 tensor products among
// them): 64 ragged sequences to 16K (633 MB) take 104 us, 6.1 TB/s or 90% of a
// copy's 6.77.  Each warp streams its own 16-token tiles through a private ring of
// asynchronous copies; no barrier is met inside a segment.
#include <cuda_runtime.h>

#include <atomic>
#include <cfloat>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "bsfa.h"
#include "bsfa_cache4.h"
#include "fp4.cuh"

namespace bsfa {

namespace {

constexpr int WARPS = 4;
constexpr int THREADS = 32 * WARPS;
constexpr int TOK = 16;             // tokens of a warp's tile
constexpr int UNIT = TOK * WARPS;   // tokens of a work unit
constexpr float HEADROOM = 5.f;     // log2 a score may pass the reference by
constexpr float SHIFT = 10.f;       // log2 of the factor that p carries: p < 2^15
constexpr int MIN_UNITS = 4;        // shortest piece of the line worth a CTA
constexpr int SEGMENT_UNITS = 8;    // a segment's fixed cost, in units
constexpr int RUN_UNITS = 256;      // units of a segment summed at once, at most
constexpr int JOIN_THREADS = 256;   // of the kernel that joins parts
constexpr int JOIN_ROWS_PARTS = 8;  // a warp to a row below, a block above
constexpr int MAX_PARTS = 768;      // parts of a segment, at most: CTAs of a cut call
constexpr int MAX_CLUSTER = 8;      // CTAs that share a segment, at most
constexpr int CLUSTER_UNITS = 16;   // units of a segment per CTA of a cluster, at most
constexpr int SMALL_WARPS = 2;      // warps of a CTA where there are many segments
constexpr int SMALL_UNITS = 32;     // units of a segment per CTA of that size, at most
constexpr int WIDE_WARPS = 16;      // warps of a CTA where there are few segments
constexpr int WIDE_GRID = 152;      // CTAs of that size: the GPU's SMs
constexpr int WIDE_GRID_OF_8 = 64;  // ... in clusters of eight
constexpr int WIDE_LEAST = 8;       // units of a segment worth one
constexpr int WIDE_UNITS = 32;      // units of a segment per CTA of that size, at most

// Query rows of a CTA: NT tiles of 8, or four (NT = 0, "half": see the values'
// product).
constexpr int rows_of(int nt) { return nt == 0 ? 4 : 8 * nt; }

// Per row-tile width: CTAs per SM, ring stages, whether the main loop goes around
// the ring in one piece (64 ragged sequences to 16K, four and eight query rows:
// 105.4 and 119.4 us by single tiles, 104.0 and 111.2 unrolled, with five stages
// 106.2 and 111.9; five tokens over 16 to 32K, NT = 3: 119.6, unrolled 123.6), and
// the most CTAs a launch has (the workspace holds two partial results each).
template <int NT>
struct Shape;
template <>
struct Shape<0> {
  static constexpr int CTAS = 4, STAGES = 4, MAX_GRID = 640;
  static constexpr bool UNROLL = true;
};
template <>
struct Shape<1> {
  static constexpr int CTAS = 4, STAGES = 4, MAX_GRID = 640;
  static constexpr bool UNROLL = true;
};
template <>
struct Shape<2> {
  static constexpr int CTAS = 3, STAGES = 4, MAX_GRID = 480;
  static constexpr bool UNROLL = true;
};
template <>
struct Shape<3> {
  static constexpr int CTAS = 2, STAGES = 4, MAX_GRID = 320;
  static constexpr bool UNROLL = false;
};
template <>
struct Shape<4> {
  static constexpr int CTAS = 2, STAGES = 4, MAX_GRID = 320;
  static constexpr bool UNROLL = false;
};

struct DecArgs {
  const uint8_t *kc, *vc, *ks, *vs;
  const int32_t *kexp, *vexp;
  long long kc_sh, vc_sh, ks_sh, vs_sh;        // head strides in bytes
  uint32_t kc_sp4, vc_sp4, ks_sp4, vs_sp4;     // page strides in units of 4 bytes
  int kc_st, vc_st, ks_st, vs_st;              // token strides in bytes
  const int32_t* table;
  int table_stride, num_pages, tiles_per_page;
  const uint16_t* q;
  uint16_t* o;
  long long q_s[3], o_s[3];
  const int32_t* seqlens;
  int batch, heads_kv, group, q_len, rows, row_tiles, max_len;
  int causal, f16, split, cluster, join_by_segment;
  float sigma_log2;
  float* lse;
  long long lse_pitch;
  float* part_o;    // [grid][2][rows of a CTA][d]
  float2* part_ml;  // [grid][2][rows of a CTA]
  int4* joins;      // [jobs]: {sequence, kvh * row_tiles + row tile, first, last CTA}, or x < 0
};

// The sequence length that the call sees.
__device__ __forceinline__ int clamp_len(const DecArgs& a, int b) {
  return max(0, min(__ldg(a.seqlens + b), a.max_len));
}
// Units of a segment on the line: its tokens', and what a CTA spends on any
// segment (queries, the first copies' latency, the join of its warps): without it
// the CTAs with many short sequences end last (64 ragged sequences to 16K: 106.2 us
// at 5, 103.6 at 8, 105.0 at 11; an earlier kernel 136 at 0, 124 at 5).
__device__ __forceinline__ int units_of(int len) { return SEGMENT_UNITS + (len + UNIT - 1) / UNIT; }

// Byte offset in a warp's stage of row `t` (0..15), 16-byte chunk `c`.  Rows
// are paired into 128-byte lines and chunks permuted so that both readers --
// for keys the rows {0,4,1,5,2,6,3,7}, two (four at d = 64) at a time, for
// values rows 4e..4e+3 at once -- touch every bank once.
template <int D>
__device__ __forceinline__ uint32_t swizzle(int t, int c) {
  if constexpr (D == 128)
    return ((t >> 1) << 7) + (((t ^ (t >> 2)) & 1) << 6) + ((c ^ (t & 2)) << 4);
  else
    return ((t >> 2) << 7) + (((t ^ ((t >> 2) << 1)) & 3) << 5) + (c << 4);
}

template <int D>
struct Stage {
  static constexpr int CODES = TOK * D / 2;           // bytes of 16 rows of codes
  static constexpr int SCALES = TOK * D / FP4_GROUP;  // ... of scales
  static constexpr int BYTES = 2 * CODES + 2 * SCALES;
};

// Row stride of a merged partial result in shared memory: d floats with one
// more after every 16 (D/8 at d = 64), rounded so that the eight row groups and
// four columns of a fragment fall into different banks.
template <int D>
__device__ __forceinline__ int merge_pos(int d) {
  return d + d / (D / 8);
}
template <int D>
constexpr int MERGE_ROW = D + 12;

// Dynamic shared memory: the rings, whose place the warps' sums take later, and
// behind them what the CTAs of a cluster send each other, or what a CTA carries
// from one run of a segment to the next.
template <int D, int NT, int W>
constexpr int ring_bytes() {
  constexpr int ring = W * Shape<NT>::STAGES * Stage<D>::BYTES;
  constexpr int merge = W * MERGE_ROW<D> * rows_of(NT) * 4;
  return ring > merge ? ring : merge;
}
template <int D, int NT, int W>
constexpr int smem_bytes(bool more) {
  return ring_bytes<D, NT, W>() + (more ? rows_of(NT) * D * 4 : 0);
}

// Where a CTA's piece of the line begins.
struct Piece {
  int begin, end;   // units
  int b, base;      // sequence of `begin`, and the units before it
  int per_cta;
};

// Cuts the line.  Every CTA adds up the lengths by itself: a few loads per
// thread, no extra launch.
__device__ __forceinline__ Piece cut(const DecArgs& a, int* sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = (a.batch + THREADS - 1) / THREADS;
  const int b0 = min(a.batch, tid * chunk), b1 = min(a.batch, b0 + chunk);
  const int per_unit = a.heads_kv * a.row_tiles;
  int sum = 0;
  for (int b = b0; b < b1; ++b) sum += units_of(clamp_len(a, b));
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) sh[warp] = incl;
  __syncthreads();
  int before = incl - sum, total = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += sh[w];
    total += sh[w];
  }
  Piece p;
  const int all = total * per_unit;
  p.per_cta = max(MIN_UNITS, (all + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x));
  p.begin = static_cast<int>(min(static_cast<long long>(all),
                                 static_cast<long long>(blockIdx.x) * p.per_cta));
  p.end = min(all, p.begin + p.per_cta);
  const int at = p.begin / per_unit;
  if (at >= before && at < before + sum) {
    int base = before;
    for (int b = b0; b < b1; ++b) {
      const int n = units_of(clamp_len(a, b));
      if (at < base + n) {
        sh[WARPS] = b;
        sh[WARPS + 1] = base * per_unit;
        break;
      }
      base += n;
    }
  }
  __syncthreads();
  p.b = sh[WARPS];
  p.base = sh[WARPS + 1];
  return p;
}

// Four elements of an output row, and with the first of them its log-sum-exp:
// `row` is the query row within the KV head's group, y and l are relative to m.
__device__ __forceinline__ void store_row4(const DecArgs& a, int b, int kvh, int row, int d0,
                                           float m, float l, float4 y) {
  const int i = row / a.group, h = kvh * a.group + (row - i * a.group);
  const float inv = l == 0.f ? 0.f : pow2f(head_exp(a.vexp, kvh)) / l;
  uint2 w;
  w.x = f32_to_x2(y.x * inv, y.y * inv, a.f16);
  w.y = f32_to_x2(y.z * inv, y.w * inv, a.f16);
  *reinterpret_cast<uint2*>(a.o + b * a.o_s[0] + h * a.o_s[1] + i * a.o_s[2] + d0) = w;
  if (a.lse != nullptr && d0 == 0)
    a.lse[h * a.lse_pitch + static_cast<long long>(b) * a.q_len + i] =
        l == 0.f ? -INFINITY : (m - SHIFT + log2f(l)) * 0.6931471805599453f;
}

// DENSE: the tokens of a page lie together in each pool, so that the strides of
// the copies are constants.
//
// RUNS: of a call whose pieces may be longer than RUN_UNITS.  The tensor cores cut
// off what they add to a sum instead of rounding it, so O falls behind by about
// 2^-24 of itself with each of a warp's tiles where values have one sign (640
// histories of 1M tokens, each in about one piece: 1.35e-3, three half steps of
// fp16).  So no more than RUN_UNITS of a segment are summed at once, 256 tiles to
// a warp (2^-16), and a CTA adds its runs in fp32.  (A kernel of its own: in one
// for all, shorter pieces paid for it, 64 x 4K 39.0 -> 39.6 us, five tokens over 16
// to 32K 119.6 -> 120.9; as it is 39.1 and 120.0.)
template <int D, int NTILES, bool DENSE, int W, bool RUNS>
__global__ void __launch_bounds__(32 * W, W <= WARPS ? Shape<NTILES>::CTAS * WARPS / W : 1)
    decode4_kernel(const DecArgs a) {
  constexpr bool HALF = NTILES == 0;
  constexpr int NT = HALF ? 1 : NTILES;       // tiles of 8 product columns
  constexpr int COLS = HALF ? 1 : 2;          // query rows of a lane in each
  constexpr int WARPS = W, THREADS = 32 * W;  // of this CTA
  constexpr int UNIT_TILES = UNIT / TOK;
  constexpr int STAGES = Shape<NTILES>::STAGES;
  constexpr int KSTEPS = D / 16;              // 16-element steps of K Q^T
  constexpr int MT = HALF ? D / 32 : D / 16;  // 16-row tiles of V^T P^T
  constexpr int ROWS = rows_of(NTILES);
  using St = Stage<D>;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ int sh_cut[WARPS + 2];
  __shared__ uint2 sh_q[NT * KSTEPS * 32];
  __shared__ float sh_sc[ROWS];
  __shared__ int sh_lim[ROWS];  // positions below it are visible to the row
  __shared__ float2 sh_ml[WARPS][ROWS];
  __shared__ float2 sh_cluster[MAX_CLUSTER][ROWS];  // of a cluster's CTAs, or carried

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  // The query row (of the CTA's) of this lane's column e of tile nt, 2c + e of the
  // tile's 8; where the rows are four, each takes two columns.
  auto col_row = [&](int nt, int e) { return HALF ? c : nt * 8 + 2 * c + e; };

  if (a.cluster > 1) cluster_arrive();
  Piece piece;
  if (W == bsfa::WARPS && a.split) {
    if (tid == 0 && !a.join_by_segment) a.joins[blockIdx.x] = make_int4(-1, 0, 0, 0);
    piece = cut(a, sh_cut);
  } else {  // one segment per cluster; u walks over it once
    const int seg = static_cast<int>(blockIdx.x) / a.cluster, per_b = a.heads_kv * a.row_tiles;
    piece.b = seg / per_b;
    const int n = units_of(clamp_len(a, piece.b));
    piece.base = 0;
    piece.begin = (seg - piece.b * per_b) * n;
    piece.end = piece.begin + n;
    piece.per_cta = n;
  }

  const uint32_t my_ring = smem_u32(ring) + warp * STAGES * St::BYTES;
  int u = piece.begin, b = piece.b, base = piece.base;
  while (u < piece.end) {
    const int len = clamp_len(a, b);
    const int n_units = units_of(len);
    const int seg = (u - base) / n_units;  // kvh * row_tiles + row tile
    const int u0 = u - base - seg * n_units;
    const int left = RUNS ? min(RUN_UNITS, piece.end - u) : piece.end - u;
    const int u1 = min(n_units, u0 + left);
    const int kvh = seg / a.row_tiles;
    const int r0 = (seg - kvh * a.row_tiles) * ROWS;  // first query row
    const int n_rows = min(ROWS, a.rows - r0);

    // Positions that the rows of this tile see: each row its own limit, all of
    // them below max_lim, and everything below min_lim by all.
    const int first_i = r0 / a.group, last_i = (r0 + n_rows - 1) / a.group;
    const int min_lim = a.causal ? max(0, len - a.q_len + first_i + 1) : len;
    const int max_lim = a.causal ? max(0, len - a.q_len + last_i + 1) : len;

    // ---- this warp's tiles: an equal run of the piece's
    int t0 = max(0, u0 - SEGMENT_UNITS) * UNIT_TILES;
    int t1 = min(max(0, u1 - SEGMENT_UNITS) * UNIT_TILES, (max_lim + TOK - 1) / TOK);
    if (a.cluster > 1) {  // this CTA's share of the segment
      const int share = (t1 + a.cluster - 1) / a.cluster;
      t0 = min(t1, static_cast<int>(cluster_rank()) * share);
      t1 = min(t1, t0 + share);
    }
    const int run = (max(0, t1 - t0) + WARPS - 1) / WARPS;
    const int t_begin = t0 + warp * run, t_end = min(t1, t_begin + run);
    const int n_tiles = max(0, t_end - t_begin);

    // ---- copies: each lane keeps its source addresses, which step through a
    // page and are formed anew where one begins; the next page's table entry is
    // in flight meanwhile.  Lanes 0-15 copy the keys' scales of a token each,
    // lanes 16-31 the values'.
    constexpr int CHUNKS = D / 32;  // 16-byte chunks of a row of codes
    const int cp_tok = lane / CHUNKS, cp_chunk = lane % CHUNKS;
    const bool cp_val = lane >= 16;
    const int32_t* table = a.table + static_cast<long long>(b) * a.table_stride;
    const int kc_st = DENSE ? D / 2 : a.kc_st, vc_st = DENSE ? D / 2 : a.vc_st;
    const int z_st = DENSE ? D / FP4_GROUP : cp_val ? a.vs_st : a.ks_st;
    const uint8_t* k_base = a.kc + kvh * a.kc_sh + (cp_tok * kc_st + cp_chunk * 16);
    const uint8_t* v_base = a.vc + kvh * a.vc_sh + (cp_tok * vc_st + cp_chunk * 16);
    const uint32_t z_sp4 = cp_val ? a.vs_sp4 : a.ks_sp4;
    const uint8_t* z_base =
        (cp_val ? a.vs + kvh * a.vs_sh : a.ks + kvh * a.ks_sh) + (lane & 15) * z_st;
    const uint32_t cp_dst = swizzle<D>(cp_tok, cp_chunk);
    int cp_left = n_tiles;                  // tiles of pages not opened yet
    int cp_col = t_begin / a.tiles_per_page;
    int cp_run = 0;                         // tiles of the open page still to copy
    int cp_entry = cp_left > 0 ? __ldg(table + cp_col) : -1;
    bool cp_ok = false;
    const uint8_t *k_src = k_base, *v_src = v_base, *z_src = z_base;
    auto open_page = [&](int off) {  // the page cp_entry names, from its tile `off`
      const bool ok = static_cast<uint32_t>(cp_entry) < static_cast<uint32_t>(a.num_pages);
      const uint32_t page = ok ? cp_entry : 0;
      const int row = off * TOK;
      cp_ok = ok;
      k_src = k_base + (static_cast<uint64_t>(page) * a.kc_sp4 << 2) + row * kc_st;
      v_src = v_base + (static_cast<uint64_t>(page) * a.vc_sp4 << 2) + row * vc_st;
      z_src = z_base + (static_cast<uint64_t>(page) * z_sp4 << 2) + row * z_st;
      cp_run = min(cp_left, a.tiles_per_page - off);
      cp_left -= cp_run;
      if (cp_left > 0) cp_entry = __ldg(table + ++cp_col);
    };
    if (cp_left > 0) open_page(t_begin - cp_col * a.tiles_per_page);
    auto copy_tile = [&](uint32_t dst) {
      if (cp_run > 0) {
        const uint32_t at = dst + cp_dst;
        if constexpr (D == 128)  // rows 8 .. 15: swizzle(t + 8) = swizzle(t) + 512
          cp_async_tile<St::CODES, D / FP4_GROUP>(at, dst + 2 * St::CODES + lane * (D / FP4_GROUP),
                                                  k_src, k_src + 8 * kc_st, v_src,
                                                  v_src + 8 * vc_st, z_src, cp_ok);
        else
          cp_async_tile<St::CODES, D / FP4_GROUP>(at, dst + 2 * St::CODES + lane * (D / FP4_GROUP),
                                                  k_src, v_src, z_src, cp_ok);
        k_src += TOK * kc_st;
        v_src += TOK * vc_st;
        z_src += TOK * z_st;
        if (--cp_run == 0 && cp_left > 0) open_page(0);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) copy_tile(my_ring + s * St::BYTES);

    // ---- queries: fragments of Q^T (fp16, a row's largest element scaled to
    // [2^14, 2^15)) and the factor that turns a product into a score in log2 units
    for (int nt = warp; nt < NT; nt += WARPS) {
      const int q_row = HALF ? g >> 1 : nt * 8 + g, r = r0 + q_row;
      float f[D / 4];
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < D / 4; ++j) f[j] = 0.f;
      if (r < a.rows) {
        const int i = r / a.group, h = kvh * a.group + (r - i * a.group);
        const uint4* src = reinterpret_cast<const uint4*>(a.q + b * a.q_s[0] + h * a.q_s[1] +
                                                          i * a.q_s[2] + c * (D / 4));
#pragma unroll
        for (int j = 0; j < D / 32; ++j) {
          const uint4 x = __ldg(src + j);
          const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 y = x2_to_f32(w[e], a.f16);
            f[8 * j + 2 * e] = y.x;
            f[8 * j + 2 * e + 1] = y.y;
            amax = fmaxf(amax, fmaxf(fabsf(y.x), fabsf(y.y)));
          }
        }
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // A row with an infinity or a NaN stays as it is: its scores are not
      // numbers in any scaling.  2^126 is the largest factor whose inverse is a
      // normal number, and it is enough: it turns bf16's least subnormal into
      // 2^-7, so a row that stays below 2^14 for it is exact in fp16.  Elsewhere
      // an element is exact that is scaled to 2^-14 or more (bf16 has 8 bits,
      // fp16 11), and one below is off by 2^-25 at most, 2^-39 of the row's
      // largest.
      const int ex = (__float_as_int(amax) >> 23) - 127;
      const int up = amax == 0.f || ex > 127 ? 0 : min(14 - ex, 126);
      const float mul = pow2f(up);
      if (c == 0) {
        // The power of two in two factors of the same sign: only a result beyond
        // fp32's range leaves it, and is cut to its largest number there, so that
        // products of zero stay scores of zero.
        const int e = head_exp(a.kexp, kvh) - up;
        sh_sc[q_row] = fminf(a.sigma_log2 * pow2f(e / 2) * pow2f(e - e / 2), FLT_MAX);
        // Rows past the last are computed along with the rest and not stored.
        sh_lim[q_row] = !a.causal || r >= a.rows ? len : len - a.q_len + r / a.group + 1;
      }
#pragma unroll
      for (int j = 0; j < KSTEPS; ++j)
        sh_q[(nt * KSTEPS + j) * 32 + lane] =
            make_uint2(pack_f16x2(f[4 * j] * mul, f[4 * j + 1] * mul),
                       pack_f16x2(f[4 * j + 2] * mul, f[4 * j + 3] * mul));
    }
    __syncthreads();

    // ---- per-lane columns: 2c and 2c + 1 of each row tile
    float acc[NT][MT][4];
    float sum[NT][COLS], sc[NT][COLS];
    float zn[NT][COLS];  // SHIFT - reference: a weight is 2^(sc * product + zn)
    uint2 qf[NT == 1 ? KSTEPS : 1];  // one row tile's queries stay in registers
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][mt][e] = 0.f;
#pragma unroll
      for (int e = 0; e < COLS; ++e) {
        zn[nt][e] = INFINITY;
        sum[nt][e] = 0.f;
        sc[nt][e] = sh_sc[col_row(nt, e)];
      }
    }
    if constexpr (NT == 1) {
#pragma unroll
      for (int j = 0; j < KSTEPS; ++j) qf[j] = sh_q[j * 32 + lane];
    }
    const uint32_t q_addr = smem_u32(sh_q) + lane * 8;
    // Row m of a 8-token half tile is token 4 (m & 1) + (m >> 1), the order in
    // which the values' fragments pair tokens.
    const int my_tok = ((g & 1) << 2) + (g >> 1);
    // This lane's places in a stage: its d/4 codes of key my_tok (key my_tok + 8
    // lies half a tile on), its d/8 codes of values c, c + 4, c + 8, c + 12 (each
    // a quarter tile on, the odd ones in the other 64 bytes of their lines).
    const uint32_t k_at = D == 128 ? swizzle<D>(my_tok, c)
                                   : swizzle<D>(my_tok, c >> 1) + (c & 1) * 8;
    const uint32_t v_at = St::CODES + (D == 128 ? swizzle<D>(c, g >> 1) + (g & 1) * 8
                                                : swizzle<D>(c, g >> 2) + (g & 3) * 4);
    const uint32_t v_at1 = v_at ^ 64u;
    const uint32_t zk_at = 2 * St::CODES + (D == 128 ? my_tok * 8 + 2 * c : my_tok * 4 + c);
    const uint32_t zv_at = 2 * St::CODES + St::SCALES + (D == 128 ? c * 8 + g : c * 4 + (g >> 1));

    auto tile = [&](const uint32_t st, const int tok0, auto masked_tag) {
      constexpr bool MASKED = decltype(masked_tag)::value;
      // ---- S^T = K Q^T.  Three row tiles leave registers for two sums per tile,
      // which halves the chain of dependent products (five tokens over 16 to 32K:
      // 121.6 -> 119.9 us).  One row tile gains nothing by it, two and four lose (64
      // ragged sequences to 16K with twelve rows 145.6 and 154.6, eight tokens over
      // 16 to 32K 148.4 and 149.8).
      constexpr int SUMS = NT == 3 ? 2 : 1;
      float s[NT][4], s2[SUMS == 2 ? NT : 1][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[nt][e] = 0.f;
          if constexpr (SUMS == 2) s2[nt][e] = 0.f;
        }
      {
        uint32_t ka[D / 32], kb[D / 32];  // d/4 codes of tokens my_tok, my_tok + 8
        uint32_t sa[2], sb[2];            // their scales, each twice
        if constexpr (D == 128) {
          const uint4 x = lds128(st + k_at), y = lds128(st + k_at + 512);
          ka[0] = x.x, ka[1] = x.y, ka[2] = x.z, ka[3] = x.w;
          kb[0] = y.x, kb[1] = y.y, kb[2] = y.z, kb[3] = y.w;
          const uint32_t za = e4m3x2_to_f16(lds16(st + zk_at));
          const uint32_t zb = e4m3x2_to_f16(lds16(st + zk_at + 64));
          sa[0] = __byte_perm(za, 0, 0x1010), sa[1] = __byte_perm(za, 0, 0x3232);
          sb[0] = __byte_perm(zb, 0, 0x1010), sb[1] = __byte_perm(zb, 0, 0x3232);
        } else {
          const uint2 x = lds64(st + k_at), y = lds64(st + k_at + 256);
          ka[0] = x.x, ka[1] = x.y;
          kb[0] = y.x, kb[1] = y.y;
          const uint32_t za = e4m3x2_to_f16(lds8(st + zk_at));
          const uint32_t zb = e4m3x2_to_f16(lds8(st + zk_at + 32));
          sa[0] = sa[1] = __byte_perm(za, 0, 0x1010);
          sb[0] = sb[1] = __byte_perm(zb, 0, 0x1010);
        }
#pragma unroll
        for (int w = 0; w < D / 32; ++w) {
          uint32_t fa[4], fb[4];
          e2m1x8_to_f16(ka[w], fa);
          e2m1x8_to_f16(kb[w], fb);
          const uint32_t xa = sa[w >> 1], xb = sb[w >> 1];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            fa[j] = mul_f16x2(fa[j], xa);
            fb[j] = mul_f16x2(fb[j], xb);
          }
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint2 q2 = NT == 1 ? qf[NT == 1 ? 2 * w + j : 0]
                                       : lds64(q_addr + (nt * KSTEPS + 2 * w + j) * 256);
              mma_f16_16816(SUMS == 2 && j ? s2[SUMS == 2 ? nt : 0] : s[nt], fa[2 * j], fb[2 * j],
                            fa[2 * j + 1], fb[2 * j + 1], q2.x, q2.y);
            }
        }
        if constexpr (SUMS == 2) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[nt][e] += s2[nt][e];
        }
      }

      // ---- weights; the reference moves where one would pass 2^(SHIFT + HEADROOM)
      float y[NT][4];
      auto lim = [&](int nt, int e) { return sh_lim[col_row(nt, e)]; };
      auto weigh = [&]() {
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; e += 3 - COLS) {  // a half tile's odd columns repeat the even
            const int col = HALF ? 0 : e & 1;
            y[nt][e] = fmaf(s[nt][e], sc[nt][col], zn[nt][col]);
            if (MASKED && tok0 + my_tok + (e & 2) * 4 >= lim(nt, col)) y[nt][e] = -INFINITY;
            over |= y[nt][e] > SHIFT + HEADROOM;
          }
        return over;
      };
      if (__any_sync(0xffffffffu, weigh())) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < COLS; ++e) {
            float lo = s[nt][e] * sc[nt][e], hi = s[nt][e + 2] * sc[nt][e];
            if (MASKED) {
              if (tok0 + my_tok >= lim(nt, e)) lo = -INFINITY;
              if (tok0 + my_tok + 8 >= lim(nt, e)) hi = -INFINITY;
            }
            const float m0 = SHIFT - zn[nt][e];
            float m1 = fmaxf(m0, fmaxf(lo, hi));
            m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, 4));
            m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, 8));
            m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, 16));
            const float f = m1 == -INFINITY ? 1.f : ex2_approx(m0 - m1);
            zn[nt][e] = SHIFT - m1;
            sum[nt][e] *= f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              acc[nt][mt][e] *= f;
              acc[nt][mt][e + 2] *= f;
              if constexpr (HALF) {
                acc[nt][mt][1] *= f;
                acc[nt][mt][3] *= f;
              }
            }
          }
        weigh();
      }
      // The products take 16-bit factors, so a weight is rounded to fp16, 2^-11 of
      // it at most; the sum l, and with it the log-sum-exp, is that of the weights
      // before.  Against 64 bits an fp16 O is off by 2.6e-4 (2-norm, 256 ragged
      // sequences to 600) where its own rounding alone is 2.1e-4, a bf16 O by its
      // rounding, 1.66e-3.  A second product with the weights' remainders makes O as
      // exact as fp32 weights do, for 104 -> 117 us at 64 ragged sequences to 16K and
      // 120 -> 151 for five tokens.
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; e += 3 - COLS) {
          y[nt][e] = ex2_approx(y[nt][e]);
          sum[nt][HALF ? 0 : e & 1] += y[nt][e];
        }
        pb[nt][0] = movmatrix_trans(pack_f16x2(y[nt][0], y[nt][HALF ? 0 : 1]));
        pb[nt][1] = movmatrix_trans(pack_f16x2(y[nt][2], y[nt][HALF ? 2 : 3]));
      }

      // ---- O^T += V^T P^T; this lane: elements [g d/8, (g + 1) d/8) of tokens c + 4j
      {
        constexpr int STEP = St::CODES / 4;  // bytes from token c + 4j to the next
        uint32_t v[4][D / 64], z[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t at = st + (j & 1 ? v_at1 : v_at) + j * STEP;
          if constexpr (D == 128) {
            const uint2 x = lds64(at);
            v[j][0] = x.x, v[j][1] = x.y;
          } else {
            v[j][0] = lds32(at);
          }
          z[j] = lds8(st + zv_at + j * (St::SCALES / 4));
        }
        if (MASKED) {
          // A hidden value weighs nothing even where it is not a number: past
          // max_lim the scale becomes 0.  Below it, a NaN that only some rows
          // see is taken out and put into those rows.
          uint32_t nans = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int t = c + 4 * j;
            if (tok0 + t >= max_lim) z[j] = 0;
            if ((z[j] & 0x7fu) == 0x7fu) {
              z[j] = 0;
              nans |= 1u << t;
            }
          }
          if (__any_sync(0xffffffffu, nans != 0)) {
            nans |= __shfl_xor_sync(0xffffffffu, nans, 1);
            nans |= __shfl_xor_sync(0xffffffffu, nans, 2);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int seen = min(max(lim(nt, e) - tok0, 0), TOK);
                if (nans & ((1u << seen) - 1u)) {
#pragma unroll
                  for (int mt = 0; mt < MT; ++mt)
                    acc[nt][mt][e] = acc[nt][mt][e + 2] = NAN;
                }
              }
          }
        }
        if constexpr (HALF) {
          // Neighbouring elements of a value stay paired: the rows of a product are
          // such pairs, its inner index is (token, which of the two), and column
          // 2r + p weighs query row r for the elements p of the pairs, with zeros at
          // the others.  No nibbles are merged, the columns that four rows leave
          // idle carry the second elements, and the products are as many.
          // After the transposition a lane of column g holds the weights of tokens
          // val_tok(0), val_tok(1) (and 2, 3) for row g / 2.
          const uint32_t first = g & 1 ? 0x1044u : 0x4410u, second = g & 1 ? 0x3244u : 0x4432u;
          uint32_t zz[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) zz[j] = e4m3x2_to_f16(z[j] * 0x101u);
#pragma unroll
          for (int step = 0; step < 2; ++step) {
            const uint32_t b0 = __byte_perm(pb[0][step], 0, first);
            const uint32_t b1 = __byte_perm(pb[0][step], 0, second);
#pragma unroll
            for (int w = 0; w < D / 64; ++w) {
              uint32_t lo[4], hi[4];
              e2m1x8_to_f16(v[2 * step][w], lo);
              e2m1x8_to_f16(v[2 * step + 1][w], hi);
#pragma unroll
              for (int j = 0; j < 2; ++j)
                mma_f16_16816(acc[0][2 * w + j], mul_f16x2(lo[2 * j], zz[2 * step]),
                              mul_f16x2(lo[2 * j + 1], zz[2 * step]),
                              mul_f16x2(hi[2 * j], zz[2 * step + 1]),
                              mul_f16x2(hi[2 * j + 1], zz[2 * step + 1]), b0, b1);
            }
          }
        } else {
          const uint32_t z01 = e4m3x2_to_f16(z[0] | z[1] << 8);
          const uint32_t z23 = e4m3x2_to_f16(z[2] | z[3] << 8);
#pragma unroll
          for (int w = 0; w < D / 64; ++w) {
            // f16x2 fragments want {token 4j', token 4j' + 4} of one element.
            const uint32_t even01 = select_low_nibbles(v[0][w], v[1][w] << 4);
            const uint32_t odd01 = select_low_nibbles(v[0][w] >> 4, v[1][w]);
            const uint32_t even23 = select_low_nibbles(v[2][w], v[3][w] << 4);
            const uint32_t odd23 = select_low_nibbles(v[2][w] >> 4, v[3][w]);
            uint32_t a0[4], a1[4], a2[4], a3[4];
            e2m1x8_to_f16(even01, a0);
            e2m1x8_to_f16(odd01, a1);
            e2m1x8_to_f16(even23, a2);
            e2m1x8_to_f16(odd23, a3);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t x0 = mul_f16x2(a0[j], z01), x1 = mul_f16x2(a1[j], z01);
              const uint32_t x2 = mul_f16x2(a2[j], z23), x3 = mul_f16x2(a3[j], z23);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16_16816(acc[nt][4 * w + j], x0, x1, x2, x3, pb[nt][0], pb[nt][1]);
            }
          }
        }
      }
    };

    uint32_t rd = my_ring, wr = my_ring + (STAGES - 1) * St::BYTES;
    const uint32_t ring_end = my_ring + STAGES * St::BYTES;
    auto next_tile = [&]() {
      cp_async_wait<STAGES - 2>();
      __syncwarp();  // every lane's copies of this tile are in, and the last one is read
      copy_tile(wr);
      const uint32_t st = rd;
      rd = rd + St::BYTES == ring_end ? my_ring : rd + St::BYTES;
      wr = wr + St::BYTES == ring_end ? my_ring : wr + St::BYTES;
      return st;
    };
    // Tiles that every row sees in whole come first; the few others take the
    // masked path in a loop of their own (one loop with a branch would move the
    // sums between registers at every join of the two).
    const int t_full = max(t_begin, min(t_end, min_lim / TOK));
    int t = t_begin;
    if constexpr (Shape<NTILES>::UNROLL) {  // the ring once around, its places constants
      for (; t + STAGES <= t_full; t += STAGES) {
#pragma unroll
        for (int x = 0; x < STAGES; ++x) {
          cp_async_wait<STAGES - 2>();
          __syncwarp();
          copy_tile(my_ring + (x + STAGES - 1) % STAGES * St::BYTES);
          tile(my_ring + x * St::BYTES, 0, std::false_type{});
        }
      }
    }
    for (; t < t_full; ++t) tile(next_tile(), 0, std::false_type{});
    for (; t < t_end; ++t) tile(next_tile(), t * TOK, std::true_type{});
    cp_async_wait<0>();

    // ---- join the warps: common reference, then one sum of the scaled parts
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < COLS; ++e) {
        float l = sum[nt][e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (g == 0) sh_ml[warp][col_row(nt, e)] = make_float2(SHIFT - zn[nt][e], l);
      }
    __syncthreads();  // also: every warp is done with its ring, which the sums reuse
    float* merge = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < COLS; ++e) {
        const int r = col_row(nt, e);
        float m = sh_ml[0][r].x;
#pragma unroll
        for (int w = 1; w < WARPS; ++w) m = fmaxf(m, sh_ml[w][r].x);
        const float f = m == -INFINITY ? 1.f : ex2_approx(SHIFT - zn[nt][e] - m);
        float* dst = merge + (warp * ROWS + r) * MERGE_ROW<D>;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if constexpr (HALF) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
              dst[merge_pos<D>(g * (D / 8) + 4 * mt + x)] = acc[nt][mt][x] * f;
          } else {
            dst[merge_pos<D>(g * (D / 8) + 2 * mt)] = acc[nt][mt][e] * f;
            dst[merge_pos<D>(g * (D / 8) + 2 * mt + 1)] = acc[nt][mt][e + 2] * f;
          }
        }
      }
    __syncthreads();
    if (a.cluster > 1) {
      // Output x of the segment (four elements) is joined by CTA x % cluster: each
      // CTA stores its sums, and the references, straight into the joining CTAs'
      // shared memory, and after one barrier every CTA adds what it got, over the
      // CTAs in order.  (Sums left in place and read remotely need a second
      // barrier and wait for the loads: 8 x 2K tokens 10.8 us, pushed 10.3.)
      const int items = ROWS * (D / 4) / a.cluster;  // the cluster is a power of two
      const uint32_t rank = cluster_rank(), got = smem_u32(ring) + ring_bytes<D, NTILES, W>();
      cluster_wait();  // the one of the kernel's beginning: every CTA runs
      for (int x = tid; x < n_rows * (D / 4); x += THREADS) {
        const int r = x / (D / 4), d0 = (x % (D / 4)) * 4;
        const float* src = merge + r * MERGE_ROW<D> + merge_pos<D>(d0);
        float4 y = make_float4(src[0], src[1], src[2], src[3]);
#pragma unroll
        for (int w = 1; w < WARPS; ++w) {
          src += ROWS * MERGE_ROW<D>;
          y.x += src[0], y.y += src[1], y.z += src[2], y.w += src[3];
        }
        cluster_st4(got + (rank * items + x / a.cluster) * 16, x % a.cluster, y);
      }
      for (int x = tid; x < n_rows * a.cluster; x += THREADS) {
        const int r = x / a.cluster;
        float m = sh_ml[0][r].x, l = 0.f;
#pragma unroll
        for (int w = 1; w < WARPS; ++w) m = fmaxf(m, sh_ml[w][r].x);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
          const float2 ml = sh_ml[w][r];
          l += m == -INFINITY ? ml.y : ml.y * ex2_approx(ml.x - m);
        }
        cluster_st2(smem_u32(&sh_cluster[rank][r]), x % a.cluster, make_float2(m, l));
      }
      cluster_arrive();
      cluster_wait();
      const float4* parts =
          reinterpret_cast<const float4*>(ring + ring_bytes<D, NTILES, W>());
      for (int k = tid; k * a.cluster + rank < n_rows * (D / 4); k += THREADS) {
        const int x = k * a.cluster + rank, r = x / (D / 4), d0 = (x % (D / 4)) * 4;
        float m = sh_cluster[0][r].x;
        for (int c1 = 1; c1 < a.cluster; ++c1) m = fmaxf(m, sh_cluster[c1][r].x);
        float l = 0.f;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c1 = 0; c1 < a.cluster; ++c1) {
          const float2 ml = sh_cluster[c1][r];
          const float4 p = parts[c1 * items + k];
          const float f = m == -INFINITY ? 1.f : ex2_approx(ml.x - m);
          l += ml.y * f;
          y.x += p.x * f, y.y += p.y * f, y.z += p.z * f, y.w += p.w * f;
        }
        store_row4(a, b, kvh, r0 + r, d0, m, l, y);
      }
      return;
    }
    // Whether the segment began in this CTA, the runs of it that the CTA has
    // summed before this one, and whether one follows.
    const int seg_begin = u - u0;
    const int cta_begin = static_cast<int>(blockIdx.x) * piece.per_cta;
    const bool began = RUNS ? seg_begin >= cta_begin : u0 == 0;
    const int carried = RUNS ? (u - max(seg_begin, cta_begin)) / RUN_UNITS : 0;
    const bool more = RUNS && u1 < n_units && u + (u1 - u0) < piece.end;
    float4* carry = reinterpret_cast<float4*>(ring + ring_bytes<D, NTILES, W>());
    float2* const carry_ml = sh_cluster[carried & 1];  // and the next run's in the other
    const bool whole = began && u1 == n_units;
    const int part = 2 * static_cast<int>(blockIdx.x) + (began ? 1 : 0);
    for (int x = tid; x < n_rows * (D / 4); x += THREADS) {
      const int r = x / (D / 4), d0 = (x % (D / 4)) * 4;
      float m = sh_ml[0][r].x;
#pragma unroll
      for (int w = 1; w < WARPS; ++w) m = fmaxf(m, sh_ml[w][r].x);
      float l = 0.f;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float2 ml = sh_ml[w][r];
        l += m == -INFINITY ? ml.y : ml.y * ex2_approx(ml.x - m);
        const float* src = merge + (w * ROWS + r) * MERGE_ROW<D> + merge_pos<D>(d0);
        y.x += src[0], y.y += src[1], y.z += src[2], y.w += src[3];
      }
      if (RUNS && carried > 0) {
        const float2 ml = carry_ml[r];
        const float4 z = carry[x];
        const float m1 = fmaxf(m, ml.x);
        const float f = m1 == -INFINITY ? 1.f : ex2_approx(m - m1);
        const float fz = m1 == -INFINITY ? 1.f : ex2_approx(ml.x - m1);
        m = m1;
        l = l * f + ml.y * fz;
        y.x = y.x * f + z.x * fz, y.y = y.y * f + z.y * fz;
        y.z = y.z * f + z.z * fz, y.w = y.w * f + z.w * fz;
      }
      if (more) {
        carry[x] = y;
        if (d0 == 0) sh_cluster[(carried & 1) ^ 1][r] = make_float2(m, l);
      } else if (whole) {
        store_row4(a, b, kvh, r0 + r, d0, m, l, y);
      } else {
        *reinterpret_cast<float4*>(
            a.part_o + (static_cast<long long>(part) * ROWS + r) * D + d0) = y;
        if (d0 == 0) a.part_ml[static_cast<long long>(part) * ROWS + r] = make_float2(m, l);
      }
    }
    if (began && !more && tid == 0) {
      const int4 job =
          make_int4(whole ? -1 : b, seg, blockIdx.x, (seg_begin + n_units - 1) / piece.per_cta);
      if (a.join_by_segment)
        a.joins[b * a.heads_kv * a.row_tiles + seg] = job;
      else if (!whole)
        a.joins[blockIdx.x] = job;
    }
    __syncthreads();  // the ring and sh_ml are free again

    u += u1 - u0;
    if (u1 == n_units && seg == a.heads_kv * a.row_tiles - 1) {
      base += n_units * a.heads_kv * a.row_tiles;
      ++b;
    }
  }
}

// Joins the parts of the segments that a cut crossed: block (x, r) takes row r
// of job x, which is segment x, or where there are more segments than CTAs the
// one that CTA x began and did not finish -- if that was cut.  The parts lie in
// the CTAs first (its second slot) .. last (their first slots).  The references
// come first, all at once, so that the sums' loads wait for nothing.  Four blocks
// to an SM are asked for: left to itself the compiler keeps to 32 registers and
// spills at d = 128 (61 registers; 1 x 128K: 34.4 -> 32.9 us).
template <int D, int ROWS>
__global__ void __launch_bounds__(JOIN_THREADS, 4) decode4_join_kernel(const DecArgs a) {
  constexpr int LANES = D / 4;                 // threads that cover a row, four elements each
  constexpr int PARTS = JOIN_THREADS / LANES;  // parts read at once
  __shared__ float4 sh_y[PARTS][LANES];
  __shared__ float2 sh_ml[JOIN_THREADS / 32];
  __shared__ float sh_w[MAX_PARTS];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 job = a.joins[blockIdx.x];
  if (job.x < 0) return;
  const int b = job.x, kvh = job.y / a.row_tiles;
  const int r = blockIdx.y, row = (job.y - kvh * a.row_tiles) * ROWS + r;
  if (row >= a.rows) return;
  const int first = job.z, count = job.w - first + 1;  // at most the CTAs, so MAX_PARTS
  const int tid = threadIdx.x;
  auto slot = [&](int p) { return 2LL * (first + p) + (p == 0 ? 1 : 0); };

  float2 mine[MAX_PARTS / JOIN_THREADS];
  float m = -INFINITY;
#pragma unroll
  for (int x = 0; x < MAX_PARTS / JOIN_THREADS; ++x) {
    const int p = tid + x * JOIN_THREADS;
    mine[x] = p < count ? a.part_ml[slot(p) * ROWS + r] : make_float2(-INFINITY, 0.f);
    m = fmaxf(m, mine[x].x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((tid & 31) == 0) sh_ml[tid >> 5].x = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < JOIN_THREADS / 32; ++w) m = fmaxf(m, sh_ml[w].x);
  float l = 0.f;
#pragma unroll
  for (int x = 0; x < MAX_PARTS / JOIN_THREADS; ++x) {
    const float w = m == -INFINITY ? 1.f : ex2_approx(mine[x].x - m);
    l += mine[x].y * w;
    sh_w[tid + x * JOIN_THREADS] = w;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if ((tid & 31) == 0) sh_ml[tid >> 5].y = l;
  __syncthreads();
  l = 0.f;
#pragma unroll
  for (int w = 0; w < JOIN_THREADS / 32; ++w) l += sh_ml[w].y;

  const int lane = tid % LANES, p0 = tid / LANES;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int p = p0; p < count; p += PARTS) {
    const float4 x = reinterpret_cast<const float4*>(a.part_o + (slot(p) * ROWS + r) * D)[lane];
    const float w = sh_w[p];
    y.x += x.x * w, y.y += x.y * w, y.z += x.z * w, y.w += x.w * w;
  }
  sh_y[p0][lane] = y;
  __syncthreads();
  if (p0 != 0) return;
#pragma unroll
  for (int p = 1; p < PARTS; ++p) {
    const float4 x = sh_y[p][lane];
    y.x += x.x, y.y += x.y, y.z += x.z, y.w += x.w;
  }
  store_row4(a, b, kvh, row, 4 * lane, m, l, y);
}

// The same where segments have few parts: a warp takes a row of job x by itself,
// 32 parts' references at a time (by rows and by blocks: 64 ragged sequences to
// 16K, about one part to a row, 104.1 and 106.8 us; five tokens over 16 ragged
// sequences to 32K, two, 119.3 and 122.7; 12 x 32K, six, 76.4 and 75.9; 8 x 64K,
// ten, 99.3 and 98.0; 4 x 64K, 19, 57.6 and 55.2; 1 x 128K, 76, 44.4 and 34.4).  The
// choice goes by the average, which one long history among many short ones
// misleads: 300 of 20 tokens and one of 128K on one KV head take 47.4 us, by blocks
// 21.1.
template <int D, int ROWS>
__global__ void __launch_bounds__(JOIN_THREADS) decode4_join_rows_kernel(const DecArgs a) {
  constexpr int E = D / 32;  // elements of a lane
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 job = a.joins[blockIdx.x];
  if (job.x < 0) return;
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.y * (JOIN_THREADS / 32) + (threadIdx.x >> 5);
  const int b = job.x, kvh = job.y / a.row_tiles;
  const int row = (job.y - kvh * a.row_tiles) * ROWS + r;
  if (r >= ROWS || row >= a.rows) return;
  const int first = job.z, count = job.w - first + 1;
  auto slot = [&](int p) { return 2LL * (first + p) + (p == 0 ? 1 : 0); };
  float m = -INFINITY, l = 0.f, y[E];
#pragma unroll
  for (int e = 0; e < E; ++e) y[e] = 0.f;
  for (int p0 = 0; p0 < count; p0 += 32) {
    const float2 ml = p0 + lane < count ? a.part_ml[slot(p0 + lane) * ROWS + r]
                                        : make_float2(-INFINITY, 0.f);
    float m1 = fmaxf(m, ml.x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
    const float f = m1 == -INFINITY ? 1.f : ex2_approx(m - m1);
    const float w = m1 == -INFINITY ? 1.f : ex2_approx(ml.x - m1);
    float sum = ml.y * w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    m = m1;
    l = l * f + sum;
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] *= f;
#pragma unroll 4
    for (int p = p0; p < min(count, p0 + 32); ++p) {
      const float wp = __shfl_sync(0xffffffffu, w, p - p0);
      const float* x = a.part_o + (slot(p) * ROWS + r) * D + lane * E;
      if constexpr (E == 4) {
        const float4 z = *reinterpret_cast<const float4*>(x);
        y[0] += z.x * wp, y[1] += z.y * wp, y[2] += z.z * wp, y[3] += z.w * wp;
      } else {
        const float2 z = *reinterpret_cast<const float2*>(x);
        y[0] += z.x * wp, y[1] += z.y * wp;
      }
    }
  }
  if constexpr (E == 4) {
    store_row4(a, b, kvh, row, 4 * lane, m, l, make_float4(y[0], y[1], y[2], y[3]));
  } else {  // two lanes' elements to one store
    const float z0 = __shfl_down_sync(0xffffffffu, y[0], 1);
    const float z1 = __shfl_down_sync(0xffffffffu, y[1], 1);
    if ((lane & 1) == 0)
      store_row4(a, b, kvh, row, 2 * lane, m, l, make_float4(y[0], y[1], z0, z1));
  }
}

// Query row tiles of a call: as few tensor-core columns as hold its rows, up
// to 32 to a CTA, and equal shares where one CTA does not hold them.
struct Plan {
  int nt, row_tiles, units, max_grid, warps, cluster;
  long long segments, all_units;
  bool split;
};

Plan plan_of(const bsfa_cache4* c, const bsfa_decode4_params* p) {
  Plan pl;
  const long long rows = static_cast<long long>(p->num_heads_q / c->num_heads_kv) * p->q_len;
  const long long eights = rows > 0 ? (rows + 7) / 8 : 1;
  pl.row_tiles = static_cast<int>((eights + 3) / 4);
  pl.nt = static_cast<int>((eights + pl.row_tiles - 1) / pl.row_tiles);
  pl.units = (p->max_seqlen + UNIT - 1) / UNIT;
  if (pl.units < 1) pl.units = 1;
  pl.segments = static_cast<long long>(p->batch) * c->num_heads_kv * pl.row_tiles;
  // (Beyond 2^31 segments, which are refused, the product could overflow.)
  pl.all_units =
      pl.segments >> 31 ? pl.segments : pl.segments * (pl.units + SEGMENT_UNITS);
  if (rows <= 4) pl.nt = 0;
  constexpr int grids[5] = {Shape<0>::MAX_GRID, Shape<1>::MAX_GRID, Shape<2>::MAX_GRID,
                            Shape<3>::MAX_GRID, Shape<4>::MAX_GRID};
  pl.max_grid = grids[pl.nt];
  // CTAs of other sizes than four warps are for eight query rows at most: a thread
  // of more needs over 128 registers, which a CTA of 16 warps does not have, and
  // CTAs of two were not tried there.
  // Few segments, of half a thousand tokens or more: a CTA of 16 warps to an SM
  // (19 ragged sequences to 1024: 13.8 -> 9.5 us; 1 x 4097: 9.4 -> 8.8; 1 x 300
  // would go from 6.6 to 7.1).  Otherwise CTAs of four, or where those would not
  // all be resident at once of two (256 ragged sequences to 128, 8 heads: 21.3 ->
  // 16.0 us; 128 to 512: 21.6 -> 17.9; of one: 17.9, 18.1).
  // Of CTAs of four and sixteen a segment gets as many as keep them all resident
  // at once; eight of sixteen only up to 64 CTAs in all (2 x 16K, 128 of them: 27
  // us, cut 19), since a cluster lies within one GPC.
  pl.warps = WARPS;
  if (pl.nt <= 1) {
    if (pl.segments <= WIDE_GRID && pl.units >= WIDE_LEAST)
      pl.warps = WIDE_WARPS;
    else if (pl.segments > pl.max_grid)
      pl.warps = SMALL_WARPS;
  }
  pl.cluster = 1;
  while (pl.warps >= WARPS && pl.cluster < MAX_CLUSTER && pl.units >= 2 * pl.cluster) {
    const int next = 2 * pl.cluster;
    const int resident = pl.warps == WARPS       ? pl.max_grid
                         : next == MAX_CLUSTER ? WIDE_GRID_OF_8
                                                 : WIDE_GRID;
    if (pl.segments * next > resident) break;
    pl.cluster = next;
  }
  // Longer segments are cut.  Wide CTAs stay ahead of the cut for twice as long
  // where they fill more than half of the GPU (4 x 16K: 21.8 and 24.4 us, 1 x 32K:
  // 20.5 and 18.8).
  int most = pl.warps == SMALL_WARPS ? SMALL_UNITS : CLUSTER_UNITS;
  if (pl.warps == WIDE_WARPS)
    most = 2 * pl.segments * pl.cluster > WIDE_GRID ? 2 * WIDE_UNITS : WIDE_UNITS;
  pl.split = pl.units > most * pl.cluster;
  if (pl.split) pl.cluster = 1, pl.warps = WARPS;
  return pl;
}

struct Carve {
  size_t part_o, part_ml, joins, bytes;
};

Carve carve(const Plan& pl, int d) {
  Carve c{};
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  const size_t grid = pl.split ? static_cast<size_t>(pl.max_grid) : 0, rows = rows_of(pl.nt);
  c.part_o = 0;
  c.part_ml = up(c.part_o + grid * 2 * rows * d * sizeof(float));
  c.joins = up(c.part_ml + grid * 2 * rows * sizeof(float2));
  c.bytes = up(c.joins + grid * sizeof(int4));
  return c;
}

bsfa_status validate_sizes(const bsfa_cache4* c, const bsfa_decode4_params* p) {
  if (c == nullptr || p == nullptr) return BSFA_ERR_INVALID_ARG;
  if (p->batch < 0 || p->q_len < 0 || p->max_seqlen < 0) return BSFA_ERR_INVALID_ARG;
  const bsfa_status v = validate_cache4(c);
  if (v != BSFA_OK) return v;
  if (p->num_heads_q <= 0 || p->num_heads_q % c->num_heads_kv) return BSFA_ERR_INVALID_ARG;
  if (p->dtype != BSFA_DTYPE_BF16 && p->dtype != BSFA_DTYPE_F16) return BSFA_ERR_UNSUPPORTED;
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

// The status of a runtime call.  The runtime keeps the error of one that failed
// until it is asked for it: asked here, a later launch does not report it as its
// own.
bsfa_status status_of(cudaError_t e) {
  if (e == cudaSuccess) return BSFA_OK;
  cudaGetLastError();
  return BSFA_ERR_CUDA;
}

// Sets a kernel's shared-memory size, once per device.
template <int D, int NT, bool DENSE, int W, bool RUNS>
bsfa_status prepare(int dev) {
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (ready.load(std::memory_order_relaxed) & bit) return BSFA_OK;
  const bsfa_status v = status_of(cudaFuncSetAttribute(decode4_kernel<D, NT, DENSE, W, RUNS>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       smem_bytes<D, NT, W>(true)));
  if (v == BSFA_OK) ready.fetch_or(bit, std::memory_order_relaxed);
  return v;
}

// The first kernel of a call that cuts.
template <int D, int NT, bool DENSE, bool RUNS>
bsfa_status launch_cut(const DecArgs& a, int grid, int dev, cudaStream_t stream) {
  const bsfa_status v = prepare<D, NT, DENSE, WARPS, RUNS>(dev);
  if (v != BSFA_OK) return v;
  decode4_kernel<D, NT, DENSE, WARPS, RUNS>
      <<<static_cast<unsigned>(grid), THREADS, smem_bytes<D, NT, WARPS>(RUNS), stream>>>(a);
  return status_of(cudaGetLastError());
}

template <int D, int NT, bool DENSE, int W = WARPS>
bsfa_status launch(const DecArgs& args, const Plan& pl, int sms, int dev, cudaStream_t stream) {
  static_assert(Shape<NT>::MAX_GRID <= MAX_PARTS, "the join's weights");
  if (!pl.split) {
    const bsfa_status v = prepare<D, NT, DENSE, W, false>(dev);
    if (v != BSFA_OK) return v;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(pl.segments * pl.cluster));
    cfg.blockDim = dim3(32 * W);
    cfg.dynamicSmemBytes = smem_bytes<D, NT, W>(pl.cluster > 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = pl.cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return status_of(cudaLaunchKernelEx(&cfg, decode4_kernel<D, NT, DENSE, W, false>, args));
  }
  if constexpr (W == WARPS) {  // other CTAs never cut
    const long long full = static_cast<long long>(sms) * Shape<NT>::CTAS;
    int grid = static_cast<int>(full < pl.max_grid ? full : pl.max_grid);
    const long long most = (pl.all_units + MIN_UNITS - 1) / MIN_UNITS;
    if (most < grid) grid = static_cast<int>(most);
    DecArgs a = args;
    a.join_by_segment = pl.segments <= grid;
    // The lengths' bound bounds the pieces.
    const bool runs = (pl.all_units + grid - 1) / grid > RUN_UNITS;
    const bsfa_status v = runs ? launch_cut<D, NT, DENSE, true>(a, grid, dev, stream)
                               : launch_cut<D, NT, DENSE, false>(a, grid, dev, stream);
    if (v != BSFA_OK) return v;
    // About grid / segments parts to a segment.
    const bool by_rows = grid < JOIN_ROWS_PARTS * pl.segments;
    constexpr int ROWS = rows_of(NT);
    const int rows = a.rows < ROWS ? a.rows : ROWS, per_block = by_rows ? JOIN_THREADS / 32 : 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(a.join_by_segment ? pl.segments : grid),
                       (rows + per_block - 1) / per_block);
    cfg.blockDim = dim3(JOIN_THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return status_of(by_rows ? cudaLaunchKernelEx(&cfg, decode4_join_rows_kernel<D, ROWS>, a)
                             : cudaLaunchKernelEx(&cfg, decode4_join_kernel<D, ROWS>, a));
  }
  return BSFA_ERR_CUDA;
}

}  // namespace

}  // namespace bsfa

using namespace bsfa;

extern "C" {

size_t bsfa_decode4_workspace_size(const bsfa_cache4* cache, const bsfa_decode4_params* p) {
  if (validate_sizes(cache, p) != BSFA_OK) return 0;
  return carve(plan_of(cache, p), cache->head_dim).bytes;
}

bsfa_status bsfa_decode4(const bsfa_cache4* cache, const bsfa_decode4_params* p,
                         bsfa_stream_t stream_) {
  bsfa_status v = validate_sizes(cache, p);
  if (v != BSFA_OK) return v;
  if (p->batch == 0 || p->q_len == 0) return BSFA_OK;
  v = validate_cache4_pointers(cache);
  if (v != BSFA_OK) return v;
  if (!p->q || !p->o || !p->seqlens) return BSFA_ERR_INVALID_ARG;
  const int64_t extent[3] = {p->batch, p->num_heads_q, p->q_len};
  if (!rows_aligned(p->q, p->q_stride, extent) || !rows_aligned(p->o, p->o_stride, extent))
    return BSFA_ERR_UNSUPPORTED;
  const Plan pl = plan_of(cache, p);
  const Carve cv = carve(pl, cache->head_dim);
  if (pl.split && (p->workspace == nullptr || (reinterpret_cast<uintptr_t>(p->workspace) & 255u) ||
                   p->workspace_bytes < cv.bytes))
    return BSFA_ERR_WORKSPACE;

  DecArgs a{};
  a.kc = cache->k;
  a.vc = cache->v;
  a.ks = cache->k_scale;
  a.vs = cache->v_scale;
  a.kexp = cache->k_exp;
  a.vexp = cache->v_exp;
  auto strides = [](const int64_t (&s)[3], uint32_t& page, long long& head, int& token) {
    page = static_cast<uint32_t>(s[0] >> 2);  // validate_cache4_pointers() bounds both
    head = s[1];
    token = static_cast<int>(s[2]);
  };
  strides(cache->k_stride, a.kc_sp4, a.kc_sh, a.kc_st);
  strides(cache->v_stride, a.vc_sp4, a.vc_sh, a.vc_st);
  strides(cache->k_scale_stride, a.ks_sp4, a.ks_sh, a.ks_st);
  strides(cache->v_scale_stride, a.vs_sp4, a.vs_sh, a.vs_st);
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
  a.lse = p->lse;
  a.lse_pitch = static_cast<long long>(p->batch) * p->q_len;
  uint8_t* ws = static_cast<uint8_t*>(p->workspace);
  a.part_o = reinterpret_cast<float*>(ws + cv.part_o);
  a.part_ml = reinterpret_cast<float2*>(ws + cv.part_ml);
  a.joins = reinterpret_cast<int4*>(ws + cv.joins);

  int dev = 0, sms = 0;
  v = status_of(cudaGetDevice(&dev));
  if (v != BSFA_OK) return v;
  v = status_of(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
  if (v != BSFA_OK || sms <= 0) return BSFA_ERR_CUDA;
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  const int row = cache->head_dim / 2, z = cache->head_dim / FP4_GROUP;
  const bool dense = cache->k_stride[2] == row && cache->v_stride[2] == row &&
                     cache->k_scale_stride[2] == z && cache->v_scale_stride[2] == z;
  using Launch = bsfa_status (*)(const DecArgs&, const Plan&, int, int, cudaStream_t);
#define BSFA_LAUNCHES(D, DENSE)                                                          \
  {launch<D, 0, DENSE>,    launch<D, 1, DENSE>, launch<D, 2, DENSE>, launch<D, 3, DENSE>, \
   launch<D, 4, DENSE>,    launch<D, 0, DENSE, SMALL_WARPS>,                              \
   launch<D, 1, DENSE, SMALL_WARPS>, launch<D, 0, DENSE, WIDE_WARPS>,                     \
   launch<D, 1, DENSE, WIDE_WARPS>}
  static const Launch launches[2][2][9] = {
      // [d = 128][dense][tiles of 8 query rows (0: half a one), or small or wide CTAs]
      {BSFA_LAUNCHES(64, false), BSFA_LAUNCHES(64, true)},
      {BSFA_LAUNCHES(128, false), BSFA_LAUNCHES(128, true)}};
#undef BSFA_LAUNCHES
  const int which = pl.nt + (pl.warps == WARPS ? 0 : pl.warps == SMALL_WARPS ? 5 : 7);
  return launches[cache->head_dim == 128][dense][which](a, pl, sms, dev, stream);
}

}  // extern "C"
