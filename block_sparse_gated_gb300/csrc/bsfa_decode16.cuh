// bsfa_decode16.cuh -- the kernels of bsfa_decode16: attention of a few new tokens
// per sequence over the 16-bit paged cache.
//
// Mathematics.  S^T = K Q^T and O^T = V^T P^T are tensor-core products of 16-bit
// factors with fp32 sums.  The softmax is streamed: a weight is p = 2^(y + z) with y
// the score in log2 units and z the row's offset, which falls, with O and the sum l
// rescaled, only when some weight would pass 2^(shift + HEADROOM).  The factor 2^shift
// that p carries cancels in O / l.  In fp16 it keeps small weights out of the
// subnormals: 2^10, with values up to 2^16 far from fp32's end.  bf16 values reach to
// that end: there it is 2^-(HEADROOM + log2 of the lengths' bound), so that the weights
// of all tokens add up to one at most and O stays within the largest value.
//
// Layout.  Cached tokens are the rows (M) of the products and query rows
// (Hq/Hkv heads times q_len tokens) the columns (N = 8 per tile), so that a decode
// step of up to 8 query heads per KV head wastes no tensor work.  Each warp streams
// its own 16-token tiles through a private ring of asynchronous copies; no barrier
// is met inside a segment.
//
// Work split.  A segment is one (sequence, KV head, row tile).  Where it is short by
// the caller's bound, a CTA takes it, or a cluster of up to sixteen, which joins its
// sums through distributed shared memory: one launch, no workspace.  Longer ones are
// counted in units of 64 tokens; the units of all segments form one line, which is
// cut into equal pieces, one per CTA, from the lengths on the device.  Long and
// short sequences balance without the host knowing them, and a captured call stays
// right as they grow.  A segment that a cut crosses leaves partial sums in the
// workspace, which a second kernel joins in a fixed order.
//
// Bound.  512 bytes per (token, KV head) at d = 128, and 4 flops of a query row to
// each two of them: HBM.  64 ragged sequences to 16K (2.25 GB) take 321 us, 7.0 TB/s
// where a copy runs at 6.79; the issue slots are 18% used there, the tensor pipe 14%.
// Twenty rows leave 255 registers to a thread and eight warps to an SM, so that fixed
// latencies show: five tokens over 16 ragged sequences to 32K 226 us, 6.2 TB/s.  More
// than 32 rows are bsfa_decode16_wide.cuh's.
#pragma once
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "bsfa.h"
#include "fp4.cuh"

namespace bsfa {

namespace decode16 {

constexpr int WARPS = 4;
constexpr int THREADS = 32 * WARPS;
constexpr int TOK = 16;             // tokens of a warp's tile
constexpr int UNIT = TOK * WARPS;   // tokens of a work unit
constexpr float HEADROOM = 5.f;     // log2 a weight may pass 2^shift by
constexpr float SHIFT_F16 = 10.f;   // log2 of the factor that a weight carries in fp16
constexpr float NO_SCORE = 3e38f;   // a row's offset before its first score
constexpr int MIN_UNITS = 4;        // shortest piece of the line worth a CTA
// A segment's fixed cost, in units (128 ragged sequences to 2K, cut, and 1 x 128K: 90.2
// and 84.0 us; at 1 96.4 and 85.5, at 5 89.6 and 84.7).
constexpr int SEGMENT_UNITS = 3;
// A call is wide from that many query rows of a KV head on, if the lengths' bound and
// the segments allow (64 ragged sequences to 16K with 16 rows 335 us, wide 347; five
// tokens of four heads over 16 to 32K, 20 rows, 227 and 232; 32 rows 224 and 226; 33
// rows, two row tiles, 172 and 102; 128 rows over 4 x 300 tokens 21.9 and 23.3, over
// 16 x 600 35.0 and 32.5).
constexpr int WIDE_ROWS = 32;
constexpr int WIDE_LEAST = 512;
constexpr int WIDE_SEGMENTS = 1 << 16;
constexpr int JOIN_THREADS = 256;   // of the kernel that joins parts
constexpr int JOIN_ROWS_PARTS = 8;  // a warp to a row below, a block above
constexpr int MAX_PARTS = 768;      // parts of a segment, at most: CTAs of a cut call
constexpr int SMS = 152;            // of the GPU
constexpr int MAX_SMS = 160;        // that a workspace is good for
constexpr int MAX_CLUSTER = 16;     // CTAs that share a segment, at most
constexpr int GRID_OF_16 = 128;     // CTAs of a call in clusters of that size, at most
constexpr int CLUSTER_UNITS = 16;   // units of a segment per CTA of a cluster, at most
constexpr int SMALL_WARPS = 1;      // warps of a CTA where there are many segments
constexpr int SMALL_NT = 2;         // ... and at most so many tiles of query rows
constexpr int SMALL_UNITS = 4;      // ... and units of a segment

// Per head dimension and row-tile width: CTAs of four warps on an SM, tiles in a
// warp's ring, and the most CTAs a cut call has (the workspace holds two partial
// results each).  At d = 64 two CTAs with rings of six tiles leave 256 sequences of 600
// tokens on two heads a second wave, 15.8 us, four with three tiles 12.3.  At d = 128 a
// third CTA with rings of two tiles gains nothing (64 ragged sequences to 16K 320 us
// both), and two with them lose (324).
template <int CTAS_, int STAGES_>
struct ShapeOf {
  static constexpr int CTAS = CTAS_, STAGES = STAGES_, MAX_GRID = MAX_SMS * CTAS;
};
template <int D, int NT>
struct Shape : ShapeOf<2, 3> {};
template <>
struct Shape<64, 1> : ShapeOf<4, 3> {};
template <>
struct Shape<64, 2> : ShapeOf<3, 4> {};
template <>
struct Shape<64, 3> : ShapeOf<2, 6> {};
template <>
struct Shape<64, 4> : ShapeOf<2, 6> {};

template <int D>
constexpr int HALF_BYTES = TOK * D * 2;  // of a tile's keys, or values
template <int D>
constexpr int STAGE_BYTES = 2 * HALF_BYTES<D>;

// Row stride of a warp's sums in shared memory, in floats: the eight elements and
// four columns of a fragment fall into different banks.
template <int D>
constexpr int MERGE_ROW = D + 4;

// Dynamic shared memory: the rings, whose place the warps' sums take later, and
// behind them what the CTAs of a cluster send each other.
template <int D, int NT, int W>
constexpr int ring_bytes() {
  constexpr int ring = W * Shape<D, NT>::STAGES * STAGE_BYTES<D>;
  constexpr int merge = W * MERGE_ROW<D> * 8 * NT * 4;
  return ring > merge ? ring : merge;
}
template <int D, int NT, int W>
constexpr int smem_bytes(bool cluster) {
  return ring_bytes<D, NT, W>() + (cluster ? 8 * NT * D * 4 : 0);
}

struct DecArgs {
  const uint8_t *k, *v;
  long long k_sp, k_sh, v_sp, v_sh;  // page and head strides in bytes
  int k_st, v_st;                    // token strides in bytes
  const int32_t* table;
  int table_stride, num_pages, tiles_per_page;
  const uint16_t* q;
  uint16_t* o;
  long long q_s[3], o_s[3];
  const int32_t* seqlens;
  int batch, heads_kv, group, q_len, rows, row_tiles, max_len;
  int causal, f16, split, cluster, join_by_segment;
  float sigma_log2;
  float shift, most;  // log2 of the factor that a bf16 weight carries, and of the largest one
  float* lse;
  long long lse_pitch;
  float* part_o;    // [grid][2][rows of a CTA][d]
  float2* part_ml;  // [grid][2][rows of a CTA]
  unsigned* err;    // the device error word (wide calls)
  int box;          // tokens of a copy (wide calls)
  int in_place;     // o is q
  // [jobs]: {sequence, kvh * row_tiles + row tile, first, last CTA}; x < 0: none, w < 0: the
  // segment lies within its first CTA.
  int4* joins;
  // Wide calls, of segments that lie within a CTA: [segments][4], a bit for each row that is
  // formed anew (form_anew), and where the output is the queries [batch][KV heads][rows][d],
  // the queries of such rows.
  uint32_t* anew;
  uint16_t* kept;
};

// log2 of the factor that a weight carries, and of the largest weight before the
// offset falls.
template <bool F16>
__device__ __forceinline__ float shift_of(const DecArgs& a) {
  return F16 ? SHIFT_F16 : a.shift;
}
template <bool F16>
__device__ __forceinline__ float most_of(const DecArgs& a) {
  return F16 ? SHIFT_F16 + HEADROOM : a.most;
}

// The sequence length that the call sees.
__device__ __forceinline__ int clamp_len(const DecArgs& a, int b) {
  return max(0, min(__ldg(a.seqlens + b), a.max_len));
}
// Units of a segment on the line: its tokens', and what a CTA spends on any segment
// (queries, the first copies' latency, the join of its warps).
template <int U = UNIT, int FIXED = SEGMENT_UNITS>
__device__ __forceinline__ int units_of(int len) {
  return FIXED + (len + U - 1) / U;
}

// Where a CTA's piece of the line begins.
struct Piece {
  int begin, end;   // units
  int b, base;      // sequence of `begin`, and the units before it
  int per_cta;
};

// Cuts the line.  Every CTA adds up the lengths by itself: a few loads per
// thread, no extra launch.
template <int U, int FIXED, int LEAST, int WARPS>
__device__ __forceinline__ Piece cut(const DecArgs& a, int* sh) {
  constexpr int THREADS = 32 * WARPS;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int chunk = (a.batch + THREADS - 1) / THREADS;
  const int b0 = min(a.batch, tid * chunk), b1 = min(a.batch, b0 + chunk);
  const int per_unit = a.heads_kv * a.row_tiles;
  int sum = 0;
  for (int b = b0; b < b1; ++b) sum += units_of<U, FIXED>(clamp_len(a, b));
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
  p.per_cta = max(LEAST, (all + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x));
  p.begin = static_cast<int>(min(static_cast<long long>(all),
                                 static_cast<long long>(blockIdx.x) * p.per_cta));
  p.end = min(all, p.begin + p.per_cta);
  const int at = p.begin / per_unit;
  if (at >= before && at < before + sum) {
    int base = before;
    for (int b = b0; b < b1; ++b) {
      const int n = units_of<U, FIXED>(clamp_len(a, b));
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

// An output row: `row` is the query row within the KV head's group.
__device__ __forceinline__ uint16_t* output_row(const DecArgs& a, int b, int kvh, int row) {
  const int i = row / a.group, h = kvh * a.group + (row - i * a.group);
  return a.o + b * a.o_s[0] + h * a.o_s[1] + i * a.o_s[2];
}

// A row's log-sum-exp, where the call wants it; l is relative to 2^m.
__device__ __forceinline__ void store_lse(const DecArgs& a, int b, int kvh, int row, float m,
                                          float l) {
  if (a.lse == nullptr) return;
  const int i = row / a.group, h = kvh * a.group + (row - i * a.group);
  a.lse[h * a.lse_pitch + static_cast<long long>(b) * a.q_len + i] =
      l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Four elements of an output row, and with the first of them its log-sum-exp:
// y and l are relative to 2^m.
__device__ __forceinline__ void store_row4(const DecArgs& a, int b, int kvh, int row, int d0,
                                           float m, float l, float4 y) {
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint2 w;
  w.x = f32_to_x2(y.x * inv, y.y * inv, a.f16);
  w.y = f32_to_x2(y.z * inv, y.w * inv, a.f16);
  *reinterpret_cast<uint2*>(output_row(a, b, kvh, row) + d0) = w;
  if (d0 == 0) store_lse(a, b, kvh, row, m, l);
}

template <bool F16>
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  if constexpr (F16)
    mma_f16_16816(c, a[0], a[1], a[2], a[3], b0, b1);
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four 8 x 8 matrices of 16-bit elements, row pointers from the lanes in order;
// transposed, or as they lie.
__device__ __forceinline__ void ldmatrix(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// Two elements, those that are not finite as zeros.
template <bool F16>
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t x) {
  constexpr uint32_t LOW = F16 ? 0x7c00u : 0x7f80u, HIGH = LOW << 16;
  if ((x & LOW) == LOW) x &= 0xffff0000u;
  if ((x & HIGH) == HIGH) x &= 0xffffu;
  return x;
}

// Four 16-byte copies, `step` bytes of global memory apart; `ok` false reads
// nothing and writes zeros.
__device__ __forceinline__ void cp_async4(uint32_t d0, uint32_t d1, uint32_t d2, uint32_t d3,
                                          const uint8_t* src, int step, bool ok) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %8, 0;\n\t"
      "cp.async.cg.shared.global [%0], [%4], 16, p;\n\t"
      "cp.async.cg.shared.global [%1], [%5], 16, p;\n\t"
      "cp.async.cg.shared.global [%2], [%6], 16, p;\n\t"
      "cp.async.cg.shared.global [%3], [%7], 16, p;\n\t}" ::"r"(d0),
      "r"(d1), "r"(d2), "r"(d3), "l"(src), "l"(src + step), "l"(src + 2 * step),
      "l"(src + 3 * step), "r"(static_cast<uint32_t>(ok))
      : "memory");
}

template <int D, int NT, bool F16, int W>
__global__ void __launch_bounds__(32 * W, Shape<D, NT>::CTAS * decode16::WARPS / W)
    decode16_kernel(const __grid_constant__ DecArgs a) {
  constexpr int WARPS = W, THREADS = 32 * W;  // of this CTA
  constexpr int UNIT_TILES = UNIT / TOK;
  constexpr int STAGES = Shape<D, NT>::STAGES, STAGE = STAGE_BYTES<D>, HALF = HALF_BYTES<D>;
  constexpr int KSTEPS = D / 16;  // 16-element steps of K Q^T
  constexpr int MT = D / 16;      // 16-row tiles of V^T P^T
  constexpr int ROWS = 8 * NT;
  constexpr int PITCH = 2 * D;    // bytes of a row
  constexpr int CHUNKS = D / 8;   // ... in pieces of 16
  extern __shared__ __align__(1024) uint8_t ring[];
  __shared__ int sh_cut[WARPS + 2];
  __shared__ uint2 sh_q[NT * KSTEPS * 32];
  __shared__ int sh_lim[ROWS];  // positions below it are visible to the row
  __shared__ float2 sh_ml[WARPS][ROWS];
  __shared__ float2 sh_cluster[MAX_CLUSTER][ROWS];

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  // The query row (of the CTA's) of this lane's column e of tile nt.
  auto col_row = [&](int nt, int e) { return nt * 8 + 2 * c + e; };

  // The next kernel's blocks (the join's, after a cut) take their places and wait there
  // for this kernel's end (1 x 16K, cut: 19.2 -> 18.5 us).
  allow_next_kernel();
  if (a.cluster > 1) cluster_arrive();
  wait_for_kernels_before();
  Piece piece;
  if (W == decode16::WARPS && a.split) {
    if (tid == 0 && !a.join_by_segment) a.joins[blockIdx.x] = make_int4(-1, 0, 0, 0);
    piece = cut<UNIT, SEGMENT_UNITS, MIN_UNITS, WARPS>(a, sh_cut);
  } else {  // one segment per cluster; u walks over it once
    const int seg = static_cast<int>(blockIdx.x) / a.cluster, per_b = a.heads_kv * a.row_tiles;
    piece.b = seg / per_b;
    const int n = units_of<>(clamp_len(a, piece.b));
    piece.base = 0;
    piece.begin = (seg - piece.b * per_b) * n;
    piece.end = piece.begin + n;
    piece.per_cta = n;
  }

  const uint32_t my_ring = smem_u32(ring) + warp * STAGES * STAGE;
  int u = piece.begin, b = piece.b, base = piece.base;
  while (u < piece.end) {
    const int len = clamp_len(a, b);
    const int n_units = units_of<>(len);
    const int seg = (u - base) / n_units;  // kvh * row_tiles + row tile
    const int u0 = u - base - seg * n_units;
    const int u1 = min(n_units, u0 + piece.end - u);
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

    // ---- copies: a lane copies piece cp_chunk of rows cp_row, cp_row + 32 / CHUNKS
    // and so on; its source addresses step through a page and are formed anew where
    // one begins, with the next page's table entry in flight meanwhile.  Piece c of
    // row t lies at place c ^ (t & 7) of its row: eight rows' pieces at once, what
    // ldmatrix reads, fall into different banks.
    constexpr int COPIES = TOK * CHUNKS / 32;  // of a lane, of the keys of a tile
    constexpr int STEP = 32 / CHUNKS;          // rows that a copy of all lanes covers
    const int cp_row = lane / CHUNKS, cp_chunk = lane % CHUNKS;
    // The first copy's place in a stage; copy i's is i * STEP rows on, with the bits of
    // i * STEP exclusive-ored into its piece.
    const uint32_t cp_at = cp_row * PITCH + ((cp_chunk ^ cp_row) << 4);
    const int32_t* table = a.table + static_cast<long long>(b) * a.table_stride;
    int cp_left = n_tiles;  // tiles of pages not opened yet
    int cp_col = 0, cp_entry = -1;
    int cp_run = 0;  // tiles of the open page still to copy
    bool cp_ok = false;
    const uint8_t *k_src = a.k, *v_src = a.v;
    auto open_page = [&](int off) {  // the page cp_entry names, from its tile `off`
      cp_ok = static_cast<uint32_t>(cp_entry) < static_cast<uint32_t>(a.num_pages);
      const long long page = cp_ok ? cp_entry : 0;
      const int row = off * TOK + cp_row;
      k_src = a.k + (page * a.k_sp + kvh * a.k_sh + row * a.k_st + cp_chunk * 16);
      v_src = a.v + (page * a.v_sp + kvh * a.v_sh + row * a.v_st + cp_chunk * 16);
      cp_run = min(cp_left, a.tiles_per_page - off);
      cp_left -= cp_run;
      if (cp_left > 0) cp_entry = __ldg(table + ++cp_col);
    };
    auto copy_tile = [&](uint32_t dst) {
      if (cp_run > 0) {
        const uint32_t at = dst + cp_at;
        auto place = [&](int i) {
          return (at ^ (((i * STEP) & 7) << 4)) + static_cast<uint32_t>(i * STEP * PITCH);
        };
#pragma unroll
        for (int i = 0; i < COPIES; i += 4)
          cp_async4(place(i), place(i + 1), place(i + 2), place(i + 3), k_src + i * STEP * a.k_st,
                    STEP * a.k_st, cp_ok);
#pragma unroll
        for (int i = 0; i < COPIES; i += 4)
          cp_async4(place(i) + HALF, place(i + 1) + HALF, place(i + 2) + HALF, place(i + 3) + HALF,
                    v_src + i * STEP * a.v_st, STEP * a.v_st, cp_ok);
        k_src += TOK * a.k_st;
        v_src += TOK * a.v_st;
        if (--cp_run == 0 && cp_left > 0) open_page(0);
      }
      cp_async_commit();
    };
    auto start = [&]() {  // the first copies of this warp's run
      cp_left = n_tiles;
      cp_col = t_begin / a.tiles_per_page;
      cp_entry = cp_left > 0 ? __ldg(table + cp_col) : -1;
      if (cp_left > 0) open_page(t_begin - cp_col * a.tiles_per_page);
#pragma unroll
      for (int s = 0; s < STAGES - 1; ++s) copy_tile(my_ring + s * STAGE);
    };
    start();

    // ---- queries: fragments of Q^T
    for (int nt = warp; nt < NT; nt += WARPS) {
      const int q_row = nt * 8 + g, r = r0 + q_row;
      uint2 f[KSTEPS];
#pragma unroll
      for (int j = 0; j < KSTEPS; ++j) f[j] = make_uint2(0u, 0u);
      if (r < a.rows) {
        const int i = r / a.group, h = kvh * a.group + (r - i * a.group);
        const uint32_t* src = reinterpret_cast<const uint32_t*>(
            a.q + b * a.q_s[0] + h * a.q_s[1] + i * a.q_s[2] + 2 * c);
#pragma unroll
        for (int j = 0; j < KSTEPS; ++j) f[j] = make_uint2(__ldg(src + 8 * j), __ldg(src + 8 * j + 4));
      }
      // Rows past the last are computed along with the rest and not stored.
      if (c == 0) sh_lim[q_row] = !a.causal || r >= a.rows ? len : len - a.q_len + r / a.group + 1;
#pragma unroll
      for (int j = 0; j < KSTEPS; ++j) sh_q[(nt * KSTEPS + j) * 32 + lane] = f[j];
    }
    __syncthreads();

    // ---- per-lane columns: 2c and 2c + 1 of each row tile
    float acc[NT][MT][4];
    float sum[NT][2];
    float zn[NT][2];  // a weight is 2^(score + zn)
    uint2 qf[NT == 1 ? KSTEPS : 1];  // one row tile's queries stay in registers
    auto clear = [&]() {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nt][mt][e] = 0.f;
#pragma unroll
        for (int e = 0; e < 2; ++e) zn[nt][e] = NO_SCORE, sum[nt][e] = 0.f;
      }
    };
    clear();
    if constexpr (NT == 1) {
#pragma unroll
      for (int j = 0; j < KSTEPS; ++j) qf[j] = sh_q[j * 32 + lane];
    }
    const uint32_t q_addr = smem_u32(sh_q) + lane * 8;
    // This lane's row pointers in a stage: of keys, token lane & 15, element 8 (lane
    // >> 4); of values, token (lane & 7) + 8 (lane >> 4), element 8 (lane >> 3 & 1).
    // Pieces 2j on are an exclusive or away.
    const uint32_t k_at = (lane & 15) * PITCH + (((lane >> 4) ^ (lane & 7)) << 4);
    const uint32_t v_at = HALF + ((lane & 7) + (lane >> 4) * 8) * PITCH +
                          ((((lane >> 3) & 1) ^ (lane & 7)) << 4);

    // MASKED: some row does not see the whole tile.  EXACT: values that are not finite
    // stay out of the products and are added one by one, see below.
    auto tile = [&](const uint32_t st, const int tok0, auto masked_tag, auto exact_tag) {
      constexpr bool MASKED = decltype(masked_tag)::value, EXACT = decltype(exact_tag)::value;
      // ---- S^T = K Q^T; up to two row tiles leave registers for two sums each, which
      // halves the chain of dependent products
      constexpr int SUMS = NT <= 2 ? 2 : 1;
      float s[NT][4], s2[SUMS == 2 ? NT : 1][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[nt][e] = s2[SUMS == 2 ? nt : 0][e] = 0.f;
#pragma unroll
      for (int j = 0; j < KSTEPS; ++j) {
        uint32_t k[4];
        ldmatrix(k, (st + k_at) ^ (j << 5));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint2 q2 = NT == 1 ? qf[NT == 1 ? j : 0] : lds64(q_addr + (nt * KSTEPS + j) * 256);
          mma_16816<F16>(SUMS == 2 && (j & 1) ? s2[SUMS == 2 ? nt : 0] : s[nt], k, q2.x, q2.y);
        }
      }
      // ---- weights; the offset falls where one would pass 2^(shift + HEADROOM)
      float y[NT][4];
      auto hidden = [&](int nt, int e) {
        return tok0 + g + (e & 2) * 4 >= sh_lim[col_row(nt, e & 1)];
      };
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if constexpr (SUMS == 2) s[nt][e] += s2[nt][e];
          s[nt][e] *= a.sigma_log2;
          if (MASKED && hidden(nt, e)) s[nt][e] = -INFINITY;
        }
      bool over = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[nt][e] = s[nt][e] + zn[nt][e & 1];
          over |= y[nt][e] > most_of<F16>(a);
        }
      if (__any_sync(0xffffffffu, over)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float m = fmaxf(s[nt][e], s[nt][e + 2]);
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
            const float z = fminf(zn[nt][e], shift_of<F16>(a) - m);
            const float f = ex2_approx(z - zn[nt][e]);
            zn[nt][e] = z;
            sum[nt][e] *= f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              acc[nt][mt][e] *= f;
              acc[nt][mt][e + 2] *= f;
            }
            y[nt][e] = s[nt][e] + z;
            y[nt][e + 2] = s[nt][e + 2] + z;
          }
      }
      // The products take 16-bit factors: a weight goes in as two, itself rounded and
      // the remainder rounded, which leaves 2^-16 of it (bf16; fp16 2^-22) and makes
      // O as good as its own rounding.  The second product costs nothing at one or two
      // row tiles and 1.5% at three (five tokens over 16 ragged sequences to 32K: 218 us
      // without it, 221).
      uint32_t hi[NT][2], lo[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[nt][e] = ex2_approx(y[nt][e]);
          sum[nt][e & 1] += y[nt][e];
        }
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t w = pack_x2<F16>(y[nt][2 * x], y[nt][2 * x + 1]);
          const float2 r = x2_to_f32(w, F16);
          hi[nt][x] = movmatrix_trans(w);
          lo[nt][x] = movmatrix_trans(pack_x2<F16>(y[nt][2 * x] - r.x, y[nt][2 * x + 1] - r.y));
        }
      }
      if (MASKED && tok0 + TOK > max_lim) {
        // A hidden value weighs nothing even where it is not a number.
        const int first = max(0, max_lim - tok0);
        for (int x = first * CHUNKS + lane; x < TOK * CHUNKS; x += 32)
          asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(st + HALF + x * 16), "r"(0)
                       : "memory");
        __syncwarp();
      }
      // ---- O^T += V^T P^T.  The tensor cores cut off what they add to a sum instead
      // of rounding it, so a tile's sum starts at zero and is added in fp32.
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t v[4];
        ldmatrix_trans(v, (st + v_at) ^ (mt << 5));
        if constexpr (EXACT) {
#pragma unroll
          for (int x = 0; x < 4; ++x) v[x] = finite_or_zero<F16>(v[x]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float o[4] = {0.f, 0.f, 0.f, 0.f};
          mma_16816<F16>(o, v, lo[nt][0], lo[nt][1]);
          mma_16816<F16>(o, v, hi[nt][0], hi[nt][1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nt][mt][e] += o[e];
        }
      }
      if constexpr (EXACT) {
#pragma unroll 1
        for (int t = 0; t < TOK; ++t) {
          float p[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float w =
                  __shfl_sync(0xffffffffu, t < 8 ? y[nt][e] : y[nt][e + 2], 4 * (t & 7) + c);
              p[nt][e] = tok0 + t < sh_lim[col_row(nt, e)] ? w : -1.f;  // a weight is not negative
            }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t at = st + HALF + t * PITCH + (((2 * mt + x) ^ (t & 7)) << 4) + 2 * g;
              const float v = x2_to_f32(lds16(at), F16).x;
              if (fabsf(v) < INFINITY) continue;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (!(p[nt][e] < 0.f))
                    acc[nt][mt][e + 2 * x] = fmaf(p[nt][e], v, acc[nt][mt][e + 2 * x]);
            }
        }
      }
    };

    uint32_t rd = my_ring, wr = my_ring + (STAGES - 1) * STAGE;
    const uint32_t ring_end = my_ring + STAGES * STAGE;
    auto next_tile = [&]() {
      cp_async_wait<STAGES - 2>();
      __syncwarp();  // every lane's copies of this tile are in, and the last one is read
      copy_tile(wr);
      const uint32_t st = rd;
      rd = rd + STAGE == ring_end ? my_ring : rd + STAGE;
      wr = wr + STAGE == ring_end ? my_ring : wr + STAGE;
      return st;
    };
    // Tiles that every row sees in whole come first; the few others take the
    // masked path in a loop of their own.
    const int t_full = max(t_begin, min(t_end, min_lim / TOK));
    int t = t_begin;
    for (; t < t_full; ++t) tile(next_tile(), 0, std::false_type{}, std::false_type{});
    for (; t < t_end; ++t) tile(next_tile(), t * TOK, std::true_type{}, std::false_type{});
    cp_async_wait<0>();

    // A value that is not finite makes the products of every row NaN: of those that
    // do not see its token (weight 0), and of those whose weight leaves no remainder
    // or a negative one.  So sums that are not finite are formed once more, with such
    // values apart; the others' sums are the same bit for bit.
    bool finite = true;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) finite = finite && fabsf(acc[nt][mt][e]) < INFINITY;
    if (!__all_sync(0xffffffffu, finite)) {
      clear();
      __syncwarp();
      start();
      rd = my_ring, wr = my_ring + (STAGES - 1) * STAGE;
      for (t = t_begin; t < t_end; ++t) tile(next_tile(), t * TOK, std::true_type{}, std::true_type{});
      cp_async_wait<0>();
    }

    // ---- join the warps: common offset, then one sum of the scaled parts
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = sum[nt][e];
        l += __shfl_xor_sync(0xffffffffu, l, 4);
        l += __shfl_xor_sync(0xffffffffu, l, 8);
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (g == 0) sh_ml[warp][col_row(nt, e)] = make_float2(-zn[nt][e], l);
      }
    __syncthreads();  // also: every warp is done with its ring, which the sums reuse
    float* merge = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = col_row(nt, e);
        float m = sh_ml[0][r].x;
#pragma unroll
        for (int w = 1; w < WARPS; ++w) m = fmaxf(m, sh_ml[w][r].x);
        const float f = ex2_approx(-zn[nt][e] - m);
        float* dst = merge + (warp * ROWS + r) * MERGE_ROW<D> + g;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          dst[16 * mt] = acc[nt][mt][e] * f;
          dst[16 * mt + 8] = acc[nt][mt][e + 2] * f;
        }
      }
    __syncthreads();
    // Row r's offset and sum, and the sum of four elements of it, over the warps.
    auto joined_ml = [&](int r) {
      float m = sh_ml[0][r].x, l = 0.f;
#pragma unroll
      for (int w = 1; w < WARPS; ++w) m = fmaxf(m, sh_ml[w][r].x);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) l += sh_ml[w][r].y * ex2_approx(sh_ml[w][r].x - m);
      return make_float2(m, l);
    };
    auto joined = [&](int r, int d0) {
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float4 x =
            *reinterpret_cast<const float4*>(merge + (w * ROWS + r) * MERGE_ROW<D> + d0);
        y.x += x.x, y.y += x.y, y.z += x.z, y.w += x.w;
      }
      return y;
    };
    if (a.cluster > 1) {
      // Output x of the segment (four elements) is joined by CTA x % cluster: each
      // CTA stores its sums, and the offsets, straight into the joining CTAs' shared
      // memory, and after one barrier every CTA adds what it got, over the CTAs in
      // order.
      const int items = ROWS * (D / 4) / a.cluster;  // the cluster is a power of two
      const uint32_t rank = cluster_rank(), got = smem_u32(ring) + ring_bytes<D, NT, W>();
      cluster_wait();  // the one of the kernel's beginning: every CTA runs
      for (int x = tid; x < n_rows * (D / 4); x += THREADS) {
        const int r = x / (D / 4), d0 = (x % (D / 4)) * 4;
        cluster_st4(got + (rank * items + x / a.cluster) * 16, x % a.cluster, joined(r, d0));
      }
      for (int x = tid; x < n_rows * a.cluster; x += THREADS) {
        const int r = x / a.cluster;
        cluster_st2(smem_u32(&sh_cluster[rank][r]), x % a.cluster, joined_ml(r));
      }
      cluster_arrive();
      cluster_wait();
      const float4* parts = reinterpret_cast<const float4*>(ring + ring_bytes<D, NT, W>());
      for (int k = tid; k * a.cluster + rank < n_rows * (D / 4); k += THREADS) {
        const int x = k * a.cluster + rank, r = x / (D / 4), d0 = (x % (D / 4)) * 4;
        float m = sh_cluster[0][r].x;
        for (int c1 = 1; c1 < a.cluster; ++c1) m = fmaxf(m, sh_cluster[c1][r].x);
        float l = 0.f;
        float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c1 = 0; c1 < a.cluster; ++c1) {
          const float2 ml = sh_cluster[c1][r];
          const float4 p = parts[c1 * items + k];
          const float f = ex2_approx(ml.x - m);
          l += ml.y * f;
          y.x += p.x * f, y.y += p.y * f, y.z += p.z * f, y.w += p.w * f;
        }
        store_row4(a, b, kvh, r0 + r, d0, m, l, y);
      }
      return;
    }
    const bool began = u0 == 0, whole = began && u1 == n_units;
    const int part = 2 * static_cast<int>(blockIdx.x) + (began ? 1 : 0);
    for (int x = tid; x < n_rows * (D / 4); x += THREADS) {
      const int r = x / (D / 4), d0 = (x % (D / 4)) * 4;
      const float2 ml = joined_ml(r);
      const float4 y = joined(r, d0);
      if (whole) {
        store_row4(a, b, kvh, r0 + r, d0, ml.x, ml.y, y);
      } else {
        *reinterpret_cast<float4*>(a.part_o + (static_cast<long long>(part) * ROWS + r) * D + d0) =
            y;
        if (d0 == 0) a.part_ml[static_cast<long long>(part) * ROWS + r] = ml;
      }
    }
    if (began && tid == 0) {
      const int4 job =
          make_int4(whole ? -1 : b, seg, blockIdx.x, (u + n_units - 1) / piece.per_cta);
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

// Whether the kernel after a join may be placed early (1 x 128K: 82.8 -> 82.0 us; at d =
// 64, where an SM holds four of its CTAs, they are spread unevenly: 47.0 -> 50.4).
template <int D>
constexpr bool EARLY_AFTER_JOIN = D == 128;

// Place of part p of a segment that began in CTA `first`.
template <int PER>
__device__ __forceinline__ long long slot_of(int first, int p) {
  const int c = p / PER;
  return (2LL * (first + c) + (c == 0 ? 1 : 0)) * PER + (p - c * PER);
}

// A row whose sums are not finite though its weights are, which may be due to a value
// that the row does not see, once more: y takes the place of the elements that are not
// finite in it.  Scores and sums are formed in fp32, in two walks over the tokens (the
// largest score and the sum of weights, then O), 32 of them at a time to a warp and by
// WARPS warps in turn, whose sums are added in order; weights are divided by their sum
// first, so that O cannot overflow.  (Rows of wide calls alone, and here, where nobody
// waits for them: 160 histories of 2^18 tokens, 40 rows each, all formed anew: 0.28 s.)
//
// Lane x of a warp holds elements E x on, E = D / 32, of what it is given and returns.
template <int D, int WARPS>
__device__ __noinline__ void form_anew(const DecArgs& a, int b, int kvh, int row, bool from_kept,
                                       int warp, float (*sh)[D], float (&y)[D / 32]) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int i = row / a.group, h = kvh * a.group + (row - i * a.group);
  const uint16_t* q = from_kept
                          ? a.kept + ((static_cast<long long>(b) * a.heads_kv + kvh) * a.rows + row) * D
                          : a.q + b * a.q_s[0] + h * a.q_s[1] + i * a.q_s[2];
  const uint4* q4 = reinterpret_cast<const uint4*>(q);
  const int len = clamp_len(a, b), lim = a.causal ? len - a.q_len + i + 1 : len;
  const int page_size = a.tiles_per_page * TOK;
  const int32_t* table = a.table + static_cast<long long>(b) * a.table_stride;
  const uint8_t *k = a.k + kvh * a.k_sh, *v = a.v + kvh * a.v_sh;
  // The score of a token, in log2 units, and where its value lies (no page: zeros).
  auto score = [&](int tok, const uint8_t*& value) {
    const int col = tok / page_size, at = tok - col * page_size, page = __ldg(table + col);
    value = nullptr;
    if (page < 0 || page >= a.num_pages) return 0.f;
    value = v + (page * a.v_sp + static_cast<long long>(at) * a.v_st);
    const uint4* k4 = reinterpret_cast<const uint4*>(k + (page * a.k_sp +
                                                          static_cast<long long>(at) * a.k_st));
    float s = 0.f;
#pragma unroll 2
    for (int e = 0; e < D / 8; ++e) {
      const uint4 x = q4[e], z = __ldg(k4 + e);
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, zs[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float2 f = x2_to_f32(xs[w], a.f16), g = x2_to_f32(zs[w], a.f16);
        s = fmaf(f.x, g.x, s);
        s = fmaf(f.y, g.y, s);
      }
    }
    return s * a.sigma_log2;
  };
  auto of_warps = [&](float x, bool largest) {  // the largest, or the sum, over all tokens
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float z = __shfl_xor_sync(0xffffffffu, x, o);
      x = largest ? fmaxf(x, z) : x + z;
    }
    if constexpr (WARPS > 1) {
      __syncthreads();
      if (lane == 0) sh[warp][0] = x;
      __syncthreads();
      x = sh[0][0];
      for (int w = 1; w < WARPS; ++w) x = largest ? fmaxf(x, sh[w][0]) : x + sh[w][0];
    }
    return x;
  };

  const uint8_t* value;
  float m = -NO_SCORE, l = 0.f;
  for (int tok = 32 * warp + lane; tok < lim; tok += 32 * WARPS) {
    const float s = score(tok, value), m1 = fmaxf(m, s);
    l = fmaf(l, ex2_approx(m - m1), ex2_approx(s - m1));
    m = m1;
  }
  const float most = of_warps(m, true);
  const float inv = 1.f / of_warps(l * ex2_approx(m - most), false);
  float o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  for (int t0 = 32 * warp; t0 < lim; t0 += 32 * WARPS) {
    value = nullptr;
    float p = 0.f;
    if (t0 + lane < lim) p = ex2_approx(score(t0 + lane, value) - most) * inv;
#pragma unroll 2
    for (int t = 0; t < 32; ++t) {
      const float pt = __shfl_sync(0xffffffffu, p, t);
      const uint8_t* vt = reinterpret_cast<const uint8_t*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(value), t));
      if (vt == nullptr) continue;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 f =
            x2_to_f32(__ldg(reinterpret_cast<const uint32_t*>(vt) + (lane * E + e) / 2), a.f16);
        o[e] = fmaf(pt, f.x, o[e]);
        o[e + 1] = fmaf(pt, f.y, o[e + 1]);
      }
    }
  }
  if constexpr (WARPS > 1) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) sh[warp][lane * E + e] = o[e];
    __syncthreads();
#pragma unroll
    for (int e = 0; e < E; ++e) {
      o[e] = sh[0][lane * E + e];
      for (int w = 1; w < WARPS; ++w) o[e] += sh[w][lane * E + e];
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (!(fabsf(y[e]) < INFINITY)) y[e] = o[e];
}

// Stores such a row; its log-sum-exp is of the weights alone, and stored with the rest.
template <int D>
__device__ __forceinline__ void store_anew(const DecArgs& a, int b, int kvh, int row,
                                           const float (&y)[D / 32]) {
  uint32_t* o = reinterpret_cast<uint32_t*>(output_row(a, b, kvh, row));
#pragma unroll
  for (int e = 0; e < D / 32; e += 2)
    o[((threadIdx.x & 31) * (D / 32) + e) / 2] = f32_to_x2(y[e], y[e + 1], a.f16);
}

// A stored row, as fp32.
template <int D>
__device__ __forceinline__ void load_stored(const DecArgs& a, int b, int kvh, int row,
                                            float (&y)[D / 32]) {
  const uint32_t* o = reinterpret_cast<const uint32_t*>(output_row(a, b, kvh, row));
#pragma unroll
  for (int e = 0; e < D / 32; e += 2) {
    const float2 f = x2_to_f32(o[((threadIdx.x & 31) * (D / 32) + e) / 2], a.f16);
    y[e] = f.x, y[e + 1] = f.y;
  }
}

// Whether row r of segment x, which lies within a CTA, is to be formed anew.  (Of other
// segments it says nothing; read all the same, so that the load waits for no other.)
template <int PER>
__device__ __forceinline__ bool is_anew(const DecArgs& a, int x, int r) {
  return PER > 1 && (a.anew[4 * x + (r >> 5)] >> (r & 31) & 1u);
}

// Joins the parts of the segments that a cut crossed: block (x, r) takes row r
// of job x, which is segment x, or where there are more segments than CTAs the
// one that CTA x began and did not finish -- if that was cut.  The parts lie in
// the CTAs first (its second slot) .. last (their first slots), PER in each.  The
// offsets come first, all at once, so that the sums' loads wait for nothing.
template <int D, int ROWS, int PER>
__global__ void __launch_bounds__(JOIN_THREADS, 4)
    decode16_join_kernel(const __grid_constant__ DecArgs a) {
  constexpr int LANES = D / 4;                 // threads that cover a row, four elements each
  constexpr int PARTS = JOIN_THREADS / LANES;  // parts read at once
  __shared__ float4 sh_y[PARTS][LANES];
  __shared__ float2 sh_ml[JOIN_THREADS / 32];
  __shared__ float sh_w[MAX_PARTS];
  if constexpr (EARLY_AFTER_JOIN<D>) allow_next_kernel();
  wait_for_kernels_before();
  const int4 job = a.joins[blockIdx.x];
  const int r = blockIdx.y;
  const bool anew = is_anew<PER>(a, blockIdx.x, r);
  if (job.x < 0 || (job.w < 0 && !anew)) return;
  const int b = job.x, kvh = job.y / a.row_tiles;
  const int row = (job.y - kvh * a.row_tiles) * ROWS + r;
  if (row >= a.rows) return;
  const int tid = threadIdx.x;
  constexpr int JOIN_WARPS = JOIN_THREADS / 32;
  float(*sh_o)[D] = reinterpret_cast<float(*)[D]>(sh_y);  // of each warp, in form_anew
  static_assert(JOIN_WARPS * D * 4 <= sizeof(sh_y), "shared memory");
  if constexpr (PER > 1) {
    if (job.w < 0) {
      float y[D / 32];
      load_stored<D>(a, b, kvh, row, y);
      form_anew<D, JOIN_WARPS>(a, b, kvh, row, a.in_place, tid >> 5, sh_o, y);
      if (tid < 32) store_anew<D>(a, b, kvh, row, y);
      return;
    }
  }
  const int first = job.z, count = PER * (job.w - first + 1);  // at most MAX_PARTS
  auto slot = [&](int p) { return slot_of<PER>(first, p); };

  float2 mine[MAX_PARTS / JOIN_THREADS];
  float m = -NO_SCORE;
#pragma unroll
  for (int x = 0; x < MAX_PARTS / JOIN_THREADS; ++x) {
    const int p = tid + x * JOIN_THREADS;
    mine[x] = p < count ? a.part_ml[slot(p) * ROWS + r] : make_float2(-NO_SCORE, 0.f);
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
    const float w = ex2_approx(mine[x].x - m);
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
  if (PER == 1 && p0 != 0) return;
  if (p0 == 0) {
#pragma unroll
    for (int p = 1; p < PARTS; ++p) {
      const float4 x = sh_y[p][lane];
      y.x += x.x, y.y += x.y, y.z += x.z, y.w += x.w;
    }
  }
  if constexpr (PER > 1) {
    const bool finite = fabsf(y.x) < INFINITY && fabsf(y.y) < INFINITY && fabsf(y.z) < INFINITY &&
                        fabsf(y.w) < INFINITY;
    if (__syncthreads_or(p0 == 0 && !finite && l < INFINITY)) {
      const float inv = 1.f / l;
      if (p0 == 0)
        reinterpret_cast<float4*>(sh_o[0])[lane] =
            make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
      __syncthreads();
      float z[D / 32];
#pragma unroll
      for (int e = 0; e < D / 32; ++e) z[e] = sh_o[0][(tid & 31) * (D / 32) + e];
      form_anew<D, JOIN_WARPS>(a, b, kvh, row, false, tid >> 5, sh_o, z);
      if (tid < 32) store_anew<D>(a, b, kvh, row, z);
      if (tid == 0) store_lse(a, b, kvh, row, m, l);
      return;
    }
    if (p0 != 0) return;
  }
  store_row4(a, b, kvh, row, 4 * lane, m, l, y);
}

// The same where segments have few parts: a warp takes a row of job x by itself,
// 32 parts' offsets at a time.
template <int D, int ROWS, int PER>
__global__ void __launch_bounds__(JOIN_THREADS)
    decode16_join_rows_kernel(const __grid_constant__ DecArgs a) {
  constexpr int E = D / 32;  // elements of a lane
  if constexpr (EARLY_AFTER_JOIN<D>) allow_next_kernel();
  wait_for_kernels_before();
  const int4 job = a.joins[blockIdx.x];
  const int lane = threadIdx.x & 31;
  const int r = blockIdx.y * (JOIN_THREADS / 32) + (threadIdx.x >> 5);
  const bool anew = r < ROWS && is_anew<PER>(a, blockIdx.x, r);
  if (job.x < 0 || (job.w < 0 && !anew)) return;
  const int b = job.x, kvh = job.y / a.row_tiles;
  const int row = (job.y - kvh * a.row_tiles) * ROWS + r;
  if (r >= ROWS || row >= a.rows) return;
  if constexpr (PER > 1) {
    if (job.w < 0) {
      float y[E];
      load_stored<D>(a, b, kvh, row, y);
      form_anew<D, 1>(a, b, kvh, row, a.in_place, 0, nullptr, y);
      store_anew<D>(a, b, kvh, row, y);
      return;
    }
  }
  const int first = job.z, count = PER * (job.w - first + 1);
  auto slot = [&](int p) { return slot_of<PER>(first, p); };
  float m = -NO_SCORE, l = 0.f, y[E];
#pragma unroll
  for (int e = 0; e < E; ++e) y[e] = 0.f;
  for (int p0 = 0; p0 < count; p0 += 32) {
    const float2 ml = p0 + lane < count ? a.part_ml[slot(p0 + lane) * ROWS + r]
                                        : make_float2(-NO_SCORE, 0.f);
    float m1 = fmaxf(m, ml.x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
    const float f = ex2_approx(m - m1), w = ex2_approx(ml.x - m1);
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
  if constexpr (PER > 1) {
    bool finite = true;
#pragma unroll
    for (int e = 0; e < E; ++e) finite = finite && fabsf(y[e]) < INFINITY;
    if (l < INFINITY && !__all_sync(0xffffffffu, finite)) {
      const float inv = 1.f / l;
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] *= inv;
      form_anew<D, 1>(a, b, kvh, row, false, 0, nullptr, y);
      store_anew<D>(a, b, kvh, row, y);
      if (lane == 0) store_lse(a, b, kvh, row, m, l);
      return;
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

// How a call is run: see plan_of().
struct Plan {
  int nt, row_tiles, units, warps, cluster, max_grid;
  long long segments, all_units;
  bool split;
  bool wide;  // bsfa_decode16_wide.cuh
};

// The status of a runtime call.  The runtime keeps the error of one that failed
// until it is asked for it: asked here, a later launch does not report it as its
// own.
inline bsfa_status status_of(cudaError_t e) {
  if (e == cudaSuccess) return BSFA_OK;
  cudaGetLastError();
  return BSFA_ERR_CUDA;
}

// Sets a kernel's shared-memory size and largest cluster, once per device.
template <int D, int NT, bool F16, int W>
bsfa_status prepare(int dev) {
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (ready.load(std::memory_order_relaxed) & bit) return BSFA_OK;
  bsfa_status v = status_of(cudaFuncSetAttribute(decode16_kernel<D, NT, F16, W>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 smem_bytes<D, NT, W>(true)));
  if (v == BSFA_OK)
    v = status_of(cudaFuncSetAttribute(decode16_kernel<D, NT, F16, W>,
                                       cudaFuncAttributeNonPortableClusterSizeAllowed, 1));
  if (v == BSFA_OK) ready.fetch_or(bit, std::memory_order_relaxed);
  return v;
}

// For kernels that wait by themselves for those before them.
inline cudaLaunchAttribute after_kernels() {
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}

// The join of what `grid` CTAs left of `segments` segments, in `jobs` jobs.
template <int D, int ROWS, int PER>
bsfa_status launch_join(const DecArgs& a, long long segments, int grid, long long jobs,
                        cudaStream_t stream) {
  // About grid / segments parts to a segment.
  const bool by_rows = grid * PER < JOIN_ROWS_PARTS * segments;
  const int rows = a.rows < ROWS ? a.rows : ROWS, per_block = by_rows ? JOIN_THREADS / 32 : 1;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr = after_kernels();
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(jobs), (rows + per_block - 1) / per_block);
  cfg.blockDim = dim3(JOIN_THREADS);
  return status_of(by_rows ? cudaLaunchKernelEx(&cfg, decode16_join_rows_kernel<D, ROWS, PER>, a)
                           : cudaLaunchKernelEx(&cfg, decode16_join_kernel<D, ROWS, PER>, a));
}

template <int D, int NT, bool F16, int W = WARPS>
bsfa_status launch(const DecArgs& args, const Plan& pl, int sms, int dev, cudaStream_t stream) {
  static_assert(Shape<D, NT>::MAX_GRID <= MAX_PARTS, "the join's weights");
  const bsfa_status v = prepare<D, NT, F16, W>(dev);
  if (v != BSFA_OK) return v;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attrs[2] = {after_kernels(), {}};
  cfg.stream = stream;
  cfg.attrs = attrs;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(32 * W);
  cfg.dynamicSmemBytes = smem_bytes<D, NT, W>(pl.cluster > 1);
  if (!pl.split) {
    cfg.gridDim = dim3(static_cast<unsigned>(pl.segments * pl.cluster));
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = pl.cluster;
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    return status_of(cudaLaunchKernelEx(&cfg, decode16_kernel<D, NT, F16, W>, args));
  }
  if constexpr (W == WARPS) {  // other CTAs never cut
    const long long full = static_cast<long long>(sms) * Shape<D, NT>::CTAS;
    int grid = static_cast<int>(full < pl.max_grid ? full : pl.max_grid);
    const long long most = (pl.all_units + MIN_UNITS - 1) / MIN_UNITS;
    if (most < grid) grid = static_cast<int>(most);
    DecArgs a = args;
    a.join_by_segment = pl.segments <= grid;
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    const bsfa_status first = status_of(cudaLaunchKernelEx(&cfg, decode16_kernel<D, NT, F16, W>, a));
    if (first != BSFA_OK) return first;
    return launch_join<D, 8 * NT, 1>(a, pl.segments, grid,
                                     a.join_by_segment ? pl.segments : grid, stream);
  }
  return BSFA_ERR_CUDA;
}

// The call of one head dimension and element type (inst_decode16_*.cu).
template <int D, bool F16>
bsfa_status run(const DecArgs& a, const Plan& pl, int sms, int dev, cudaStream_t stream) {
  using Launch = bsfa_status (*)(const DecArgs&, const Plan&, int, int, cudaStream_t);
  // [tiles of 8 query rows], then CTAs of one warp
  static const Launch launches[4 + SMALL_NT] = {
      launch<D, 1, F16>,              launch<D, 2, F16>,
      launch<D, 3, F16>,              launch<D, 4, F16>,
      launch<D, 1, F16, SMALL_WARPS>, launch<D, 2, F16, SMALL_WARPS>};
  return launches[pl.nt - 1 + (pl.warps == SMALL_WARPS ? 4 : 0)](a, pl, sms, dev, stream);
}

}  // namespace decode16

}  // namespace bsfa
