// bsfa_cache16.cu -- bsfa_rotary and bsfa_cache16_write: rows of queries and keys
// rotated by their positions, and keys and values written into 16-bit pages.
//
// Mathematics.  A pair (a, b) at position p is turned by the angle p * f.  With s
// the integer nearest below f / 2pi * 2^64, the product p * s modulo 2^64 is the
// angle's fraction of a turn: whole turns fall off as the product wraps, and no
// digit of a far position is lost (in fp32 the angle 131071 * 1 is off by 2^-8).
//
// One thread owns eight pairs of a row: 16 elements in two 16-byte pieces, so that
// the threads of a row read and write whole lines.  It forms its eight sines and
// cosines once and walks over the heads it is given, of the queries, the keys or
// the values.  Both calls move each byte once and are bound by HBM: 32 query and 8 KV
// heads of 32768 tokens, d = 128 (671 MB), are rotated in 100 us, 6.7 TB/s (a copy runs
// at 6.79); 131072 tokens of them rotated and written to pages (3.22 GB) in 459 us, 7.0.
#include <cuda_runtime.h>

#include <cstdint>

#include "bsfa.h"
#include "bsfa_cache16.h"
#include "bsfa_cache4.h"
#include "fp4.cuh"

namespace bsfa {

namespace {

constexpr int THREADS = 128;
constexpr int CHUNK = 16;  // elements of a row that a thread owns: eight pairs
// Heads whose loads a thread issues at once (that prompt, a gradient of 15009 tokens,
// 10396 packed tokens of 32 heads of d = 64: 99.6, 49.0 and 18.5 us; at 4 100.2, 50.1
// and 18.1, at 2 100.1, 50.6 and 19.0).
constexpr int AHEAD = 3;
// Blocks that a call with few rows is spread over.  More of them form the same angles
// more often, fewer leave SMs idle (the packed tokens, and one token of 256 sequences:
// 18.1 and 4.3 us; at 2048 20.9 and 5.1).
constexpr int FILL = 600;

enum Kind { QUERIES, KEYS, VALUES };

// Rows in, rows out; for keys and values of a cache `out` is a pool and its
// first stride the pages'.
struct Part {
  const uint16_t* in;
  uint16_t* out;
  long long in_s[3], out_s[3];  // {batch, head, token} elements; {page, head, token}
  int heads;
  int blocks;  // of blockIdx.y, heads_per_block heads each
};

struct RowsArgs {
  Part part[3];
  const int32_t *table, *cu, *start;
  int table_stride, table_width, page_size, num_pages;
  int paged;  // keys and values go to pages
  int batch, seqlen;
  long long rows;       // batch * seqlen, or the packed rows; below 2^31
  int heads_per_block;  // heads that one thread walks over
  // The rotation; pairs is 0 where there is none.
  const float* inv_freq;
  const int32_t* positions;
  long long pos_s[2];  // {axis, batch}
  int pairs, inverse, num_axes;
  uint8_t axis[64];
};

// Where row t of the call lies.
struct Row {
  int b;          // its sequence; negative: none (packed rows outside every sequence)
  int i;          // its row of the tensors (within the sequence, or packed)
  long long pos;  // its position (offsets below zero put rows beyond 2^31)
};

// The sequence and position of packed row r.i.
__device__ __forceinline__ void find_sequence(const RowsArgs& a, Row& r) {
  // The last sequence that begins at or before it.
  int lo = 0, hi = a.batch;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a.cu + mid) <= r.i)
      lo = mid + 1;
    else
      hi = mid;
  }
  r.b = lo - 1;
  if (r.b >= 0 && r.i >= __ldg(a.cu + r.b + 1)) r.b = -1;
  if (r.b >= 0) r.pos = static_cast<long long>(r.i) - __ldg(a.cu + r.b);
}

// The page of a row and its token there; false where the position names no row.
__device__ __forceinline__ bool find_page(const RowsArgs& a, const Row& r, int& page, int& token) {
  if (r.pos < 0 || r.pos >= static_cast<long long>(a.table_width) * a.page_size) return false;
  const int p = static_cast<int>(r.pos), col = p / a.page_size;
  page = __ldg(a.table + static_cast<long long>(r.b) * a.table_stride + col);
  token = p - col * a.page_size;
  return page >= 0 && page < a.num_pages;
}

// |f| / 2pi in units of 2^-64 turn, modulo one turn: f is m * 2^(e - 150) with a
// 24-bit m, and the 88 bits of m * floor(2^66 / 2pi) are shifted by e - 152.
__device__ __forceinline__ uint64_t turns_per_position(float f) {
  constexpr uint64_t INV_2PI = 0xA2F9836E4E441529ull;  // floor(2^66 / (2 pi))
  const uint32_t bits = __float_as_uint(f);
  const int e = max(1, static_cast<int>(bits >> 23 & 0xffu));
  const uint32_t m = (bits & 0x7fffffu) | (bits & 0x7f800000u ? 0x800000u : 0u);
  const uint64_t low = static_cast<uint64_t>(m) * static_cast<uint32_t>(INV_2PI);
  const uint64_t high = static_cast<uint64_t>(m) * static_cast<uint32_t>(INV_2PI >> 32) +
                        (low >> 32);  // the upper 56 bits
  const int down = 152 - e;
  if (down >= 32) return down < 96 ? high >> (down - 32) : 0;
  const uint64_t lowest = low & 0xffffffffu;
  if (down >= 0) return high << (32 - down) | lowest >> down;
  return down > -64 ? (high << 32 | lowest) << -down : 0;  // beyond: whole turns only
}

// cos and sin of position * f.
__device__ __forceinline__ void turn(float f, long long position, float& c, float& s) {
  uint64_t phase = turns_per_position(f) * static_cast<uint64_t>(position);
  if (f < 0.f) phase = 0 - phase;
  const uint32_t p = static_cast<uint32_t>((phase + (1ull << 31)) >> 32);
  const uint32_t quarter = (p + (1u << 29)) >> 30;
  // The angle beyond the nearest quarter turn, at most pi / 4 and three roundings off
  // (an integer's, the constant's, the product's), and the Taylor series there: sin to
  // x^9 / 9!, cos to x^10 / 10!, which leave 2^-29 and 2^-33.
  const float x = static_cast<float>(static_cast<int32_t>(p - (quarter << 30))) * 0x1.921fb6p-30f;
  const float y = x * x;
  float s0 = fmaf(y, 1.f / 362880.f, -1.f / 5040.f);
  s0 = fmaf(y, s0, 1.f / 120.f);
  s0 = fmaf(y, s0, -1.f / 6.f);
  s0 = fmaf(x * y, s0, x);
  float c0 = fmaf(y, -1.f / 3628800.f, 1.f / 40320.f);
  c0 = fmaf(y, c0, -1.f / 720.f);
  c0 = fmaf(y, c0, 1.f / 24.f);
  c0 = fmaf(y, c0, -0.5f);
  c0 = fmaf(y, c0, 1.f);
  const bool odd = quarter & 1u;
  c = odd ? s0 : c0;
  s = odd ? c0 : s0;
  if ((quarter + 1u) & 2u) c = -c;
  if (quarter & 2u) s = -s;
  if (!isfinite(f)) c = s = f - f;
}

template <int D, bool F16, bool INTERLEAVED>
__global__ void __launch_bounds__(THREADS) rows16_kernel(const __grid_constant__ RowsArgs a) {
  constexpr int GROUPS = D / CHUNK;  // threads of a row
  // (Without allow_next_kernel(): blocks of the next call that take their places early are
  // spread unevenly over the SMs, 14.0 -> 15.7 us for the packed rows of a chunked prompt.)
  wait_for_kernels_before();
  const int g = threadIdx.x & (GROUPS - 1);
  const long long t =
      static_cast<long long>(blockIdx.x) * (THREADS / GROUPS) + threadIdx.x / GROUPS;
  if (t >= a.rows) return;
  int y = blockIdx.y, kind = QUERIES;
  while (y >= a.part[kind].blocks) y -= a.part[kind++].blocks;
  const Part& part = a.part[kind];
  const int h0 = y * a.heads_per_block, h1 = min(h0 + a.heads_per_block, part.heads);

  // This thread's two pieces of eight elements: of the rotated part, of what
  // passes behind it, or of a row that is copied.
  const bool rotated = kind != VALUES && g < a.pairs / 8;
  int lo, hi;
  if (kind == VALUES) {
    lo = 8 * g, hi = D / 2 + 8 * g;
  } else if (rotated) {
    lo = 8 * g, hi = a.pairs + 8 * g;
  } else {
    const int x = 8 * (g - a.pairs / 8), passing = D / 2 - a.pairs;
    lo = 2 * a.pairs + x, hi = lo + passing;
  }
  const int gap = hi - lo;
  Row r;
  r.i = static_cast<int>(t), r.b = 0;
  if (a.cu == nullptr) {
    r.b = r.i / a.seqlen;
    r.i -= r.b * a.seqlen;
    r.pos = r.i;
  }
  const long long batch = r.b;
  const uint16_t* in =
      part.in + batch * part.in_s[0] + h0 * part.in_s[1] + r.i * part.in_s[2] + lo;
  uint4 x[AHEAD], z[AHEAD];
  auto load = [&](int h) {
#pragma unroll
    for (int n = 0; n < AHEAD; ++n)
      if (h + n < h1) {
        const uint16_t* src = in + n * part.in_s[1];
        x[n] = *reinterpret_cast<const uint4*>(src);
        z[n] = *reinterpret_cast<const uint4*>(src + gap);
      }
    in += AHEAD * part.in_s[1];
  };
  // In flight while the sequence, the page and the angles are found (of a packed row
  // outside every sequence for nothing).
  load(h0);

  if (a.cu != nullptr) find_sequence(a, r);
  if (r.b < 0) return;
  if (a.start) r.pos += __ldg(a.start + r.b);
  long long at;
  if (kind != QUERIES && a.paged) {
    int page, token;
    if (!find_page(a, r, page, token)) return;
    at = page * part.out_s[0] + token * part.out_s[2];
  } else {
    at = batch * part.out_s[0] + r.i * part.out_s[2];
  }
  uint16_t* out = part.out + at + h0 * part.out_s[1] + lo;

  // Eight pairs: elements e of both pieces, or the neighbours of the first piece
  // and then of the second.
  float c[8], s[8];
  if (rotated) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = INTERLEAVED ? 4 * g + (e & 3) + (e < 4 ? 0 : a.pairs / 2) : 8 * g + e;
      long long position = r.pos;
      if (a.positions != nullptr)
        position = __ldg(a.positions + a.axis[j] * a.pos_s[0] + batch * a.pos_s[1] + r.i);
      turn(__ldg(a.inv_freq + j), position, c[e], s[e]);
      if (a.inverse) s[e] = -s[e];
    }
  }

  for (int h = h0;;) {
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      if (h + n >= h1) return;
      if (rotated) {
        uint32_t p[4] = {x[n].x, x[n].y, x[n].z, x[n].w}, q[4] = {z[n].x, z[n].y, z[n].z, z[n].w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const float2 u = x2_to_f32(p[w], F16), v = x2_to_f32(q[w], F16);
          if constexpr (INTERLEAVED) {
            p[w] = f32_to_x2(fmaf(u.x, c[w], -(u.y * s[w])), fmaf(u.y, c[w], u.x * s[w]), F16);
            q[w] = f32_to_x2(fmaf(v.x, c[w + 4], -(v.y * s[w + 4])),
                             fmaf(v.y, c[w + 4], v.x * s[w + 4]), F16);
          } else {
            const int e = 2 * w;
            p[w] = f32_to_x2(fmaf(u.x, c[e], -(v.x * s[e])),
                             fmaf(u.y, c[e + 1], -(v.y * s[e + 1])), F16);
            q[w] = f32_to_x2(fmaf(v.x, c[e], u.x * s[e]), fmaf(v.y, c[e + 1], u.y * s[e + 1]),
                             F16);
          }
        }
        x[n] = make_uint4(p[0], p[1], p[2], p[3]);
        z[n] = make_uint4(q[0], q[1], q[2], q[3]);
      }
      *reinterpret_cast<uint4*>(out) = x[n];
      *reinterpret_cast<uint4*>(out + gap) = z[n];
      out += part.out_s[1];
    }
    h += AHEAD;
    if (h >= h1) return;
    load(h);
  }
}

// What both entry points check of the rows, the rotation and which tensors a
// call needs: `pool` where keys and values go to pages.
bsfa_status validate_rows(const bsfa_rope* rope, const bsfa_rows16* r, bool pool) {
  if (r == nullptr) return BSFA_ERR_INVALID_ARG;
  if (r->batch < 0 || r->seqlen < 0) return BSFA_ERR_INVALID_ARG;
  if (r->head_dim != 64 && r->head_dim != 128) return BSFA_ERR_UNSUPPORTED;
  if (r->dtype != BSFA_DTYPE_BF16 && r->dtype != BSFA_DTYPE_F16) return BSFA_ERR_UNSUPPORTED;
  if (r->q && r->num_heads_q <= 0) return BSFA_ERR_INVALID_ARG;
  if (r->k && r->num_heads_kv <= 0) return BSFA_ERR_INVALID_ARG;
  if (r->batch > CACHE4_MAX_BATCH || (r->q && r->num_heads_q > CACHE4_MAX_HEADS) ||
      (r->k && r->num_heads_kv > CACHE4_MAX_HEADS))
    return BSFA_ERR_UNSUPPORTED;
  if (!r->cu_seqlens && static_cast<long long>(r->batch) * r->seqlen > 0x7fffffffLL)
    return BSFA_ERR_UNSUPPORTED;
  if (rope != nullptr) {
    if (rope->pairs <= 0 || rope->num_axes < 1) return BSFA_ERR_INVALID_ARG;
    if (rope->pairs % 8 || 2 * rope->pairs > r->head_dim || rope->num_axes > BSFA_ROPE_MAX_AXES)
      return BSFA_ERR_UNSUPPORTED;
    for (int j = 0; j < rope->pairs; ++j)
      if (rope->axis[j] >= rope->num_axes) return BSFA_ERR_INVALID_ARG;
    if (pool && rope->inverse) return BSFA_ERR_INVALID_ARG;
  }
  if (r->batch == 0 || r->seqlen == 0) return BSFA_OK;
  if (rope != nullptr && !rope->inv_freq) return BSFA_ERR_INVALID_ARG;
  if (pool ? !r->k || !r->v || (r->q && !rope) : !r->q && !r->k) return BSFA_ERR_INVALID_ARG;
  if ((r->q && !r->q_out) || (!pool && r->k && !r->k_out)) return BSFA_ERR_INVALID_ARG;
  const int64_t n = r->cu_seqlens ? 1 : r->batch;
  const int64_t q[3] = {n, r->num_heads_q, r->seqlen}, k[3] = {n, r->num_heads_kv, r->seqlen};
  if (r->q && (!rows_aligned(r->q, r->q_stride, q) || !rows_aligned(r->q_out, r->q_out_stride, q)))
    return BSFA_ERR_UNSUPPORTED;
  if (r->k && !rows_aligned(r->k, r->k_stride, k)) return BSFA_ERR_UNSUPPORTED;
  if (!pool && r->k && !rows_aligned(r->k_out, r->k_out_stride, k)) return BSFA_ERR_UNSUPPORTED;
  if (pool && !rows_aligned(r->v, r->v_stride, k)) return BSFA_ERR_UNSUPPORTED;
  return BSFA_OK;
}

Part part_of(const void* in, const int64_t (&in_s)[3], void* out, const int64_t (&out_s)[3],
             int heads) {
  Part p{};
  if (in == nullptr) return p;
  p.in = static_cast<const uint16_t*>(in);
  p.out = static_cast<uint16_t*>(out);
  for (int i = 0; i < 3; ++i) p.in_s[i] = in_s[i], p.out_s[i] = out_s[i];
  p.heads = heads;
  return p;
}

bsfa_status launch_rows(const bsfa_cache16* c, const bsfa_rope* rope, const bsfa_rows16* r,
                        bsfa_stream_t stream_) {
  RowsArgs a{};
  a.part[QUERIES] = part_of(r->q, r->q_stride, r->q_out, r->q_out_stride, r->num_heads_q);
  if (c != nullptr) {
    a.part[KEYS] = part_of(r->k, r->k_stride, c->k, c->k_stride, r->num_heads_kv);
    a.part[VALUES] = part_of(r->v, r->v_stride, c->v, c->v_stride, r->num_heads_kv);
    a.paged = 1;
    a.table = c->block_table;
    a.table_stride = c->block_table_stride;
    a.table_width = c->block_table_width;
    a.page_size = c->page_size;
    a.num_pages = c->num_pages;
  } else {
    a.part[KEYS] = part_of(r->k, r->k_stride, r->k_out, r->k_out_stride, r->num_heads_kv);
  }
  a.cu = r->cu_seqlens;
  a.start = r->start;
  a.batch = r->batch;
  a.seqlen = r->seqlen;
  a.rows = r->cu_seqlens ? r->seqlen : static_cast<long long>(r->batch) * r->seqlen;
  bool interleaved = false;
  if (rope != nullptr) {
    a.inv_freq = rope->inv_freq;
    a.positions = rope->positions;
    a.pos_s[0] = rope->position_stride[0];
    a.pos_s[1] = rope->position_stride[1];
    a.pairs = rope->pairs;
    a.inverse = rope->inverse != 0;
    a.num_axes = rope->num_axes;
    for (int j = 0; j < rope->pairs; ++j) a.axis[j] = rope->axis[j];
    interleaved = rope->interleaved != 0;
  }
  const int per_block = THREADS / (r->head_dim / CHUNK);
  const long long blocks = (a.rows + per_block - 1) / per_block;
  // A thread that walks over more heads forms its sines and finds its page once
  // for all of them; with few rows the heads go to separate blocks, so that the
  // call still fills the GPU.
  const int heads = a.part[0].heads + a.part[1].heads + a.part[2].heads;
  long long split = (FILL + blocks - 1) / blocks;
  split = split < 1 ? 1 : split > heads ? heads : split;
  a.heads_per_block = static_cast<int>((heads + split - 1) / split);
  unsigned y = 0;
  for (Part& p : a.part) {
    p.blocks = (p.heads + a.heads_per_block - 1) / a.heads_per_block;
    y += p.blocks;
  }
  using Kernel = void (*)(RowsArgs);
  static const Kernel kernels[2][2][2] = {  // [fp16][d = 128][interleaved]
      {{rows16_kernel<64, false, false>, rows16_kernel<64, false, true>},
       {rows16_kernel<128, false, false>, rows16_kernel<128, false, true>}},
      {{rows16_kernel<64, true, false>, rows16_kernel<64, true, true>},
       {rows16_kernel<128, true, false>, rows16_kernel<128, true, true>}}};
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), y);
  cfg.blockDim = dim3(THREADS);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream_);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg,
                         kernels[r->dtype == BSFA_DTYPE_F16][r->head_dim == 128][interleaved],
                         a) == cudaSuccess)
    return BSFA_OK;
  cudaGetLastError();  // taken here, so that a later launch does not report it as its own
  return BSFA_ERR_CUDA;
}

}  // namespace

bsfa_status validate_cache16(const bsfa_cache16* c) {
  if (c->num_heads_kv <= 0 || c->num_pages < 1 || c->page_size <= 0 || c->block_table_width < 0 ||
      c->block_table_stride < c->block_table_width)
    return BSFA_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return BSFA_ERR_UNSUPPORTED;
  if (c->dtype != BSFA_DTYPE_BF16 && c->dtype != BSFA_DTYPE_F16) return BSFA_ERR_UNSUPPORTED;
  if (c->page_size % 16) return BSFA_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->block_table_width) * c->page_size > (1LL << 30))
    return BSFA_ERR_UNSUPPORTED;
  if (c->num_heads_kv > CACHE4_MAX_HEADS) return BSFA_ERR_UNSUPPORTED;
  return BSFA_OK;
}

bsfa_status validate_cache16_pointers(const bsfa_cache16* c) {
  if (!c->k || !c->v || (!c->block_table && c->block_table_width > 0)) return BSFA_ERR_INVALID_ARG;
  const int64_t extent[3] = {c->num_pages, c->num_heads_kv, c->page_size};
  if (!rows_aligned(c->k, c->k_stride, extent) || !rows_aligned(c->v, c->v_stride, extent))
    return BSFA_ERR_UNSUPPORTED;
  // Offsets within a page are 32-bit bytes in the attention kernel.
  const int64_t most = ((1LL << 30) - 1) / c->page_size;
  if (c->k_stride[2] > most || c->v_stride[2] > most) return BSFA_ERR_UNSUPPORTED;
  return BSFA_OK;
}

}  // namespace bsfa

using namespace bsfa;

extern "C" {

bsfa_status bsfa_rotary(const bsfa_rope* rope, const bsfa_rows16* rows, bsfa_stream_t stream) {
  if (rope == nullptr) return BSFA_ERR_INVALID_ARG;
  const bsfa_status v = validate_rows(rope, rows, false);
  if (v != BSFA_OK || rows->batch == 0 || rows->seqlen == 0) return v;
  return launch_rows(nullptr, rope, rows, stream);
}

bsfa_status bsfa_cache16_write(const bsfa_cache16* cache, const bsfa_rope* rope,
                               const bsfa_rows16* rows, bsfa_stream_t stream) {
  if (cache == nullptr) return BSFA_ERR_INVALID_ARG;
  bsfa_status v = validate_rows(rope, rows, true);
  if (v != BSFA_OK) return v;
  v = validate_cache16(cache);
  if (v != BSFA_OK) return v;
  if (rows->num_heads_kv != cache->num_heads_kv || rows->head_dim != cache->head_dim ||
      rows->dtype != cache->dtype)
    return BSFA_ERR_INVALID_ARG;
  if (rows->batch == 0 || rows->seqlen == 0) return BSFA_OK;
  v = validate_cache16_pointers(cache);
  if (v != BSFA_OK) return v;
  return launch_rows(cache, rope, rows, stream);
}

}  // extern "C"
