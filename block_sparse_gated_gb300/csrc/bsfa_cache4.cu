// bsfa_cache4.cu -- bsfa_cache4_write and bsfa_cache4_read: 16-bit keys and
// values quantised into the pages of a 4-bit cache, and read back.
//
// One thread owns 16 consecutive elements of a row (one scale) and walks over
// the heads it is given, of the keys or of the values.
// Both kernels move each byte once and are bound by HBM: the write reads 32
// and stores 9 bytes per 16 elements, the read the other way round.  Measured
// for 131072 tokens of 8 heads, d = 128 (688 MB each): write 101 us, read 105 us,
// 6.8 and 6.5 TB/s (a copy runs at 6.77).
#include <cuda_runtime.h>

#include <cstdint>

#include "bsfa.h"
#include "bsfa_cache4.h"
#include "fp4.cuh"

namespace bsfa {

namespace {

constexpr int THREADS = 128;
// Heads whose loads a thread issues at once (128K tokens written and read: 207.7,
// 211.0, 205.7 us at 1, 2, 4).
constexpr int AHEAD = 4;

struct RowsArgs {
  const uint8_t *kc, *vc, *ks, *vs;  // written by the write, read by the read
  const int32_t *kexp, *vexp;
  long long kc_s[3], vc_s[3], ks_s[3], vs_s[3];  // {page, head, token} bytes
  const uint16_t *k, *v;
  long long k_s[3], v_s[3];  // {batch, head, token} elements
  const int32_t *table, *cu, *start;
  int table_stride, table_width, page_size, num_pages;
  int heads, batch, seqlen;
  long long rows;       // batch * seqlen, or the packed rows; below 2^31
  int heads_per_block;  // heads that one thread walks over
};

// Where row t of the call lies.
struct Slot {
  int b;         // its sequence; negative: none (packed rows outside every sequence)
  int i;         // its row of the 16-bit tensors (within the sequence, or packed)
  int page;      // negative: the position names no cache row
  int token;     // within the page
};

__device__ __forceinline__ Slot find_slot(const RowsArgs& a, int t) {
  Slot s;
  long long pos;  // offsets below zero put rows of a sequence beyond 2^31
  if (a.cu == nullptr) {
    s.b = t / a.seqlen;
    s.i = t - s.b * a.seqlen;
    pos = s.i;
  } else {
    // The last sequence that begins at or before row t.
    int lo = 0, hi = a.batch;
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.cu + mid) <= t)
        lo = mid + 1;
      else
        hi = mid;
    }
    s.b = lo - 1;
    s.i = t;
    if (s.b >= 0 && t >= __ldg(a.cu + s.b + 1)) s.b = -1;
    if (s.b < 0) return s;
    pos = static_cast<long long>(t) - __ldg(a.cu + s.b);
  }
  s.page = -1;
  s.token = 0;
  const long long p = pos + (a.start ? __ldg(a.start + s.b) : 0);
  if (p >= 0 && p < static_cast<long long>(a.table_width) * a.page_size) {
    const int col = static_cast<int>(p) / a.page_size;
    const int page = __ldg(a.table + static_cast<long long>(s.b) * a.table_stride + col);
    if (page >= 0 && page < a.num_pages) {
      s.page = page;
      s.token = static_cast<int>(p) - col * a.page_size;
    }
  }
  return s;
}

// 16 elements -> 16 codes and a scale.
//
// scale = e4m3(a / 6), formed as a * fp32(1/6): a has at most 11 significant
// bits, so where a / 6 lies halfway between two e4m3 values the product is
// exactly that, and elsewhere it stays on its side (checked for every bf16 and
// fp16 magnitude).  1 / scale is the approximate reciprocal after one Newton
// step.  x / scale as x * (1 / scale) is off by less than 2^-20 up to 6.5, so it
// is rounded to a multiple of 2^-16 by adding and subtracting 1.5 * 2^7: a
// quotient halfway between two codes becomes exactly that, and any other stays
// on its side of it, because the short x and scale keep it at least 2^-13 away.
template <bool F16>
__device__ __forceinline__ void quantise16(const uint32_t (&x)[8], float down, uint2& codes,
                                           uint32_t& scale) {
  // Largest magnitude: 16-bit patterns without the sign order like the values,
  // with infinity and NaN above every finite one.
  uint32_t m = x[0] & 0x7fff7fffu;
#pragma unroll
  for (int i = 1; i < 8; ++i) m = __vmaxu2(m, x[i] & 0x7fff7fffu);
  m = max(m & 0xffffu, m >> 16);
  const bool finite = m < (F16 ? 0x7c00u : 0x7f80u);
  const float a = x2_to_f32(m, F16).x * down;
  const uint32_t byte = max(f32_to_e4m3(__fmul_rn(a, 1.f / 6.f)), 1u);  // 1: the scale 2^-9
  const float s = f16x2_to_f32(e4m3x2_to_f16(byte)).x;
  float r = rcp_approx(s);
  r = __fmaf_rn(r, __fmaf_rn(-s, r, 1.f), r) * down;
  const uint64_t r2 = f2_pack(r, r), up = f2_pack(192.f, 192.f), back = f2_pack(-192.f, -192.f);
  float y[16];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = x2_to_f32(x[i], F16);
    f2_unpack(f2_add(f2_fma(f2_pack(f.x, f.y), r2, up), back), y[2 * i], y[2 * i + 1]);
  }
  codes.x = finite ? f32x8_to_e2m1(y) : 0u;
  codes.y = finite ? f32x8_to_e2m1(y + 8) : 0u;
  scale = finite ? byte : 0x7fu;
}

// 16 elements of 16 bits: one 32-byte access where the rows begin on 32 bytes
// (WIDE), else two of 16.
template <bool WIDE>
__device__ __forceinline__ void load16(const uint16_t* p, uint32_t (&x)[8]) {
  if constexpr (WIDE) {
    asm volatile("ld.global.nc.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3]), "=r"(x[4]), "=r"(x[5]),
                   "=r"(x[6]), "=r"(x[7])
                 : "l"(p));
  } else {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
    const uint4 b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
    x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
}
template <bool WIDE>
__device__ __forceinline__ void store16(uint16_t* p, const uint32_t (&x)[8]) {
  if constexpr (WIDE) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(x[0]),
                 "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
  } else {
    reinterpret_cast<uint4*>(p)[0] = make_uint4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<uint4*>(p)[1] = make_uint4(x[4], x[5], x[6], x[7]);
  }
}

// This thread's group of the keys (or values) of its row, head by head.
struct Walk {
  uint16_t* wide;
  uint8_t *codes, *scale;
  long long wide_step, codes_step, scale_step;
  const int32_t* exp;
};

__device__ __forceinline__ Walk walk(const RowsArgs& a, const Slot& s, bool value, int h, int g) {
  const long long* ws = value ? a.v_s : a.k_s;
  const long long* cs = value ? a.vc_s : a.kc_s;
  const long long* ss = value ? a.vs_s : a.ks_s;
  const long long b = a.cu == nullptr ? s.b : 0, page = s.page < 0 ? 0 : s.page;
  Walk w;
  w.wide = const_cast<uint16_t*>(value ? a.v : a.k) + b * ws[0] + h * ws[1] + s.i * ws[2] +
           g * FP4_GROUP;
  w.codes = const_cast<uint8_t*>(value ? a.vc : a.kc) + page * cs[0] + h * cs[1] +
            s.token * cs[2] + g * 8;
  w.scale = const_cast<uint8_t*>(value ? a.vs : a.ks) + page * ss[0] + h * ss[1] +
            s.token * ss[2] + g;
  w.wide_step = ws[1], w.codes_step = cs[1], w.scale_step = ss[1];
  w.exp = value ? a.vexp : a.kexp;
  return w;
}
__device__ __forceinline__ void step(Walk& w) {
  w.wide += w.wide_step;
  w.codes += w.codes_step;
  w.scale += w.scale_step;
}

// The row and group of a thread, and its page.  A block takes the keys or the
// values (blockIdx.z) of heads_per_block heads.
template <int D>
__device__ __forceinline__ bool place(const RowsArgs& a, int& g, Slot& s) {
  constexpr int groups = D / FP4_GROUP;
  g = threadIdx.x & (groups - 1);
  const long long row =
      static_cast<long long>(blockIdx.x) * (THREADS / groups) + threadIdx.x / groups;
  if (row >= a.rows) return false;
  s = find_slot(a, static_cast<int>(row));
  return s.b >= 0;
}

template <int D, bool F16, bool WIDE>
__global__ void __launch_bounds__(THREADS) cache4_write_kernel(const RowsArgs a) {
  int g;
  Slot s;
  if (!place<D>(a, g, s) || s.page < 0) return;
  const int h0 = blockIdx.y * a.heads_per_block, h1 = min(h0 + a.heads_per_block, a.heads);
  Walk w = walk(a, s, blockIdx.z != 0, h0, g);
  for (int h = h0; h < h1; h += AHEAD) {
    uint32_t x[AHEAD][8];
#pragma unroll
    for (int n = 0; n < AHEAD; ++n)
      if (h + n < h1) load16<WIDE>(w.wide + n * w.wide_step, x[n]);
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      if (h + n >= h1) return;
      uint2 codes;
      uint32_t scale;
      quantise16<F16>(x[n], pow2f(-head_exp(w.exp, h + n)), codes, scale);
      *reinterpret_cast<uint2*>(w.codes) = codes;
      *w.scale = static_cast<uint8_t>(scale);
      step(w);
    }
  }
}

template <int D, bool F16, bool WIDE>
__global__ void __launch_bounds__(THREADS) cache4_read_kernel(const RowsArgs a) {
  int g;
  Slot s;
  if (!place<D>(a, g, s)) return;
  const int h0 = blockIdx.y * a.heads_per_block, h1 = min(h0 + a.heads_per_block, a.heads);
  Walk w = walk(a, s, blockIdx.z != 0, h0, g);
  for (int h = h0; h < h1; h += AHEAD) {
    uint2 codes[AHEAD];
    uint32_t scale[AHEAD];
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      codes[n] = make_uint2(0u, 0u);
      scale[n] = 0u;
      if (h + n < h1 && s.page >= 0) {
        codes[n] = __ldg(reinterpret_cast<const uint2*>(w.codes + n * w.codes_step));
        scale[n] = __ldg(w.scale + n * w.scale_step);
      }
    }
#pragma unroll
    for (int n = 0; n < AHEAD; ++n) {
      if (h + n >= h1) return;
      // code * scale has 6 significant bits: exact in fp32, and so is the power
      // of two; one rounding, to the output's type.
      const float f =
          f16x2_to_f32(e4m3x2_to_f16(scale[n])).x * pow2f(head_exp(w.exp, h + n));
      uint32_t out[8];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t e[4];
        e2m1x8_to_f16(half ? codes[n].y : codes[n].x, e);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 y = f16x2_to_f32(e[j]);
          out[4 * half + j] = f32_to_x2(y.x * f, y.y * f, F16);
        }
      }
      store16<WIDE>(w.wide, out);
      step(w);
    }
  }
}

bsfa_status validate_rows(const bsfa_cache4* c, const bsfa_cache4_rows* r) {
  if (c == nullptr || r == nullptr) return BSFA_ERR_INVALID_ARG;
  if (r->batch < 0 || r->seqlen < 0) return BSFA_ERR_INVALID_ARG;
  const bsfa_status v = validate_cache4(c);
  if (v != BSFA_OK) return v;
  if (r->dtype != BSFA_DTYPE_BF16 && r->dtype != BSFA_DTYPE_F16) return BSFA_ERR_UNSUPPORTED;
  if (r->batch > CACHE4_MAX_BATCH) return BSFA_ERR_UNSUPPORTED;
  if (!r->cu_seqlens && static_cast<long long>(r->batch) * r->seqlen > 0x7fffffffLL)
    return BSFA_ERR_UNSUPPORTED;
  if (r->batch == 0 || r->seqlen == 0) return BSFA_OK;
  const bsfa_status q = validate_cache4_pointers(c);
  if (q != BSFA_OK) return q;
  if (!r->k || !r->v) return BSFA_ERR_INVALID_ARG;
  const int64_t extent[3] = {r->cu_seqlens ? 1 : r->batch, c->num_heads_kv, r->seqlen};
  if (!rows_aligned(r->k, r->k_stride, extent) || !rows_aligned(r->v, r->v_stride, extent))
    return BSFA_ERR_UNSUPPORTED;
  return BSFA_OK;
}

bsfa_status launch_rows(const bsfa_cache4* c, const bsfa_cache4_rows* r, bool write,
                        bsfa_stream_t stream_) {
  const bsfa_status v = validate_rows(c, r);
  if (v != BSFA_OK || r->batch == 0 || r->seqlen == 0) return v;
  RowsArgs a{};
  a.kc = c->k;
  a.vc = c->v;
  a.ks = c->k_scale;
  a.vs = c->v_scale;
  a.kexp = c->k_exp;
  a.vexp = c->v_exp;
  for (int i = 0; i < 3; ++i) {
    a.kc_s[i] = c->k_stride[i];
    a.vc_s[i] = c->v_stride[i];
    a.ks_s[i] = c->k_scale_stride[i];
    a.vs_s[i] = c->v_scale_stride[i];
    a.k_s[i] = r->k_stride[i];
    a.v_s[i] = r->v_stride[i];
  }
  a.k = static_cast<const uint16_t*>(r->k);
  a.v = static_cast<const uint16_t*>(r->v);
  a.table = c->block_table;
  a.cu = r->cu_seqlens;
  a.start = r->start;
  a.table_stride = c->block_table_stride;
  a.table_width = c->block_table_width;
  a.page_size = c->page_size;
  a.num_pages = c->num_pages;
  a.heads = c->num_heads_kv;
  a.batch = r->batch;
  a.seqlen = r->seqlen;
  a.rows = r->cu_seqlens ? r->seqlen : static_cast<long long>(r->batch) * r->seqlen;
  const int per_block = THREADS / (c->head_dim / FP4_GROUP);
  const long long blocks = (a.rows + per_block - 1) / per_block;
  // A thread that walks over more heads finds its page once for all of them;
  // with few rows the heads go to separate blocks, so that the call still fills
  // the GPU.
  const int heads = c->num_heads_kv;
  long long split = (2048 + blocks - 1) / blocks;
  split = split < 1 ? 1 : split > heads ? heads : split;
  a.heads_per_block = static_cast<int>((heads + split - 1) / split);
  const dim3 grid(static_cast<unsigned>(blocks),
                  (heads + a.heads_per_block - 1) / a.heads_per_block, 2);
  cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_);
  bool wide = ((reinterpret_cast<uintptr_t>(r->k) | reinterpret_cast<uintptr_t>(r->v)) & 31u) == 0;
  for (int i = 0; i < 3; ++i) wide = wide && r->k_stride[i] % 16 == 0 && r->v_stride[i] % 16 == 0;
  using Kernel = void (*)(RowsArgs);
  static const Kernel kernels[2][2][2][2] = {  // [write][fp16][d = 128][wide]
      {{{cache4_read_kernel<64, false, false>, cache4_read_kernel<64, false, true>},
        {cache4_read_kernel<128, false, false>, cache4_read_kernel<128, false, true>}},
       {{cache4_read_kernel<64, true, false>, cache4_read_kernel<64, true, true>},
        {cache4_read_kernel<128, true, false>, cache4_read_kernel<128, true, true>}}},
      {{{cache4_write_kernel<64, false, false>, cache4_write_kernel<64, false, true>},
        {cache4_write_kernel<128, false, false>, cache4_write_kernel<128, false, true>}},
       {{cache4_write_kernel<64, true, false>, cache4_write_kernel<64, true, true>},
        {cache4_write_kernel<128, true, false>, cache4_write_kernel<128, true, true>}}}};
  kernels[write][r->dtype == BSFA_DTYPE_F16][c->head_dim == 128][wide]<<<grid, THREADS, 0,
                                                                          stream>>>(a);
  return cudaGetLastError() == cudaSuccess ? BSFA_OK : BSFA_ERR_CUDA;
}

}  // namespace

bsfa_status validate_cache4(const bsfa_cache4* c) {
  if (c->num_heads_kv <= 0 || c->num_pages < 1 || c->page_size <= 0 || c->block_table_width < 0 ||
      c->block_table_stride < c->block_table_width)
    return BSFA_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return BSFA_ERR_UNSUPPORTED;
  if (c->page_size % 16) return BSFA_ERR_UNSUPPORTED;
  if (static_cast<long long>(c->block_table_width) * c->page_size > (1LL << 30))
    return BSFA_ERR_UNSUPPORTED;
  if (c->num_heads_kv > CACHE4_MAX_HEADS) return BSFA_ERR_UNSUPPORTED;
  return BSFA_OK;
}

bsfa_status validate_cache4_pointers(const bsfa_cache4* c) {
  if (!c->k || !c->v || !c->k_scale || !c->v_scale ||
      (!c->block_table && c->block_table_width > 0))
    return BSFA_ERR_INVALID_ARG;
  const int64_t unit = c->head_dim / FP4_GROUP;  // bytes of a row's scales
  const uintptr_t code_bits = reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v);
  const uintptr_t scale_bits =
      reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale);
  if ((code_bits & 15u) || (scale_bits & (unit - 1))) return BSFA_ERR_UNSUPPORTED;
  const int extent[3] = {c->num_pages, c->num_heads_kv, c->page_size};
  for (int i = 0; i < 3; ++i) {
    if (extent[i] == 1) continue;  // only ever multiplied by 0
    if (c->k_stride[i] <= 0 || c->v_stride[i] <= 0 || c->k_scale_stride[i] <= 0 ||
        c->v_scale_stride[i] <= 0)
      return BSFA_ERR_UNSUPPORTED;
    // The attention kernel's address arithmetic: page strides below 2^34 bytes,
    // offsets within a page below 2^31.
    const int64_t most = i == 0   ? (1LL << 34) - 1
                         : i == 2 ? 0x7fffffffLL / c->page_size
                                  : INT64_MAX;
    if (c->k_stride[i] > most || c->v_stride[i] > most || c->k_scale_stride[i] > most ||
        c->v_scale_stride[i] > most)
      return BSFA_ERR_UNSUPPORTED;
    if (c->k_stride[i] % 16 || c->v_stride[i] % 16 || c->k_scale_stride[i] % unit ||
        c->v_scale_stride[i] % unit)
      return BSFA_ERR_UNSUPPORTED;
  }
  return BSFA_OK;
}

}  // namespace bsfa

extern "C" {

bsfa_status bsfa_cache4_write(const bsfa_cache4* cache, const bsfa_cache4_rows* rows,
                              bsfa_stream_t stream) {
  return bsfa::launch_rows(cache, rows, true, stream);
}

bsfa_status bsfa_cache4_read(const bsfa_cache4* cache, const bsfa_cache4_rows* rows,
                             bsfa_stream_t stream) {
  return bsfa::launch_rows(cache, rows, false, stream);
}

}  // extern "C"
