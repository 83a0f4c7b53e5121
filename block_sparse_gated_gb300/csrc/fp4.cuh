// fp4.cuh -- one-instruction wrappers for the 4-bit cache kernels: e2m1 and
// e4m3 conversions, the warp-level fp16 matrix product, 16-byte asynchronous
// copies.
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace bsfa {

constexpr int FP4_GROUP = 16;  // elements that share an e4m3 scale

// Eight e2m1 codes (element 0 in the low bits) as four f16x2: r[i] = {element
// 2i (low half), element 2i + 1}.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

// Eight floats as e2m1 codes, element 0 in the low bits; nearest, ties to the
// even code, magnitudes saturate at 6.
__device__ __forceinline__ uint32_t f32x8_to_e2m1(const float* f) {
  uint32_t w;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(w)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return w;
}

// Two e4m3 bytes (low byte first) as f16x2; 0x7f and 0xff become NaN.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two_bytes) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.u16.u32 h, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}"
      : "=r"(r)
      : "r"(two_bytes));
  return r;
}

// A float as an e4m3 byte, nearest, ties to even, saturating at 448.
__device__ __forceinline__ uint32_t f32_to_e4m3(float x) {
  uint32_t r;
  asm("{\n\t.reg .b16 h;\n\tcvt.rn.satfinite.e4m3x2.f32 h, %2, %1;\n\tcvt.u32.u16 %0, h;\n\t}"
      : "=r"(r)
      : "f"(x), "f"(0.f));
  return r & 0xffu;
}

// The low nibble of each byte from `low`, the high one from `high`.
__device__ __forceinline__ uint32_t select_low_nibbles(uint32_t low, uint32_t high) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xe4;" : "=r"(r) : "r"(low), "r"(high), "r"(0x0f0f0f0fu));
  return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t x) {
  float2 r;
  asm("{\n\t.reg .f16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(x));
  return r;
}

// The two 16-bit elements of a word as floats (bf16, or fp16 where `f16`).
__device__ __forceinline__ float2 x2_to_f32(uint32_t x, bool f16) {
  if (f16) return f16x2_to_f32(x);
  return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

// Two floats rounded to 16 bits.
__device__ __forceinline__ uint32_t f32_to_x2(float lo, float hi, bool f16) {
  return f16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
}

// 2^k as a float, k in [-126, 127].
__device__ __forceinline__ float pow2f(int k) { return __int_as_float((k + 127) << 23); }

// A head's exponent, clamped to the documented range; 0 where there is none.
__device__ __forceinline__ int head_exp(const int32_t* e, int head) {
  return e == nullptr ? 0 : max(-100, min(100, __ldg(e + head)));
}

// c += A (16 x 16, row major) * B (16 x 8, column major) in fp16 with fp32 sums.
// Lane 4g + c holds A rows g, g + 8 at columns {2c, 2c+1}, {2c+8, 2c+9}
// (a0, a1: rows at the first pair; a2, a3: at the second), B column g at the
// same rows (b0, b1), and C rows g, g + 8 at columns {2c, 2c+1}.
__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transposes an 8 x 8 matrix of 16-bit elements held two to a lane.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Shared-memory loads by 32-bit address.
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "r"(a)
               : "memory");
  return r;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(a) : "memory");
  return r;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(r) : "r"(a) : "memory");
  return r;
}

// One lane's share of a tile, global -> shared, asynchronously: 16 bytes of keys
// (k1: also of the tile's second half, 512 bytes on), of values `V` bytes on, and
// `Z` bytes of scales.  `ok` false reads nothing and writes zeros.  (One block with
// one predicate: a byte count in a register costs about eight instructions more
// per copy, a predicate of its own one.)
template <int V, int Z>
__device__ __forceinline__ void cp_async_tile(uint32_t dst, uint32_t dst_z, const void* k0,
                                              const void* k1, const void* v0, const void* v1,
                                              const void* z, bool ok) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %7, 0;\n\t"
      "cp.async.cg.shared.global [%0], [%2], 16, p;\n\t"
      "cp.async.cg.shared.global [%0+512], [%3], 16, p;\n\t"
      "cp.async.cg.shared.global [%0+%8], [%4], 16, p;\n\t"
      "cp.async.cg.shared.global [%0+%9], [%5], 16, p;\n\t"
      "cp.async.ca.shared.global [%1], [%6], %10, p;\n\t}" ::"r"(dst),
      "r"(dst_z), "l"(k0), "l"(k1), "l"(v0), "l"(v1), "l"(z), "r"(static_cast<uint32_t>(ok)),
      "n"(V), "n"(V + 512), "n"(Z)
      : "memory");
}
template <int V, int Z>
__device__ __forceinline__ void cp_async_tile(uint32_t dst, uint32_t dst_z, const void* k0,
                                              const void* v0, const void* z, bool ok) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %5, 0;\n\t"
      "cp.async.cg.shared.global [%0], [%2], 16, p;\n\t"
      "cp.async.cg.shared.global [%0+%6], [%3], 16, p;\n\t"
      "cp.async.ca.shared.global [%1], [%4], %7, p;\n\t}" ::"r"(dst),
      "r"(dst_z), "l"(k0), "l"(v0), "l"(z), "r"(static_cast<uint32_t>(ok)), "n"(V), "n"(Z)
      : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Thread-block clusters: this CTA's rank, the two halves of a barrier over all
// threads (release and acquire), and stores into the CTA of rank k at a local
// address's offset.
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_st4(uint32_t addr, uint32_t k, float4 x) {
  asm volatile(
      "{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.v4.f32 [a], {%2,%3,%4,%5};\n\t}" ::"r"(addr),
      "r"(k), "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w)
      : "memory");
}
__device__ __forceinline__ void cluster_st2(uint32_t addr, uint32_t k, float2 x) {
  asm volatile(
      "{\n\t.reg .u32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.v2.f32 [a], {%2,%3};\n\t}" ::"r"(addr),
      "r"(k), "f"(x.x), "f"(x.y)
      : "memory");
}

}  // namespace bsfa
