// bsfa_decode16_wide.cuh -- attention over the 16-bit cache for calls of many query
// rows per KV head (several tokens of many heads): up to 128 rows to a CTA on the
// fifth-generation tensor cores, so that each key and value is read once for all of
// them.
//
// Mathematics and work split are those of bsfa_decode16.cuh; query rows are the rows
// (M = 128) of S = Q K^T and O = P V here, and a tile is 128 tokens.  A weight goes
// into the products as two 16-bit numbers, as there.
//
// Two softmax warpgroups take the tiles in turn, each with a score buffer, an O and a
// row offset of its own: neither waits for the other, and their results are two parts
// of the segment, which the join adds along with those of other CTAs.  Of a segment
// that lies within one CTA the second warpgroup adds them.  Sums that are not finite
// are formed anew by the join, where nobody waits for them.
//
// Roles (384 threads, one CTA per SM):
//   warp 0      copies K and V tiles through TMA, one box per lane: a box lies within
//               a page.
//   warp 1      issues the products, owns TMEM.
//   warp 2      writes what the join is to do.
//   warps 4-7   softmax of the even tiles, a thread to a row.
//   warps 8-11  ... of the odd ones.
// Bound.  At 128 rows a tile's products take 1900 cycles and its 64 KB (d = 128) 2790 at
// a copy's rate; between them stands the chain of a warpgroup (scores, weights, O), two
// of which overlap.  16 ragged sequences to 32K on four heads (570 MB) take 103 us with
// 64 rows and 109 with 128, 5.5 and 5.2 TB/s (by row tiles of 32 on mma.sync 173 and
// 320); d = 64, 128 rows, 70 us, bound by the weights' arithmetic.  512 new tokens of
// four heads over 16K on eight KV heads: 156 us, 865 TFLOP/s, and half as much again
// for the weights' second numbers.
//
// TMEM: scores at columns 0 and 128, O at 256 and 384.  The weights of 32 keys take
// the columns of their scores: 16 for the first numbers, 16 for the second.
#pragma once
#include "bsfa_decode16.cuh"
#include "bsfa_fwd.cuh"

namespace bsfa {

namespace decode16 {

constexpr int WIDE_UNIT = TILE;        // tokens of a work unit
// A segment's fixed cost, in units (100 ragged sequences to 1K, 64 rows: 89.9 us at 6,
// 91.1 at 3, 95.7 at 10, before segments overlapped).
constexpr int WIDE_SEGMENT_UNITS = 6;
constexpr int WIDE_MIN_UNITS = 1;  // shortest piece of the line worth a CTA (1 x 1K with 64
                                   // rows: 13.0 us; at 4 16.1)
constexpr int WIDE_THREADS = 384;
// Tiles that a warpgroup sums in TMEM, at most: the tensor cores cut off what they add
// instead of rounding it, up to 2^-23 of the sum at each of a tile's sixteen steps, so
// 2^-13 of a run's O at worst (values of one sign over 40000 tokens, fp16: 2^-14 on
// average).  Longer runs are added in fp32, in the workspace.
constexpr int WIDE_RUN = 64;
// Of the key and of the value ring (16 ragged sequences to 32K with 64 rows: 104.7 us; at
// 2 110.1).
constexpr int WIDE_STAGES = 3;
constexpr int WIDE_PARTS = 2;          // that a CTA leaves of a segment

struct WideCtrl {
  uint64_t q_full, q_empty;
  uint64_t k_full[WIDE_STAGES], k_empty[WIDE_STAGES];
  uint64_t v_full[WIDE_STAGES], v_empty[WIDE_STAGES];
  uint64_t s_full[2], p_full[2], pv_done[2];  // of each warpgroup
  uint64_t x_full, x_empty;  // the first warpgroup's part of a segment: there, read
  float2 part[TILE];         // ... its offsets and sums
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int cut[WIDE_THREADS / 32 + 2];
};

template <int D>
struct WideLayout {
  static constexpr int TB = TILE * D * 2;  // bytes of a tile
  static constexpr int K_OFF = TB, V_OFF = K_OFF + WIDE_STAGES * TB;
  static constexpr int C_OFF = V_OFF + WIDE_STAGES * TB;
  static constexpr int RAW = C_OFF + static_cast<int>(sizeof(WideCtrl)) + 1024;
  // At least 120 KB, so that one CTA is resident per SM (it takes all of TMEM).
  static constexpr int BYTES = RAW > 120 * 1024 ? RAW : 120 * 1024;
  static_assert(BYTES <= 227 * 1024, "shared memory");
};

// One segment's part in a CTA's piece.
struct WideWork {
  int b, kvh, seg, r0, n_rows, len, min_lim, max_lim;
  int t0, n;            // first tile, tiles
  bool began, whole;    // the segment begins in this CTA, and ends there as well
  int last_cta;         // ... or in that one
};

struct WideWalk {
  const DecArgs& a;
  Piece p;
  int u, b, base;
  __device__ __forceinline__ WideWalk(const DecArgs& a_, const Piece& p_)
      : a(a_), p(p_), u(p_.begin), b(p_.b), base(p_.base) {}
  __device__ __forceinline__ bool next(WideWork& w) {
    if (u >= p.end) return false;
    const int per_b = a.heads_kv * a.row_tiles;
    w.b = b;
    w.len = clamp_len(a, b);
    const int n_units = units_of<WIDE_UNIT, WIDE_SEGMENT_UNITS>(w.len);
    w.seg = (u - base) / n_units;
    const int u0 = u - base - w.seg * n_units, u1 = min(n_units, u0 + p.end - u);
    w.kvh = w.seg / a.row_tiles;
    w.r0 = (w.seg - w.kvh * a.row_tiles) * TILE;
    w.n_rows = min(TILE, a.rows - w.r0);
    const int first_i = w.r0 / a.group, last_i = (w.r0 + w.n_rows - 1) / a.group;
    w.min_lim = a.causal ? max(0, w.len - a.q_len + first_i + 1) : w.len;
    w.max_lim = a.causal ? max(0, w.len - a.q_len + last_i + 1) : w.len;
    w.t0 = max(0, u0 - WIDE_SEGMENT_UNITS);
    w.n = max(0, min(max(0, u1 - WIDE_SEGMENT_UNITS), (w.max_lim + TILE - 1) / TILE) - w.t0);
    w.began = u0 == 0;
    w.whole = w.began && u1 == n_units;
    w.last_cta = (u + n_units - 1) / p.per_cta;
    u += u1 - u0;
    if (u1 == n_units && w.seg == per_b - 1) {
      base += n_units * per_b;
      ++b;
    }
    return true;
  }
};

template <int D, bool F16>
__global__ void __launch_bounds__(WIDE_THREADS, 1)
    decode16_wide_kernel(const __grid_constant__ CUtensorMap tmK,
                         const __grid_constant__ CUtensorMap tmV,
                         const __grid_constant__ DecArgs a) {
  using LY = WideLayout<D>;
  constexpr int TB = LY::TB, NHALF = D / 64, HB = TILE * 128;  // 64-column halves of a tile
  constexpr int ST = WIDE_STAGES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t *sQ = base, *sK = base + LY::K_OFF, *sV = base + LY::V_OFF;
  WideCtrl* c = reinterpret_cast<WideCtrl*>(base + LY::C_OFF);
  volatile int* abort = &c->abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&c->q_full, 128);
    mbar_init(&c->q_empty, 1);
    for (int i = 0; i < ST; ++i) {
      mbar_init(&c->k_full[i], 1);
      mbar_init(&c->k_empty[i], 1);
      mbar_init(&c->v_full[i], 1);
      mbar_init(&c->v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c->s_full[i], 1);
      mbar_init(&c->p_full[i], 128);
      mbar_init(&c->pv_done[i], 1);
    }
    mbar_init(&c->x_full, 128);
    mbar_init(&c->x_empty, 128);
    mbar_init(&c->drain, 1);
    c->abort = 0;
    fence_mbarrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&tmK);
    prefetch_tensormap(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(&c->tmem_base, 512);
    tmem_relinquish();
  }
  allow_next_kernel();
  wait_for_kernels_before();
  const Piece piece = cut<WIDE_UNIT, WIDE_SEGMENT_UNITS, WIDE_MIN_UNITS, WIDE_THREADS / 32>(a, c->cut);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem_base;

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    const int box = a.box, boxes = TILE / box;
    uint32_t kc = 0;  // tiles so far
    bool ok = true;
    WideWork w;
    for (WideWalk walk(a, piece); ok && walk.next(w);) {
      const int32_t* table = a.table + static_cast<long long>(w.b) * a.table_stride;
      const int page_size = a.tiles_per_page * TOK;
      for (int t = 0; t < w.n; ++t, ++kc) {
        // This lane's box; those past what any row sees stay as they are: their scores
        // are masked and their values zeroed.
        const int pos = (w.t0 + t) * TILE + lane * box;
        const bool mine = lane < boxes && pos < w.max_lim;
        const int loaded = __popc(__ballot_sync(0xffffffffu, mine));
        int page = a.num_pages, at = 0;  // a page that is none reads as zeros
        if (mine) {
          const int entry = __ldg(table + pos / page_size);
          at = pos % page_size;
          if (entry >= 0 && entry < a.num_pages) page = entry;
        }
        const uint32_t st = kc % ST, par = ((kc / ST) & 1) ^ 1;
        auto copy = [&](uint64_t* full, uint8_t* tile, const CUtensorMap* map) {
          if (lane == 0) mbar_arrive_expect_tx(full, loaded * box * D * 2);
          __syncwarp();
          if (mine)
            for (int hf = 0; hf < NHALF; ++hf)
              tma_load_4d(tile + hf * HB + lane * box * 128, map, full, hf * 64, at, w.kvh, page);
          __syncwarp();
        };
        if (!(ok = wait_all(&c->k_empty[st], par, abort, a.err, ERR_WAIT_K_EMPTY))) break;
        copy(&c->k_full[st], sK + st * TB, &tmK);
        if (!(ok = wait_all(&c->v_empty[st], par, abort, a.err, ERR_WAIT_V_EMPTY))) {
          drain_wait(&c->k_full[st], (kc / ST) & 1);
          break;
        }
        copy(&c->v_full[st], sV + st * TB, &tmV);
      }
    }
    if (!ok) {  // let every copy already issued land before the CTA can exit
      for (uint32_t i = 0; i < ST && i < kc; ++i) {
        const uint32_t f = kc - 1 - i;
        drain_wait(&c->k_full[f % ST], (f / ST) & 1);
        drain_wait(&c->v_full[f % ST], (f / ST) & 1);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ products
    constexpr uint32_t IDESC_QK = idesc_f32acc<F16>(128, TILE, false, false);
    constexpr uint32_t IDESC_PV = idesc_f32acc<F16>(128, D, false, true);
    const uint64_t dQ = smem_desc_sw128(smem_u32(sQ), 16, 1024);
    const uint64_t dK = smem_desc_sw128(smem_u32(sK), 16, 1024);
    const uint64_t dV = smem_desc_sw128(smem_u32(sV), HB, 1024);
    uint32_t kc = 0, vc = 0, uc = 0, pc[2] = {0, 0};
    bool ok = true;
    WideWork w;
    for (WideWalk walk(a, piece); ok && walk.next(w);) {
      if (w.n == 0) continue;
      if (!(ok = wait_all(&c->q_full, uc & 1, abort, a.err, ERR_WAIT_Q_FULL))) break;
      ++uc;
      auto scores = [&](int t) -> bool {  // S of tile t
        const uint32_t st = kc % ST;
        if (!wait_all(&c->k_full[st], (kc / ST) & 1, abort, a.err, ERR_WAIT_K_FULL)) return false;
        tc_fence_after();
        if (elect_one()) {
          issue_qk<D, 1>(tmem + (t & 1) * 128, dQ, dK + ((st * TB) >> 4), IDESC_QK);
          umma_commit(&c->s_full[t & 1]);
          umma_commit(&c->k_empty[st]);
          if (t == w.n - 1) umma_commit(&c->q_empty);
        }
        __syncwarp();
        ++kc;
        return true;
      };
      for (int t = 0; t < 2 && t < w.n; ++t)
        if (!(ok = scores(t))) break;
      for (int t = 0; ok && t < w.n; ++t, ++vc) {
        const int wg = t & 1;
        const uint32_t st = vc % ST;
        if (!(ok = wait_all(&c->v_full[st], (vc / ST) & 1, abort, a.err, ERR_WAIT_V_FULL))) break;
        const int seen = w.max_lim - (w.t0 + t) * TILE;  // a hidden value may be anything
        if (seen < TILE) zero_tile_rows<D>(sV + st * TB, seen, lane);
        if (!(ok = wait_all(&c->p_full[wg], pc[wg] & 1, abort, a.err, ERR_WAIT_P_FULL))) break;
        ++pc[wg];
        tc_fence_after();
        if (elect_one()) {
          const uint32_t d_o = tmem + 256 + wg * 128, d_p = tmem + wg * 128;
          const uint64_t dv = dV + ((st * TB) >> 4);
          const bool fresh = (t >> 1) % WIDE_RUN == 0;  // a run begins
#pragma unroll
          for (int kk = 0; kk < TILE / 16; ++kk) {
            const uint32_t p = d_p + 32 * (kk >> 1) + 8 * (kk & 1);
            umma_ts(d_o, p + 16, dv + ((kk * 2048) >> 4), IDESC_PV, fresh && kk == 0 ? 0u : 1u);
            umma_ts(d_o, p, dv + ((kk * 2048) >> 4), IDESC_PV, 1u);
          }
          umma_commit(&c->pv_done[wg]);
          umma_commit(&c->v_empty[st]);
        }
        __syncwarp();
        if (t + 2 < w.n && !(ok = scores(t + 2))) break;
      }
    }
    // Drain: every issued product completes before TMEM is given back.
    if (elect_one()) umma_commit(&c->drain);
    __syncwarp();
    drain_wait(&c->drain, 0);
  } else if (warp == 2) {
    // ------------------------------------------------------------ the join's table
    // Of every segment that begins in this piece, by a warp that waits for nothing: the
    // join follows it even where a wait of the others has run out and they have left.
    WideWork w;
    for (WideWalk walk(a, piece); walk.next(w);)
      if (w.began && lane == 0)
        a.joins[w.b * a.heads_kv * a.row_tiles + w.seg] =
            make_int4(w.b, w.seg, static_cast<int>(blockIdx.x), w.whole ? -1 : w.last_cta);
  } else if (warp >= 4) {
    // ------------------------------------------------------------ softmax
    const int wg = (warp - 4) >> 2, wq = warp & 3, row = wq * 32 + lane;
    const uint32_t tlane = tmem + (static_cast<uint32_t>(wq * 32) << 16);
    const uint32_t tS = tlane + wg * 128, tO = tlane + 256 + wg * 128;
    const float sc = a.sigma_log2;
    uint32_t sc_n = 0, pv_n = 0;  // tiles of this warpgroup, its products
    uint32_t uc = 0, xc = 0;      // queries so far, segments within this CTA
    uint32_t read = 0;            // ... and those whose first part is known to have been read
    bool ok = true;
    // The second warpgroup may have yet to read the first one's O and part of the segment
    // before, which are written from here on.
    auto part_is_free = [&]() -> bool {
      if (wg != 0 || read == xc) return true;
      read = xc;
      return wait_all(&c->x_empty, (xc - 1) & 1, abort, a.err, ERR_WAIT_WG);
    };
    WideWork w;
    for (WideWalk walk(a, piece); ok && walk.next(w);) {
      const int r = w.r0 + row;
      const bool real = row < w.n_rows;
      const int i = real ? r / a.group : 0;
      const int lim = !real ? 0 : a.causal ? w.len - a.q_len + i + 1 : w.len;
      const int slot = WIDE_PARTS * (2 * static_cast<int>(blockIdx.x) + (w.began ? 1 : 0)) + wg;
      const long long at = static_cast<long long>(slot) * TILE + row;
      if (w.n > 0 && wg == 0) {
        // ---- this thread's query row, swizzled as TMA would (by the first warpgroup: the
        // second may still be joining the segment before)
        const int h = w.kvh * a.group + (r - i * a.group);
        const uint4* src = reinterpret_cast<const uint4*>(a.q + w.b * a.q_s[0] + h * a.q_s[1] +
                                                          i * a.q_s[2]);
        uint4 y[D / 8];
#pragma unroll
        for (int x = 0; x < D / 8; ++x) y[x] = real ? __ldg(src + x) : make_uint4(0u, 0u, 0u, 0u);
        if (uc > 0 &&
            !(ok = wait_all(&c->q_empty, (uc - 1) & 1, abort, a.err, ERR_WAIT_Q_EMPTY)))
          break;
        ++uc;
#pragma unroll
        for (int x = 0; x < D / 8; ++x)
          *reinterpret_cast<uint4*>(sQ + (x >> 3) * HB + row * 128 +
                                    (((x & 7) ^ (row & 7)) << 4)) = y[x];
        fence_proxy_async_shared();
        mbar_arrive(&c->q_full);
      }
      float z = NO_SCORE, l = 0.f;        // of the run
      float z_c = NO_SCORE, l_c = 0.f;    // of the runs before it
      bool carried = false;
      int in_run = 0;                     // tiles of the run so far
      // Adds the run's O to what the part holds.
      auto flush = [&](bool any) -> bool {
        if (any && !wait_all(&c->pv_done[wg], (pv_n - 1) & 1, abort, a.err, ERR_WAIT_O_FULL))
          return false;
        tc_fence_after();
        const float both = fminf(z, z_c);
        const float f = ex2_approx(both - z), f_c = ex2_approx(both - z_c);
        float4* dst = reinterpret_cast<float4*>(a.part_o + at * D);
#pragma unroll 1
        for (int x = 0; x < D / 32; ++x) {
          uint32_t o[32];
          if (any) {
            tmem_ld32(tO + 32 * x, o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          if (!real) continue;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float4 y = make_float4(__uint_as_float(o[4 * e]) * f, __uint_as_float(o[4 * e + 1]) * f,
                                   __uint_as_float(o[4 * e + 2]) * f,
                                   __uint_as_float(o[4 * e + 3]) * f);
            if (carried) {
              const float4 old = dst[8 * x + e];
              y.x = fmaf(old.x, f_c, y.x), y.y = fmaf(old.y, f_c, y.y);
              y.z = fmaf(old.z, f_c, y.z), y.w = fmaf(old.w, f_c, y.w);
            }
            dst[8 * x + e] = y;
          }
        }
        tc_fence_before();
        l_c = fmaf(l_c, f_c, l * f);
        z_c = both;
        l = 0.f;
        carried = true;
        in_run = 0;
        return true;
      };

      for (int t = wg; t < w.n; t += 2) {
        if (in_run == WIDE_RUN && !(ok = flush(true))) break;
        if (!(ok = wait_all(&c->s_full[wg], sc_n & 1, abort, a.err, ERR_WAIT_S_FULL))) break;
        ++sc_n;
        tc_fence_after();
        const int tok0 = (w.t0 + t) * TILE;
        const bool masked = tok0 + TILE > w.min_lim;
        const int seen = lim - tok0;  // keys of the tile that this row sees
        // ---- the largest score
        float m = -INFINITY;
        if (!masked) {
#pragma unroll 1
          for (int x = 0; x < 4; ++x) {
            uint32_t s[32];  // not looked at: the load gives their maximum
            float mx;
            tmem_ld32_max(tS + 32 * x, s, mx);
            tmem_wait_ld();
            m = fmaxf(m, mx);
          }
        } else {
#pragma unroll 1
          for (int x = 0; x < 4; ++x) {
            uint32_t s[32];
            tmem_ld32(tS + 32 * x, s);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (32 * x + e < seen) m = fmaxf(m, __uint_as_float(s[e]));
          }
        }
        m *= sc;
        const bool over = m + z > most_of<F16>(a);
        if (__any_sync(0xffffffffu, over)) {
          const float z1 = over ? fminf(z, shift_of<F16>(a) - m) : z;
          const float f = ex2_approx(z1 - z);
          z = z1;
          l *= f;
          if (in_run > 0) {  // O of the run's tiles before
            if (!(ok = wait_all(&c->pv_done[wg], (pv_n - 1) & 1, abort, a.err, ERR_WAIT_O_FULL)))
              break;
            tc_fence_after();
#pragma unroll 1
            for (int x = 0; x < D / 32; ++x) {
              uint32_t o[32];
              tmem_ld32(tO + 32 * x, o);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(tO + 32 * x, o);
            }
            tmem_wait_st();
          }
        }
        // ---- weights, in place of their scores
        const uint64_t sc2 = f2_pack(sc, sc), z2 = f2_pack(z, z);
        uint64_t sum2[2] = {0, 0};
        auto weights = [&](auto masked_tag) {
#pragma unroll 1
          for (int x = 0; x < 4; ++x) {
            uint32_t s[32], hi[16], lo[16];
            tmem_ld32(tS + 32 * x, s);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float p0, p1;
              f2_unpack(
                  f2_fma(f2_pack(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), sc2, z2),
                  p0, p1);
              p0 = ex2_approx(p0), p1 = ex2_approx(p1);
              if constexpr (decltype(masked_tag)::value) {
                if (32 * x + 2 * e >= seen) p0 = 0.f;
                if (32 * x + 2 * e + 1 >= seen) p1 = 0.f;
              }
              const uint64_t p = f2_pack(p0, p1);
              sum2[e & 1] = f2_add(sum2[e & 1], p);
              hi[e] = pack_x2<F16>(p0, p1);
              const float2 q = x2_to_f32(hi[e], F16);
              f2_unpack(f2_add(p, f2_pack(-q.x, -q.y)), p0, p1);
              lo[e] = pack_x2<F16>(p0, p1);
            }
            tmem_st16(tS + 32 * x, hi);
            tmem_st16(tS + 32 * x + 16, lo);
          }
        };
        if (masked)
          weights(std::true_type{});
        else
          weights(std::false_type{});
        float l0, l1;
        f2_unpack(f2_add(sum2[0], sum2[1]), l0, l1);
        l += l0 + l1;
        tmem_wait_st();
        tc_fence_before();
        if (!(ok = part_is_free())) break;
        mbar_arrive(&c->p_full[wg]);
        ++pv_n;
        ++in_run;
      }
      if (!ok || !(ok = part_is_free())) break;
      if (!w.whole || carried) {
        if (!(ok = flush(in_run > 0))) break;
        if (!w.whole) {
          if (real) a.part_ml[at] = make_float2(-z_c, l_c);
          continue;
        }
      }
      // ---- a segment within this CTA: both parts from where they are, TMEM or (after
      // more than one run) global memory
      const bool any = in_run > 0;
      if (any && !(ok = wait_all(&c->pv_done[wg], (pv_n - 1) & 1, abort, a.err, ERR_WAIT_O_FULL)))
        break;
      if (wg == 0) {
        c->part[row] = carried ? make_float2(z_c, l_c) : make_float2(z, l);
        tc_fence_before();
        mbar_arrive(&c->x_full);
      } else {
        if (!(ok = wait_all(&c->x_full, xc & 1, abort, a.err, ERR_WAIT_WG))) break;
        tc_fence_after();
        const float2 other = c->part[row];
        const int tiles0 = (w.n + 1) / 2;  // of the other warpgroup
        const float my_z = carried ? z_c : z, my_l = carried ? l_c : l;
        const float both = fminf(my_z, other.x);
        const float f = ex2_approx(both - my_z), f0 = ex2_approx(both - other.x);
        const float sum = fmaf(my_l, f, other.y * f0);
        const float4 *own = reinterpret_cast<const float4*>(a.part_o + at * D),
                     *first = own - TILE * D / 4;
        auto joined = [&](int x, float (&y)[32]) {  // 32 elements
          float o0[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = o0[e] = 0.f;
          auto load = [&](uint32_t from, const float4* held, bool in_memory, bool there,
                          float (&to)[32]) {
            if (in_memory) {
#pragma unroll
              for (int e = 0; e < 8 && real; ++e)
                *reinterpret_cast<float4*>(to + 4 * e) = __ldcg(held + 8 * x + e);
            } else if (there) {
              uint32_t v[32];
              tmem_ld32(from + 32 * x, v);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) to[e] = __uint_as_float(v[e]);
            }
          };
          load(tO, own, carried, any, y);
          load(tO - 128, first, tiles0 > WIDE_RUN, tiles0 > 0, o0);
#pragma unroll
          for (int e = 0; e < 32; ++e) y[e] = fmaf(y[e], f, o0[e] * f0);
        };
        auto store = [&](int x, const float (&y)[32]) {
#pragma unroll
          for (int e = 0; e < 32 && real; e += 4)
            store_row4(a, w.b, w.kvh, r, 32 * x + e, -both, sum,
                       make_float4(y[e], y[e + 1], y[e + 2], y[e + 3]));
        };
        bool finite = true;
#pragma unroll 1
        for (int x = 0; x < D / 32; ++x) {
          float y[32];
          joined(x, y);
#pragma unroll
          for (int e = 0; e < 32; ++e) finite = finite && fabsf(y[e]) < INFINITY;
          if (!a.in_place) store(x, y);
        }
        // What is not finite is formed anew by the join, from the queries: where the output
        // takes their place, nothing is stored before they have been kept.
        const bool anew = real && !finite && sum < INFINITY;
        if (a.in_place) {
          if (anew) {
            const uint4* src = reinterpret_cast<const uint4*>(output_row(a, w.b, w.kvh, r));
            uint4* dst = reinterpret_cast<uint4*>(
                a.kept + ((static_cast<long long>(w.b) * a.heads_kv + w.kvh) * a.rows + r) * D);
#pragma unroll
            for (int x = 0; x < D / 8; ++x) dst[x] = src[x];
          }
#pragma unroll 1
          for (int x = 0; x < D / 32; ++x) {
            float y[32];
            joined(x, y);
            store(x, y);
          }
        }
        const uint32_t rows_anew = __ballot_sync(0xffffffffu, anew);
        if (lane == 0)
          a.anew[4 * (w.b * a.heads_kv * a.row_tiles + w.seg) + wq] = rows_anew;
        tc_fence_before();
        mbar_arrive(&c->x_empty);
      }
      ++xc;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, 512);
}

// One call: the kernel and the join of its parts.
template <int D, bool F16>
bsfa_status run_wide(const CUtensorMap& tmK, const CUtensorMap& tmV, const DecArgs& a,
                     const Plan& pl, int sms, int dev, cudaStream_t stream) {
  static_assert(WIDE_PARTS * MAX_SMS <= MAX_PARTS, "the join's weights");
  static std::atomic<uint64_t> ready{0};
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (!(ready.load(std::memory_order_relaxed) & bit)) {
    const bsfa_status v = status_of(cudaFuncSetAttribute(
        decode16_wide_kernel<D, F16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
        WideLayout<D>::BYTES));
    if (v != BSFA_OK) return v;
    ready.fetch_or(bit, std::memory_order_relaxed);
  }
  int grid = sms < MAX_SMS ? sms : MAX_SMS;
  const long long most = (pl.all_units + WIDE_MIN_UNITS - 1) / WIDE_MIN_UNITS;
  if (most < grid) grid = static_cast<int>(most);
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr = after_kernels();
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(WIDE_THREADS);
  cfg.dynamicSmemBytes = WideLayout<D>::BYTES;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const bsfa_status first =
      status_of(cudaLaunchKernelEx(&cfg, decode16_wide_kernel<D, F16>, tmK, tmV, a));
  if (first != BSFA_OK) return first;
  return launch_join<D, TILE, WIDE_PARTS>(a, pl.segments, grid, pl.segments, stream);
}

}  // namespace decode16

}  // namespace bsfa
