// The 4-bit paged cache: page layout and the quantiser (include/kvs.h, kvs_page_pool).
//
// Every 32 channels of a row have one half-precision scale s, the smallest half >= max|x| / 7,
// and 4-bit codes c + 8 with c = x / s rounded to the nearest integer, ties to even; the row
// reads back as c s. s >= max|x| / 7 keeps c within [-7, 7] without a clamp, in the subnormal
// halves too. A block that has no such s (a non-finite element, max|x| > 7 * 65504) gets a NaN
// scale, so that it reads back as NaN.
#pragma once

#include <cuda_fp16.h>

#include "kvs_common.cuh"

namespace kvs {

constexpr int kPageRows = KVS_PAGE_ROWS;
static_assert(kPageRows == 32, "one lane per row");

// Byte offsets inside a page of D channels (nb = D / 32 scale blocks a row).
//  K codes  [nb][32 rows][16 B]: the 32 channels of a block in order, low nibble first. Four
//           lanes read a row's block as four words, and eight rows of it are 128 contiguous
//           bytes: the A fragment of an m16n8k16 MMA without bank conflicts.
//  V codes  [nb][16 row pairs][8 quads][2 rows][2 B]: the same two bytes of a channel quad, the
//           rows of a pair side by side, so that one word holds a pair of consecutive rows (the
//           MMA's k index) of four channels; each row still owns whole 16-bit pieces, so rows
//           can be written one at a time.
//  K scales [32 rows][nb] half: a lane takes all blocks of its row with one load.
//  V scales [nb][32 rows] half: a lane takes a row pair of one block with one load.
//  log-counts [32] fp32.
template <int D>
struct PageLayout {
  static constexpr int nb = D / 32;
  static constexpr int kK = 0;
  static constexpr int kV = 16 * D;
  static constexpr int kKs = 32 * D;
  static constexpr int kVs = 34 * D;
  static constexpr int kLn = 36 * D;
  static constexpr int kBytes = 36 * D + 4 * kPageRows;
  static_assert(kBytes % 16 == 0, "bulk copies");
  // offsets of row r: the 16 B of K block b; the 16-bit V piece of quad `quad` of block b
  __host__ __device__ static constexpr int k_code(int b, int r) { return kK + b * 512 + r * 16; }
  __host__ __device__ static constexpr int v_piece(int b, int r, int quad) {
    return kV + b * 512 + (r >> 1) * 32 + quad * 4 + (r & 1) * 2;
  }
  __host__ __device__ static constexpr int k_scale(int b, int r) { return kKs + (r * nb + b) * 2; }
  __host__ __device__ static constexpr int v_scale(int b, int r) { return kVs + (b * kPageRows + r) * 2; }
  __host__ __device__ static constexpr int logn(int r) { return kLn + r * 4; }
};

// Smallest half >= amax / 7, as bits; NaN when there is none. A product and a conversion that both
// round up give it or the one above it; 7 h is exact in fp32 (3 + 11 bits), so the comparison that
// tells is too.
__device__ __forceinline__ uint32_t scale_bits(float amax) {
  constexpr float kSeventh = 0.14285715f;            // the next fp32 above 1/7
  static_assert(7.0 * kSeventh > 1.0, "rounded up");
  uint32_t h = __half_as_ushort(__float2half_ru(__fmul_ru(amax, kSeventh)));
  if (7.f * __half2float(__ushort_as_half((unsigned short)(h - 1))) >= amax) h -= 1;   // (NaN for h = 0: no)
  return h > 0x7bffu ? 0x7fffu : h;
}

// The 8 codes of x[0..7] as nibbles, low first, for the scale with bits `sb`.
//
// bf16 rows: x = m 2^e with m < 2^8, and a rounding border is (2k + 1) n 2^(f - 1) with
// s = n 2^f, n < 2^11. Off a border, x is at least 2^(f - 1) or 2^e away from it, in units of s
// at least 1 / 2n or 2^-8 x / s: more than 2^-12. x * (1/s) is off by at most 6.5 * 2^-23, so
// adding 48 (last place 2^-18) puts a value on a border exactly back onto it and leaves the
// others on their side; the second sum rounds to an integer, ties to even, and leaves c + 8 in
// the low bits. fp32 rows: x and a border may be 2^-24 apart relative to each other, so the
// quotient is rounded correctly by a division (a quotient off a border never rounds onto it: a
// border has 4 bits).
template <typename T>
__device__ __forceinline__ uint32_t quantise8(const float* x, uint32_t sb) {
  const float s = __half2float(__ushort_as_half((unsigned short)sb));
  uint32_t w = 0;
  if constexpr (sizeof(T) == 2) {
    float inv;                                         // off by a last place at most
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
    // the bits of the second sum are 0x4b400000 + code: all eight go into place by shift and add,
    // and the eight constants come off in one piece (modulo 2^32)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = fmaf(x[i], inv, 48.f);
      w += __float_as_uint(__fadd_rn(t, 12582912.f + 8.f - 48.f)) << (4 * i);
    }
    w -= 0x4b400000u * 0x11111111u;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) w |= (uint32_t)(__float2int_rn(__fdiv_rn(x[i], s)) + 8) << (4 * i);
  }
  return sb == 0u || sb == 0x7fffu ? 0x88888888u : w;      // nothing but zeros, or not representable
}

// 8 channels of a row as they are in the cache.
template <typename T> struct Raw8;
template <> struct Raw8<bf16> {
  uint4 v;
  __device__ __forceinline__ void load(const bf16* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
  // the largest magnitude; as integers, magnitudes order like their values, with infinities and
  // NaN on top
  __device__ __forceinline__ float amax() const {
    const uint32_t m = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
    return __uint_as_float(max(m << 16, m & 0xffff0000u));
  }
  __device__ __forceinline__ void widen(float* x) const {
    x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
    x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z); x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
  }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __ldcs(reinterpret_cast<const float4*>(p));
    b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ float amax() const {
    auto u = [](float f) { return __float_as_uint(f) & 0x7fffffffu; };
    return __uint_as_float(max(max(max(u(a.x), u(a.y)), max(u(a.z), u(a.w))),
                               max(max(u(b.x), u(b.y)), max(u(b.z), u(b.w)))));
  }
  __device__ __forceinline__ void widen(float* x) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};

// Codes and scale of 8 channels of a row held by this lane, the 32 channels of a block being
// held by four consecutive lanes (a multiple of 4 on). Whole warps take part.
template <typename T>
__device__ __forceinline__ uint32_t quantise_lane(const Raw8<T>& raw, uint32_t& sb) {
  uint32_t a = __float_as_uint(raw.amax());
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
  sb = scale_bits(__uint_as_float(a));
  float x[8];
  raw.widen(x);
  return quantise8<T>(x, sb);
}

// c = u - 8 of the 8 codes of a word, low nibble first. A code put into the low bits of 2^23 adds
// u 16^j to it, and one fused multiply-add takes 2^23 and 8 off again, exactly; an integer
// conversion would run at a quarter of the rate.
__device__ __forceinline__ void centred8(uint32_t w, float* c) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int j = i & 3;
    const uint32_t v = i < 4 ? w : w >> 16;
    const float f = __uint_as_float((v & (15u << (4 * j))) | 0x4b000000u);
    c[i] = fmaf(f, 1.f / (float)(1 << (4 * j)), -(8388608.f / (float)(1 << (4 * j)) + 8.f));
  }
}

// The 8 channels of a word of codes at scale s.
__device__ __forceinline__ void dequantise8(uint32_t w, float s, float* x) {
  centred8(w, x);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] *= s;
}

// Pages that `rows` >= 0 rows fill (no overflow for the largest int).
__host__ __device__ __forceinline__ int pages_of(int rows) {
  return (int)(((unsigned)rows + kPageRows - 1) / kPageRows);
}

}  // namespace kvs
