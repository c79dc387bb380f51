// GQA decode attention over the 4-bit paged cache (kvs_page_decode_attn).
//
// Attention of the KVSlimmer deep dive ("论文专题讲解：KVSlimmer：非对称 KV 合并的数学与工程",
// §数学主线三) with the log-count bias of merged rows, over rows held in pages (pages.cuh):
//   x_t = q . k_t / sqrt(d) + logn_t,  out = sum_t 2^(x_t log2 e - M) v_t / sum_t 2^(x_t log2 e - M)
//
// Work split. The pages of all units (KV heads of all sequences) are numbered one unit after
// another, and CTA i takes pages [i c, (i + 1) c): lengths are ragged and known on the device
// only, so every CTA sums them up for itself. A unit that lies in one CTA is finished there; one
// that spans several gets a partial row per CTA in the workspace, and the last of them to arrive
// (a counter per unit) combines. No CTA waits for another.
//
// A page is one contiguous block, so a single bulk copy (untiled, no tensor map) brings it into
// the ring of the warp that works on it; each warp issues its own copies and needs no other
// warp until the end of a unit.
#include "decode_common.cuh"
#include "kvs_common.cuh"
#include "kvs_kernels.h"
#include "pages.cuh"
#include "ptx.cuh"

namespace kvs {

constexpr int kPdWarps = 8;
constexpr int kPdThreads = kPdWarps * 32;
constexpr int kPdStages = 2;

template <int D, int G>
struct PageDecodeShape {
  static constexpr int kRing = kPdWarps * kPdStages * PageLayout<D>::kBytes;
  // the warps' partial outputs [NW][G][D]; the CTA that finishes a unit reuses them for the
  // factors of the splits [G][CTAs] and the sums of all groups of threads but the first
  static constexpr int kUnits = G * D / 4;                       // 4-column units of an output
  static constexpr int kGroups = kPdThreads / kUnits;
  static_assert(kUnits * kGroups == kPdThreads, "one thread per unit and group");
  static constexpr int kFac = G * kPageDecodeCtas * 4;
  static constexpr int kSums = (kGroups - 1) * kUnits * 16;
  static constexpr int kPart = kPdWarps * G * D * 4;
  static constexpr int kAcc = kPart > kFac + kSums ? kPart : kFac + kSums;
  static_assert(kFac % 16 == 0 && kAcc % 16 == 0, "alignment");
  static constexpr int kSmem = kRing + kAcc + kPdWarps * kPdStages * 8;
};

// Weight of a partial (m, l, acc) against the reference M. One without a row that counts has
// l = 0; NaN logits leave m at -inf and l NaN, which has to go through.
__device__ __forceinline__ float part_weight(float m, float l, float M) {
  return l != 0.f ? exp2f(m - M) : 0.f;
}

// Pages of a unit in the numbering: an empty one has one, so that a CTA finishes it.
__device__ __forceinline__ int unit_span(int L) { return L > 0 ? pages_of(L) : 1; }

// One warp's share of a unit: its softmax state over the pages it has taken. begin() loads the
// unit's queries, take() adds the first nval rows of a page, end() writes the partial output
// [G][D] and (m, l) per query head (log2 domain; m is a reference, not always the maximum).

// fp32: CUDA cores, every product and sum in fp32. Logits with a lane per row, values with a lane
// per channel quad. Not tuned: the fp32 cache is the accuracy path, and this kernel stays within
// an fp32 softmax attention's own error.
template <typename T, int D, int G>
struct PageWarp {
  using P = PageLayout<D>;
  static constexpr int QL = D / 4, RPS = 32 / QL;       // lanes per row of V, rows at a time
  const float (*qs)[D];
  float m[G], l[G], acc[G][4];

  __device__ __forceinline__ void begin(const T*, const float (*qs_)[D], int) {
    qs = qs_;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      m[g] = -INFINITY;
      l[g] = acc[g][0] = acc[g][1] = acc[g][2] = acc[g][3] = 0.f;
    }
  }

  __device__ __forceinline__ void take(unsigned char* pg, int nval, int lane) {
    float x[G];
#pragma unroll
    for (int g = 0; g < G; ++g) x[g] = 0.f;
#pragma unroll
    for (int b = 0; b < P::nb; ++b) {
      const uint4 w4 = *reinterpret_cast<const uint4*>(pg + P::k_code(b, lane));
      const float s = __half2float(*reinterpret_cast<const __half*>(pg + P::k_scale(b, lane)));
      const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
      float y[G];
#pragma unroll
      for (int g = 0; g < G; ++g) y[g] = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float k[8];
        dequantise8(w[i], 1.f, k);
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int c = 0; c < 8; ++c) y[g] = fmaf(qs[g][b * 32 + i * 8 + c], k[c], y[g]);
      }
#pragma unroll
      for (int g = 0; g < G; ++g) x[g] = fmaf(y[g], s, x[g]);
    }
    const float ln = *reinterpret_cast<const float*>(pg + P::logn(lane)) * kLog2e;
    float p[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float xg = lane < nval ? x[g] + ln : -INFINITY;
      const float M = fmaxf(m[g], warp_max(xg));
      const float base = M == -INFINITY ? 0.f : M;
      const float f = exp2f(m[g] - base);
      p[g] = exp2f(xg - base);
      l[g] = fmaf(l[g], f, p[g]);
      m[g] = M;
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[g][c] *= f;
    }
    const int quad = lane % QL, b = quad / 8;
    for (int r0 = 0; r0 < nval; r0 += RPS) {
      const int r = r0 + lane / QL;
      const uint32_t w = *reinterpret_cast<const uint16_t*>(pg + P::v_piece(b, r, quad % 8));
      float s = __half2float(*reinterpret_cast<const __half*>(pg + P::v_scale(b, r)));
      if (r >= nval) s = 0.f;                  // whatever the rest of the page holds
      float v[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = (float)((int)(w >> (4 * c) & 15u) - 8) * s;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float pr = __shfl_sync(0xffffffffu, p[g], r);
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[g][c] = fmaf(pr, v[c], acc[g][c]);
      }
    }
  }

  __device__ __forceinline__ void end(float* sa, float* sm, float* sl, int lane) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float ls = warp_sum(l[g]);
      if (lane == 0) {
        sm[g] = m[g];
        sl[g] = ls;
      }
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (RPS == 2) acc[g][c] += __shfl_xor_sync(0xffffffffu, acc[g][c], 16);
      if (lane < QL)
        *reinterpret_cast<float4*>(sa + g * D + lane * 4) =
            make_float4(acc[g][0], acc[g][1], acc[g][2], acc[g][3]);
    }
  }
};

// bf16: m16n8k16 MMAs on half operands, the rows of the page in the M (or K) dimension and the
// query heads in the N = 8 columns, as in the bf16 cache's decode (S^T = K Q^T, O^T = V^T P^T).
//
// The codes are never converted. A 4-bit code u in bits 0-3 or 4-7 of a 16-bit half IS the
// subnormal half u 2^-24 or 16 u 2^-24, which the MMA multiplies exactly; so one AND makes an A
// register out of a word of codes. The offset of 8 and the factors are put right outside:
//   K: acc_b = sum_c u q' over a block of 32 channels, started at -8 2^-24 sum_c q' (so it ends as
//      2^-24 sum c q'), then x += scale_b acc_b in fp32. q' is the query times a power of two that
//      puts its largest element into [2^14, 2^15): exact in half, as are the 1/16 of the
//      channels in bits 4-7, down to 2^-28 of the largest element.
//   V: the block's scale goes onto the weights (B), w = half(half(p) scale), and
//      sum_t (u - 8) w = sum_t u w - 8 sum_t w. The second sum is one more MMA per block whose A
//      is 8 2^-24 in row b: all blocks share one accumulator. Both sums see the same rounded w,
//      so the offset cancels to fp32 accuracy.
// p and w are rounded to half (2^-11 each); the reference m keeps p scale <= 2^15 and the largest
// p at 2^7 (over scales above 1) or more when it was set, so weights down to 2^-21 of the largest
// stay normal halves, and below that the error is at most 2^-25 / 2^7 of it.
// Instead of the 8 conversions and 8 products a word of codes would cost, it costs 5 integer
// operations; per 16 rows x 128 channels about 190 instructions against the 2368 bytes read.
template <int D, int G>
struct PageWarp<bf16, D, G> {
  using P = PageLayout<D>;
  static constexpr int NB = P::nb;
  uint32_t qb[2 * NB][2];      // B of S^T: [2 b + i], k slots (8 t + 2 i, + 4) and (8 t + 2 i + 1, + 5)
  float c0[NB], c1[NB];        // -8 2^-24 sum q' of block b for the heads 2 t and 2 t + 1
  float f0, f1;                // logit (log2) per unit of the scaled accumulators
  float m0, m1, l0, l1;
  float O[NB][2][4];           // rows: channels 4 g, 4 g + 1 | 4 g + 2, 4 g + 3 of block b
  float off[4];                // row b: 8 2^-24 sum_t w of block b

  __device__ __forceinline__ void begin(const bf16* q, const float (*)[D], int lane) {
    const int g = lane >> 2, t = lane & 3;
    uint4 raw[NB];
    uint32_t top = 0;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      raw[b] = g < G ? *reinterpret_cast<const uint4*>(q + g * D + b * 32 + t * 8) : make_uint4(0, 0, 0, 0);
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(raw[b].x & 0x7fff7fffu, raw[b].y & 0x7fff7fffu),
                                   __vmaxu2(raw[b].z & 0x7fff7fffu, raw[b].w & 0x7fff7fffu)));
    }
    top = max(top & 0xffffu, top >> 16);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = top == 0u ? 0 : max(-102, min(126, 14 + 127 - (int)(top >> 7)));
    const float up = __uint_as_float((uint32_t)(127 + e) << 23);
    const float f = __uint_as_float((uint32_t)(127 + 24 - e) << 23) * (kLog2e / sqrtf((float)D));
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float x[8] = {bf16_lo(raw[b].x), bf16_hi(raw[b].x), bf16_lo(raw[b].y), bf16_hi(raw[b].y),
                    bf16_lo(raw[b].z), bf16_hi(raw[b].z), bf16_lo(raw[b].w), bf16_hi(raw[b].w)};
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float w = i & 1 ? up * 0.0625f : up;
        const __half2 h = __floats2half2_rn(x[i] * w, x[i + 4] * w);
        qb[2 * b + i / 2][i & 1] = *reinterpret_cast<const uint32_t*>(&h);
        const float2 back = __half22float2(h);
        sum += (back.x + back.y) * (i & 1 ? 16.f : 1.f);
      }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      sum *= -8.f / 16777216.f;
      c0[b] = __shfl_sync(0xffffffffu, sum, t * 8);
      c1[b] = __shfl_sync(0xffffffffu, sum, t * 8 + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) O[b][0][i] = O[b][1][i] = 0.f;
    }
    f0 = __shfl_sync(0xffffffffu, f, t * 8);
    f1 = __shfl_sync(0xffffffffu, f, t * 8 + 4);
    m0 = m1 = -INFINITY;
    l0 = l1 = 0.f;
    off[0] = off[1] = off[2] = off[3] = 0.f;
  }

  __device__ __forceinline__ void take(unsigned char* pg, int nval, int lane) {
    constexpr uint32_t LO = 0x000f000fu, HI = 0x00f000f0u;
    const int g = lane >> 2, t = lane & 3;
    if (nval < kPageRows) {
      // the page's other rows may hold anything: their weights are 0, so no scale may be NaN
      if (lane >= nval)
#pragma unroll
        for (int b = 0; b < NB; ++b) *reinterpret_cast<uint16_t*>(pg + P::v_scale(b, lane)) = 0;
      fence_proxy_async_smem();      // the stage's next copy comes after these stores
      __syncwarp();
    }
    float x[2][4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = i * 16 + g;
      __half2 sa[NB / 2], sb[NB / 2];            // K scales of rows r and r + 8
#pragma unroll
      for (int b = 0; b < NB / 2; ++b) {
        sa[b] = *reinterpret_cast<const __half2*>(pg + P::k_scale(2 * b, r));
        sb[b] = *reinterpret_cast<const __half2*>(pg + P::k_scale(2 * b, r + 8));
      }
      float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t wa = *reinterpret_cast<const uint32_t*>(pg + P::k_code(b, r) + t * 4);
        const uint32_t wb = *reinterpret_cast<const uint32_t*>(pg + P::k_code(b, r + 8) + t * 4);
        float a[4];
        mma_f16_16816(a, wa & LO, wb & LO, wa & HI, wb & HI, qb[2 * b][0], qb[2 * b][1], c0[b],
                      c1[b], c0[b], c1[b]);
        const uint32_t ua = wa >> 8, ub = wb >> 8;
        mma_f16_16816(a, ua & LO, ub & LO, ua & HI, ub & HI, qb[2 * b + 1][0], qb[2 * b + 1][1],
                      a[0], a[1], a[2], a[3]);
        const float s = b & 1 ? __high2float(sa[b / 2]) : __low2float(sa[b / 2]);
        const float z = b & 1 ? __high2float(sb[b / 2]) : __low2float(sb[b / 2]);
        y[0] = fmaf(s, a[0], y[0]);
        y[1] = fmaf(s, a[1], y[1]);
        y[2] = fmaf(z, a[2], y[2]);
        y[3] = fmaf(z, a[3], y[3]);
      }
      const float na = *reinterpret_cast<const float*>(pg + P::logn(r)) * kLog2e;
      const float nb = *reinterpret_cast<const float*>(pg + P::logn(r + 8)) * kLog2e;
      x[i][0] = fmaf(y[0], f0, na);
      x[i][1] = fmaf(y[1], f1, na);
      x[i][2] = fmaf(y[2], f0, nb);
      x[i][3] = fmaf(y[3], f1, nb);
      if (nval < kPageRows) {
        if (r >= nval) x[i][0] = x[i][1] = -INFINITY;
        if (r + 8 >= nval) x[i][2] = x[i][3] = -INFINITY;
      }
    }
    // 2^ev > every V scale of the page (at least 1): p 2^ev stays below 2^15
    uint32_t smax;
    if constexpr (NB == 4) {
      const uint2 w = *reinterpret_cast<const uint2*>(pg + P::kVs + lane * 8);
      smax = __vmaxu2(w.x, w.y);
    } else {
      smax = *reinterpret_cast<const uint32_t*>(pg + P::kVs + lane * 4);
    }
    smax = __reduce_max_sync(0xffffffffu, max(smax & 0xffffu, smax >> 16));
    const float ev = (float)max(0, (int)(smax >> 10) - 14);
    const bool poison = smax > 0x7c00u;          // a block that reads as NaN
    // The reference of a column moves only when a weight would pass 2^15, to where the largest is
    // 2^7: after the first pages that is rare, and so are the maxima over the rows (the 8 lanes
    // sharing t) and the rescale.
    const float lim0 = m0 + (15.f - ev), lim1 = m1 + (15.f - ev);
    const bool up = fmaxf(fmaxf(x[0][0], x[0][2]), fmaxf(x[1][0], x[1][2])) > lim0 ||
                    fmaxf(fmaxf(x[0][1], x[0][3]), fmaxf(x[1][1], x[1][3])) > lim1;
    if (__any_sync(0xffffffffu, up)) {
      float h0 = fmaxf(fmaxf(x[0][0], x[0][2]), fmaxf(x[1][0], x[1][2]));
      float h1 = fmaxf(fmaxf(x[0][1], x[0][3]), fmaxf(x[1][1], x[1][3]));
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        h0 = fmaxf(h0, __shfl_xor_sync(0xffffffffu, h0, o));
        h1 = fmaxf(h1, __shfl_xor_sync(0xffffffffu, h1, o));
      }
      const float n0 = h0 > lim0 ? h0 + (ev - 7.f) : m0, n1 = h1 > lim1 ? h1 + (ev - 7.f) : m1;
      // factors of the old reference (0 when there was none: l and O are still 0)
      const float e0 = n0 == m0 ? 1.f : ex2_ftz(m0 - n0), e1 = n1 == m1 ? 1.f : ex2_ftz(m1 - n1);
      l0 *= e0;
      l1 *= e1;
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          O[b][j][0] *= e0; O[b][j][1] *= e1; O[b][j][2] *= e0; O[b][j][3] *= e1;
        }
      off[0] *= e0; off[1] *= e1; off[2] *= e0; off[3] *= e1;
      m0 = n0;
      m1 = n1;
    }
    const float b0 = m0 == -INFINITY ? 0.f : m0, b1 = m1 == -INFINITY ? 0.f : m1;
    __half2 pb[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float p0 = ex2_ftz(x[i][0] - b0), p1 = ex2_ftz(x[i][1] - b1);
      const float p2 = ex2_ftz(x[i][2] - b0), p3 = ex2_ftz(x[i][3] - b1);
      l0 += p0 + p2;
      l1 += p1 + p3;
      const __half2 u = __floats2half2_rn(p0, p1), v = __floats2half2_rn(p2, p3);
      const uint32_t ut = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&u));
      const uint32_t vt = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&v));
      pb[i][0] = *reinterpret_cast<const __half2*>(&ut);
      pb[i][1] = *reinterpret_cast<const __half2*>(&vt);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int r = i * 16 + 2 * t;
        const __half2 wu = __hmul2(pb[i][0], *reinterpret_cast<const __half2*>(pg + P::v_scale(b, r)));
        const __half2 wv = __hmul2(pb[i][1], *reinterpret_cast<const __half2*>(pg + P::v_scale(b, r + 8)));
        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(&wu);
        const uint32_t w1 = *reinterpret_cast<const uint32_t*>(&wv);
        const uint32_t va = *reinterpret_cast<const uint32_t*>(pg + P::v_piece(b, r, g));
        const uint32_t vb = *reinterpret_cast<const uint32_t*>(pg + P::v_piece(b, r + 8, g));
        float(&X)[4] = O[b][0];
        mma_f16_16816(X, va & LO, va & HI, vb & LO, vb & HI, w0, w1, X[0], X[1], X[2], X[3]);
        const uint32_t ua = va >> 8, ub = vb >> 8;
        float(&Y)[4] = O[b][1];
        mma_f16_16816(Y, ua & LO, ua & HI, ub & LO, ub & HI, w0, w1, Y[0], Y[1], Y[2], Y[3]);
        uint32_t z0 = w0, z1 = w1;
        if (poison) {       // 0 x NaN would reach the other blocks' rows; X and Y have it already
          z0 &= __heq2_mask(wu, wu);
          z1 &= __heq2_mask(wv, wv);
        }
        const uint32_t one = g == b ? 0x00080008u : 0u;
        mma_f16_16816(off, one, 0u, one, 0u, z0, z1, off[0], off[1], off[2], off[3]);
      }
  }

  __device__ __forceinline__ void end(float* sa, float* sm, float* sl, int lane) {
    const int g = lane >> 2, t = lane & 3;
    constexpr float kUp = 16777216.f;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float z0 = __shfl_sync(0xffffffffu, off[0], b * 4 + t) * kUp;
      const float z1 = __shfl_sync(0xffffffffu, off[1], b * 4 + t) * kUp;
      const float(&X)[4] = O[b][0], (&Y)[4] = O[b][1];
      if (2 * t < G)
        *reinterpret_cast<float4*>(sa + 2 * t * D + b * 32 + g * 4) =
            make_float4(fmaf(X[0], kUp, -z0), fmaf(X[2], kUp / 16, -z0), fmaf(Y[0], kUp, -z0),
                        fmaf(Y[2], kUp / 16, -z0));
      if (2 * t + 1 < G)
        *reinterpret_cast<float4*>(sa + (2 * t + 1) * D + b * 32 + g * 4) =
            make_float4(fmaf(X[1], kUp, -z1), fmaf(X[3], kUp / 16, -z1), fmaf(Y[1], kUp, -z1),
                        fmaf(Y[3], kUp / 16, -z1));
    }
    if (g == 0) {
      if (2 * t < G) {
        sm[2 * t] = m0;
        sl[2 * t] = l0;
      }
      if (2 * t + 1 < G) {
        sm[2 * t + 1] = m1;
        sl[2 * t + 1] = l1;
      }
    }
  }
};

template <typename T, int D, int G>
__global__ void __launch_bounds__(kPdThreads, 2)
page_decode_kernel(const T* __restrict__ q, unsigned char* pages, const int32_t* __restrict__ table,
                   int n_pages, int max_pages, int32_t* len, const T* __restrict__ k_new,
                   const T* __restrict__ v_new, T* __restrict__ out, int units, int32_t* counters,
                   int32_t* done, float* part, int32_t* flags) {
  using P = PageLayout<D>;
  using S = PageDecodeShape<D, G>;
  constexpr int NW = kPdWarps, ST = kPdStages, RS = D + kPartPad;
  extern __shared__ __align__(128) unsigned char dsm[];
  unsigned char* ring = dsm + (threadIdx.x / 32) * ST * P::kBytes;          // this warp's stages
  float* s_acc = reinterpret_cast<float*>(dsm + S::kRing);                  // [NW][G][D]
  uint64_t* full = reinterpret_cast<uint64_t*>(dsm + S::kRing + S::kAcc) + (threadIdx.x / 32) * ST;
  __shared__ __align__(16) float qs[G][D];
  __shared__ float s_m[NW][G], s_l[NW][G], s_new[G], s_stat[G][2];
  __shared__ float s_fac[G * NW];
  __shared__ long long s_sum[NW];
  __shared__ int s_unit, s_last;
  __shared__ long long s_at;

  griddep_wait();                 // launched with programmatic stream serialisation
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool want_append = k_new != nullptr;
  const long long cap = (long long)max_pages * kPageRows;
  auto length = [&](int u) {
    const int L = len[u];
    return L < 0 || L > cap ? 0 : L;
  };
  if (lane == 0) {
    for (int s = 0; s < ST; ++s) mbar_init(&full[s], 1);
    fence_mbar_init();
  }

  // the numbering: total pages, and the unit and page this CTA starts with
  const int per = (units + kPdThreads - 1) / kPdThreads;
  const int u0 = min(units, tid * per), u1 = min(units, u0 + per);
  long long mine = 0;
  for (int u = u0; u < u1; ++u) {
    const int L = len[u];
    if ((L < 0 || L > cap) && blockIdx.x == 0) set_flag(flags, KVS_FLAG_BAD_LENGTH);
    mine += unit_span(length(u));
  }
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) s_sum[warp] = inc;
  __syncthreads();
  long long total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
  }
  // at least one page per warp of a CTA: short caches gain nothing from more partial rows
  long long chunk = (total + gridDim.x - 1) / gridDim.x;
  if (chunk < NW) chunk = NW;
  const long long f0 = blockIdx.x * chunk, f1 = min(total, f0 + chunk);
  if (f0 < f1) {
    long long at = before + inc - mine;
    if (at <= f0 && f0 < at + mine) {
      int u = u0;
      for (; at + unit_span(length(u)) <= f0; ++u) at += unit_span(length(u));
      s_unit = u;
      s_at = at;
    }
  }
  __syncthreads();

  if (f0 < f1) {
    // This warp's pages are f0 + warp, f0 + warp + NW, ... The issuing side runs ST pages ahead
    // of the consuming side, each with its own place in the numbering.
    struct Place {
      int u, L;
      long long at, end;           // the unit's pages are [at, end)
    };
    auto move_to = [&](Place& p, long long f) {
      while (f >= p.end) {
        ++p.u;
        p.L = length(p.u);
        p.at = p.end;
        p.end = p.at + unit_span(p.L);
      }
    };
    Place ip{s_unit, length(s_unit), s_at, 0};
    ip.end = ip.at + unit_span(ip.L);
    long long fi = f0 + warp;      // next page to issue
    uint32_t loaded = 0;           // bit s: stage s holds (or is getting) a page
    auto issue = [&](int s) {
      loaded &= ~(1u << s);
      if (fi < f1) {
        move_to(ip, fi);
        const long long j = fi - ip.at;
        if (j * kPageRows < ip.L) {
          const int id = table[(size_t)ip.u * max_pages + j];
          if (id >= 0 && id < n_pages) {
            loaded |= 1u << s;
            if (lane == 0) {
              mbar_arrive_expect_tx(&full[s], P::kBytes);
              bulk_load(ring + s * P::kBytes, pages + (size_t)id * P::kBytes, P::kBytes, &full[s]);
            }
          } else if (lane == 0) {
            set_flag(flags, KVS_FLAG_BAD_PAGE);
          }
        }
      }
      fi += NW;
    };
    for (int s = 0; s < ST; ++s) issue(s);

    const float qscale = kLog2e / sqrtf((float)D);
    Place cp{s_unit, length(s_unit), s_at, 0};
    cp.end = cp.at + unit_span(cp.L);
    long long fc = f0 + warp;      // next page to consume
    int stage = 0;
    uint32_t phase = 0;            // bit s: parity of stage s
    for (long long seg = f0; seg < f1;) {
      move_to(cp, seg);
      const int u = cp.u, L = cp.L;
      const long long seg_end = min(f1, cp.end);
      for (int i = tid; i < G * D; i += kPdThreads)
        qs[i / D][i % D] = to_f32(q[(size_t)u * G * D + i]) * qscale;
      __syncthreads();

      PageWarp<T, D, G> pw;
      pw.begin(q + (size_t)u * G * D, qs, lane);
      for (; fc < seg_end; fc += NW) {
        const int nval = (int)min((long long)kPageRows, L - (fc - cp.at) * kPageRows);
        if (loaded >> stage & 1u) {
          if (!__all_sync(0xffffffffu, mbar_wait(&full[stage], phase >> stage & 1u))) {
            // give up: give every copy in flight one more bound, then take no further page
            set_flag(flags, KVS_FLAG_TIMEOUT);
            for (int s = 0; s < ST; ++s)
              if (loaded >> s & 1u) mbar_wait(&full[s], phase >> s & 1u);
            loaded = 0;
            fi = f1;
            continue;
          }
          phase ^= 1u << stage;
          pw.take(ring + stage * P::kBytes, nval, lane);
          __syncwarp();
        }
        issue(stage);
        stage = stage + 1 == ST ? 0 : stage + 1;
      }
      pw.end(s_acc + warp * G * D, s_m[warp], s_l[warp], lane);

      // ---- the end of the unit in this CTA ----
      const long long lp = L / kPageRows;            // the page a new row goes to
      int new_id = -1;
      if (want_append && len[u] == L && lp < max_pages) new_id = table[(size_t)u * max_pages + lp];
      const bool fits = new_id >= 0 && new_id < n_pages;
      if (fits)
        for (int g = warp; g < G; g += NW) {
          float sp = 0.f;
          for (int c = lane; c < D; c += 32) sp = fmaf(qs[g][c], to_f32(k_new[(size_t)u * D + c]), sp);
          sp = warp_sum(sp);
          if (lane == 0) s_new[g] = sp;
        }
      __syncthreads();
      const long long first = cp.at / chunk, last = (cp.end - 1) / chunk;
      const int nsplit = (int)(last - first) + 1;
      bool finish = true;
      if (nsplit > 1) {
        // slot 1 of the CTA the unit begins in, slot 0 of the others
        float* row0 = part + ((size_t)blockIdx.x * 2 + (blockIdx.x == first ? 1 : 0)) * G * RS;
        for (int i = tid; i < G * D; i += kPdThreads) {
          const int g = i / D, c = i % D;
          float M = -INFINITY, A = 0.f, Ls = 0.f;
          for (int w = 0; w < NW; ++w) M = fmaxf(M, s_m[w][g]);
          for (int w = 0; w < NW; ++w) {
            const float f = part_weight(s_m[w][g], s_l[w][g], M);
            A = fmaf(s_acc[(w * G + g) * D + c], f, A);
            Ls = fmaf(s_l[w][g], f, Ls);
          }
          row0[g * RS + c] = A;
          if (c == 0) {
            row0[g * RS + D] = M;
            row0[g * RS + D + 1] = Ls;
          }
        }
        __syncthreads();
        if (tid == 0) s_last = atom_add_acq_rel_gpu(&counters[u], 1) == nsplit - 1;
        __syncthreads();
        finish = s_last != 0;
      }
      if (finish) {
        // Sum the partials (the splits' rows in the workspace, or the warps' in shared memory):
        // four columns a thread, the partials dealt out over NGRP threads for each four. The
        // workspace rows are loaded in batches ahead of the factors, one round trip a batch.
        constexpr int NU = S::kUnits, NGRP = S::kGroups;
        constexpr int kBatch = 8;
        const int grp = tid / NU, unit = tid % NU, g = unit * 4 / D, c = unit * 4 % D;
        const int np = nsplit > 1 ? nsplit : NW;
        auto row_of = [&](int s) {
          return part + ((size_t)(first + s) * 2 + (s == 0 ? 1 : 0)) * G * RS;
        };
        float4 v[kBatch];
        if (nsplit > 1) {
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            if (grp + i * NGRP < np)
              v[i] = __ldcg(reinterpret_cast<const float4*>(row_of(grp + i * NGRP) + g * RS + c));
        }
        float* fac = nsplit > 1 ? s_acc : s_fac;     // [G][np]
        for (int gg = warp; gg < G; gg += NW) {
          const float sn = fits ? s_new[gg] : -INFINITY;
          constexpr int kMaxPer = (kPageDecodeCtas + 31) / 32;
          float ms[kMaxPer], ls[kMaxPer], M = sn;
#pragma unroll
          for (int i = 0; i < kMaxPer; ++i) {
            const int s = lane + i * 32;
            ms[i] = -INFINITY;
            ls[i] = 0.f;
            if (s < np) {
              if (nsplit > 1) {
                const float2 ml = __ldcg(reinterpret_cast<const float2*>(row_of(s) + gg * RS + D));
                ms[i] = ml.x;
                ls[i] = ml.y;
              } else {
                ms[i] = s_m[s][gg];
                ls[i] = s_l[s][gg];
              }
            }
          }
#pragma unroll
          for (int i = 0; i < kMaxPer; ++i) M = fmaxf(M, ms[i]);
          M = warp_max(M);
          float Ls = 0.f;
#pragma unroll
          for (int i = 0; i < kMaxPer; ++i) {
            const int s = lane + i * 32;
            const float f = part_weight(ms[i], ls[i], M);
            Ls = fmaf(ls[i], f, Ls);
            if (s < np) fac[gg * np + s] = f;
          }
          Ls = warp_sum(Ls);
          if (sn > -INFINITY) Ls += exp2f(sn - M);
          if (lane == 0) {
            s_stat[gg][0] = M;
            s_stat[gg][1] = Ls;
          }
        }
        __syncthreads();
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s0 = grp; s0 < np; s0 += kBatch * NGRP) {
          if (nsplit > 1) {
            if (s0 != grp) {
#pragma unroll
              for (int i = 0; i < kBatch; ++i)
                if (s0 + i * NGRP < np)
                  v[i] = __ldcg(reinterpret_cast<const float4*>(row_of(s0 + i * NGRP) + g * RS + c));
            }
          } else {
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
              if (s0 + i * NGRP < np)
                v[i] = *reinterpret_cast<const float4*>(s_acc + ((s0 + i * NGRP) * G + g) * D + c);
          }
#pragma unroll
          for (int i = 0; i < kBatch; ++i)
            if (s0 + i * NGRP < np) {
              const float f = fac[g * np + s0 + i * NGRP];
              A.x = fmaf(v[i].x, f, A.x);
              A.y = fmaf(v[i].y, f, A.y);
              A.z = fmaf(v[i].z, f, A.z);
              A.w = fmaf(v[i].w, f, A.w);
            }
        }
        if constexpr (NGRP > 1) {
          __syncthreads();                           // the warps' partials have been read
          if (grp > 0) *reinterpret_cast<float4*>(s_acc + S::kFac / 4 + ((grp - 1) * NU + unit) * 4) = A;
          __syncthreads();
          if (grp == 0)
#pragma unroll
            for (int i = 0; i < NGRP - 1; ++i) {
              const float4 w = *reinterpret_cast<const float4*>(s_acc + S::kFac / 4 + (i * NU + unit) * 4);
              A.x += w.x; A.y += w.y; A.z += w.z; A.w += w.w;
            }
        }
        if (grp == 0) {
          const float M = s_stat[g][0], Ls = s_stat[g][1];
          if (fits) {
            const float f = exp2f(s_new[g] - M);
            const T* vn = v_new + (size_t)u * D + c;
            A.x = fmaf(to_f32(vn[0]), f, A.x); A.y = fmaf(to_f32(vn[1]), f, A.y);
            A.z = fmaf(to_f32(vn[2]), f, A.z); A.w = fmaf(to_f32(vn[3]), f, A.w);
          }
          T* o = out + (size_t)u * G * D + unit * 4;
          const bool none = Ls == 0.f;               // nothing attended: zeros
          store_out<T>(o, none ? 0.f : A.x / Ls);
          store_out<T>(o + 1, none ? 0.f : A.y / Ls);
          store_out<T>(o + 2, none ? 0.f : A.z / Ls);
          store_out<T>(o + 3, none ? 0.f : A.w / Ls);
        }
        if (want_append && len[u] == L) {
          if (fits) {
            if (warp < 2) {
              // warp 0 the key, warp 1 the value: 8 channels a lane
              const T* src = (warp == 0 ? k_new : v_new) + (size_t)u * D;
              float x[8];
#pragma unroll
              for (int c = 0; c < 8; ++c) x[c] = lane < D / 8 ? to_f32(src[lane * 8 + c]) : 0.f;
              uint32_t sb;
              const uint32_t w = quantise_lane<T>(x, sb);
              unsigned char* pg = pages + (size_t)new_id * P::kBytes;
              const int r = L % kPageRows, b = lane / 4, sub = lane % 4;
              if (lane < D / 8) {
                if (warp == 0) {
                  *reinterpret_cast<uint32_t*>(pg + P::k_code(b, r) + sub * 4) = w;
                  if (sub == 0) *reinterpret_cast<uint16_t*>(pg + P::k_scale(b, r)) = (uint16_t)sb;
                  if (lane == 0) *reinterpret_cast<float*>(pg + P::logn(r)) = 0.f;
                } else {
                  *reinterpret_cast<uint16_t*>(pg + P::v_piece(b, r, sub * 2)) = (uint16_t)w;
                  *reinterpret_cast<uint16_t*>(pg + P::v_piece(b, r, sub * 2 + 1)) = (uint16_t)(w >> 16);
                  if (sub == 0) *reinterpret_cast<uint16_t*>(pg + P::v_scale(b, r)) = (uint16_t)sb;
                }
              }
            }
          } else if (tid == 0) {
            set_flag(flags, KVS_FLAG_OUT_CAPACITY);
          }
        }
        if (tid == 0 && nsplit > 1) counters[u] = 0;
      }
      seg = seg_end;
      __syncthreads();            // the shared arrays are free for the next unit
    }
  }
  if (want_append) {
    // every CTA reads every length: they move on once the last CTA is through
    __syncthreads();
    if (tid == 0) s_last = atom_add_acq_rel_gpu(done, 1) == (int)gridDim.x - 1;
    __syncthreads();
    if (s_last) {
      for (int u = tid; u < units; u += kPdThreads) {
        const int L = len[u];
        if (L < 0 || L >= cap) continue;
        const int id = table[(size_t)u * max_pages + L / kPageRows];
        if (id >= 0 && id < n_pages) len[u] = L + 1;
      }
      if (tid == 0) *done = 0;
    }
  }
}

template <typename T, int D, int G>
static cudaError_t launch_t(const kvs_cache_desc& d, const void* q, const kvs_page_pool& pool,
                            int32_t* len, const void* k_new, const void* v_new, void* out,
                            char* ws, cudaStream_t st) {
  using S = PageDecodeShape<D, G>;
  auto kfn = page_decode_kernel<T, D, G>;
  if (!ensure_smem_attr((const void*)kfn, S::kSmem)) return cudaErrorInvalidValue;
  const int units = d.B * d.H_kv;
  const PageLayoutWs Ly = page_layout_ws(d);
  const cudaError_t e = launch_pdl(
      kfn, dim3(kPageDecodeCtas), dim3(kPdThreads), S::kSmem, st, (const T*)q,
      (unsigned char*)pool.pages, (const int32_t*)pool.table, pool.n_pages, pool.max_pages, len,
      (const T*)k_new, (const T*)v_new, (T*)out, units, reinterpret_cast<int32_t*>(ws + Ly.counters),
      reinterpret_cast<int32_t*>(ws + Ly.done), reinterpret_cast<float*>(ws + Ly.part),
      reinterpret_cast<int32_t*>(ws));
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_page_decode(const kvs_cache_desc& d, const void* q, const kvs_page_pool& pool,
                               int32_t* len, const void* k_new, const void* v_new, void* out,
                               char* ws, cudaStream_t st) {
  const int G = d.H_q / d.H_kv;
#define KVS_PD(TT, DD, GG) return launch_t<TT, DD, GG>(d, q, pool, len, k_new, v_new, out, ws, st)
#define KVS_PD_G(TT, DD)        \
  if (G == 1) KVS_PD(TT, DD, 1); \
  if (G == 2) KVS_PD(TT, DD, 2); \
  if (G == 4) KVS_PD(TT, DD, 4); \
  if (G == 8) KVS_PD(TT, DD, 8)
  if (d.dtype == KVS_BF16) {
    if (d.d == 128) { KVS_PD_G(bf16, 128); }
    else { KVS_PD_G(bf16, 64); }
  } else {
    if (d.d == 128) { KVS_PD_G(float, 128); }
    else { KVS_PD_G(float, 64); }
  }
#undef KVS_PD_G
#undef KVS_PD
  return cudaErrorInvalidValue;
}

}  // namespace kvs
