// GQA decode attention over the 4-bit paged cache (kvs_page_decode_attn).
//
// Attention of the KVSlimmer deep dive ("论文专题讲解：KVSlimmer：非对称 KV 合并的数学与工程",
// §数学主线三) with the log-count bias of merged rows, over rows held in pages (pages.cuh):
//   x_t = q . k_t / sqrt(d) + logn_t,  out = sum_t 2^(x_t log2 e - M) v_t / sum_t 2^(x_t log2 e - M)
//
// A page is one contiguous block, so a single bulk copy (untiled, no tensor map) brings it into
// the ring of the warp that works on it; each warp issues its own copies and needs no other
// warp until the end of a unit. Two kernels share the work on a page (PageWarp, PageRing):
//  - split kernel: lengths are ragged and known on the device only, so every CTA sums them up for
//    itself. The pages of all units (KV heads of all sequences) are numbered one unit after
//    another and dealt out in even runs, or a fixed number of CTAs goes to each unit. A unit that
//    lies in one CTA is finished there; one that spans several gets a partial row per CTA in the
//    workspace, and the last of them to arrive (a counter at the first of them) combines. No CTA
//    waits for another.
//  - cluster kernel: one thread-block cluster per unit, combined in distributed shared memory (one
//    or two units with wide tables: several, joined through the workspace).
//
// Measured on one B200 (G = 4, d = 128, bf16; device time of captured back-to-back launches over
// three caches in turn, so that pages come from L2 up to 8 x 16384 rows; bytes are 148 a row):
//   cluster   8 units x  2048 rows    6.8 us (2.4 MB: launch, three round trips and the combine)
//             8 units x 16384 rows   11.7 us, 1.7 TB/s
//             8 units x 32768 rows   17.1 us, 2.3 TB/s (80 SMs: ten CTAs are the largest cluster
//                                    of which eight fit the GPU at once)
//             1 unit x 131072 rows   13.2 us (8 clusters), 1.5 TB/s
//   split    64 units x 11K..22K     39.0 us, 4.0 TB/s = 0.61 of the measured copy peak
//           128 units x 1K..8K       29.9 us, 2.9 TB/s
// The same kernels without the arithmetic take 4.1, 5.7, 10.2 us for 8 units, 31.5 and 23.1 us: the
// split kernel is bound first by how it brings the pages in (the lengths, the numbering and the page
// numbers before the first of them; barriers of all warps at the end of every unit; the ends), and
// its bf16 instances of d = 128 spill (188 bytes a thread at G = 4).
#include <atomic>

#include "decode_common.cuh"
#include "kvs_common.cuh"
#include "kvs_kernels.h"
#include "pages.cuh"
#include "ptx.cuh"

namespace kvs {

// Split kernel: two CTAs of 8 warps an SM (128 registers a thread, 100 to 115 KB of shared memory),
// so that one streams while the other ends a unit; two stages a warp are 150 KB of copies in
// flight per SM (a prefetch of the pages after those into L2 measured 3% to 15% slower).
constexpr int kPdWarps = 8;
constexpr int kPdThreads = kPdWarps * 32;
constexpr int kPdStages = 2;
constexpr int kPdLens = kPdThreads;    // units of a CTA whose lengths it keeps in shared memory

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
// l = 0; where logits are NaN l is, which has to go through.
__device__ __forceinline__ float part_weight(float m, float l, float M) {
  return l != 0.f ? ex2_ftz(m - M) : 0.f;
}

// Log-counts are taken relative to a `base`, one of a page that the warp has met, so that neither
// logits nor differences of log-counts are lost beside ones far from zero. One further than this
// from the base moves it: the distance to those that matter then costs a logit 2^-14 at most.
constexpr float kFarLogn = 710.f;

__device__ __forceinline__ float logn_over(float ln, float base) { return (ln - base) * kLog2e; }
// Whether a log-count leaves its row out.
__device__ __forceinline__ bool logn_masked(float ln) { return ln * kLog2e == -INFINITY; }

// Partials (m relative to base b) that are joined get the highest base of those with rows that count
// as their common one B: their m become relative to it. Bases are 0 but beside log-counts far from
// zero, and a call where all are skips this.
struct CommonBase {
  float B = -INFINITY;
  __device__ __forceinline__ void see(float l, float b) {
    if (l != 0.f) B = fmaxf(B, b);
  }
  __device__ __forceinline__ float settle() {
    if (B == -INFINITY) B = 0.f;
    return B;
  }
  __device__ __forceinline__ float over(float m, float l, float b) const {
    return l != 0.f ? m + logn_over(b, B) : m;
  }
};

// Cluster kernel: one CTA of 16 warps an SM (all of its clusters have to fit at once).
constexpr int kPcWarps = 16;
constexpr int kPcStages = 2;

template <int D, int G>
struct PageClusterShape {
  static constexpr int kRing = kPcWarps * kPcStages * PageLayout<D>::kBytes;
  static constexpr int kAcc = kPcWarps * G * D * 4;   // the warps' partial outputs
  static constexpr int kSum = G * D * 4;              // their sum
  static constexpr int kSmem = kRing + kAcc + kSum + kPcWarps * kPcStages * 8;
};

// A cluster per unit, or the split kernel? The cluster's launch costs 4 to 5 us less (no numbering,
// no round trip to the workspace), but the longest unit sets its time, and the host knows only
// how many pages a unit may have. Measured (us, G = 4, d = 128, equal lengths; cluster | split):
//   8 units (C = 10)   2048 rows  6.8 | 10.9   16384 rows 11.7 | 14.0   65536 rows 26.9 | 25.5
//   32 units (C = 4)   2048 rows  7.8 | 11.6   16384 rows 20.1 | 24.7
//   64 units (C = 2)    512 rows  7.3 | 10.4    8192 rows 20.5 | 24.7
// A lone full unit of 64 C pages among empty ones takes the cluster 12 us and the split kernel 9 to
// 12; one of 128 C pages 18 us, a risk that is taken for the few units that C >= 8 means, as they are
// mostly the heads of one sequence.
constexpr int kPcMaxPages = 128;                     // of a unit in one CTA
static_assert(kPcMaxPages <= kPcWarps * 32, "a lane of the cluster kernel has one page at most");
static bool use_cluster(int C, int clusters, int max_pages) {
  return C >= 2 && max_pages <= (C >= 8 ? kPcMaxPages : kPcMaxPages / 2) * C * clusters;
}

// Clusters of a unit: one or two units with wide tables have 8 in all. A cluster has at most 16
// CTAs, and 8 clusters of 10 run side by side. Measured (us, G = 4, d = 128; several clusters | what
// it would be else): one unit with a table of 1025 pages 9.1 | 12.1 at 32768 rows, 8.1 | 6.2 at 2048;
// with 4097 pages (else the split kernel) 13.2 | 26.6 at 131072 rows, 8.1 | 9.4 at 2048; two units of
// 4097 pages 18.5 | 25.7 and 8.1 | 9.8. With 513 pages it is 7.9 | 8.2 when they are full and
// 7.6 | 5.6 at 2048 rows, and four units of 1025 pages lose (12.5 | 11.7): the workspace's round
// trip costs 1.6 us. The table's width decides, not a length: a unit's CTAs could read different
// lengths once one of them has appended.
constexpr int kPcWide = 1024;
static_assert(8 * kMaxClusterSize <= kPageDecodeCtas, "a counter for every slice");
static int clusters_of(int units, int max_pages) {
  return units <= 2 && max_pages > kPcWide ? 8 / units : 1;
}

// How many pages more than the mean the longest unit may have in a CTA for a split by units.
// Measured (us, equal lengths; by units | even runs): 16 units x 8192 rows 12.5 | 15.4, 128 x 2048
// 17.8 | 20.0, 256 x 512 11.9 | 17.1, 64 x 16384 39.0 | 38.0; on the ragged batches of 64 and 128
// units, which the rule leaves to the even runs, 45.7 | 38.3 and 37.3 | 29.2.
constexpr int kByUnit = 40;

// Places of a unit in the numbering: its pages, and some padding for the work at its end (an
// empty unit has a place, so that a CTA finishes it). Measured on the ragged batches of 64 and 128
// units: 4 places 40.4 and 31.4 us, 8: 40.0 and 30.8, 12: 39.4 and 30.1, 24: 39.5 and 30.6.
constexpr int kUnitPages = 12;
__device__ __forceinline__ int unit_span(int L) { return pages_of(L) + kUnitPages; }

__device__ __forceinline__ __half2 as_half2(uint32_t u) { return *reinterpret_cast<const __half2*>(&u); }
__device__ __forceinline__ uint32_t as_u32(__half2 h) { return *reinterpret_cast<const uint32_t*>(&h); }

// One warp's share of a unit: its softmax state over the pages it has taken. load() and prepare()
// make the unit's operands from its queries (share() and fetch() hand them from one warp to the
// others), reset() starts a unit, take() adds the first nval rows of a page, end() writes the
// partial output [G][D], (m, l) per query head (log2 domain; m is a reference, not always the
// maximum, relative to the base of the log-counts, and -inf where no row counts; -l for a base other
// than 0) and the base.

// fp32: CUDA cores, every product and sum in fp32 (two at a time where they come in pairs), so
// that it stays within an fp32 softmax attention's own error. Logits with a lane per row, values
// with a lane per channel quad. 8 units x 32768 rows (G = 4, d = 128) take 54 us, about 1000 cycles a
// page and SM, of which the arithmetic issues in about 330. The rest goes through shared memory:
// every lane reads every query element again for each page (128 loads of 16 bytes), and the weights
// travel by 128 shuffles.
template <typename T, int D, int G>
struct PageWarp {
  using P = PageLayout<D>;
  static constexpr int QL = D / 4, RPS = 32 / QL;       // lanes per row of V, rows at a time
  const float (*qs)[D];        // scaled queries, in shared memory
  float base;                  // of the log-counts; the maxima are relative to it too
  float m[G], l[G];
  float2 acc[G][2];

  const T* q;
  static constexpr int kShare = G * D * 4;
  __device__ __forceinline__ void init(__half*, int) {}
  __device__ __forceinline__ void load(const T* q_, int) { q = q_; }
  __device__ __forceinline__ void prepare(int) {}
  __device__ __forceinline__ void share(void* to, int lane) const {
    for (int i = lane; i < G * D; i += 32) reinterpret_cast<float*>(to)[i] = q[i] * (kLog2e / sqrtf((float)D));
  }
  __device__ __forceinline__ void fetch(const void* from, int) { qs = reinterpret_cast<const float(*)[D]>(from); }
  __device__ __forceinline__ void reset() {
    base = 0.f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      m[g] = -INFINITY;
      l[g] = 0.f;
      acc[g][0] = acc[g][1] = make_float2(0.f, 0.f);
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
      float2 y[G];
#pragma unroll
      for (int g = 0; g < G; ++g) y[g] = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float k[8];
        centred8(w[i], k);
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
          for (int c = 0; c < 8; c += 4) {
            const float4 v = *reinterpret_cast<const float4*>(&qs[g][b * 32 + i * 8 + c]);
            y[g] = ffma2(make_float2(v.x, v.y), make_float2(k[c], k[c + 1]), y[g]);
            y[g] = ffma2(make_float2(v.z, v.w), make_float2(k[c + 2], k[c + 3]), y[g]);
          }
      }
#pragma unroll
      for (int g = 0; g < G; ++g) x[g] = fmaf(y[g].x + y[g].y, s, x[g]);
    }
    // rows that count: one whose log-count is -inf does not, whatever it holds
    const float ln = *reinterpret_cast<const float*>(pg + P::logn(lane));
    const bool counts = lane < nval && !logn_masked(ln);
    const uint32_t live = __ballot_sync(0xffffffffu, counts);
    if (__any_sync(0xffffffffu, counts && fabsf(ln - base) > kFarLogn)) {
      const float top = redux_max(counts ? ln : -INFINITY);
      bool none = true;
#pragma unroll
      for (int g = 0; g < G; ++g) none = none && m[g] == -INFINITY;
      if (fabsf(top) < INFINITY && (top - base > kFarLogn || (none && base - top > kFarLogn))) {
#pragma unroll
        for (int g = 0; g < G; ++g) m[g] += logn_over(base, top);
        base = top;
      }
    }
    float p[G];
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float xg = counts ? x[g] + logn_over(ln, base) : -INFINITY;
      if (__any_sync(0xffffffffu, xg > m[g])) {      // a new maximum: rare after the first pages
        const float M = fmaxf(m[g], warp_max(xg));
        const float f = exp2f(m[g] - M);
        l[g] *= f;
        acc[g][0].x *= f; acc[g][0].y *= f; acc[g][1].x *= f; acc[g][1].y *= f;
        m[g] = M;
      }
      p[g] = exp2f(xg - (m[g] == -INFINITY ? 0.f : m[g]));
      l[g] += p[g];
    }
    // a pair of rows at a time: one word holds the quad's channels of both
    const int quad = lane % QL, b = quad / 8;
#pragma unroll 2
    for (int r0 = 0; r0 < nval; r0 += 2 * RPS) {
      const int r = r0 + 2 * (lane / QL);
      const uint32_t w = *reinterpret_cast<const uint32_t*>(pg + P::v_piece(b, r, quad % 8));
      float2 s = __half22float2(*reinterpret_cast<const __half2*>(pg + P::v_scale(b, r)));
      if (!(live >> r & 1u)) s.x = 0.f;              // (also what the rest of the page holds)
      if (!(live >> r & 2u)) s.y = 0.f;
      float v[8];
      centred8(w, v);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v[c] *= s.x;
        v[4 + c] *= s.y;
      }
#pragma unroll
      for (int g = 0; g < G; ++g)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float pr = __shfl_sync(0xffffffffu, p[g], r + i);
#pragma unroll
          for (int c = 0; c < 2; ++c)
            acc[g][c] = ffma2(make_float2(pr, pr), make_float2(v[4 * i + 2 * c], v[4 * i + 2 * c + 1]), acc[g][c]);
        }
    }
  }

  __device__ __forceinline__ void end(float* sa, float* sm, float* sl, float* sb, int lane) {
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float ls = warp_sum(l[g]);
      if (lane == 0) {
        sm[g] = m[g];
        sl[g] = base == 0.f ? ls : -ls;
        *sb = base;
      }
      float4 v = make_float4(acc[g][0].x, acc[g][0].y, acc[g][1].x, acc[g][1].y);
      if (RPS == 2) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, 16);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, 16);
        v.z += __shfl_xor_sync(0xffffffffu, v.z, 16);
        v.w += __shfl_xor_sync(0xffffffffu, v.w, 16);
      }
      if (lane < QL) *reinterpret_cast<float4*>(sa + g * D + lane * 4) = v;
    }
  }
};

// bf16: m16n8k16 MMAs on half operands, the rows of the page in the M (or K) dimension and the
// query heads in the N = 8 columns, as in the bf16 cache's decode (S^T = K Q^T, O^T = V^T P^T).
//
// The codes are never converted. A 4-bit code u in bits 0-3 or 4-7 of a 16-bit half IS the
// subnormal half u 2^-24 or 16 u 2^-24, which the MMA multiplies exactly (and a byte of two codes
// the sum of the two); so one AND or byte permutation makes an A register out of a word of codes.
// The offset of 8 and the factors are put right outside:
//   K: a_b = 2^-24 sum_c u q' over a block of 32 channels, x = sum_b scale_b (a_b - 8 2^-24 sum_c q').
//      q' is the query times a power of two that puts its largest element into [2^14, 2^15): exact
//      in half, as are the 1/16 of the channels in bits 4-7, down to 2^-28 of the largest
//      element. The second sum is one more MMA: A is the rows' scales (their k slots repeated),
//      B the blocks' sums of q' in three half parts (down to 2^-24, the last place of halves); it
//      starts x.
//   V: the block's scale goes onto the weights (B), w = half(half(p) scale), and
//      sum_t (u - 8) scale p = sum_t u w - 8 sum_t scale p. The second sum is one MMA for all
//      blocks, with the scales as A and the weights half(p) as B (and a row of ones, for the sum
//      of the weights); it does not see the rounding of w, which therefore counts on |u| <= 15
//      instead of |u - 8| <= 7. Of two channels in a byte one is summed alone and the other as
//      u + 16 u'; the difference is taken at the end.
// p and w are rounded to half (2^-11 each); the reference m keeps p <= 2^15 and the largest p at 2^7
// or more when it was set, so weights down to 2^-21 of the largest stay normal halves, and below
// that the error is at most 2^-25 / 2^7 of it. For w the same holds with the scales in units of
// scale_values (with scales taken as they are, those of 2^-17 lost a third of their range, and
// what a row lost of u w stayed in 8 scale p).
//
// What bounds it: 462 instructions a page (32 rows, d = 128), of which 207 on the integer pipe,
// which takes one every other cycle, and 36 MMAs of 8 cycles on the tensor pipe of the legacy
// MMAs; the two hardly overlap. About 197 cycles a page and SM, from 12 warps an SM on (20 warps
// at 96 registers gain nothing), where an SM's share of the copy peak brings a page in 203: both
// bounds at once. Converting the codes to half instead costs 8 conversions and 8 products a word
// where this takes 4 or 5 integer operations; unpacking for tcgen05 would have to write every
// unpacked register to tensor memory first. Fragments by ldmatrix instead of 27 more loads and the
// weight sums by MMA took the page from 507 to 450. The reference in two parts, the units of the V
// scales and the bases of the partials cost 0.5 us a launch, nearly all of it at the first page of a
// warp and at the end of a unit; with the scales of every page out of range 64 units take 8% (values
// of 1e-4) to 16% longer (of 30).

template <int D, int G>
struct PageWarp<bf16, D, G> {
  using P = PageLayout<D>;
  static constexpr int NB = P::nb;
  uint4 raw[NB];               // the queries as loaded: lane (g, t) has channels 8 t.. of each block
  uint32_t qb[2 * NB][2];      // B of S^T: [2 b + i], k slots (8 t + 2 i, + 4) and (8 t + 2 i + 1, + 5)
  uint32_t cb[2];              // B of the offset: -8 2^-24 sum q' of the blocks, in three half parts
  float f0, f1;                // logit (log2) per unit of the scaled accumulators
  // The reference of a column (log2) is base log2 e - c f: the base of the log-counts (0 unless they
  // are far from zero), and what the accumulators start from.
  float base, c0, c1;
  // a logit over the reference by more than this moves it: 15, -inf while there is none
  float lim0, lim1;
  float O[NB][2][4];           // sums of u w, of channels 4 g (+ 2) and of 4 g + 1 (+ 3) times 16 plus it
  float off[4];                // row b: sum_t p scale of block b; row 4: sum_t p
  // where this lane's row of `za` in take() is: 1 and an offset in the page, or 0 and an address
  uint32_t za_page, za_off;
  // V scales are taken times 2^k, k of each block's own (kNoUnit: no scale but 0 yet); see scale_values.
  // k + 32 of block b from bit kAt(b) on; bit 12 (13, 28, 29): block 0 (1, 2, 3) of some row reads as
  // NaN; bit 31: some k is not 0.
  uint32_t units;
  static constexpr int kNoUnit = 24;
  static __host__ __device__ constexpr int kAt(int b) { return (b & 1) * 6 + (b >> 1) * 16; }
  static __host__ __device__ constexpr uint32_t kNan(int b) { return 1u << (12 + (b & 1) + (b >> 1) * 16); }
  static __host__ __device__ constexpr uint32_t kAll(int k) {
    uint32_t u = k != 0 ? 1u << 31 : 0u;
    for (int b = 0; b < NB; ++b) u |= (uint32_t)(k + 32) << kAt(b);
    return u;
  }
  __device__ __forceinline__ int unit(int at) const { return (int)(units >> at & 63u) - 32; }
  static __device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }

  // `ones_`: 32 bytes of shared memory of this warp's own
  __device__ __forceinline__ void init(__half* ones_, int lane) {
    if (lane < 16) ones_[lane] = __float2half_rn(lane < 8 ? 1.f : 0.f);
    const int row = lane & 7;
    za_page = row < NB ? 1u : 0u;
    za_off = row < NB ? P::kVs + row * 64 + (lane >> 3) * 16 : smem_u32(ones_) + (row == 4 ? 0u : 16u);
  }

  __device__ __forceinline__ void load(const bf16* q, int lane) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int b = 0; b < NB; ++b)
      raw[b] = g < G ? *reinterpret_cast<const uint4*>(q + g * D + b * 32 + t * 8) : make_uint4(0, 0, 0, 0);
  }

  // The unit's operands from `raw`.
  __device__ __forceinline__ void prepare(int lane) {
    const int t = lane & 3;
    uint32_t top = 0;
#pragma unroll
    for (int b = 0; b < NB; ++b)
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(raw[b].x & 0x7fff7fffu, raw[b].y & 0x7fff7fffu),
                                   __vmaxu2(raw[b].z & 0x7fff7fffu, raw[b].w & 0x7fff7fffu)));
    top = max(top & 0xffffu, top >> 16);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
    const int e = top == 0u ? 0 : max(-102, min(126, 14 + 127 - (int)(top >> 7)));
    const float up = __uint_as_float((uint32_t)(127 + e) << 23);
    const float f = __uint_as_float((uint32_t)(127 + 24 - e) << 23) * (kLog2e / sqrtf((float)D));
    uint32_t part[NB / 2][4];                        // of blocks 2 b and 2 b + 1; the fourth is 0
#pragma unroll
    for (int b2 = 0; b2 < NB / 2; ++b2) {
      float c[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int b = 2 * b2 + k;
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
        c[k] = sum * (-8.f / 16777216.f);
      }
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const __half2 h = __floats2half2_rn(c[0], c[1]);
        part[b2][i] = *reinterpret_cast<const uint32_t*>(&h);
        const float2 back = __half22float2(h);
        c[0] -= back.x;
        c[1] -= back.y;
      }
      part[b2][3] = 0u;
    }
    // k slots: part after part, the blocks of a part in order
    if constexpr (NB == 4) {
      const uint32_t lo = t & 2 ? part[0][1] : part[0][0], hi = t & 2 ? part[1][1] : part[1][0];
      cb[0] = t & 1 ? hi : lo;
      cb[1] = t & 2 ? 0u : t & 1 ? part[1][2] : part[0][2];
    } else {
      cb[0] = t == 0 ? part[0][0] : t == 1 ? part[0][1] : t == 2 ? part[0][2] : 0u;
      cb[1] = 0u;
    }
    f0 = __shfl_sync(0xffffffffu, f, t * 8);
    f1 = __shfl_sync(0xffffffffu, f, t * 8 + 4);
  }
  // One warp prepares for the others (kShare bytes, 16-byte aligned).
  static constexpr int kShare = (NB + 1) * 512;
  __device__ __forceinline__ void share(void* to, int lane) const {
    uint4* p = reinterpret_cast<uint4*>(to) + lane;
#pragma unroll
    for (int b = 0; b < NB; ++b) p[b * 32] = make_uint4(qb[2 * b][0], qb[2 * b][1], qb[2 * b + 1][0], qb[2 * b + 1][1]);
    p[NB * 32] = make_uint4(cb[0], cb[1], __float_as_uint(f0), __float_as_uint(f1));
  }
  __device__ __forceinline__ void fetch(const void* from, int lane) {
    const uint4* p = reinterpret_cast<const uint4*>(from) + lane;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint4 v = p[b * 32];
      qb[2 * b][0] = v.x; qb[2 * b][1] = v.y; qb[2 * b + 1][0] = v.z; qb[2 * b + 1][1] = v.w;
    }
    const uint4 v = p[NB * 32];
    cb[0] = v.x; cb[1] = v.y;
    f0 = __uint_as_float(v.z); f1 = __uint_as_float(v.w);
  }
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) O[b][0][i] = O[b][1][i] = 0.f;
    base = c0 = c1 = 0.f;
    lim0 = lim1 = -INFINITY;
    off[0] = off[1] = off[2] = off[3] = 0.f;
    units = kAll(kNoUnit);
  }

  // Logits (log2) of a page's rows relative to the references: rows g, g + 8 of 16 i .., columns 2 t, 2 t + 1.
  __device__ __forceinline__ void logits(const unsigned char* pg, int lane, float (&x)[2][4]) const {
    constexpr uint32_t LO = 0x000f000fu, HI = 0x00f000f0u;
    const int g = lane >> 2, t = lane & 3;
    // the two groups of 16 rows side by side: each step's MMAs are independent of one another
    __half2 sa[2][NB / 2], sb[2][NB / 2];        // K scales of rows r and r + 8
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = i * 16 + g;
      if constexpr (NB == 4) {
        const uint2 u = *reinterpret_cast<const uint2*>(pg + P::k_scale(0, r));
        const uint2 v = *reinterpret_cast<const uint2*>(pg + P::k_scale(0, r + 8));
        sa[i][0] = as_half2(u.x); sa[i][1] = as_half2(u.y);
        sb[i][0] = as_half2(v.x); sb[i][1] = as_half2(v.y);
      } else {
        sa[i][0] = *reinterpret_cast<const __half2*>(pg + P::k_scale(0, r));
        sb[i][0] = *reinterpret_cast<const __half2*>(pg + P::k_scale(0, r + 8));
      }
      const uint32_t za = as_u32(t & 1 ? sa[i][NB / 2 - 1] : sa[i][0]);
      const uint32_t zb = as_u32(t & 1 ? sb[i][NB / 2 - 1] : sb[i][0]);
      mma_f16_16816_cols(x[i], za, zb, za, zb, cb[0], cb[1], c0, c1);
    }
    const uint32_t at = smem_u32(pg);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      uint32_t wa[2], wb[2];                       // word t of rows g, g + 8, g + 16, g + 24
      ldsm_x4(at + P::k_code(b, 0) + lane * 16, wa[0], wb[0], wa[1], wb[1]);
      float a[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        mma_f16_16816_zero(a[i], wa[i] & LO, wb[i] & LO, wa[i] & HI, wb[i] & HI, qb[2 * b][0],
                           qb[2 * b][1]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t ua = wa[i] >> 8, ub = wb[i] >> 8;
        mma_f16_16816(a[i], ua & LO, ub & LO, ua & HI, ub & HI, qb[2 * b + 1][0], qb[2 * b + 1][1]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float s = b & 1 ? __high2float(sa[i][b / 2]) : __low2float(sa[i][b / 2]);
        const float z = b & 1 ? __high2float(sb[i][b / 2]) : __low2float(sb[i][b / 2]);
        x[i][0] = fmaf(s, a[i][0], x[i][0]);
        x[i][1] = fmaf(s, a[i][1], x[i][1]);
        x[i][2] = fmaf(z, a[i][2], x[i][2]);
        x[i][3] = fmaf(z, a[i][3], x[i][3]);
      }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = i * 16 + g;
      const float na = logn_over(*reinterpret_cast<const float*>(pg + P::logn(r)), base);
      const float nb = logn_over(*reinterpret_cast<const float*>(pg + P::logn(r + 8)), base);
      x[i][0] = fmaf(x[i][0], f0, na);
      x[i][1] = fmaf(x[i][1], f1, na);
      x[i][2] = fmaf(x[i][2], f0, nb);
      x[i][3] = fmaf(x[i][3], f1, nb);
    }
  }

  __device__ __forceinline__ void take(unsigned char* pg, int nval, int lane) {
    constexpr uint32_t LO = 0x000f000fu, BOTH = 0x00ff00ffu;
    const int g = lane >> 2, t = lane & 3;
    if (nval < kPageRows) {
      // the page's other rows may hold anything: a logit of 0 - inf, and a weight of 0 for a value of 0
      if (lane >= nval) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          *reinterpret_cast<uint16_t*>(pg + P::k_scale(b, lane)) = 0;
          *reinterpret_cast<uint16_t*>(pg + P::v_scale(b, lane)) = 0;
        }
        *reinterpret_cast<float*>(pg + P::logn(lane)) = -INFINITY;
      }
      fence_proxy_async_smem();      // the stage's next copy comes after these stores
      __syncwarp();
    }
    float x[2][4];
    for (bool again = false;;) {
      logits(pg, lane, x);
      // The reference of a column moves only when a weight would pass 2^15, to where the largest is
      // 2^7: after the first pages that is rare. Scales out of range are rare too: above 1 (adding
      // 0x43ff carries a half above 1.0 into its sign bit; NaN as well), or, while a warp has met
      // small ones only, all of them.
      uint32_t odd = units;
      if constexpr (NB == 4) {
        const uint2 w = *reinterpret_cast<const uint2*>(pg + P::kVs + lane * 8);
        odd |= (w.x + 0x43ff43ffu) | (w.y + 0x43ff43ffu);
      } else {
        odd |= *reinterpret_cast<const uint32_t*>(pg + P::kVs + lane * 4) + 0x43ff43ffu;
      }
      const float h0 = max_nan(max3_nan(x[0][0], x[0][2], x[1][0]), x[1][2]);
      const float h1 = max_nan(max3_nan(x[0][1], x[0][3], x[1][1]), x[1][3]);
      const bool far = !(h0 <= lim0 && h1 <= lim1);        // (a NaN too)
      if (!again && !__any_sync(0xffffffffu, (odd & 0x80008000u) != 0u || far)) break;
      const bool move = again || __any_sync(0xffffffffu, far);
      if (move && !again && move_base(pg, lane)) {
        again = true;                                      // the logits are made anew
        continue;
      }
      if (__any_sync(0xffffffffu, (odd & 0x80008000u) != 0u)) scale_values(pg, lane);
      if (move) move_reference(pg, x, h0, h1, lane);
      break;
    }
    __half2 pb[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2 u = __floats2half2_rn(ex2_ftz(x[i][0]), ex2_ftz(x[i][1]));
      const __half2 v = __floats2half2_rn(ex2_ftz(x[i][2]), ex2_ftz(x[i][3]));
      const uint32_t ut = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&u));
      const uint32_t vt = movmatrix_trans(*reinterpret_cast<const uint32_t*>(&v));
      pb[i][0] = *reinterpret_cast<const __half2*>(&ut);
      pb[i][1] = *reinterpret_cast<const __half2*>(&vt);
    }
    // V scales of row pairs t, t + 4, t + 8, t + 12 of every block: each matrix eight times the same
    // 16 bytes. As A (`za`): row b the scales of block b, row 4 ones, so that the sums of weights
    // come with the sums of scaled weights.
    const uint32_t at = smem_u32(pg);
    uint32_t sv[NB][4], za[4];
#pragma unroll
    for (int b = 0; b < NB; ++b)
      ldsm_x4(at + P::v_scale(b, 0) + (lane >> 3) * 16, sv[b][0], sv[b][1], sv[b][2], sv[b][3]);
    ldsm_x4(at * za_page + za_off, za[0], za[1], za[2], za[3]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = i * 16 + 2 * t;
      mma_f16_16816(off, za[2 * i], 0u, za[2 * i + 1], 0u, as_u32(pb[i][0]), as_u32(pb[i][1]));
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint32_t w0 = as_u32(__hmul2(pb[i][0], as_half2(sv[b][2 * i])));
        const uint32_t w1 = as_u32(__hmul2(pb[i][1], as_half2(sv[b][2 * i + 1])));
        const uint32_t va = *reinterpret_cast<const uint32_t*>(pg + P::v_piece(b, r, g));
        const uint32_t vb = *reinterpret_cast<const uint32_t*>(pg + P::v_piece(b, r + 8, g));
        mma_f16_16816(O[b][0], va & LO, va & BOTH, vb & LO, vb & BOTH, w0, w1);
        const uint32_t ua = __byte_perm(va, 0u, 0x4341), ub = __byte_perm(vb, 0u, 0x4341);
        mma_f16_16816(O[b][1], ua & LO, ua, ub & LO, ub, w0, w1);
      }
    }
  }

  // A row whose log-count is -inf is left out whatever it holds: where keys or values read as NaN,
  // move_reference and scale_values ask for it.
  static __device__ __forceinline__ bool masked(const unsigned char* pg, int r) {
    return logn_masked(*reinterpret_cast<const float*>(pg + P::logn(r)));
  }

  // Takes the base to the page's largest log-count if that is far above it, or if it is far below
  // and no row has counted yet. The old reference, which the new logits would be lost against, is
  // left in lim (relative to the new base, so far below 0) for move_reference to join with them.
  __device__ __forceinline__ bool move_base(const unsigned char* pg, int lane) {
    const float ln = *reinterpret_cast<const float*>(pg + P::logn(lane));
    const float top = redux_max(logn_masked(ln) ? -INFINITY : ln);
    if (!(fabsf(top - base) > kFarLogn)) return false;
    if (fabsf(top) == INFINITY || (top < base && __any_sync(0xffffffffu, fmaxf(lim0, lim1) > 0.f))) return false;
    const float d = logn_over(base, top), r0 = d - c0 * f0, r1 = d - c1 * f1;
    base = top;
    // a reference that logits put so high that it is near the new base, or above it, stays
    c0 = lim0 > 0.f && r0 > -kFarLogn ? -r0 / f0 : 0.f;
    c1 = lim1 > 0.f && r1 > -kFarLogn ? -r1 / f1 : 0.f;
    if (lim0 > 0.f && r0 <= -kFarLogn) lim0 = r0;
    if (lim1 > 0.f && r1 <= -kFarLogn) lim1 = r1;
    return true;
  }

  // How far the reference of a column moves for a page whose largest logit over it is h: up to where
  // the largest weight is 2^7, if one would pass 2^15. lim < 0: there is none yet, or one left by
  // move_base.
  static __device__ __forceinline__ float move_of(float h, float lim) {
    return lim < 0.f ? fmaxf(h - 7.f, lim) : h > lim ? h - 7.f : 0.f;
  }

  static __device__ __forceinline__ float advance(float& c, float f, float u) {
    const float dc = u > -INFINITY ? __fdividef(u, f) : 0.f;
    c -= dc;
    return dc * f;
  }

  // Brings the page's V scales into range. A weight times a scale is rounded to half, which holds
  // 2^-25 to 2^16: the weights use all of that, so the scales have to stay near 1. Those of a block
  // are taken times a power of two 2^k (exactly, but for scales below 2^-14 of the largest), which
  // goes down when a larger scale comes: 0 for a largest scale in [2^-6, 1), else what brings it
  // into [1/2, 1). O and the block's row of off are in units of 2^-k. NaN scales go too: 0 x NaN
  // would reach the other blocks through the shared sum of weights; end() puts the NaN where it
  // belongs.
  __device__ __forceinline__ void scale_values(unsigned char* pg, int lane) {
    constexpr int LB = 32 / NB, NW = NB / 2;         // lanes of a block, words of a lane
    uint32_t* at = reinterpret_cast<uint32_t*>(pg + P::kVs) + lane * NW;
    uint32_t w[NW], top = 0u;
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      w[i] = at[i];
      top = __vmaxu2(top, w[i]);
    }
    top = max(top & 0xffffu, top >> 16);
    // the usual first page: 2^-6 to 1 in every lane
    if (units == kAll(kNoUnit) && __all_sync(0xffffffffu, top >= 0x2400u && top <= 0x3c00u)) {
      units = kAll(0);
      return;
    }
    // 2^ev > every scale (of the lane's)
    auto above = [](uint32_t h) {
      return (int)(__float_as_uint(__half2float(__ushort_as_half((unsigned short)h))) >> 23) - 126;
    };
    int k = unit(kAt(lane / LB));
    if (__any_sync(0xffffffffu, top > 0x7bffu || above(top) + k > 0)) {
      uint32_t bad = 0u;
      top = 0u;
#pragma unroll
      for (int i = 0; i < NW; ++i) {
        const int r = (lane % LB * NW + i) * 2;
        if (masked(pg, r)) w[i] &= 0xffff0000u;
        if (masked(pg, r + 1)) w[i] &= 0xffffu;
        const uint32_t m = __vcmpgtu2(w[i], 0x7bff7bffu);
        w[i] &= ~m;
        bad |= m;
        top = __vmaxu2(top, w[i]);
      }
      top = max(top & 0xffffu, top >> 16);
#pragma unroll
      for (int o = 1; o < LB; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      const uint32_t nan = __ballot_sync(0xffffffffu, bad != 0u);
      const int ev = above(top);
      if (ev + k > 0) k = ev >= -5 && ev <= 0 ? 0 : -ev;
      uint32_t now = 0u;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const int kb = __shfl_sync(0xffffffffu, k, b * LB);
        now |= (uint32_t)(kb + 32) << kAt(b) | (kb != 0 ? 1u << 31 : 0u) | (units & kNan(b));
        if (nan >> (b * LB) & ((1u << LB) - 1u)) now |= kNan(b);
        const float f = pow2(kb - unit(kAt(b)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          O[b][0][i] *= f;
          O[b][1][i] *= f;
        }
        if (lane >> 2 == b) {
          off[0] *= f;
          off[1] *= f;
        }
      }
      units = now;
    }
    const __half2 f = __float2half2_rn(pow2(k / 2)), h = __float2half2_rn(pow2(k - k / 2));
#pragma unroll
    for (int i = 0; i < NW; ++i) at[i] = as_u32(__hmul2(__hmul2(as_half2(w[i]), f), h));
    fence_proxy_async_smem();        // the stage's next copy comes after these stores
    __syncwarp();
  }

  // The references for a page whose logits over them are x, the largest in this lane's columns and
  // rows h0, h1 (NaN if one is). x becomes relative to the new references.
  __device__ __forceinline__ void move_reference(const unsigned char* pg, float (&x)[2][4], float h0, float h1,
                                                 int lane) {
    if (__any_sync(0xffffffffu, h0 != h0 || h1 != h1)) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; j += 2)
          if (masked(pg, i * 16 + (lane >> 2) + j * 4)) x[i][j] = x[i][j + 1] = -INFINITY;
      h0 = fmaxf(fmaxf(x[0][0], x[0][2]), fmaxf(x[1][0], x[1][2]));
      h1 = fmaxf(fmaxf(x[0][1], x[0][3]), fmaxf(x[1][1], x[1][3]));
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {               // the 8 lanes sharing t
      h0 = fmaxf(h0, __shfl_xor_sync(0xffffffffu, h0, o));
      h1 = fmaxf(h1, __shfl_xor_sync(0xffffffffu, h1, o));
    }
    // the moves as the accumulators will hold them (0 where no row counts in the column yet)
    const float u0 = advance(c0, f0, move_of(h0, lim0)), u1 = advance(c1, f1, move_of(h1, lim1));
    const float e0 = ex2_ftz((lim0 < 0.f ? lim0 : 0.f) - u0), e1 = ex2_ftz((lim1 < 0.f ? lim1 : 0.f) - u1);
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        O[b][j][0] *= e0; O[b][j][1] *= e1; O[b][j][2] *= e0; O[b][j][3] *= e1;
      }
    off[0] *= e0; off[1] *= e1; off[2] *= e0; off[3] *= e1;
    if (fmaxf(h0, lim0) > -INFINITY) lim0 = 15.f;
    if (fmaxf(h1, lim1) > -INFINITY) lim1 = 15.f;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // (a move far from 0 is rounded; a weight may not pass 2^15 for that)
        const float y = x[i][j] - (j & 1 ? u1 : u0);
        x[i][j] = y > 15.f ? 15.f : y;               // (a NaN stays)
      }
  }

  __device__ __forceinline__ void end(float* sa, float* sm, float* sl, float* sb, int lane) {
    const int g = lane >> 2, t = lane & 3;
    const float l0 = __shfl_sync(0xffffffffu, off[0], 16 + t), l1 = __shfl_sync(0xffffffffu, off[1], 16 + t);
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int k = unit(kAt(b));
      const float kUp = pow2(24 - k), kOff = pow2(3 - k);
      float z0 = __shfl_sync(0xffffffffu, off[0], b * 4 + t) * kOff;
      float z1 = __shfl_sync(0xffffffffu, off[1], b * 4 + t) * kOff;
      if (units & kNan(b)) z0 = z1 = NAN;
      const float(&X)[4] = O[b][0], (&Y)[4] = O[b][1];
      if (2 * t < G)
        *reinterpret_cast<float4*>(sa + 2 * t * D + b * 32 + g * 4) =
            make_float4(fmaf(X[0], kUp, -z0), fmaf(X[2] - X[0], kUp / 16, -z0), fmaf(Y[0], kUp, -z0),
                        fmaf(Y[2] - Y[0], kUp / 16, -z0));
      if (2 * t + 1 < G)
        *reinterpret_cast<float4*>(sa + (2 * t + 1) * D + b * 32 + g * 4) =
            make_float4(fmaf(X[1], kUp, -z1), fmaf(X[3] - X[1], kUp / 16, -z1), fmaf(Y[1], kUp, -z1),
                        fmaf(Y[3] - Y[1], kUp / 16, -z1));
    }
    if (lane == 0) *sb = base;
    if (g == 0) {
      if (2 * t < G) {
        sm[2 * t] = l0 != 0.f ? -c0 * f0 : -INFINITY;
        sl[2 * t] = base == 0.f ? l0 : -l0;
      }
      if (2 * t + 1 < G) {
        sm[2 * t + 1] = l1 != 0.f ? -c1 * f1 : -INFINITY;
        sl[2 * t + 1] = base == 0.f ? l1 : -l1;
      }
    }
  }
};

// The pages one warp works through, in its own ring of ST stages of shared memory. Page k of the
// warp is entry k mod 32 (one per lane) of list k / 32: page number << 6 | rows that count, 0 for
// nothing to read. Two lists are held, the one being worked on and the next; `fill` makes them.
template <int D, int ST>
struct PageRing {
  using P = PageLayout<D>;
  unsigned char* pages;
  unsigned char* ring;
  uint64_t* full;
  uint32_t list, next;           // the list that page k + ST is on, and the one after it
  uint32_t due[ST];              // entries of the pages from k on
  uint32_t parity[ST];           // of their stages
  int k, stage, ahead;           // the next page, its stage, the place of page k + ST - 1 in its list

  __device__ __forceinline__ void issue(int s, uint32_t e, int lane) {
    if (e != 0u && lane == 0) {
      mbar_arrive_expect_tx(&full[s], P::kBytes);
      bulk_load(ring + s * P::kBytes, pages + (size_t)(e >> 6) * P::kBytes, P::kBytes, &full[s]);
    }
  }
  // `first` is list 0. The copies of the first ST pages go out; then the caller sets `next`.
  __device__ __forceinline__ void start(unsigned char* pages_, unsigned char* ring_, uint64_t* full_,
                                        uint32_t first, int lane) {
    pages = pages_;
    ring = ring_;
    full = full_;
    list = first;
    k = stage = 0;
    ahead = ST - 1;
    if (lane == 0) {
      for (int s = 0; s < ST; ++s) mbar_init(&full[s], 1);
      fence_mbar_init();
    }
    __syncwarp();
#pragma unroll
    for (int s = 0; s < ST; ++s) {
      due[s] = __shfl_sync(0xffffffffu, list, s);
      parity[s] = 0u;
      issue(s, due[s], lane);
    }
  }
  // Hands the pages up to (not including) page `kend` to take(page in shared memory, rows).
  // False when a copy did not arrive: the warp's other copies have had their bound by then, and
  // none is issued any more.
  template <typename Fill, typename Take>
  __device__ __forceinline__ bool run(int kend, int lane, Fill&& fill, Take&& take) {
    for (; k < kend; ++k) {
      const uint32_t cur = due[0];
      if (cur != 0u) {
        if (!__all_sync(0xffffffffu, mbar_wait(full + stage, parity[0]))) {
#pragma unroll
          for (int i = 0; i < ST; ++i) {
            if (due[i] != 0u) mbar_wait(full + (stage + i) % ST, parity[i]);
            due[i] = 0u;
          }
          list = next = 0u;
          return false;
        }
        parity[0] ^= 1u;
        take(ring + stage * P::kBytes, (int)(cur & 63u));
        __syncwarp();
      }
      ahead = (ahead + 1) & 31;
      if (ahead == 0) {
        list = next;
        next = fill();
      }
      const uint32_t par = parity[0];
#pragma unroll
      for (int i = 0; i + 1 < ST; ++i) {
        due[i] = due[i + 1];
        parity[i] = parity[i + 1];
      }
      parity[ST - 1] = par;
      due[ST - 1] = __shfl_sync(0xffffffffu, list, ahead);
      issue(stage, due[ST - 1], lane);
      stage = stage + 1 == ST ? 0 : stage + 1;
    }
    return true;
  }
};

// What a decode call works on.
template <typename T>
struct PageArgs {
  const T* q;
  unsigned char* pages;
  const int32_t* table;
  int n_pages, max_pages;
  int32_t* len;
  const T* k_new;              // nullptr: nothing to append
  const T* v_new;
  T* out;
  int units;
  int32_t* counters;           // [kPageDecodeCtas]
  int32_t* done;
  float* part;
  int32_t* flags;

  __device__ __forceinline__ int legal(int L) const {
    return L < 0 || L > (long long)max_pages * kPageRows ? 0 : L;
  }
  // The page a new row of unit u goes to, -1 when it has none (or its length is out of range).
  __device__ __forceinline__ int new_page(int u, int L) const {
    if (k_new == nullptr || L < 0 || L / kPageRows >= max_pages) return -1;
    const int id = table[(size_t)u * max_pages + L / kPageRows];
    return id >= 0 && id < n_pages ? id : -1;
  }
};

// Logit (log2) of the new row for query head g of unit u; count 1, so no bias. A whole warp.
template <typename T, int D, int G>
__device__ __forceinline__ float new_logit(const PageArgs<T>& a, int u, int g, int lane) {
  float sp = 0.f;
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
    sp = fmaf(to_f32(a.q[((size_t)u * G + g) * D + c * 32 + lane]),
              to_f32(a.k_new[(size_t)u * D + c * 32 + lane]), sp);
  return warp_sum(sp) * (kLog2e / sqrtf((float)D));
}

// Four columns of an output from the sum A over a unit's rows (weights against M over the base B,
// their sum Ls) and the new row (logit sn, -inf for none).
template <typename T>
__device__ __forceinline__ void finish_columns(float4 A, float M, float Ls, float B, float sn, const T* vn, T* o) {
  if (sn > -INFINITY || sn != sn) {
    sn += logn_over(0.f, B);
    const float R = fmaxf(M, sn);
    const float fo = Ls != 0.f ? ex2_ftz(M - R) : 0.f, fn = ex2_ftz(sn - R);
    Ls = fmaf(Ls, fo, fn);
    A.x = fmaf(A.x, fo, to_f32(vn[0]) * fn);
    A.y = fmaf(A.y, fo, to_f32(vn[1]) * fn);
    A.z = fmaf(A.z, fo, to_f32(vn[2]) * fn);
    A.w = fmaf(A.w, fo, to_f32(vn[3]) * fn);
  }
  const float inv = Ls == 0.f ? 0.f : 1.f / Ls;      // 0: nothing attended, zeros
  store_out<T>(o, A.x * inv);
  store_out<T>(o + 1, A.y * inv);
  store_out<T>(o + 2, A.z * inv);
  store_out<T>(o + 3, A.w * inv);
}

// Writes the new row of unit u quantised to row L of page `id`: warp 0 the key, warp 1 the value.
template <typename T, int D>
__device__ __forceinline__ void write_new_row(const PageArgs<T>& a, int u, int L, int id, int warp, int lane) {
  using P = PageLayout<D>;
  if (warp >= 2) return;
  const T* src = (warp == 0 ? a.k_new : a.v_new) + (size_t)u * D;
  float x[8];                    // element loads: these rows need not be 16-byte aligned
#pragma unroll
  for (int c = 0; c < 8; ++c) x[c] = lane < D / 8 ? to_f32(src[lane * 8 + c]) : 0.f;
  Raw8<float> raw;
  raw.a = make_float4(x[0], x[1], x[2], x[3]);
  raw.b = make_float4(x[4], x[5], x[6], x[7]);
  uint32_t sb;
  const uint32_t w = quantise_lane<float>(raw, sb);
  if (lane >= D / 8) return;
  unsigned char* pg = a.pages + (size_t)id * P::kBytes;
  const int r = L % kPageRows, b = lane / 4, sub = lane % 4;
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

// Sum of the warps' partial outputs over their common base B, four columns from column c of query
// head g on.
template <int D, int G, int NW>
__device__ __forceinline__ float4 merge_warps(const float* s_acc, const float (*s_m)[G], const float (*s_l)[G],
                                              const float* s_b, int g, int c, float& M, float& Ls, float& B) {
  uint32_t any = 0u;
  M = -INFINITY;
  Ls = B = 0.f;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    M = fmaxf(M, s_m[w][g]);
    any |= __float_as_uint(s_l[w][g]);
  }
  float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
  auto add = [&](int w, float m) {
    const float l = fabsf(s_l[w][g]), f = part_weight(m, l, M);
    const float4 v = *reinterpret_cast<const float4*>(s_acc + (w * G + g) * D + c);
    A.x = fmaf(v.x, f, A.x); A.y = fmaf(v.y, f, A.y);
    A.z = fmaf(v.z, f, A.z); A.w = fmaf(v.w, f, A.w);
    Ls = fmaf(l, f, Ls);
  };
  if ((int)any >= 0) {
#pragma unroll
    for (int w = 0; w < NW; ++w) add(w, s_m[w][g]);
  } else {
    CommonBase cb;
    for (int w = 0; w < NW; ++w) cb.see(s_l[w][g], s_b[w]);
    B = cb.settle();
    M = -INFINITY;
    for (int w = 0; w < NW; ++w) M = fmaxf(M, cb.over(s_m[w][g], s_l[w][g], s_b[w]));
#pragma unroll 1
    for (int w = 0; w < NW; ++w) add(w, cb.over(s_m[w][g], s_l[w][g], s_b[w]));
  }
  return A;
}

template <typename T, int D, int G>
__global__ void __launch_bounds__(kPdThreads, 2)
page_decode_kernel(const PageArgs<T> a) {
  using P = PageLayout<D>;
  using S = PageDecodeShape<D, G>;
  constexpr int NW = kPdWarps, ST = kPdStages, RS = D + kPartPad;
  extern __shared__ __align__(128) unsigned char dsm[];
  float* s_acc = reinterpret_cast<float*>(dsm + S::kRing);                  // [NW][G][D]
  __shared__ __align__(16) unsigned char s_q[PageWarp<T, D, G>::kShare];    // a unit's operands
  __shared__ __align__(16) __half s_ones[NW][16];                           // bf16: PageWarp::init
  __shared__ float s_m[NW][G], s_l[NW][G], s_stat[G][3];
  __shared__ float s_b[NW];
  __shared__ float s_new[3][G];   // the new row's logits, for the units of s_split and a whole one
  __shared__ int s_len[kPdLens];  // lengths (as they are in memory) of units from the first one on
  // the unit that began in an earlier CTA (0) and the one that goes on in a later one (1): unit,
  // first CTA, CTAs, length
  __shared__ int4 s_split[2];
  __shared__ int s_last[2];

  griddep_wait();                 // launched with programmatic stream serialisation
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid < 2) s_split[tid].x = -1;

  // Every warp reads all lengths and settles for itself what this CTA does, so no barrier comes
  // before the first copies. The host keeps the total below 2^31.
  uint32_t sum = 0, most = 0;
#pragma unroll 4
  for (int u = lane; u < a.units; u += 32) {
    const int L = a.len[u];
    if (L != a.legal(L) && blockIdx.x == 0 && warp == 0) set_flag(a.flags, KVS_FLAG_BAD_LENGTH);
    sum += unit_span(a.legal(L));
    most = max(most, (uint32_t)pages_of(a.legal(L)));
  }
  const int total = (int)__reduce_add_sync(0xffffffffu, sum);
  const int longest = (int)__reduce_max_sync(0xffffffffu, most);
  // Two ways to split the pages. Even runs of the numbering: the same work for every CTA, but a
  // unit begins and ends anywhere in a CTA. Or `per_unit` CTAs for each unit, which saves the
  // boundaries (about 8 us of a launch, 40 pages of a CTA) and costs what the longest unit is
  // longer than the mean.
  const int per_unit = (int)gridDim.x / a.units;
  const bool by_unit = per_unit > 0 && (longest + per_unit - 1) / per_unit <= total / (int)gridDim.x + kByUnit;
  // at least one page per warp of a CTA: short caches gain nothing from more partial rows
  const int chunk = max(NW, (total + (int)gridDim.x - 1) / (int)gridDim.x);
  int f0, f1, part = 0, parts = 1;                     // this CTA's places
  if (by_unit) {
    const int u = blockIdx.x / per_unit;
    part = blockIdx.x % per_unit;
    const int np = u < a.units ? pages_of(a.legal(a.len[u])) : 0;
    parts = max(1, min(per_unit, np / (2 * NW)));      // two pages per warp at least
    f0 = (int)((long long)np * part / parts);
    f1 = u < a.units && part < parts ? max(f0 + 1, (int)((long long)np * (part + 1) / parts)) : f0;
  } else {
    f0 = (int)min((long long)total, (long long)blockIdx.x * chunk);
    f1 = (int)min((long long)total, (long long)f0 + chunk);
  }
  // Lengths move on when every CTA has read them, so this CTA says when it has: once the ones
  // of its own units are in shared memory, while the first pages are on their way. (A CTA with
  // more units than fit there reads on from memory, and says so at its end.)
  bool told = false;
  auto tell = [&]() {                                  // one warp
    int last = 0;
    if (lane == 0) last = atom_add_acq_rel_gpu(a.done, 1) == (int)gridDim.x - 1;
    if (!__shfl_sync(0xffffffffu, last, 0)) return;
    for (int u = lane; u < a.units; u += 32) {
      const int L = a.len[u];
      if (a.new_page(u, L) >= 0) a.len[u] = L + 1;
    }
    if (lane == 0) *a.done = 0;
  };

  if (f0 < f1) {
    struct Place {
      int u, L;
      int at, end;                 // the unit's pages are [at, end)
    };
    // The new row of a unit that is being finished: its page (-1: none) with its logits in s_new
    // after the next barrier, and its place in the cache.
    // (`len`: the unit's length as it is in memory, which may be out of range)
    auto new_row = [&](int u, int len, int slot) {
      const int id = a.k_new != nullptr ? a.new_page(u, len) : -1;
      if (id >= 0 && warp < G) {
        const float sn = new_logit<T, D, G>(a, u, warp, lane);
        if (lane == 0) s_new[slot][warp] = sn;
      }
      return id;
    };
    auto append = [&](int u, int len, int id) {
      if (id >= 0)
        write_new_row<T, D>(a, u, len, id, warp, lane);
      else if (a.k_new != nullptr && tid == 0 && a.legal(len) == len)
        set_flag(a.flags, KVS_FLAG_OUT_CAPACITY);
    };
    int u_first = 0;
    auto len_of = [&](int u) { return told ? s_len[u - u_first] : a.len[u]; };
    auto move_to = [&](Place& p, int f) {
      while (f >= p.end) {
        ++p.u;
        p.L = a.legal(len_of(p.u));
        p.at = p.end;
        p.end = p.at + unit_span(p.L);
      }
    };
    Place cp;
    if (by_unit) {
      cp.u = blockIdx.x / per_unit;
      cp.L = a.legal(a.len[cp.u]);
      cp.at = 0;
      cp.end = unit_span(cp.L);
    } else {
      int base = 0, acc = 0, w, n;                 // the 32 units that page f0 falls among
      for (;; base += 32, acc += n) {
        w = base + lane < a.units ? unit_span(a.legal(a.len[base + lane])) : 0;
        n = (int)__reduce_add_sync(0xffffffffu, (uint32_t)w);
        if (f0 < acc + n) break;
      }
      int inc = w;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += x;
      }
      const int who = __ffs(__ballot_sync(0xffffffffu, f0 < acc + inc)) - 1;
      cp.u = base + who;
      cp.L = a.legal(a.len[cp.u]);
      cp.end = acc + __shfl_sync(0xffffffffu, inc, who);
      cp.at = cp.end - unit_span(cp.L);
    }

    // a run that begins in the padding of a unit leaves that unit to others
    auto live_end = [&](const Place& p) { return p.at + max(1, pages_of(p.L)); };
    if (f0 >= live_end(cp)) {
      f0 = min(f1, cp.end);
      if (f0 < f1) move_to(cp, f0);
    }

    // This warp's pages are f0 + warp, f0 + warp + NW, ...
    Place lp = cp;                 // this lane's place in the list that comes next
    int lf = f0 + warp + NW * lane;
    auto fill = [&]() -> uint32_t {
      uint32_t e = 0;
      if (lf < f1) {
        move_to(lp, lf);
        const int n = min(kPageRows, lp.L - (lf - lp.at) * kPageRows);
        if (n > 0) {
          const int id = a.table[(size_t)lp.u * a.max_pages + (lf - lp.at)];
          if (id >= 0 && id < a.n_pages)
            e = (uint32_t)id << 6 | (uint32_t)n;
          else
            set_flag(a.flags, KVS_FLAG_BAD_PAGE);
        }
        lf += 32 * NW;
      }
      return e;
    };
    // the queries ahead of the pages: behind 150 KB of copies per SM they would come
    // microseconds later
    PageWarp<T, D, G> pw;
    pw.init(s_ones[warp], lane);
    const bool first_warp = warp == 0, last_warp = warp == NW - 1;
    if (first_warp) pw.load(a.q + (size_t)cp.u * G * D, lane);
    PageRing<D, ST> pr;
    pr.start(a.pages, dsm + warp * ST * P::kBytes,
             reinterpret_cast<uint64_t*>(dsm + S::kRing + S::kAcc) + warp * ST, fill(), lane);
    if (first_warp) {
      pw.prepare(lane);
      pw.share(s_q, lane);
    }
    u_first = cp.u;
    const int n = by_unit ? 1 : (f1 - cp.at) / kUnitPages + 1;     // no more units than that begin before f1
    const bool keeps = a.k_new != nullptr && n <= kPdLens;
    if (keeps && tid < n && cp.u + tid < a.units) s_len[tid] = a.len[cp.u + tid];
    __syncthreads();
    told = keeps;
    if (told && last_warp) tell();
    pr.next = fill();

    for (int seg = f0; seg < f1;) {
      move_to(cp, seg);
      const int u = cp.u;
      const int seg_end = min(f1, cp.end);
      const int first = by_unit ? (int)blockIdx.x - part : cp.at / chunk;
      const int nsplit = by_unit ? parts : (live_end(cp) - 1) / chunk - first + 1;
      const int slot = (int)blockIdx.x == first ? 1 : 0;
      pw.fetch(s_q, lane);
      pw.reset();
      if (a.k_new != nullptr && nsplit == 1 && tid < 2)    // wanted at the unit's end
        prefetch_l2((tid == 0 ? a.k_new : a.v_new) + (size_t)u * D);
      static_assert(G <= NW, "a warp per query head");
      if (!pr.run((seg_end - f0 - warp + NW - 1) / NW, lane, fill,
                  [&](unsigned char* pg, int n) { pw.take(pg, n, lane); })) {
        set_flag(a.flags, KVS_FLAG_TIMEOUT);
        lf = f1;
      }
      const bool more = seg_end < f1;
      if (more && first_warp) pw.load(a.q + (size_t)(u + 1) * G * D, lane);
      if (more || seg != f0) __syncthreads();      // the last unit's partials, this one's operands: read
      const int len = len_of(u);
      const int id = nsplit == 1 ? new_row(u, len, 2) : -1;
      pw.end(s_acc + warp * G * D, s_m[warp], s_l[warp], s_b + warp, lane);
      if (more && first_warp) {
        pw.prepare(lane);
        pw.share(s_q, lane);
      }
      __syncthreads();
      if (tid < G * D / 4) {
        const int g = tid * 4 / D, c = tid * 4 % D;
        float M, Ls, B;
        const float4 A = merge_warps<D, G, NW>(s_acc, s_m, s_l, s_b, g, c, M, Ls, B);
        if (nsplit == 1) {
          finish_columns<T>(A, M, Ls, B, id >= 0 ? s_new[2][g] : -INFINITY, a.v_new + (size_t)u * D + c,
                            a.out + (size_t)u * G * D + tid * 4);
        } else {
          // a row of the workspace; who finishes the unit is settled after this CTA's last page
          float* row = a.part + ((size_t)blockIdx.x * 2 + slot) * G * RS + g * RS;
          *reinterpret_cast<float4*>(row + c) = A;
          if (c == 0) *reinterpret_cast<float4*>(row + D) = make_float4(M, Ls, B, 0.f);
        }
      }
      if (nsplit == 1)
        append(u, len, id);
      else if (tid == 0)
        s_split[slot] = make_int4(u, first, nsplit, len);
      seg = seg_end;
    }

    // Who finishes the units split over several CTAs: the last of them to arrive here. (That
    // costs a round trip to L2, so it waits until this CTA's pages are through.)
    __syncthreads();
    if (tid < 2) {
      const int4 sp = s_split[tid];
      s_last[tid] = sp.x >= 0 && atom_add_acq_rel_gpu(&a.counters[sp.y], 1) == sp.z - 1;
    }
    int new_id[2];                                 // (loads that overlap the arrivals')
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int4 sp = s_split[i];
      new_id[i] = sp.x >= 0 ? new_row(sp.x, sp.w, i) : -1;
    }
    __syncthreads();
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
      if (!s_last[i]) continue;
      // Sum the splits' rows: four columns a thread, the splits dealt out over NGRP threads for
      // each four, loads in batches.
      constexpr int NU = S::kUnits, NGRP = S::kGroups, kBatch = 4, kFew = 6;
      const int4 sp = s_split[i];
      const int u = sp.x, np = sp.z;
      const int grp = tid / NU, unit = tid % NU, g = unit * 4 / D, c = unit * 4 % D;
      // slot 1 of the CTA the unit begins in, slot 0 of the others
      const float* rows = a.part + (size_t)sp.y * 2 * G * RS;
      auto row_of = [&](int s) { return rows + (2 * s + (s == 0 ? 1 : 0)) * G * RS; };
      const int id = i == 0 ? new_id[0] : new_id[1];
      if (np <= kFew) {
        // few splits (the usual case): every thread weighs them for itself, one round trip
        if (tid < NU) {
          const int g = tid * 4 / D, c = tid * 4 % D;
          float4 ml[kFew], v[kFew];
          uint32_t any = 0u;
#pragma unroll
          for (int s = 0; s < kFew; ++s) {
            ml[s] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
            v[s] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (s < np) {
              ml[s] = __ldcg(reinterpret_cast<const float4*>(row_of(s) + g * RS + D));
              v[s] = __ldcg(reinterpret_cast<const float4*>(row_of(s) + g * RS + c));
            }
          }
          float M = -INFINITY, Ls = 0.f, B = 0.f;
#pragma unroll
          for (int s = 0; s < kFew; ++s) any |= __float_as_uint(ml[s].z);
          if (any != 0u) {
            CommonBase cb;
#pragma unroll
            for (int s = 0; s < kFew; ++s) cb.see(ml[s].y, ml[s].z);
            B = cb.settle();
#pragma unroll
            for (int s = 0; s < kFew; ++s) ml[s].x = cb.over(ml[s].x, ml[s].y, ml[s].z);
          }
#pragma unroll
          for (int s = 0; s < kFew; ++s) M = fmaxf(M, ml[s].x);
          float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int s = 0; s < kFew; ++s) {
            const float f = part_weight(ml[s].x, ml[s].y, M);
            Ls = fmaf(ml[s].y, f, Ls);
            A.x = fmaf(v[s].x, f, A.x); A.y = fmaf(v[s].y, f, A.y);
            A.z = fmaf(v[s].z, f, A.z); A.w = fmaf(v[s].w, f, A.w);
          }
          finish_columns<T>(A, M, Ls, B, id >= 0 ? s_new[i][g] : -INFINITY, a.v_new + (size_t)u * D + c,
                            a.out + (size_t)u * G * D + tid * 4);
        }
        append(u, sp.w, id);
        if (tid == 0) a.counters[sp.y] = 0;
        continue;
      }
      float* fac = s_acc;                          // [G][np]
      float4 v[kBatch];
      auto load_batch = [&](int s0) {
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (s0 + j * NGRP < np)
            v[j] = __ldcg(reinterpret_cast<const float4*>(row_of(s0 + j * NGRP) + g * RS + c));
      };
      load_batch(grp);                             // with the factors' loads: one round trip for both
      if (warp < G) {
        constexpr int kPer = (kPageDecodeCtas + 31) / 32;
        float4 ml[kPer];
        float M = -INFINITY, Ls = 0.f, B = 0.f;
        uint32_t any = 0u;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int s = lane + j * 32;
          ml[j] = make_float4(-INFINITY, 0.f, 0.f, 0.f);
          if (j * 32 < np && s < np)
            ml[j] = __ldcg(reinterpret_cast<const float4*>(row_of(s) + warp * RS + D));
          any |= __float_as_uint(ml[j].z);
        }
        if (__any_sync(0xffffffffu, any != 0u)) {
          CommonBase cb;
#pragma unroll
          for (int j = 0; j < kPer; ++j) cb.see(ml[j].y, ml[j].z);
          cb.B = warp_max(cb.B);
          B = cb.settle();
#pragma unroll
          for (int j = 0; j < kPer; ++j) ml[j].x = cb.over(ml[j].x, ml[j].y, ml[j].z);
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) M = fmaxf(M, ml[j].x);
        M = warp_max(M);
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int s = lane + j * 32;
          const float f = part_weight(ml[j].x, ml[j].y, M);
          Ls = fmaf(ml[j].y, f, Ls);
          if (s < np) fac[warp * np + s] = f;
        }
        Ls = warp_sum(Ls);
        if (lane == 0) {
          s_stat[warp][0] = M;
          s_stat[warp][1] = Ls;
          s_stat[warp][2] = B;
        }
      }
      __syncthreads();
      float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int s0 = grp; s0 < np; s0 += kBatch * NGRP) {
        if (s0 != grp) load_batch(s0);
#pragma unroll
        for (int j = 0; j < kBatch; ++j)
          if (s0 + j * NGRP < np) {
            const float f = fac[g * np + s0 + j * NGRP];
            A.x = fmaf(v[j].x, f, A.x); A.y = fmaf(v[j].y, f, A.y);
            A.z = fmaf(v[j].z, f, A.z); A.w = fmaf(v[j].w, f, A.w);
          }
      }
      if constexpr (NGRP > 1) {
        float* sums = s_acc + S::kFac / 4;
        if (grp > 0) *reinterpret_cast<float4*>(sums + ((grp - 1) * NU + unit) * 4) = A;
        __syncthreads();
        if (grp == 0)
#pragma unroll
          for (int j = 0; j < NGRP - 1; ++j) {
            const float4 w = *reinterpret_cast<const float4*>(sums + (j * NU + unit) * 4);
            A.x += w.x; A.y += w.y; A.z += w.z; A.w += w.w;
          }
      }
      if (grp == 0) {
        finish_columns<T>(A, s_stat[g][0], s_stat[g][1], s_stat[g][2], id >= 0 ? s_new[i][g] : -INFINITY,
                          a.v_new + (size_t)u * D + c, a.out + (size_t)u * G * D + unit * 4);
      }
      append(u, sp.w, id);
      if (tid == 0) a.counters[sp.y] = 0;
      __syncthreads();            // the shared arrays are free for the other unit
    }
  }
  if (a.k_new != nullptr && !told) {
    __syncthreads();
    if (warp == 0) tell();
  }
}

// Weighs the partials (m over base b, l, A) of the 16 lanes of a half-warp and sums them up in every
// lane (A, l, the common base b); returns the reference.
__device__ __forceinline__ float half_warp_sum(float4& A, float m, float& l, float& b) {
  if (__any_sync(0xffffffffu, b != 0.f)) {
    CommonBase cb;
    cb.see(l, b);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) cb.B = fmaxf(cb.B, __shfl_xor_sync(0xffffffffu, cb.B, o));
    cb.settle();
    m = cb.over(m, l, b);
    b = cb.B;
  }
  float M = m;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float f = part_weight(m, l, M);
  l *= f;
  A.x *= f; A.y *= f; A.z *= f; A.w *= f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    l += __shfl_xor_sync(0xffffffffu, l, o);
    A.x += __shfl_xor_sync(0xffffffffu, A.x, o);
    A.y += __shfl_xor_sync(0xffffffffu, A.y, o);
    A.z += __shfl_xor_sync(0xffffffffu, A.z, o);
    A.w += __shfl_xor_sync(0xffffffffu, A.w, o);
  }
  return M;
}

// The same with one thread-block cluster per unit, for few units: the CTAs of the cluster take
// the unit's pages in turn, and combine through distributed shared memory. The page numbers do
// not depend on the other units' lengths, so they are loaded together with the length, and the
// combine needs neither the workspace nor a round trip to it.
//
// One or two units with wide tables have several clusters each (gridDim.y = units x `clusters`,
// clusters_of), which take the unit's pages in turn. Each CTA leaves its slice of its cluster's
// output in the workspace, and of the CTAs with the same slice the last to arrive (a counter per
// unit and slice; it is zero again then) joins them, in the clusters' order.
template <typename T, int D, int G>
__global__ void __launch_bounds__(kPcWarps * 32, 1)
page_decode_cluster_kernel(const PageArgs<T> a, int clusters) {
  using P = PageLayout<D>;
  using S = PageClusterShape<D, G>;
  constexpr int NW = kPcWarps, ST = kPcStages;
  extern __shared__ __align__(128) unsigned char dsm[];
  float* s_acc = reinterpret_cast<float*>(dsm + S::kRing);                  // [NW][G][D]
  float* s_sum = reinterpret_cast<float*>(dsm + S::kRing + S::kAcc);        // [G][D], read by peers
  __shared__ __align__(16) float s_q[sizeof(T) == 4 ? G * D : 4];           // fp32: PageWarp::share
  __shared__ __align__(16) __half s_ones[NW][16];                           // bf16: PageWarp::init
  __shared__ float s_m[NW][G], s_l[NW][G], s_new[G];
  __shared__ float s_b[NW];
  __shared__ __align__(16) float s_ml[G][4];                                // (m, l, base), read by peers

  griddep_wait();                 // launched with programmatic stream serialisation
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = gridDim.x, rank = (int)cluster_ctarank();
  const int u = blockIdx.y / clusters, part = blockIdx.y % clusters;
  const int len = a.len[u], L = a.legal(len);
  const int first = part * C + rank, step = C * clusters;
  const long long j = first + (long long)step * (warp + NW * lane);     // this lane's page
  const int id = j < a.max_pages ? a.table[(size_t)u * a.max_pages + j] : -1;
  PageWarp<T, D, G> pw;
  pw.init(s_ones[warp], lane);
  pw.load(a.q + (size_t)u * G * D, lane);
  if (L != len && part == 0 && rank == 0 && tid == 0) set_flag(a.flags, KVS_FLAG_BAD_LENGTH);
  auto entry = [&]() -> uint32_t {
    const int n = (int)min((long long)kPageRows, L - j * kPageRows);
    if (n <= 0) return 0u;
    if (id >= 0 && id < a.n_pages) return (uint32_t)id << 6 | (uint32_t)n;
    set_flag(a.flags, KVS_FLAG_BAD_PAGE);
    return 0u;
  };
  PageRing<D, ST> pr;
  pr.start(a.pages, dsm + warp * ST * P::kBytes,
           reinterpret_cast<uint64_t*>(dsm + S::kRing + S::kAcc + S::kSum) + warp * ST, entry(), lane);
  pr.next = 0u;                   // (use_cluster: there is one list)
  // (every warp for itself: there is one unit, and a barrier would cost more)
  pw.prepare(lane);
  if constexpr (sizeof(T) == 4) {
    if (warp == 0) pw.share(s_q, lane);
    __syncthreads();
    pw.fetch(s_q, lane);
  }
  pw.reset();
  const int new_id = a.k_new != nullptr ? a.new_page(u, len) : -1;
  if (new_id >= 0 && warp < G) {
    const float sn = new_logit<T, D, G>(a, u, warp, lane);
    if (lane == 0) s_new[warp] = sn;
  }
  if (!pr.run((pages_of(L) - first + step * (NW - warp) - 1) / (step * NW), lane, [] { return 0u; },
              [&](unsigned char* pg, int n) { pw.take(pg, n, lane); }))
    set_flag(a.flags, KVS_FLAG_TIMEOUT);
  pw.end(s_acc + warp * G * D, s_m[warp], s_l[warp], s_b + warp, lane);
  __syncthreads();
  for (int i = tid; i < G * D / 4; i += NW * 32) {
    const int g = i * 4 / D, c = i * 4 % D;
    float M, Ls, B;
    *reinterpret_cast<float4*>(s_sum + i * 4) = merge_warps<D, G, NW>(s_acc, s_m, s_l, s_b, g, c, M, Ls, B);
    if (c == 0) {
      *reinterpret_cast<float4*>(s_ml[g]) = make_float4(M, Ls, B, 0.f);
    }
  }
  cluster_arrive();
  cluster_wait();
  // this CTA's slice of the output: a half-warp per four columns, lane j of it taking CTA j
  constexpr int NU = G * D / 4;
  const int lo = NU * rank / C, hi = NU * (rank + 1) / C;
  for (int b0 = lo + 2 * warp; b0 < hi; b0 += 2 * NW) {
    const int b = b0 + (lane >> 4), src = lane & 15;
    const int g = min(b, NU - 1) * 4 / D, c = b * 4 % D;
    float m = -INFINITY, l = 0.f, base = 0.f;
    float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
    if (b < hi && src < C) {
      const float4 ml = ld_cluster_f32x4(cluster_map(smem_u32(&s_ml[g][0]), src));
      A = ld_cluster_f32x4(cluster_map(smem_u32(s_sum + b * 4), src));
      m = ml.x;
      l = ml.y;
      base = ml.z;
    }
    const float M = half_warp_sum(A, m, l, base);
    if (b < hi && src == 0) {
      if (clusters == 1) {
        finish_columns<T>(A, M, l, base, new_id >= 0 ? s_new[g] : -INFINITY, a.v_new + (size_t)u * D + c,
                          a.out + (size_t)u * G * D + b * 4);
      } else {
        float* row = a.part + (((size_t)u * clusters + part) * NU + b) * 8;
        *reinterpret_cast<float4*>(row) = A;
        *reinterpret_cast<float4*>(row + 4) = make_float4(M, l, base, 0.f);
      }
    }
  }
  cluster_arrive();               // this CTA has read its peers; the wait is at the end
  bool last = true;
  if (clusters > 1) {
    __shared__ int s_last;
    __syncthreads();
    if (tid == 0) s_last = atom_add_acq_rel_gpu(&a.counters[u * C + rank], 1) == clusters - 1;
    __syncthreads();
    last = s_last != 0;
    if (last) {
      for (int b0 = lo + 2 * warp; b0 < hi; b0 += 2 * NW) {
        const int b = b0 + (lane >> 4), src = lane & 15;
        const int g = min(b, NU - 1) * 4 / D, c = b * 4 % D;
        float m = -INFINITY, l = 0.f, base = 0.f;
        float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
        if (b < hi && src < clusters) {
          const float* row = a.part + (((size_t)u * clusters + src) * NU + b) * 8;
          A = __ldcg(reinterpret_cast<const float4*>(row));
          const float4 ml = __ldcg(reinterpret_cast<const float4*>(row + 4));
          m = ml.x;
          l = ml.y;
          base = ml.z;
        }
        const float M = half_warp_sum(A, m, l, base);
        if (b < hi && src == 0)
          finish_columns<T>(A, M, l, base, new_id >= 0 ? s_new[g] : -INFINITY, a.v_new + (size_t)u * D + c,
                            a.out + (size_t)u * G * D + b * 4);
      }
      if (tid == 0) a.counters[u * C + rank] = 0;
    }
  }
  if (last && rank == 0 && a.k_new != nullptr) {
    // every CTA read the length before its cluster's first barrier, and each cluster's first CTA
    // has arrived by now
    if (new_id >= 0) {
      write_new_row<T, D>(a, u, len, new_id, warp, lane);
      if (tid == 0) a.len[u] = len + 1;
    } else if (tid == 0 && len == L) {
      set_flag(a.flags, KVS_FLAG_OUT_CAPACITY);
    }
  }
  cluster_wait();                 // no CTA leaves while a peer may read its shared memory
}

// Raises a kernel's dynamic shared-memory limit. The default one counts its static arrays too, so
// it is raised whenever the sum could pass it.
static bool allow_smem(const void* fn, size_t bytes) {
  return ensure_smem_attr(fn, bytes > 48 * 1024 ? bytes : 48 * 1024 + 16);
}

// Cluster size for `clusters` of them on the current device, or 0 when the split kernel is to be
// used: the largest C <= 16 with C * clusters <= SM count for which the occupancy calculator places
// all clusters at once. Cached per device and number of clusters.
template <typename T, int D, int G>
static int page_cluster_size(int clusters) {
  using S = PageClusterShape<D, G>;
  constexpr int kDevices = 64, kMost = 74;             // (148 SMs: no more clusters of two CTAs fit)
  auto kfn = page_decode_cluster_kernel<T, D, G>;
  static std::atomic<signed char> cache[kDevices][kMost + 1];     // the size + 1, 0: not known
  int dev = 0;
  if (clusters > kMost || cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return 0;
  if (const int known = cache[dev][clusters].load(std::memory_order_relaxed)) return known - 1;
  int sms = 0;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  int C = sms / clusters;
  if (C > kMaxClusterSize) C = kMaxClusterSize;
  if (!allow_smem((const void*)kfn, S::kSmem)) C = 0;
  if (C > 8 && !ensure_nonportable_cluster((const void*)kfn)) C = 8;
  for (; C >= 2; --C) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C, clusters);
    cfg.blockDim = dim3(kPcWarps * 32);
    cfg.dynamicSmemBytes = S::kSmem;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = C;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, (const void*)kfn, &cfg) == cudaSuccess && n >= clusters) break;
  }
  (void)cudaGetLastError();   // a refused query leaves no error behind
  if (C < 2) C = 0;
  cache[dev][clusters].store((signed char)(C + 1), std::memory_order_relaxed);
  return C;
}

template <typename T, int D, int G>
static cudaError_t launch_t(const kvs_cache_desc& d, const void* q, const kvs_page_pool& pool,
                            int32_t* len, const void* k_new, const void* v_new, void* out,
                            char* ws, size_t ws_bytes, cudaStream_t st) {
  const int units = d.B * d.H_kv;
  const PageLayoutWs Ly = page_layout_ws(d);
  const PageArgs<T> a = {(const T*)q, (unsigned char*)pool.pages, pool.table, pool.n_pages,
                         pool.max_pages, len, (const T*)k_new, (const T*)v_new, (T*)out, units,
                         reinterpret_cast<int32_t*>(ws + Ly.counters),
                         reinterpret_cast<int32_t*>(ws + Ly.done),
                         reinterpret_cast<float*>(ws + ws_tail(ws_bytes, Ly.part)), reinterpret_cast<int32_t*>(ws)};
  count_launches(1);
  const int clusters = clusters_of(units, pool.max_pages);
  const int C = page_cluster_size<T, D, G>(units * clusters);
  if (use_cluster(C, clusters, pool.max_pages)) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C, units * clusters);
    cfg.blockDim = dim3(kPcWarps * 32);
    cfg.dynamicSmemBytes = PageClusterShape<D, G>::kSmem;
    cfg.stream = st;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = C;
    at[1].val.clusterDim.y = 1;
    at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, page_decode_cluster_kernel<T, D, G>, a, clusters);
    return e != cudaSuccess ? e : cudaGetLastError();
  }
  auto kfn = page_decode_kernel<T, D, G>;
  using S = PageDecodeShape<D, G>;
  if (!allow_smem((const void*)kfn, S::kSmem)) return cudaErrorInvalidValue;
  const cudaError_t e = launch_pdl(kfn, dim3(kPageDecodeCtas), dim3(kPdThreads), S::kSmem, st, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_page_decode(const kvs_cache_desc& d, const void* q, const kvs_page_pool& pool,
                               int32_t* len, const void* k_new, const void* v_new, void* out,
                               char* ws, size_t ws_bytes, cudaStream_t st) {
  const int G = d.H_q / d.H_kv;
#define KVS_PD(TT, DD, GG) return launch_t<TT, DD, GG>(d, q, pool, len, k_new, v_new, out, ws, ws_bytes, st)
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
