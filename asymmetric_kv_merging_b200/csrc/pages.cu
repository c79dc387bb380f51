// The 4-bit paged cache: page tables and slot maps, rows to pages and back.
//
// The pages bring no cache format of their own; this is the serving side of the merged cache:
// after a pooled budget every KV head has its own length, and pages let ragged heads share one
// pool while a row shrinks from 516 to 148 bytes (d = 128).
#include <cuda_runtime.h>

#include "kvs_common.cuh"
#include "kvs_kernels.h"
#include "pages.cuh"
#include "ptx.cuh"

namespace kvs {

// ---------------------------------------------------------------------------
// Page tables from lengths
// ---------------------------------------------------------------------------

constexpr int kAssignThreads = 1024;

struct UnitPages {
  int held, want;     // pages of the unit before and after (equal: nothing to do)
};

__device__ __forceinline__ UnitPages unit_pages(int rows, int held, int max_pages) {
  if (held < 0 || held > max_pages) return {0, 0};                       // left alone
  if (rows < 0 || pages_of(rows) > max_pages) return {held, held};
  return {held, pages_of(rows)};
}

// One CTA: exclusive sums of the pages each unit takes and gives back, then a warp per unit
// moves the page numbers: first those given back onto the free stack, then those taken off it.
__global__ void __launch_bounds__(kAssignThreads)
page_assign_kernel(const int32_t* __restrict__ rows, int32_t* held, int32_t* table,
                   int32_t* free_pages, int32_t* n_free, int units, int n_pages, int max_pages,
                   int2* __restrict__ offs, int32_t* flags) {
  __shared__ longlong2 s_warp[kAssignThreads / 32];   // 64 bits: garbage lengths may add up to more
  __shared__ longlong2 s_total;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (units + kAssignThreads - 1) / kAssignThreads;
  const int u0 = min(units, tid * per), u1 = min(units, u0 + per);
  longlong2 sum = make_longlong2(0, 0);
  bool bad = false;
  for (int u = u0; u < u1; ++u) {
    const int r = rows[u], h = held[u];
    const UnitPages p = unit_pages(r, h, max_pages);
    bad |= h < 0 || h > max_pages || r < 0 || pages_of(r) > max_pages;
    sum.x += max(0, p.want - p.held);
    sum.y += max(0, p.held - p.want);
  }
  if (bad) set_flag(flags, KVS_FLAG_BAD_LENGTH);
  longlong2 inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, inc.x, o);
    const long long y = __shfl_up_sync(0xffffffffu, inc.y, o);
    if (lane >= o) {
      inc.x += x;
      inc.y += y;
    }
  }
  if (lane == 31) s_warp[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const longlong2 w = s_warp[lane];
    longlong2 c = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, c.x, o);
      const long long y = __shfl_up_sync(0xffffffffu, c.y, o);
      if (lane >= o) {
        c.x += x;
        c.y += y;
      }
    }
    if (lane == 31) s_total = c;
    s_warp[lane] = make_longlong2(c.x - w.x, c.y - w.y);
  }
  __syncthreads();
  const long long taken = s_total.x, given = s_total.y;
  const int avail = *n_free;
  const bool ok = avail >= 0 && avail + given <= n_pages && taken <= avail + given;
  if (!ok) {
    if (tid == 0) set_flag(flags, KVS_FLAG_NO_PAGES);
    return;
  }
  int2 at = make_int2((int)(s_warp[warp].x + inc.x - sum.x), (int)(s_warp[warp].y + inc.y - sum.y));
  for (int u = u0; u < u1; ++u) {
    offs[u] = at;
    const UnitPages p = unit_pages(rows[u], held[u], max_pages);
    at.x += max(0, p.want - p.held);
    at.y += max(0, p.held - p.want);
  }
  __syncthreads();
  for (int u = warp; u < units; u += kAssignThreads / 32) {
    const UnitPages p = unit_pages(rows[u], held[u], max_pages);
    const int o = avail + offs[u].y;
    for (int j = p.want + lane; j < p.held; j += 32) {
      int32_t* e = table + (size_t)u * max_pages + j;
      free_pages[o + j - p.want] = *e;
      *e = -1;
    }
  }
  __syncthreads();
  const int base = avail + (int)given - (int)taken;
  for (int u = warp; u < units; u += kAssignThreads / 32) {
    const int h = held[u];
    const UnitPages p = unit_pages(rows[u], h, max_pages);
    const int o = base + offs[u].x;
    for (int j = p.held + lane; j < p.want; j += 32)
      table[(size_t)u * max_pages + j] = free_pages[o + j - p.held];
    __syncwarp();
    if (lane == 0 && h >= 0 && h <= max_pages) held[u] = p.want;
  }
  __syncthreads();
  if (tid == 0) *n_free = base;
}

// slots[u][i] = slot of row begin[u] + i, -1 past the unit's rows or where it holds no page.
__global__ void __launch_bounds__(256)
page_slots_kernel(const int32_t* __restrict__ rows, const int32_t* __restrict__ begin,
                  const int32_t* __restrict__ held, const int32_t* __restrict__ table,
                  int32_t* __restrict__ slots, int units, int max_pages, int stride) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= stride) return;
  for (int u = blockIdx.y; u < units; u += gridDim.y) {
    const int b = begin ? begin[u] : 0;
    const long long t = (long long)b + i;
    int slot = -1;
    if (b >= 0 && t < rows[u] && t / kPageRows < min(held[u], max_pages)) {
      const int pg = table[(size_t)u * max_pages + (int)(t / kPageRows)];
      if (pg >= 0) slot = pg * kPageRows + (int)(t % kPageRows);
    }
    slots[(size_t)u * stride + i] = slot;
  }
}

cudaError_t launch_page_assign(const kvs_page_pool& pool, int units, const int32_t* rows,
                               int32_t* held, int32_t* free_pages, int32_t* n_free,
                               const int32_t* begin, int32_t* slots, int stride, char* ws,
                               cudaStream_t st) {
  page_assign_kernel<<<1, kAssignThreads, 0, st>>>(
      rows, held, pool.table, free_pages, n_free, units, pool.n_pages, pool.max_pages,
      reinterpret_cast<int2*>(ws + page_persistent_bytes(units)), reinterpret_cast<int32_t*>(ws));
  count_launches(1);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !slots) return e;
  const dim3 grid((stride + 255) / 256, units < 65535 ? units : 65535);
  page_slots_kernel<<<grid, 256, 0, st>>>(rows, begin, held, pool.table, slots, units,
                                          pool.max_pages, stride);
  count_launches(1);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Rows to pages and back
// ---------------------------------------------------------------------------

// A warp takes 8 consecutive rows, lane l channels 8 (l mod 4) .. of row l / 4 of one block of 32
// channels after another. Codes of consecutive slots are then whole 128-byte lines (8 rows of 16
// bytes; 4 pairs of 32), the maximum of a block is two shuffles away, and a lane has all the
// loads of its row (8 of 16 bytes at d = 128 in bf16) in flight together.
constexpr int kRowThreads = 256;
constexpr int kRowsPerWarp = 8;
constexpr int kRowsPerBlock = kRowThreads / 32 * kRowsPerWarp;

// Whether the V codes of two neighbouring rows (lanes l and l ^ 4) share words: the rows' slots
// are a pair of the page, in order.
__device__ __forceinline__ bool paired(int slot, int lane) {
  const int other = __shfl_xor_sync(0xffffffffu, slot, 4);
  return slot >= 0 && other == (slot ^ 1) && (slot & 1) == ((lane >> 2) & 1);
}

template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads)
page_store_kernel(const T* __restrict__ K, const T* __restrict__ V, const float* __restrict__ logn,
                  const int32_t* __restrict__ slots, long long n_rows,
                  unsigned char* __restrict__ pages, int n_slots, int32_t* flags) {
  using P = PageLayout<D>;
  constexpr int NB = P::nb;
  const int lane = threadIdx.x & 31, sub = lane & 3;
  const long long r = (long long)blockIdx.x * kRowsPerBlock + threadIdx.x / 4;
  int slot = r < n_rows ? slots[r] : -1;
  if (slot >= n_slots) {
    if (sub == 0) set_flag(flags, KVS_FLAG_BAD_PAGE);
    slot = -1;
  }
  if (!__any_sync(0xffffffffu, slot >= 0)) return;
  const bool live = slot >= 0;
  Raw8<T> k[NB], v[NB];
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    if (live) {
      k[b].load(K + r * D + b * 32 + sub * 8);
      v[b].load(V + r * D + b * 32 + sub * 8);
    } else {
      k[b].zero();
      v[b].zero();
    }
  }
  const float ln = live && logn && sub == 0 ? logn[r] : 0.f;
  const bool pair = paired(slot, lane);
  const int row = slot & (kPageRows - 1);
  unsigned char* pg = pages + (size_t)(live ? slot / kPageRows : 0) * P::kBytes;
  uint32_t ks[NB], vs = 0;
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const uint32_t kw = quantise_lane<T>(k[b], ks[b]);
    uint32_t s;
    const uint32_t vw = quantise_lane<T>(v[b], s);
    if (sub == b) vs = s;
    // of a pair, the first row's lane writes both rows' pieces of quad 2 sub, the second's of 2 sub + 1
    const uint32_t ow = __shfl_xor_sync(0xffffffffu, vw, 4);
    if (live) {
      *reinterpret_cast<uint32_t*>(pg + P::k_code(b, row) + sub * 4) = kw;
      if (pair) {
        const bool odd = row & 1;
        *reinterpret_cast<uint32_t*>(pg + P::v_piece(b, row & ~1, sub * 2 + (odd ? 1 : 0))) =
            odd ? __byte_perm(ow, vw, 0x7632) : __byte_perm(vw, ow, 0x5410);
      } else {
        *reinterpret_cast<uint16_t*>(pg + P::v_piece(b, row, sub * 2)) = (uint16_t)vw;
        *reinterpret_cast<uint16_t*>(pg + P::v_piece(b, row, sub * 2 + 1)) = (uint16_t)(vw >> 16);
      }
    }
  }
  if (!live) return;
  if (sub == 0) {
    if constexpr (NB == 4)
      *reinterpret_cast<uint2*>(pg + P::k_scale(0, row)) = make_uint2(ks[0] | ks[1] << 16, ks[2] | ks[3] << 16);
    else
      *reinterpret_cast<uint32_t*>(pg + P::k_scale(0, row)) = ks[0] | ks[1] << 16;
    *reinterpret_cast<float*>(pg + P::logn(row)) = ln;
  }
  if (sub < NB) *reinterpret_cast<uint16_t*>(pg + P::v_scale(sub, row)) = (uint16_t)vs;
}

template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads)
page_load_kernel(const unsigned char* __restrict__ pages, int n_slots,
                 const int32_t* __restrict__ slots, long long n_rows, T* __restrict__ K,
                 T* __restrict__ V, float* __restrict__ logn, int32_t* flags) {
  using P = PageLayout<D>;
  constexpr int NB = P::nb;
  const int lane = threadIdx.x & 31, sub = lane & 3;
  const long long r = (long long)blockIdx.x * kRowsPerBlock + threadIdx.x / 4;
  int slot = r < n_rows ? slots[r] : -1;
  if (slot >= n_slots) {
    if (sub == 0) set_flag(flags, KVS_FLAG_BAD_PAGE);
    slot = -1;
  }
  if (!__any_sync(0xffffffffu, slot >= 0)) return;
  const bool live = slot >= 0, pair = paired(slot, lane);
  const int row = slot & (kPageRows - 1);
  const bool odd = row & 1;
  const unsigned char* pg = pages + (size_t)(live ? slot / kPageRows : 0) * P::kBytes;
  uint32_t kw[NB], vw[NB], vs = 0;
  uint2 ks = make_uint2(0u, 0u);
  float ln = 0.f;
#pragma unroll
  for (int b = 0; b < NB; ++b) kw[b] = vw[b] = 0u;
  if (live) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      kw[b] = __ldcs(reinterpret_cast<const uint32_t*>(pg + P::k_code(b, row) + sub * 4));
      if (pair)
        vw[b] = __ldcs(reinterpret_cast<const uint32_t*>(pg + P::v_piece(b, row & ~1, sub * 2 + (odd ? 1 : 0))));
      else
        vw[b] = *reinterpret_cast<const uint16_t*>(pg + P::v_piece(b, row, sub * 2)) |
                (uint32_t)*reinterpret_cast<const uint16_t*>(pg + P::v_piece(b, row, sub * 2 + 1)) << 16;
    }
    if constexpr (NB == 4)
      ks = *reinterpret_cast<const uint2*>(pg + P::k_scale(0, row));
    else
      ks.x = *reinterpret_cast<const uint32_t*>(pg + P::k_scale(0, row));
    if (sub < NB) vs = *reinterpret_cast<const uint16_t*>(pg + P::v_scale(sub, row));
    if (sub == 0 && logn) ln = *reinterpret_cast<const float*>(pg + P::logn(row));
  }
#pragma unroll
  for (int b = 0; b < NB; ++b) {
    const uint32_t ow = __shfl_xor_sync(0xffffffffu, vw[b], 4);
    if (pair) vw[b] = odd ? __byte_perm(ow, vw[b], 0x7632) : __byte_perm(vw[b], ow, 0x5410);
    const uint32_t sv = __shfl_sync(0xffffffffu, vs, (lane & ~3) + b);
    const uint32_t sk = (b & 2 ? ks.y : ks.x) >> (b & 1 ? 16 : 0);
    if (live) {
      float x[8];
      dequantise8(kw[b], __half2float(__ushort_as_half((unsigned short)sk)), x);
#pragma unroll
      for (int i = 0; i < 8; i += Vec16<T>::n) store_vec(K + r * D + b * 32 + sub * 8 + i, x + i);
      dequantise8(vw[b], __half2float(__ushort_as_half((unsigned short)sv)), x);
#pragma unroll
      for (int i = 0; i < 8; i += Vec16<T>::n) store_vec(V + r * D + b * 32 + sub * 8 + i, x + i);
    }
  }
  if (live && sub == 0 && logn) logn[r] = ln;
}

static int row_blocks(long long n_rows) { return (int)((n_rows + kRowsPerBlock - 1) / kRowsPerBlock); }

template <typename T, int D>
static cudaError_t store_t(const kvs_cache_desc& d, const void* K, const void* V,
                           const float* logn, const int32_t* slots, const kvs_page_pool& pool,
                           char* ws, cudaStream_t st) {
  const long long n = (long long)d.B * d.H_kv * d.T_cap;
  page_store_kernel<T, D><<<row_blocks(n), kRowThreads, 0, st>>>(
      (const T*)K, (const T*)V, logn, slots, n, (unsigned char*)pool.pages,
      pool.n_pages * kPageRows, reinterpret_cast<int32_t*>(ws));
  count_launches(1);
  return cudaGetLastError();
}

template <typename T, int D>
static cudaError_t load_t(const kvs_cache_desc& d, const kvs_page_pool& pool, const int32_t* slots,
                          void* K, void* V, float* logn, char* ws, cudaStream_t st) {
  const long long n = (long long)d.B * d.H_kv * d.T_cap;
  page_load_kernel<T, D><<<row_blocks(n), kRowThreads, 0, st>>>(
      (const unsigned char*)pool.pages, pool.n_pages * kPageRows, slots, n, (T*)K, (T*)V, logn,
      reinterpret_cast<int32_t*>(ws));
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_page_store(const kvs_cache_desc& d, const void* K, const void* V,
                              const float* logn, const int32_t* slots, const kvs_page_pool& pool,
                              char* ws, cudaStream_t st) {
  if (d.dtype == KVS_BF16)
    return d.d == 128 ? store_t<bf16, 128>(d, K, V, logn, slots, pool, ws, st)
                      : store_t<bf16, 64>(d, K, V, logn, slots, pool, ws, st);
  return d.d == 128 ? store_t<float, 128>(d, K, V, logn, slots, pool, ws, st)
                    : store_t<float, 64>(d, K, V, logn, slots, pool, ws, st);
}

cudaError_t launch_page_load(const kvs_cache_desc& d, const kvs_page_pool& pool,
                             const int32_t* slots, void* K, void* V, float* logn, char* ws,
                             cudaStream_t st) {
  if (d.dtype == KVS_BF16)
    return d.d == 128 ? load_t<bf16, 128>(d, pool, slots, K, V, logn, ws, st)
                      : load_t<bf16, 64>(d, pool, slots, K, V, logn, ws, st);
  return d.d == 128 ? load_t<float, 128>(d, pool, slots, K, V, logn, ws, st)
                    : load_t<float, 64>(d, pool, slots, K, V, logn, ws, st);
}

}  // namespace kvs
