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

constexpr int kAssignThreads = 256;
constexpr int kAssignLocal = 4096;    // units whose offsets fit in shared memory (32 KB)

struct UnitPages {
  int held, want;     // pages of the unit before and after (equal: nothing to do)
};

__device__ __forceinline__ bool unit_legal(int rows, int held, int max_pages) {
  return held >= 0 && held <= max_pages && rows >= 0 && pages_of(rows) <= max_pages;
}
__device__ __forceinline__ UnitPages unit_pages(int rows, int held, int max_pages) {
  if (held < 0 || held > max_pages) return {0, 0};                       // left alone
  if (rows < 0 || pages_of(rows) > max_pages) return {held, held};
  return {held, pages_of(rows)};
}

// Exclusive sums over the units of the pages they take (x) and give back (y) into pre[units];
// the totals in 64 bits (garbage lengths may add up to more). One CTA.
__device__ __forceinline__ longlong2 scan_units(const int32_t* rows, const int32_t* held, int units,
                                                int max_pages, int2* pre, bool& bad) {
  __shared__ longlong2 s_warp[kAssignThreads / 32 + 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (units + kAssignThreads - 1) / kAssignThreads;
  const int u0 = min(units, tid * per), u1 = min(units, u0 + per);
  longlong2 sum = make_longlong2(0, 0);
  for (int u = u0; u < u1; ++u) {
    const int r = rows[u], h = held[u];
    const UnitPages p = unit_pages(r, h, max_pages);
    bad |= !unit_legal(r, h, max_pages);
    sum.x += max(0, p.want - p.held);
    sum.y += max(0, p.held - p.want);
  }
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
  longlong2 before = make_longlong2(0, 0), total = before;
#pragma unroll
  for (int w = 0; w < kAssignThreads / 32; ++w) {
    if (w == warp) before = total;
    total.x += s_warp[w].x;
    total.y += s_warp[w].y;
  }
  int2 at = make_int2((int)(before.x + inc.x - sum.x), (int)(before.y + inc.y - sum.y));
  for (int u = u0; u < u1; ++u) {
    pre[u] = at;
    const UnitPages p = unit_pages(rows[u], held[u], max_pages);
    at.x += max(0, p.want - p.held);
    at.y += max(0, p.held - p.want);
  }
  __syncthreads();
  return total;
}

// The unit that taken (or given) page i belongs to: the last one whose offset is not above i.
template <bool kGiven>
__device__ __forceinline__ int unit_of(const int2* pre, int units, int i) {
  int lo = 0, hi = units - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if ((kGiven ? pre[mid].y : pre[mid].x) <= i) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kAssignThreads)
page_scan_kernel(const int32_t* __restrict__ rows, const int32_t* __restrict__ held, int units,
                 int max_pages, int2* pre, longlong2* total, int32_t* flags) {
  bool bad = false;
  const longlong2 t = scan_units(rows, held, units, max_pages, pre, bad);
  if (bad) set_flag(flags, KVS_FLAG_BAD_LENGTH);
  if (threadIdx.x == 0) *total = t;
}

// Moves the page numbers and writes the slot map, spread over the grid. The stack after the call
// is the old one, with the given pages pushed and the taken ones popped; where a taken page is
// one that is given in the same call, the thread that has it hands it on. So nothing of the
// stack that is read is also written, and no CTA waits for another; what other CTAs still read
// (the held counts, and the table entries of given pages if a slot map has to find those) is
// written by the last CTA to finish.
// Latency-bound throughout (a launch, the lengths, a page number, its slot): 128 units that give
// all pages back and take 18000 others with a slot map of a million rows, 14 us for the two calls
// (the same bytes take 0.7 us); 8 rows more for each of 128 units, 4.5 us a call. Sums and searches
// in every CTA cost less than a second launch would; one CTA for the page numbers and a second
// launch for the slots took 29 and 6.4 us.
template <bool kLocal>
__global__ void __launch_bounds__(kAssignThreads)
page_assign_kernel(const int32_t* __restrict__ rows, int32_t* held, int32_t* table,
                   int32_t* free_pages, int32_t* n_free, const int32_t* __restrict__ begin,
                   int32_t* __restrict__ slots, int stride, int units, int n_pages, int max_pages,
                   int2* ws_pre, const longlong2* ws_total, int32_t* done, int32_t* flags) {
  __shared__ int2 s_pre[kLocal ? kAssignLocal : 1];
  __shared__ int s_last;
  const int tid = threadIdx.x;
  const int avail = *n_free;
  int2* pre = kLocal ? s_pre : ws_pre;
  longlong2 total;
  if constexpr (kLocal) {
    bool bad = false;
    total = scan_units(rows, held, units, max_pages, s_pre, bad);
    if (bad && blockIdx.x == 0) set_flag(flags, KVS_FLAG_BAD_LENGTH);
  } else {
    total = *ws_total;
  }
  const bool ok = avail >= 0 && avail + total.y <= n_pages && total.x <= avail + total.y;
  const int taken = ok ? (int)total.x : 0, given = ok ? (int)total.y : 0;
  const int top = avail + given - taken;               // the stack's size afterwards
  const bool keep = slots != nullptr && taken > 0;     // given entries stay until the end
  const long long gtid = (long long)blockIdx.x * kAssignThreads + tid;
  const long long gsize = (long long)gridDim.x * kAssignThreads;
  auto entry = [&](int u, int j) -> int32_t& { return table[(size_t)u * max_pages + j]; };
  auto given_at = [&](int i) -> int32_t& {
    const int u = unit_of<true>(pre, units, i);
    return entry(u, unit_pages(rows[u], held[u], max_pages).want + i - pre[u].y);
  };
  auto taken_at = [&](int i) -> int32_t& {
    const int u = unit_of<false>(pre, units, i);
    return entry(u, held[u] + i - pre[u].x);
  };
  for (long long i = gtid; i < given; i += gsize) {
    int32_t& e = given_at((int)i);
    const int at = avail + (int)i;                     // its place on the stack
    if (at < top) free_pages[at] = e;
    else taken_at(at - top) = e;
    if (!keep) e = -1;
  }
  for (long long i = gtid; i < taken - given; i += gsize) taken_at((int)i) = free_pages[top + i];

  if (slots != nullptr) {
    // a warp takes 128 slots of a unit, a lane four of them (of at most two pages)
    const int lane = tid & 31, per = (stride + 127) / 128;
    const long long w0 = gtid / 32, nw = gsize / 32;
    const int du = (int)(nw / per), dc = (int)(nw % per);
    const bool wide = stride % 4 == 0 && (reinterpret_cast<uintptr_t>(slots) & 15) == 0;
    int c = (int)(w0 % per);
    for (long long u = w0 / per; u < units; u += du) {
      const int b = begin ? begin[u] : 0, r = rows[u], h = held[u];
      const UnitPages p = ok ? unit_pages(r, h, max_pages) : UnitPages{h, h};
      const int np = min(p.want, max_pages);           // pages that the unit has afterwards
      const int i0 = c * 128 + lane * 4;
      auto page = [&](int j) -> int {
        if (j >= np) return -1;
        if (j < p.held) return entry((int)u, j);
        const int at = top + pre[u].x + j - p.held;
        return at < avail ? free_pages[at] : given_at(at - avail);
      };
      int out[4], j_of = -1, id = -1;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const long long t = (long long)b + i0 + k;
        out[k] = -1;
        if (b >= 0 && t < r) {
          const int j = (int)((unsigned)t / kPageRows);
          if (j != j_of) {
            j_of = j;
            id = page(j);
            if (id >= n_pages) {                           // (its slots would wrap around)
              set_flag(flags, KVS_FLAG_BAD_PAGE);
              id = -1;
            }
          }
          if (id >= 0) out[k] = id * kPageRows + (int)((unsigned)t % kPageRows);
        }
      }
      int32_t* o = slots + (size_t)u * stride + i0;
      if (wide && i0 < stride) {
        *reinterpret_cast<int4*>(o) = make_int4(out[0], out[1], out[2], out[3]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (i0 + k < stride) o[k] = out[k];
      }
      c += dc;
      if (c >= per) {
        c -= per;
        ++u;
      }
    }
  }
  if (!ok) {
    if (gtid == 0) set_flag(flags, KVS_FLAG_NO_PAGES);
    return;                                            // (in every CTA)
  }
  __syncthreads();
  if (gridDim.x > 1) {
    if (tid == 0) s_last = atom_add_acq_rel_gpu(done, 1) == (int)gridDim.x - 1;
    __syncthreads();
    if (!s_last) return;
    if (tid == 0) *done = 0;
  }
  if (keep) {
    for (int i = tid; i < given; i += kAssignThreads) {
      // (a handed-on page's new entry is never one of these: those units only give)
      given_at(i) = -1;
    }
    __syncthreads();
  }
  for (int u = tid; u < units; u += kAssignThreads) {
    const int h = held[u];
    if (h >= 0 && h <= max_pages) held[u] = unit_pages(rows[u], h, max_pages).want;
  }
  if (tid == 0) *n_free = top;
}

cudaError_t launch_page_assign(const kvs_page_pool& pool, int units, const int32_t* rows,
                               int32_t* held, int32_t* free_pages, int32_t* n_free,
                               const int32_t* begin, int32_t* slots, int stride, char* ws,
                               size_t ws_bytes, cudaStream_t st) {
  const PageAssignWs Ly = page_assign_ws(units);
  longlong2* total = reinterpret_cast<longlong2*>(ws + ws_tail(ws_bytes, Ly.scratch));
  int2* pre = reinterpret_cast<int2*>(total + 1);
  int32_t* flags = reinterpret_cast<int32_t*>(ws);
  // enough CTAs for four slots (or eight page numbers, if every page moved) a thread, up to four
  // per SM (148 of 512 threads take 15.3 us where 592 of 256 take 13.9, 592 of 512 17.7)
  const long long work = (long long)units * stride / 4 > (long long)units * pool.max_pages / 8
                             ? (long long)units * stride / 4 : (long long)units * pool.max_pages / 8;
  long long ctas = (work + kAssignThreads - 1) / kAssignThreads;
  if (ctas > 2 * kTargetCtas) ctas = 2 * kTargetCtas;
  if (ctas < 1) ctas = 1;
  const bool local = units <= kAssignLocal;
  if (!local) {
    page_scan_kernel<<<1, kAssignThreads, 0, st>>>(rows, held, units, pool.max_pages, pre, total, flags);
    count_launches(1);
  }
  auto kfn = local ? page_assign_kernel<true> : page_assign_kernel<false>;
  kfn<<<(int)ctas, kAssignThreads, 0, st>>>(rows, held, pool.table, free_pages, n_free, begin, slots,
                                            stride, units, pool.n_pages, pool.max_pages, pre, total,
                                            reinterpret_cast<int32_t*>(ws + Ly.done), flags);
  count_launches(1);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// Rows to pages and back
// ---------------------------------------------------------------------------

// A warp takes 8 consecutive rows, lane l channels 8 (l mod 4) .. of row l / 4 of one block of 32
// channels after another. Codes of consecutive slots are then whole 128-byte lines (8 rows of 16
// bytes; 4 pairs of 32), the maximum of a block is two shuffles away, and a lane has all the
// loads of its row (8 of 16 bytes at d = 128 in bf16) in flight together. 262144 rows of d = 128 in
// bf16 (175 MB of rows and pages): stored in 30.7 us, 5.7 TB/s = 0.87 of the measured copy peak, and
// loaded in 29.7 us, 0.90; in fp32 (309 MB) stored in 75.3 us, 4.1 TB/s (that instance spills 60 bytes
// a thread), and loaded in 60.5, 5.1 TB/s. With two rows a warp step and the codes masked and shifted into place
// one by one the store took 61 us, the load 37; blocks of 256 threads take 0.7 us longer.
constexpr int kRowThreads = 128;
constexpr int kRowsPerWarp = 8;
constexpr int kRowsPerBlock = kRowThreads / 32 * kRowsPerWarp;

// Whether the V codes of two neighbouring rows (lanes l and l ^ 4) share words: the rows' slots
// are a pair of the page, in order.
__device__ __forceinline__ bool paired(int slot, int lane) {
  const int other = __shfl_xor_sync(0xffffffffu, slot, 4);
  return slot >= 0 && other == (slot ^ 1) && (slot & 1) == ((lane >> 2) & 1);
}

template <typename T, int D>
__global__ void __launch_bounds__(kRowThreads, 8)      // (left alone, the loads take turns in 40 registers)
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
__global__ void __launch_bounds__(kRowThreads, 12)
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
