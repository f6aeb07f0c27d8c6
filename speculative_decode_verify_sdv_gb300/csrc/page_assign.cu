// Page tables and slot maps of a paged cache from the requests' lengths (sdv_page_assign).
//
// want_b = ceil((ctx_b + n_b) / page) pages against held_b.  With R pages given back in all and
// `count` on the list, top = count + R: the k-th page given back, in the order of the table,
// goes to place top - 1 - k, and the k-th one taken comes from there; who cannot have all its
// pages, and everyone behind, takes none.  Giving the same pages back restores the list.
//
// Two exclusive sums over the requests, of what is given back and of what is needed, and a
// copy of page ids.  A round of 48 windows moves some 50 ids and writes 6 KB: latency bounds it,
// the lengths' loads and then those of the list and of the table's entries (3.5 us a call, 48
// requests of 17 rows).  So for up to 255 requests, 2560 rows to place and tables of 65,536 entries in all
// one CTA makes both sums in one scan, and takes the new pages' ids for the slots from the list itself, not
// from the table that it writes.  Beyond one of them a cluster shares the copies, and a launch of its own writes
// positions and slots (512 prompts of up to 2001 rows, 31,843 pages taken and given back: 20.5 us the
// two calls, 8 MB written).
#include <cuda_runtime.h>

#include <climits>
#include <cstdint>

#include "host_util.h"
#include "mixing.h"
#include "sdv.h"
#include "sdv_device.cuh"

namespace sdv {

namespace {

struct PageArgs {
  int32_t *free_pages, *n_free, *table, *held;
  const int32_t *ctx, *n_rows;
  int32_t *granted, *positions, *slots;  // each may be null
  int32_t *plan_held, *plan_rows;        // [B] each: pages held and rows granted after the call
  int B, T, n_pages, page, max_pages;
  int* status;
};

constexpr int kPageThreads = 1024;

struct PageNeed {
  int ctx, n, held, want;
  bool bad;
  __device__ __forceinline__ int back() const { return max(held - want, 0); }
  __device__ __forceinline__ int need() const { return max(want - held, 0); }
};

__device__ __forceinline__ PageNeed page_need(const PageArgs& a, int b) {
  PageNeed p{0, 0, 0, 0, false};
  if (b >= a.B) return p;
  const int c = __ldcg(a.ctx + b), n = a.n_rows != nullptr ? __ldcg(a.n_rows + b) : a.T, h = __ldcg(a.held + b);
  p.ctx = max(c, 0);
  p.n = min(max(n, 0), a.T);
  p.held = min(max(h, 0), a.max_pages);
  const long long want = ((long long)p.ctx + p.n + a.page - 1) / a.page;
  p.want = want > a.max_pages ? a.max_pages : (int)want;
  p.bad = p.ctx != c || p.n != n || p.held != h || want > a.max_pages;
  return p;
}

// Sum over the block's threads in front of this one; `all`: over all of them.
__device__ __forceinline__ long long block_scan(long long x, long long* warp_sums, long long& all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long incl = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += o;
  }
  __syncthreads();  // the last call's sums have been read
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  const long long mine = warp_sums[lane];
  long long s = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, s, off);
    if (lane >= off) s += o;
  }
  all = __shfl_sync(0xffffffffu, s, 31);
  return incl - x + __shfl_sync(0xffffffffu, s - mine, warp);
}

__device__ __forceinline__ unsigned cluster_rank() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ unsigned cluster_size() {
  unsigned r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
// All threads of the cluster meet; what they wrote before is seen behind it.
__device__ __forceinline__ void cluster_meet() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Position and slot of row t of sequence b; false where the table's entry is not a page.
__device__ __forceinline__ bool place_row(const PageArgs& a, int b, int t, int ctx, int rows) {
  int pos = -1, slot = -1;
  bool ok = true;
  if (t < rows) {
    pos = ctx + t;
    if (a.slots != nullptr) {
      const int id = __ldcg(a.table + (size_t)b * a.max_pages + pos / a.page);
      ok = id >= 0 && id < a.n_pages;
      if (ok) slot = id * a.page + pos % a.page;
    }
  }
  const size_t e = (size_t)b * a.T + t;
  if (a.positions != nullptr) a.positions[e] = pos;
  if (a.slots != nullptr) a.slots[e] = slot;
  return ok;
}

// One cluster: every CTA computes the sums, the warps of all share the copies.
__global__ void __launch_bounds__(kPageThreads, 1) page_assign_kernel(const PageArgs a) {
  __shared__ long long warp_sums[32], s_off[kPageThreads];
  __shared__ int s_from[kPageThreads], s_count[kPageThreads];
  const int tid = threadIdx.x, lane = tid & 31;
  const int rank = cluster_rank(), warps = cluster_size() * (kPageThreads / 32), me = rank * (kPageThreads / 32) + (tid >> 5);
  griddep_wait();
  const int listed = __ldcg(a.n_free), count = min(max(listed, 0), a.n_pages);
  bool bad = listed != count;
  PageNeed first = page_need(a, tid);  // of the first 1024 sequences, kept
  long long sum = 0, back_all, all;
  for (int b0 = 0; b0 < a.B; b0 += kPageThreads) {
    const PageNeed p = b0 == 0 ? first : page_need(a, b0 + tid);
    bad |= p.bad;
    sum += p.back();
  }
  block_scan(sum, warp_sums, back_all);
  const long long top = count + back_all;
  bad |= top > a.n_pages;
  if (back_all > 0) {
    long long before = 0;
    for (int b0 = 0; b0 < a.B; b0 += kPageThreads) {
      const PageNeed p = b0 == 0 ? first : page_need(a, b0 + tid);
      const long long off = block_scan(p.back(), warp_sums, all) + before;
      s_off[tid] = off;
      s_from[tid] = p.want;
      s_count[tid] = p.back();
      __syncthreads();
      for (int i = me; i < min(kPageThreads, a.B - b0); i += warps) {
        int32_t* const row = a.table + (size_t)(b0 + i) * a.max_pages + s_from[i];
#pragma unroll 4
        for (int j = lane; j < s_count[i]; j += 32) {
          const int id = __ldcg(row + j);
          const long long at = top - 1 - (s_off[i] + j);
          bad |= id < 0 || id >= a.n_pages;
          row[j] = -1;
          if (at < a.n_pages) a.free_pages[at] = id;
        }
      }
      before += all;
    }
    cluster_meet();
  }
  long long before = 0, taken = 0;
  for (int b0 = 0; b0 < a.B; b0 += kPageThreads) {
    const PageNeed p = b0 == 0 ? first : page_need(a, b0 + tid);
    const long long off = block_scan(p.need(), warp_sums, all) + before;
    const bool served = off + p.need() <= top;
    const int fresh = served ? p.need() : 0, held = served ? p.want : min(p.held, p.want);
    taken += fresh;
    if (rank == 0 && b0 + tid < a.B) {
      a.plan_held[b0 + tid] = held;
      a.plan_rows[b0 + tid] = (int)min((long long)p.n, max((long long)held * a.page - p.ctx, 0ll));
    }
    s_off[tid] = off;
    s_from[tid] = p.held;
    s_count[tid] = fresh;
    __syncthreads();
    if (all > 0) {
      for (int i = me; i < min(kPageThreads, a.B - b0); i += warps) {
        int32_t* const row = a.table + (size_t)(b0 + i) * a.max_pages + s_from[i];
#pragma unroll 4
        for (int j = lane; j < s_count[i]; j += 32) {
          const long long at = top - 1 - (s_off[i] + j);
          const int id = at < a.n_pages ? __ldcg(a.free_pages + at) : -1;
          bad |= id < 0 || id >= a.n_pages;
          row[j] = id;
        }
      }
    }
    before += all;
  }
  block_scan(taken, warp_sums, all);
  cluster_meet();  // every CTA has read the lengths, every copy and the plan are there
  if (rank == 0) {
    for (int b = tid; b < a.B; b += kPageThreads) {
      a.held[b] = __ldcg(a.plan_held + b);
      if (a.granted != nullptr) a.granted[b] = __ldcg(a.plan_rows + b);
    }
    if (tid == 0) *a.n_free = (int)min(top - all, (long long)a.n_pages);
  }
  if (bad) atomicOr(a.status, kDevErrIndex);
}

// ---- one CTA ----------------------------------------------------------------------------

// One CTA against the cluster and its second launch, us a call (the giving back half of the calls):
// 8 sequences of 256 rows 3.7 against 4.2, of 512 4.6 against 4.4; 32 of 64 4.2 against 4.6, of 128
// 5.2 against 4.6; 255 of 9 4.9 against 5.3, of 17 6.0 against 5.3.
//
// How many pages a call moves is only known on the device; the tables' entries bound it.  Moved pages,
// us a call without places: 48 sequences, 48 pages 3.1 against 5.5, 12,288 14.7 against 7.8, 49,152 49.7 against
// 17.1; 255, 255 pages 3.1 against 5.4, 4080 8.6 against 5.9, 65,280 72 against 8.7, 261,120 273 against 20.  At
// the limit a call that moves every entry loses some 60 us, once in the life of its sequences, and every
// round with few pages gains 2.  Of up to eight sequences the cluster copies each by one warp: of eight
// 32,768 pages take 27.7 against 39.5.
constexpr int kSmallThreads = 512, kSmallSeqs = 255, kSmallAnyTable = 8;
constexpr long long kSmallRows = 2560, kSmallEntries = 65536;

struct TwoSums {
  long long back, need;
};
__device__ __forceinline__ TwoSums up_by(TwoSums x, int off) {
  return TwoSums{__shfl_up_sync(0xffffffffu, x.back, off), __shfl_up_sync(0xffffffffu, x.need, off)};
}

// The last of n sorted numbers that is not above k, the first of them being 0: whose k-th page it is.
__device__ __forceinline__ int owner_of(const long long* sums, int n, long long k) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sums[mid] <= k) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kSmallThreads, 1) page_assign_small_kernel(const PageArgs a) {
  constexpr int W = kSmallThreads / 32;
  __shared__ TwoSums s_warp[W];
  __shared__ long long s_back[kSmallThreads], s_need[kSmallThreads], s_taken;
  __shared__ int s_ctx[kSmallThreads], s_held[kSmallThreads], s_want[kSmallThreads], s_rows[kSmallThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_wait();
  const int listed = __ldcg(a.n_free), count = min(max(listed, 0), a.n_pages);
  const PageNeed p = page_need(a, tid);
  bool bad = listed != count || p.bad;
  const TwoSums mine{p.back(), p.need()};
  TwoSums incl = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const TwoSums o = up_by(incl, off);
    if (lane >= off) incl = TwoSums{incl.back + o.back, incl.need + o.need};
  }
  if (lane == 31) s_warp[warp] = incl;
  if (tid == 0) s_taken = 0;
  __syncthreads();
  TwoSums all{0, 0}, front{0, 0};
#pragma unroll
  for (int w = 0; w < W; ++w) {
    if (w == warp) front = all;
    all = TwoSums{all.back + s_warp[w].back, all.need + s_warp[w].need};
  }
  const long long back_off = front.back + incl.back - mine.back, need_off = front.need + incl.need - mine.need;
  const long long top = count + all.back;
  bad |= top > a.n_pages;
  const bool served = need_off + mine.need <= top;
  const int held = served ? p.want : min(p.held, p.want);
  const int rows = (int)min((long long)p.n, max((long long)held * a.page - p.ctx, 0ll));
  s_back[tid] = back_off;
  s_need[tid] = need_off;
  s_ctx[tid] = p.ctx;
  s_held[tid] = p.held;
  s_want[tid] = p.want;
  s_rows[tid] = rows;
  if (all.need > top && served) atomicMax(reinterpret_cast<unsigned long long*>(&s_taken), (unsigned long long)(need_off + mine.need));
  __syncthreads();
  const long long taken = all.need > top ? s_taken : all.need;
#pragma unroll 4
  for (long long k = tid; k < all.back; k += kSmallThreads) {
    const int b = owner_of(s_back, a.B, k);
    int32_t* const entry = a.table + (size_t)b * a.max_pages + s_want[b] + (k - s_back[b]);
    const int id = __ldcg(entry);
    const long long at = top - 1 - k;
    bad |= id < 0 || id >= a.n_pages;
    *entry = -1;
    if (at < a.n_pages) a.free_pages[at] = id;
  }
  if (all.back > 0) __syncthreads();
  auto listed_id = [&](long long k) {  // the k-th page taken
    const long long at = top - 1 - k;
    const int id = at < a.n_pages ? a.free_pages[at] : -1;
    bad |= id < 0 || id >= a.n_pages;
    return id;
  };
#pragma unroll 4
  for (long long k = tid; k < taken; k += kSmallThreads) {
    const int b = owner_of(s_need, a.B, k);
    a.table[(size_t)b * a.max_pages + s_held[b] + (k - s_need[b])] = listed_id(k);
  }
  if (tid < a.B) {
    a.held[tid] = held;
    if (a.granted != nullptr) a.granted[tid] = rows;
  }
  if (tid == 0) *a.n_free = (int)min(top - taken, (long long)a.n_pages);
  if (a.positions != nullptr || a.slots != nullptr) {
    const int total = a.B * a.T;
#pragma unroll 2
    for (int e = tid; e < total; e += kSmallThreads) {
      const int b = e / a.T, t = e - b * a.T;
      int pos = -1, slot = -1;
      if (t < s_rows[b]) {
        pos = s_ctx[b] + t;
        const int j = pos / a.page;
        const int id = j < s_held[b] ? a.table[(size_t)b * a.max_pages + j] : listed_id(s_need[b] + j - s_held[b]);
        if (id >= 0 && id < a.n_pages) slot = id * a.page + pos - j * a.page;
        else bad = true;
      }
      if (a.positions != nullptr) a.positions[e] = pos;
      if (a.slots != nullptr) a.slots[e] = slot;
    }
  }
  if (bad) atomicOr(a.status, kDevErrIndex);
}

constexpr int kPlaceThreads = 256, kPlaceRows = 4;

__global__ void __launch_bounds__(kPlaceThreads) page_place_kernel(const PageArgs a) {
  griddep_wait();
  const int b = blockIdx.y, t0 = blockIdx.x * kPlaceThreads * kPlaceRows + threadIdx.x;
  const int ctx = max(__ldcg(a.ctx + b), 0), rows = __ldcg(a.plan_rows + b);
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPlaceRows; ++i) {
    const int t = t0 + i * kPlaceThreads;
    if (t < a.T) bad |= !place_row(a, b, t, ctx, rows);
  }
  if (bad) atomicOr(a.status, kDevErrIndex);
}

constexpr int kMaxPageSeqs = 65535;

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace

}  // namespace sdv

extern "C" {

size_t sdv_page_assign_workspace_bytes(int32_t B) {
  if (B < 1 || B > sdv::kMaxPageSeqs) return 0;
  return sdv::kHeaderBytes + 2 * sdv::round_256((size_t)B * 4);
}

sdv_status sdv_page_assign(const sdv_pagepool* pool, int32_t B, int32_t T, const int32_t* ctx,
                           const int32_t* n_rows_or_null, int32_t* granted_or_null, int32_t* positions_or_null,
                           int32_t* slots_or_null, void* ws, size_t ws_bytes, sdv_stream_t stream) {
  if (pool == nullptr || pool->free_pages == nullptr || pool->n_free == nullptr || pool->table == nullptr ||
      pool->held == nullptr || ctx == nullptr || B < 1 || T < 1)
    return SDV_ERR_INVALID_ARG;
  if (pool->n_pages < 1 || pool->page_size < 1 || pool->max_pages < 1) return SDV_ERR_INVALID_ARG;
  for (const void* p : {(const void*)pool->free_pages, (const void*)pool->n_free, (const void*)pool->table,
                        (const void*)pool->held, (const void*)ctx, (const void*)n_rows_or_null,
                        (const void*)granted_or_null, (const void*)positions_or_null, (const void*)slots_or_null})
    if (!sdv::aligned4(p)) return SDV_ERR_INVALID_ARG;
  // positions and slots are 32-bit numbers
  if (B > sdv::kMaxPageSeqs || (long long)pool->n_pages * pool->page_size > INT32_MAX ||
      (long long)pool->max_pages * pool->page_size > INT32_MAX)
    return SDV_ERR_UNSUPPORTED;
  if (ws == nullptr || !sdv::is_aligned16(ws) || ws_bytes < sdv_page_assign_workspace_bytes(B)) return SDV_ERR_WORKSPACE;
  sdv::PageArgs a{};
  a.free_pages = pool->free_pages;
  a.n_free = pool->n_free;
  a.table = pool->table;
  a.held = pool->held;
  a.ctx = ctx;
  a.n_rows = n_rows_or_null;
  a.granted = granted_or_null;
  a.positions = positions_or_null;
  a.slots = slots_or_null;
  a.plan_held = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + sdv::kHeaderBytes);
  a.plan_rows = a.plan_held + sdv::round_256((size_t)B * 4) / 4;
  a.B = B;
  a.T = T;
  a.n_pages = pool->n_pages;
  a.page = pool->page_size;
  a.max_pages = pool->max_pages;
  a.status = static_cast<int*>(ws);
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool maps = positions_or_null != nullptr || slots_or_null != nullptr;
  if (B <= sdv::kSmallSeqs && (!maps || (long long)B * T <= sdv::kSmallRows) &&
      (B <= sdv::kSmallAnyTable || (long long)B * pool->max_pages <= sdv::kSmallEntries))
    return sdv::status_of(sdv::launch_pdl(sdv::page_assign_small_kernel, dim3(1), dim3(sdv::kSmallThreads), 0, st, a));
  const int cluster = 8;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(cluster);
  cfg.blockDim = dim3(sdv::kPageThreads);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = sdv::counted(cudaLaunchKernelEx(&cfg, sdv::page_assign_kernel, a));
  if (e == cudaSuccess && maps) {
    const int per = sdv::kPlaceThreads * sdv::kPlaceRows;
    e = sdv::launch_pdl(sdv::page_place_kernel, dim3((unsigned)(((long long)T + per - 1) / per), B),
                        dim3(sdv::kPlaceThreads), 0, st, a);
  }
  return sdv::status_of(e);
}

}  // extern "C"
