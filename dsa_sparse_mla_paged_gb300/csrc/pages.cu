// Page operations on the paged caches: give requests new lengths (free, trim,
// grow with copy on write), fork requests, pack the pages in use to the front.
//
// The bookkeeping is exact and its result does not depend on the order in which
// threads run: free pages are ranked by number, requests by index, and the
// only atomics are additions to reference counts.
//
// Each call is a plan kernel and an apply kernel. The plan ranks the pages: one
// cluster of 8 CTAs reads page_refs twice (count, then rank; a rank needs the
// counts of the CTAs before it, exchanged through distributed shared memory), so
// the 4 bytes a page cost two launches in all instead of one per scan step. The
// apply kernel edits the tables and moves page contents: the bytes of the
// pages that are copied bound it, read once and written once.
//
// Measured: the plan 3 to 5 us (over 60,000 pages); 192 requests that copy their open
// page in 8 pools (139 MB, much of it from L2: the one shared page) 15 us; packing 64 requests
// in 8 pools (364 MB) 55 to 60 us (6.1 to 6.6 TB/s); forking 96 requests of 2,048 pages 2.6 us.
// A small call is the host's two launches.
#include <cooperative_groups.h>

#include "dsa_internal.cuh"
#include "sm103_ptx.cuh"

namespace dsa {

namespace {

constexpr int kPlanCtas = 8;
constexpr int kPlanThreads = 1024;
constexpr int kApplyThreads = 256;
constexpr int kPiece = kApplyThreads * 16 * 4;  // bytes a CTA copies at once: four 16-B loads in flight per thread

// words of the workspace's totals
enum { kHdFree = 0, kHdLive = 1, kHdFirstHigh = 2 };

struct Pools {
  char* base[kMaxPools];
  int64_t stride[kMaxPools];
  uint32_t units[kMaxPools];   // 16-B units of a page
  int first[kMaxPools + 1];    // first piece of the pool among a page's pieces
  int n;
};

struct PagesArgs {
  const int32_t* new_lens;
  const int32_t* src;
  const int32_t* dst;
  int32_t* table;
  int32_t* ctx;
  int32_t* refs;
  int32_t* page_map;
  int32_t* live_out;
  int32_t* head;
  int32_t* need;   // [batch] pages a request takes; fork: the length pair i copies, -1 if refused
  int32_t* first;  // [batch] rank of its first page; fork: claims, then pair i's rank among those of its source
  int32_t* from;   // [batch] page to copy before it is written, -1 none; fork: pairs with this source
  int32_t* list;   // [num_pages] free pages by rank; compact: destinations
  int32_t* list2;  // [num_pages] compact: live pages by rank
  int32_t* rank;   // [num_pages] compact: rank of a live page, -1 free; resize: whether the call found it live
  int32_t* err;
  int batch, max_pages, cap, num_pages, n;
};

__device__ __forceinline__ int pages_of(int len) { return (len + kPage - 1) / kPage; }

// Inclusive scan of one value per thread over the block; `total` gets the sum.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* warp_sums, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  __syncthreads();  // warp_sums of the previous call are consumed
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    T s = lane < int(blockDim.x >> 5) ? warp_sums[lane] : T(0);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  total = warp_sums[(blockDim.x >> 5) - 1];
  return v + (warp > 0 ? warp_sums[warp - 1] : T(0));
}

// ---------------------------------------------------------------- resize: the plan of the requests
__device__ void plan_requests(const PagesArgs& a, long long* warp_sums) {
  long long carry = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
    const int b = b0 + int(threadIdx.x);
    int need = 0, from = -1;
    if (b < a.batch) {
      const int old = a.ctx[b], now = a.new_lens[b];
      if (now >= 0) {
        if (old < 0 || old > a.cap || now > a.cap) {
          atomicOr(a.err, DSA_DEVERR_CTX);
          need = -1;
        } else if (now > old) {
          need = pages_of(now) - pages_of(old);
          if (old % kPage) {
            const int pg = a.table[size_t(b) * a.max_pages + old / kPage];
            if (pg < 0 || pg >= a.num_pages) {
              atomicOr(a.err, DSA_DEVERR_BLOCK_TABLE);
              need = -1;
            } else if (a.refs[pg] < 1) {  // a free page, which another request may get
              atomicOr(a.err, DSA_DEVERR_PAGES);
              need = -1;
            } else if (a.refs[pg] > 1) {
              from = pg;
              ++need;
            }
          }
        }
      }
    }
    long long total;
    const long long upto = carry + block_scan<long long>(need > 0 ? need : 0, warp_sums, total);
    carry += total;
    if (b < a.batch) {
      // a request whose pages are not all among the num_pages ranks cannot be
      // served: INT_MAX as its first rank says so
      const long long at = upto - (need > 0 ? need : 0);
      a.need[b] = need;
      a.first[b] = upto <= a.num_pages ? int(at) : 0x7FFFFFFF;
      a.from[b] = from;
    }
  }
}

// Ranks the pages in number order. Resize: list[rank] = free page, the number of
// free pages, and rank[p], whether p is live. Compact: rank[p] of every live page (-1 for a free one),
// list2[rank] = live page, list[k] = the k-th free page below the number of live
// pages, and that number with the rank of the first live page at or above it.
template <bool kCompact>
__global__ void __launch_bounds__(kPlanThreads) __cluster_dims__(kPlanCtas, 1, 1) pages_plan_kernel(PagesArgs a) {
  namespace cg = cooperative_groups;
  ptx::cluster_arrive();
  pdl_wait();
  __shared__ long long warp_sums64[32];
  __shared__ int warp_sums[32];
  __shared__ int counts[kPlanCtas];
  cg::cluster_group cl = cg::this_cluster();
  const int me = int(cl.block_rank());
  // this CTA's pages
  const int per = (a.num_pages + kPlanCtas - 1) / kPlanCtas;
  const int p0 = min(a.num_pages, me * per), p1 = min(a.num_pages, p0 + per);
  int mine = 0;
  for (int p = p0 + int(threadIdx.x); p < p1; p += kPlanThreads) mine += a.refs[p] > 0;
  int total;
  block_scan<int>(mine, warp_sums, total);
  ptx::cluster_wait();  // every CTA has started: their shared memory can be written
  if (threadIdx.x < kPlanCtas) *cl.map_shared_rank(counts + me, threadIdx.x) = total;
  cl.sync();
  int before = 0, live = 0;
  for (int i = 0; i < kPlanCtas; ++i) {
    if (i < me) before += counts[i];
    live += counts[i];
  }
  if (me == 0 && threadIdx.x == 0) {
    a.head[kHdFree] = a.num_pages - live;
    a.head[kHdLive] = live;
    if (live == a.num_pages) a.head[kHdFirstHigh] = live;
  }
  if (!kCompact && me == kPlanCtas - 1) plan_requests(a, warp_sums64);
  for (int q0 = p0; q0 < p1; q0 += kPlanThreads) {
    const int p = q0 + int(threadIdx.x);
    const int is_live = p < p1 && a.refs[p] > 0;
    const int li = before + block_scan<int>(is_live, warp_sums, total) - is_live;  // live pages before p
    before += total;
    if (p >= p1) continue;
    if constexpr (kCompact) {
      a.rank[p] = is_live ? li : -1;
      if (is_live) a.list2[li] = p;
      else if (p < live) a.list[p - li] = p;
      if (p == live) a.head[kHdFirstHigh] = li;
    } else {
      if (!is_live) a.list[p - li] = p;
      a.rank[p] = is_live;
    }
  }
}

// ---------------------------------------------------------------- page contents
// One piece of the copy of page `src` to page `dst` by the whole CTA.
__device__ __forceinline__ void copy_piece(const Pools& pools, int piece, int src, int dst) {
  int i = 0;
  while (i + 1 < pools.n && piece >= pools.first[i + 1]) ++i;
  const uint32_t u0 = uint32_t(piece - pools.first[i]) * (kPiece / 16) + threadIdx.x;
  const uint4* s = reinterpret_cast<const uint4*>(pools.base[i] + int64_t(src) * pools.stride[i]);
  uint4* d = reinterpret_cast<uint4*>(pools.base[i] + int64_t(dst) * pools.stride[i]);
  uint4 v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (u0 + k * kApplyThreads < pools.units[i]) v[k] = __ldcs(s + u0 + k * kApplyThreads);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (u0 + k * kApplyThreads < pools.units[i]) __stcs(d + u0 + k * kApplyThreads, v[k]);
}

__device__ __forceinline__ void drop_ref(const PagesArgs& a, int pg) {
  if (atomicAdd(a.refs + pg, -1) <= 0) {  // held by fewer than the tables say
    atomicAdd(a.refs + pg, 1);
    atomicOr(a.err, DSA_DEVERR_PAGES);
  }
}

// The first gridDim.x - copiers CTAs edit the requests, the others copy.
__global__ void __launch_bounds__(kApplyThreads) pages_resize_kernel(const __grid_constant__ PagesArgs a,
                                                                     const __grid_constant__ Pools pools) {
  pdl_wait();
  const int n_free = a.head[kHdFree];
  auto served = [&](int b, int need) { return need == 0 || (a.first[b] != 0x7FFFFFFF && a.first[b] + need <= n_free); };
  // the tables and counts
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    const int now = a.new_lens[b], need = a.need[b], old = a.ctx[b];
    if (now < 0 || need < 0) continue;
    if (!served(b, need)) {
      if (threadIdx.x == 0) atomicOr(a.err, DSA_DEVERR_NO_PAGES);
      continue;
    }
    int32_t* row = a.table + size_t(b) * a.max_pages;
    const int have = pages_of(old), want = pages_of(now), copy = a.from[b] >= 0;
    const int at = a.first[b];
    for (int j = have + int(threadIdx.x); j < want; j += kApplyThreads) {
      const int pg = a.list[at + copy + j - have];
      row[j] = pg;
      a.refs[pg] = 1;
    }
    for (int j = want + int(threadIdx.x); j < have; j += kApplyThreads) {
      const int pg = row[j];
      // (a page that was free may be another request's by now: its count is not touched)
      if (pg < 0 || pg >= a.num_pages) atomicOr(a.err, DSA_DEVERR_BLOCK_TABLE);
      else if (a.rank[pg]) drop_ref(a, pg);
      else atomicOr(a.err, DSA_DEVERR_PAGES);
      row[j] = -1;
    }
    __syncthreads();  // every thread has read ctx[b]
    if (threadIdx.x == 0) {
      if (copy) {
        const int pg = a.list[at];
        row[old / kPage] = pg;
        a.refs[pg] = 1;
        drop_ref(a, a.from[b]);
      }
      a.ctx[b] = now;
    }
  }
  // the open pages' contents
  const int pieces = pools.first[pools.n];
  if (pieces == 0) return;
  const int64_t items = int64_t(a.batch) * pieces;
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
    const int b = int(i / pieces);
    const int src = a.from[b];
    if (src < 0 || !served(b, a.need[b])) continue;
    copy_piece(pools, int(i - int64_t(b) * pieces), src, a.list[a.first[b]]);
  }
}

// ---------------------------------------------------------------- fork
__global__ void __launch_bounds__(kPlanThreads) fork_plan_kernel(PagesArgs a) {
  pdl_wait();
  for (int b = threadIdx.x; b < a.batch; b += kPlanThreads) {
    a.first[b] = 0x7FFFFFFF;
    a.from[b] = 0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
    const int d = a.dst[i];
    if (d >= 0 && d < a.batch) atomicMin(a.first + d, i);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
    const int s = a.src[i], d = a.dst[i];
    int len = -1;
    if (s < 0 || s >= a.batch || d < 0 || d >= a.batch || s == d || __ldcg(a.first + d) != i || a.ctx[d] != 0) {
      atomicOr(a.err, DSA_DEVERR_PAGES);
    } else {
      len = a.ctx[s];
      if (len < 0 || len > a.cap) {
        atomicOr(a.err, DSA_DEVERR_CTX);
        len = -1;
      }
    }
    a.need[i] = len;
  }
  __syncthreads();
  // how many pairs share a source, and one of them that adds for all
  for (int i = threadIdx.x; i < a.n; i += kPlanThreads)
    a.first[i] = a.need[i] >= 0 ? atomicAdd(a.from + a.src[i], 1) : 1;
}

// grid (pair, slice of the row). Of the pairs with one source, one adds to the pages' counts
// for all of them (96 forks of one prompt of 2,048 pages: 10.6 us with an addition for
// each, 2.6 so). A slot that is both a source and a destination
// was empty before the call, so nothing is read from a row that is written.
__global__ void __launch_bounds__(kApplyThreads) fork_apply_kernel(PagesArgs a) {
  pdl_wait();
  for (int i = blockIdx.x; i < a.n; i += gridDim.x) {
    const int len = a.need[i];
    if (len < 0) continue;
    const int src = a.src[i], holds = a.first[i] == 0 ? a.from[src] : 0;
    const int32_t* from = a.table + size_t(src) * a.max_pages;
    int32_t* to = a.table + size_t(a.dst[i]) * a.max_pages;
    for (int j = blockIdx.y * kApplyThreads + int(threadIdx.x); j < pages_of(len); j += gridDim.y * kApplyThreads) {
      const int pg = from[j];
      to[j] = pg;
      if (pg < 0 || pg >= a.num_pages) atomicOr(a.err, DSA_DEVERR_BLOCK_TABLE);
      else if (holds) atomicAdd(a.refs + pg, holds);
    }
    if (blockIdx.y == 0 && threadIdx.x == 0) a.ctx[a.dst[i]] = len;
  }
}

// ---------------------------------------------------------------- compact
__global__ void __launch_bounds__(kApplyThreads) compact_apply_kernel(const __grid_constant__ PagesArgs a,
                                                                      const __grid_constant__ Pools pools) {
  pdl_wait();
  const int live = a.head[kHdLive], high = a.head[kHdFirstHigh], moves = live - high;
  const int tid = blockIdx.x * kApplyThreads + threadIdx.x, step = gridDim.x * kApplyThreads;
  auto moved = [&](int pg) {  // the new number of page pg; -1 if it is free
    const int r = a.rank[pg];
    return r < 0 ? -1 : pg < live ? pg : a.list[r - high];
  };
  for (int k = tid; k < moves; k += step) {
    const int s = a.list2[high + k];
    a.refs[a.list[k]] = a.refs[s];
    a.refs[s] = 0;
  }
  if (a.page_map)
    for (int p = tid; p < a.num_pages; p += step) a.page_map[p] = moved(p);
  if (a.live_out && tid == 0) *a.live_out = live;
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    const int len = a.ctx[b];
    if (len < 0 || len > a.cap) {
      if (threadIdx.x == 0) atomicOr(a.err, DSA_DEVERR_CTX);
      continue;
    }
    int32_t* row = a.table + size_t(b) * a.max_pages;
    for (int j = threadIdx.x; j < pages_of(len); j += kApplyThreads) {
      const int pg = row[j];
      if (pg < 0 || pg >= a.num_pages) {
        atomicOr(a.err, DSA_DEVERR_BLOCK_TABLE);
        continue;
      }
      const int to = moved(pg);
      if (to < 0) atomicOr(a.err, DSA_DEVERR_PAGES);
      else if (to != pg) row[j] = to;
    }
  }
  const int pieces = pools.first[pools.n];
  if (pieces == 0) return;
  const int64_t items = int64_t(moves) * pieces;
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) {
    const int k = int(i / pieces);
    copy_piece(pools, int(i - int64_t(k) * pieces), a.list2[high + k], a.list[k]);
  }
}

PagesArgs make_args(const dsa_params_t& p, const WsLayout& L, char* ws, int32_t* table, int32_t* ctx, int32_t* refs) {
  PagesArgs a = {};
  a.table = table;
  a.ctx = ctx;
  a.refs = refs;
  a.head = reinterpret_cast<int32_t*>(ws + L.pg_head);
  a.need = reinterpret_cast<int32_t*>(ws + L.pg_req);
  a.first = a.need + p.batch;
  a.from = a.first + p.batch;
  a.list = reinterpret_cast<int32_t*>(ws + L.pg_list);
  a.list2 = a.list + p.num_pages;
  a.rank = a.list2 + p.num_pages;
  a.err = reinterpret_cast<int32_t*>(ws + L.err);
  a.batch = p.batch;
  a.max_pages = p.max_pages_per_req;
  a.cap = L.cap;
  a.num_pages = p.num_pages;
  return a;
}

Pools make_pools(const dsa_page_pool_t* pools, int n) {
  Pools q = {};
  q.n = n;
  for (int i = 0; i < n; ++i) {
    q.base[i] = static_cast<char*>(pools[i].base);
    q.stride[i] = pools[i].page_stride;
    q.units[i] = uint32_t(pools[i].page_bytes / 16);
    q.first[i + 1] = q.first[i] + int((pools[i].page_bytes + kPiece - 1) / kPiece);
  }
  return q;
}

}  // namespace

cudaError_t launch_pages_resize(const dsa_params_t& p, const WsLayout& L, char* ws, const int32_t* new_lens,
                                const dsa_page_pool_t* pools, int n_pools, int32_t* block_table, int32_t* ctx_lens,
                                int32_t* page_refs, cudaStream_t st) {
  PagesArgs a = make_args(p, L, ws, block_table, ctx_lens, page_refs);
  a.new_lens = new_lens;
  cudaError_t e = launch_pdl(pages_plan_kernel<false>, dim3(kPlanCtas), dim3(kPlanThreads), 0, st, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(pages_resize_kernel, dim3(4 * sm_count()), dim3(kApplyThreads), 0, st, a, make_pools(pools, n_pools));
}

cudaError_t launch_pages_fork(const dsa_params_t& p, const WsLayout& L, char* ws, int n, const int32_t* src,
                              const int32_t* dst, int32_t* block_table, int32_t* ctx_lens, int32_t* page_refs,
                              cudaStream_t st) {
  PagesArgs a = make_args(p, L, ws, block_table, ctx_lens, page_refs);
  a.src = src;
  a.dst = dst;
  a.n = n;
  cudaError_t e = launch_pdl(fork_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, a);
  if (e != cudaSuccess) return e;
  const int slices = (p.max_pages_per_req + kApplyThreads - 1) / kApplyThreads;
  return launch_pdl(fork_apply_kernel, dim3(n, slices < 16 ? slices : 16), dim3(kApplyThreads), 0, st, a);
}

cudaError_t launch_pages_compact(const dsa_params_t& p, const WsLayout& L, char* ws, const dsa_page_pool_t* pools,
                                 int n_pools, int32_t* block_table, const int32_t* ctx_lens, int32_t* page_refs,
                                 int32_t* page_map, int32_t* live, cudaStream_t st) {
  PagesArgs a = make_args(p, L, ws, block_table, const_cast<int32_t*>(ctx_lens), page_refs);
  a.page_map = page_map;
  a.live_out = live;
  cudaError_t e = launch_pdl(pages_plan_kernel<true>, dim3(kPlanCtas), dim3(kPlanThreads), 0, st, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(compact_apply_kernel, dim3(4 * sm_count()), dim3(kApplyThreads), 0, st, a, make_pools(pools, n_pools));
}

}  // namespace dsa
