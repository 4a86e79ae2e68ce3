// Eviction of cached tokens by accumulated attention weight: choose the tokens that stay, plan the pages,
// move the rows together.
//
// select: a cluster of 8 CTAs per request finds the k-th largest weight exactly, by three passes of histograms (11, 11
//   and 10 bits of the order key) over its slices of the weights, summed through distributed shared memory; then
//   one pass writes the kept tokens in order. The weights are read five times, from L2 after the first.
// plan: one cluster ranks the free pages (if a shared page has to be replaced) and gives every request its fresh pages
//   and its place in the list of moves.
// apply: the moves, then tables, counts, lengths and weights. A page is rewritten in place where nobody else holds
//   it, which needs no free pages, but other CTAs may still have to read its old rows. Token i of the new context is token
//   kept[i] >= i of the old one, and kept rises, so whoever reads a row that unit u of a stream (a request's rows in
//   one layer of a pool) overwrites comes no later than u in that stream. The moves are therefore done in batches, in
//   order: every CTA gathers its units of batch k into shared memory, all CTAs meet, and the units are written, while
//   those of batch k + 1 (which read behind all that batches up to k write) are already on their way into the other half of
//   shared memory. The bytes moved bound it, read once and written once.
#include <cooperative_groups.h>

#include "dsa_internal.cuh"
#include "sm103_ptx.cuh"

namespace dsa {

namespace {

constexpr int kCtas = 8;        // of a cluster
constexpr int kThreads = 1024;
constexpr int kBins = 2048;

// a unit of a move: what one warp gathers at a time
constexpr int kLatUnit = 16;    // tokens: 9,216 B (FP8)
constexpr int kSlot = kLatUnit * kLatRowFp8;
static_assert(kSlot >= kPage * (kIdxDim + 4), "a page of index keys is a unit, too");
constexpr int kMassUnit = 1024; // weights
static_assert(kSlot >= kMassUnit * 4, "weights");
constexpr int kMoveWarps = 12;
constexpr size_t kMoveSmem = size_t(2) * kMoveWarps * kSlot;
constexpr uint32_t kBarrierPolls = 1u << 22;  // 0.1 us and more each

enum { kPlanNew = 0, kPlanOld = 1, kPlanFirstPage = 2, kPlanNeed = 3, kPlanFresh = 4 };  // int32 [5][batch]
enum { kHeadItems = 0, kHeadArrived = 1 };                                 // int64 [4]

struct TokenPools {
  char* base[kMaxPools];
  int64_t page_stride[kMaxPools], layer_stride[kMaxPools];
  int layers[kMaxPools], fmt[kMaxPools];
  int n, units;  // units of a page, in all pools and layers
};

struct EvictArgs {
  const int32_t* budgets;
  float* mass;
  int32_t* table;
  int32_t* ctx;
  int32_t* refs;
  int32_t* kept;
  int32_t* list;   // [batch][cap]
  long long* head;
  long long* item; // [batch] first item of a request's moves
  int32_t* plan;   // [5][batch]: new length (-1: the request stays as it is) and old one, first page that changes, fresh
                   // pages, rank of the first of them
  int32_t* fresh;  // [batch][max_pages] rank of a page's fresh page among its request's, -1: in place
  int32_t* free;   // [num_pages]
  int* err;
  int64_t stride;  // of mass and kept
  int batch, max_pages, cap, num_pages, sinks, recent, units;
};

__device__ __forceinline__ int pages_of(int len) { return (len + kPage - 1) / kPage; }

// Inclusive scan over the block's 1,024 threads; `total` gets the sum.
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
    T s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  total = warp_sums[31];
  return v + (warp > 0 ? warp_sums[warp - 1] : T(0));
}

// Order key of a weight; a NaN is below everything.
__device__ __forceinline__ uint32_t mass_key(float f) { return f != f ? 0u : score_order_key(f); }

// ---------------------------------------------------------------- select
__global__ void __launch_bounds__(kThreads) __cluster_dims__(kCtas, 1, 1) evict_select_kernel(EvictArgs a) {
  namespace cg = cooperative_groups;
  __shared__ uint32_t hist[3][kBins];
  __shared__ uint32_t sums[32];
  __shared__ uint32_t s_bin, s_left, s_gt[kCtas], s_eq[kCtas], s_first[kCtas], s_mine;
  pdl_wait();
  const int b = blockIdx.x / kCtas, n = a.ctx[b], budget = a.budgets[b];
  if (budget < 0 || n < 0 || n > a.cap || n <= budget) {  // (the same for the whole cluster)
    if (blockIdx.x % kCtas == 0 && threadIdx.x == 0) {
      a.plan[kPlanNew * a.batch + b] = -1;
      a.plan[kPlanOld * a.batch + b] = n < 0 || n > a.cap ? 0 : n;
      a.plan[kPlanNeed * a.batch + b] = 0;
      if (budget >= 0 && (n < 0 || n > a.cap)) atomicOr(a.err, DSA_DEVERR_CTX);
    }
    return;
  }
  ptx::cluster_arrive();
  cg::cluster_group cl = cg::this_cluster();
  const int me = int(cl.block_rank()), tid = threadIdx.x;
  const int head = min(a.sinks, budget), tail = min(a.recent, budget - head);
  const int mid = n - head - tail;                  // tokens to choose from
  const int per = (mid + kCtas - 1) / kCtas, i0 = min(mid, me * per), i1 = min(mid, i0 + per);
  const float* mass = a.mass + b * a.stride + head;
  int32_t* list = a.list + size_t(b) * a.cap;
  // the ends
  for (int i = me * kThreads + tid; i < head; i += kCtas * kThreads) list[i] = i;
  for (int i = me * kThreads + tid; i < tail; i += kCtas * kThreads) list[budget - tail + i] = n - tail + i;
  for (int i = tid; i < 3 * kBins; i += kThreads) (&hist[0][0])[i] = 0;
  if (tid == 0) s_mine = 0x7FFFFFFF;
  __syncthreads();
  const uint32_t k = uint32_t(budget - head - tail);
  uint32_t tau = 0xFFFFFFFFu, left = 0;             // keys above tau stay, and the first `left` that equal it
  if (k > 0) {
    tau = 0;
    left = k;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t bins = pass == 2 ? 1024 : kBins;
      // the bits above this pass's are those of tau
      const uint64_t above = ~uint64_t(0) << (pass == 0 ? 32 : pass == 1 ? 21 : 10);
      for (int j0 = i0; j0 < i1; j0 += kThreads) {
        const int i = j0 + tid;
        const uint32_t key = i < i1 ? mass_key(mass[i]) : 0;
        const bool in = i < i1 && ((key ^ tau) & uint32_t(above)) == 0;
        const uint32_t bin = in ? (key >> shift) & (bins - 1) : ~0u;
        // many weights alike (those of tokens that nothing looked at): one addition for a warp of them
        int same;
        __match_all_sync(0xffffffffu, bin, &same);
        if (same) {
          if (in && (tid & 31) == 0) atomicAdd(&hist[pass][bin], 32u);
        } else if (in) {
          atomicAdd(&hist[pass][bin], 1u);
        }
      }
      __syncthreads();
      if (pass == 0) ptx::cluster_wait();  // every CTA has started: their shared memory can be read
      cl.sync();
      // thread t: bins from the top, 2t and 2t + 1 below it
      uint32_t c[2] = {0, 0};
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        const int bin = int(bins) - 1 - (2 * tid + d);
        if (bin >= 0)
          for (int r = 0; r < kCtas; ++r) c[d] += cl.map_shared_rank(&hist[pass][0], r)[bin];
      }
      uint32_t total;
      const uint32_t upto = block_scan<uint32_t>(c[0] + c[1], sums, total), before = upto - c[0] - c[1];
      if (before < left && upto >= left) {
        const int second = before + c[0] < left;
        s_bin = bins - 1 - (2 * tid + second);
        s_left = left - before - (second ? c[0] : 0);
      }
      __syncthreads();
      tau |= s_bin << shift;
      left = s_left;
      __syncthreads();
    }
  } else {
    ptx::cluster_wait();
  }
  // how many of each kind the slices hold
  uint32_t gt = 0, eq = 0;
  for (int i = i0 + tid; i < i1; i += kThreads) {
    const uint32_t key = mass_key(mass[i]);
    gt += k > 0 && key > tau;
    eq += k > 0 && key == tau;
  }
  uint32_t all_gt, all_eq;
  block_scan<uint32_t>(gt, sums, all_gt);
  block_scan<uint32_t>(eq, sums, all_eq);
  if (tid < kCtas) {
    *cl.map_shared_rank(s_gt + me, tid) = all_gt;
    *cl.map_shared_rank(s_eq + me, tid) = all_eq;
  }
  cl.sync();
  gt = eq = 0;
  for (int r = 0; r < me; ++r) {
    gt += s_gt[r];
    eq += s_eq[r];
  }
  // the kept tokens, in order; a tie's rank decides
  int first = 0x7FFFFFFF;  // the first that goes
  for (int j0 = i0; j0 < i1; j0 += kThreads) {
    const int i = j0 + tid;
    const uint32_t key = i < i1 ? mass_key(mass[i]) : 0;
    const bool is_gt = i < i1 && k > 0 && key > tau, is_eq = i < i1 && k > 0 && key == tau;
    uint32_t total;
    const uint32_t up = block_scan<uint32_t>(uint32_t(is_gt) | uint32_t(is_eq) << 16, sums, total);
    const uint32_t g = gt + (up & 0xFFFF) - is_gt, e = eq + (up >> 16) - is_eq;  // before this one
    gt += total & 0xFFFF;
    eq += total >> 16;
    if (is_gt || (is_eq && e < left)) list[head + g + min(e, left)] = head + i;
    else if (i < i1) first = min(first, head + i);
  }
  if (first != 0x7FFFFFFF) atomicMin(&s_mine, uint32_t(first));
  __syncthreads();
  if (tid == 0) *cl.map_shared_rank(s_first + me, 0) = s_mine;
  cl.sync();  // (also: the list is complete)
  if (me != 0) return;
  // the request's pages
  first = 0x7FFFFFFF;
  for (int r = 0; r < kCtas; ++r) first = min(first, int(s_first[r]));
  const int used = pages_of(n), want = pages_of(budget), from = first < budget ? first / kPage : want;
  const int32_t* row = a.table + size_t(b) * a.max_pages;
  uint32_t bad = 0, need = 0;
  for (int j0 = 0; j0 < used; j0 += kThreads) {
    const int j = j0 + tid;
    uint32_t shared = 0;
    if (j < used) {
      const int pg = row[j];
      if (pg < 0 || pg >= a.num_pages) bad |= DSA_DEVERR_BLOCK_TABLE;
      else if (a.refs[pg] < 1) bad |= DSA_DEVERR_PAGES;
      else shared = j >= from && j < want && a.refs[pg] > 1;
    }
    uint32_t total;
    const uint32_t up = block_scan<uint32_t>(shared, sums, total);
    if (j < used) a.fresh[size_t(b) * a.max_pages + j] = shared ? int(need + up - 1) : -1;
    need += total;
  }
  bad = uint32_t(__syncthreads_or(int(bad & DSA_DEVERR_BLOCK_TABLE)) ? DSA_DEVERR_BLOCK_TABLE : 0) |
        uint32_t(__syncthreads_or(int(bad & DSA_DEVERR_PAGES)) ? DSA_DEVERR_PAGES : 0);
  if (tid == 0) {
    if (bad) atomicOr(a.err, int(bad));
    a.plan[kPlanNew * a.batch + b] = bad ? -1 : budget;
    a.plan[kPlanOld * a.batch + b] = n;
    a.plan[kPlanFirstPage * a.batch + b] = from;
    a.plan[kPlanNeed * a.batch + b] = bad ? 0 : int(need);
  }
}

// ---------------------------------------------------------------- plan
// Items of a request's moves: its units page by page for every pool and layer, then its weights.
__device__ __forceinline__ long long items_of(int from, int len, int units) {
  const int pages = pages_of(len) - from;
  return pages > 0 ? (long long)pages * units + (len - from * kPage + kMassUnit - 1) / kMassUnit : 0;
}

__global__ void __launch_bounds__(kThreads) __cluster_dims__(kCtas, 1, 1) evict_plan_kernel(EvictArgs a) {
  namespace cg = cooperative_groups;
  __shared__ long long sums64[32];
  __shared__ uint32_t sums[32];
  __shared__ uint32_t counts[kCtas];
  ptx::cluster_arrive();
  pdl_wait();
  cg::cluster_group cl = cg::this_cluster();
  const int me = int(cl.block_rank()), tid = threadIdx.x;
  // fresh pages that the requests want, in all
  long long want = 0;
  for (int b = tid; b < a.batch; b += kThreads) want += a.plan[kPlanNeed * a.batch + b];
  long long wanted;
  block_scan<long long>(want, sums64, wanted);
  ptx::cluster_wait();
  uint32_t free = 0;
  if (wanted > 0) {  // (the same in every CTA)
    const int per = (a.num_pages + kCtas - 1) / kCtas;
    const int p0 = min(a.num_pages, me * per), p1 = min(a.num_pages, p0 + per);
    uint32_t mine = 0, total;
    for (int p = p0 + tid; p < p1; p += kThreads) mine += a.refs[p] <= 0;
    block_scan<uint32_t>(mine, sums, total);
    if (tid < kCtas) *cl.map_shared_rank(counts + me, tid) = total;
    cl.sync();
    uint32_t before = 0;
    for (int r = 0; r < kCtas; ++r) {
      if (r < me) before += counts[r];
      free += counts[r];
    }
    for (int q0 = p0; q0 < p1; q0 += kThreads) {
      const int p = q0 + tid;
      const uint32_t is_free = p < p1 && a.refs[p] <= 0;
      const uint32_t at = before + block_scan<uint32_t>(is_free, sums, total) - is_free;
      if (is_free) a.free[at] = p;
      before += total;
    }
  }
  if (me != 0) return;
  long long pages = 0, items = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    const int b = b0 + tid;
    int need = 0, len = -1;
    if (b < a.batch) {
      need = a.plan[kPlanNeed * a.batch + b];
      len = a.plan[kPlanNew * a.batch + b];
    }
    long long total;
    const long long upto = pages + block_scan<long long>(need, sums64, total);
    pages += total;
    if (need > 0 && upto > (long long)free) {
      atomicOr(a.err, DSA_DEVERR_NO_PAGES);
      a.plan[kPlanNew * a.batch + b] = len = -1;
    }
    const long long mine = len >= 0 ? items_of(a.plan[kPlanFirstPage * a.batch + b], len, a.units) : 0;
    const long long end = items + block_scan<long long>(mine, sums64, total);
    items += total;
    if (b < a.batch) {
      a.plan[kPlanFresh * a.batch + b] = int(upto - need);
      a.item[b] = end - mine;
    }
  }
  if (tid == 0) {
    a.head[kHeadItems] = items;
    a.head[kHeadArrived] = 0;
  }
}

// ---------------------------------------------------------------- apply
// What a warp needs to write a gathered unit.
struct Unit {
  char* dst;    // rows, whole 16 B each (null: none)
  char* words;  // index keys' scales, or weights (null: none)
  int bytes, n_words, words_at;  // where in the slot the words begin
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}

// Gathers tokens' rows of kChunks 16-B chunks: lane i has the addresses of rows i and i + 32.
template <int kChunks>
__device__ __forceinline__ void gather_rows(uint32_t smem, const char* r0, const char* r1, int rows, int lane) {
  const int n = rows * kChunks;
#pragma unroll 4
  for (int c0 = 0; c0 < n; c0 += 32) {  // (whole warps: the shuffles)
    const int c = c0 + lane, row = c / kChunks, off = c - row * kChunks;
    const uint64_t lo = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(r0), row & 31);
    const uint64_t hi = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(r1), row & 31);
    if (c < n) cp_async16(smem + c * 16, reinterpret_cast<const char*>(row < 32 ? lo : hi) + off * 16);
  }
}

// Starts the gathering of item `it` by a warp.
__device__ __forceinline__ Unit gather(const EvictArgs& a, const TokenPools& pools, long long it, uint32_t smem, int lane) {
  // the request: the last whose items begin at or before it (those without any share their start with the next)
  int lo = 0, hi = a.batch;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (a.item[m] <= it) lo = m;
    else hi = m;
  }
  const int b = lo, len = a.plan[kPlanNew * a.batch + b], from = a.plan[kPlanFirstPage * a.batch + b];
  const int pages = pages_of(len) - from;
  long long q = it - a.item[b];
  const int32_t* list = a.list + size_t(b) * a.cap;
  const int32_t* row = a.table + size_t(b) * a.max_pages;
  Unit u{nullptr, nullptr, 0, 0, 0};
  if (q >= (long long)pages * a.units) {  // weights
    const int i0 = from * kPage + int(q - (long long)pages * a.units) * kMassUnit, n = min(kMassUnit, len - i0);
    const float* mass = a.mass + b * a.stride;
    for (int i = lane; i < n; i += 32) cp_async4(smem + i * 4, mass + list[i0 + i]);
    u.words = reinterpret_cast<char*>(a.mass + b * a.stride + i0);
    u.n_words = n;
    return u;
  }
  // the pool, layer, page and part of it
  int pool = 0, per = 0;
  for (;; ++pool) {
    per = pools.fmt[pool] >= DSA_TOKEN_LAT_FP8 ? kPage / kLatUnit : 1;
    const long long size = (long long)pages * pools.layers[pool] * per;
    if (q < size) break;
    q -= size;
  }
  const int fmt = pools.fmt[pool], layer = int(q / ((long long)pages * per)), r = int(q - (long long)layer * pages * per);
  const int j = from + r / per, tokens = kPage / per, slot0 = (r % per) * tokens, i0 = j * kPage + slot0;
  const int n = min(tokens, len - i0);
  if (n <= 0) return u;
  char* base = pools.base[pool] + layer * pools.layer_stride[pool];
  const int rank = a.fresh[size_t(b) * a.max_pages + j];
  const int to = rank < 0 ? row[j] : a.free[a.plan[kPlanFresh * a.batch + b] + rank];
  char* dst = base + int64_t(to) * pools.page_stride[pool];
  const int width = fmt == DSA_TOKEN_KEY_FP8 ? 128 : fmt == DSA_TOKEN_KEY_MXFP4 ? 64 : fmt == DSA_TOKEN_LAT_FP8 ? 576 : 352;
  const char* src[2] = {nullptr, nullptr};
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    const int i = 32 * d + lane;
    if (i < n) {
      const int tok = list[i0 + i];
      const char* page = base + int64_t(row[tok / kPage]) * pools.page_stride[pool];
      src[d] = page + (tok % kPage) * width;
      if (fmt <= DSA_TOKEN_KEY_MXFP4)  // its scale, behind the rows
        cp_async4(smem + kPage * width + i * 4, page + kPage * width + (tok % kPage) * 4);
    }
  }
  if (fmt == DSA_TOKEN_LAT_FP8) gather_rows<36>(smem, src[0], src[1], n, lane);
  else if (fmt == DSA_TOKEN_LAT_NVFP4) gather_rows<22>(smem, src[0], src[1], n, lane);
  else if (fmt == DSA_TOKEN_KEY_FP8) gather_rows<8>(smem, src[0], src[1], n, lane);
  else gather_rows<4>(smem, src[0], src[1], n, lane);
  u.dst = dst + slot0 * width;
  u.bytes = n * width;
  if (fmt <= DSA_TOKEN_KEY_MXFP4) {
    u.words = dst + kPage * width;
    u.n_words = n;
    u.words_at = kPage * width;
  }
  return u;
}

__device__ __forceinline__ void drop_ref(const EvictArgs& a, int pg) {
  if (atomicAdd(a.refs + pg, -1) <= 0) {  // held by fewer than the tables say
    atomicAdd(a.refs + pg, 1);
    atomicOr(a.err, DSA_DEVERR_PAGES);
  }
}

// A cooperative launch (its CTAs meet).
__global__ void __launch_bounds__(32 * kMoveWarps, 1) evict_apply_kernel(const __grid_constant__ EvictArgs a,
                                                                        const __grid_constant__ TokenPools pools) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_ok;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long items = a.head[kHeadItems], per = (long long)gridDim.x * kMoveWarps;
  const long long batches = (items + per - 1) / per;
  unsigned long long* arrived = reinterpret_cast<unsigned long long*>(a.head + kHeadArrived);
  auto slot = [&](long long k) { return smem + (size_t(k & 1) * kMoveWarps + warp) * kSlot; };
  auto start = [&](long long k) {
    const long long it = k * per + (long long)blockIdx.x * kMoveWarps + warp;
    Unit u{nullptr, nullptr, 0, 0, 0};
    if (it < items) u = gather(a, pools, it, ptx::smem_u32(slot(k)), lane);
    asm volatile("cp.async.commit_group;" ::: "memory");
    return u;
  };
  Unit now = {};
  if (batches > 0) now = start(0);
  for (long long k = 0; k < batches; ++k) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // this CTA has read what it needs of batches up to k
    if (threadIdx.x == 0) {
      __threadfence();
      atomicAdd(arrived, 1ull);
    }
    Unit next = {};
    if (k + 1 < batches) {
      if (lane == 0) ptx::bulk_wait_read();  // the other half was written out from
      __syncwarp();
      next = start(k + 1);
    }
    if (threadIdx.x == 0) {
      const unsigned long long goal = (unsigned long long)(k + 1) * gridDim.x;
      int ok = 0;
      for (uint32_t i = 0; i < kBarrierPolls; ++i) {
        unsigned long long v;
        asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(arrived) : "memory");
        if (v >= goal) {
          ok = 1;
          break;
        }
        __nanosleep(64);
      }
      s_ok = ok;
    }
    __syncthreads();
    if (!s_ok) {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
      if (lane == 0) ptx::bulk_wait_read();
      if (threadIdx.x == 0) atomicOr(a.err, DSA_DEVERR_TIMEOUT);
      return;
    }
    const uint8_t* from = slot(k);
    for (int i = lane; i < now.n_words; i += 32)
      reinterpret_cast<uint32_t*>(now.words)[i] = reinterpret_cast<const uint32_t*>(from + now.words_at)[i];
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (now.dst) ptx::bulk_store(now.dst, from, uint32_t(now.bytes));
      ptx::bulk_commit();
    }
    __syncwarp();
    now = next;
  }
  if (lane == 0) ptx::bulk_wait_read();
  // Every row has been read: tables, counts and lengths, a CTA a request ...
  for (int b = blockIdx.x; b < a.batch; b += gridDim.x) {
    const int len = a.plan[kPlanNew * a.batch + b];
    if (len < 0) continue;
    int32_t* row = a.table + size_t(b) * a.max_pages;
    const int first = a.plan[kPlanFirstPage * a.batch + b], want = pages_of(len), used = pages_of(a.plan[kPlanOld * a.batch + b]);
    for (int j = first + int(threadIdx.x); j < used; j += blockDim.x) {
      const int pg = row[j], rank = a.fresh[size_t(b) * a.max_pages + j];
      if (j >= want) {
        row[j] = -1;
        drop_ref(a, pg);
      } else if (rank >= 0) {
        const int to = a.free[a.plan[kPlanFresh * a.batch + b] + rank];
        row[j] = to;
        a.refs[to] = 1;
        drop_ref(a, pg);
      }
    }
    if (threadIdx.x == 0) a.ctx[b] = len;
  }
  // ... and the old indices of what stays and the weights behind the new ends, in pieces of the requests
  const int piece = 4 * int(blockDim.x), pieces = (a.cap + piece - 1) / piece;
  for (long long q = blockIdx.x; q < (long long)a.batch * pieces; q += gridDim.x) {
    const int b = int(q / pieces), i0 = int(q - (long long)b * pieces) * piece;
    const int len = a.plan[kPlanNew * a.batch + b], old = a.plan[kPlanOld * a.batch + b];
    const int32_t* list = a.list + size_t(b) * a.cap;
    for (int i = i0 + int(threadIdx.x); i < min(i0 + piece, old); i += blockDim.x) {
      if (len < 0) {
        if (a.kept) a.kept[b * a.stride + i] = i;
      } else if (i >= len) {
        a.mass[b * a.stride + i] = 0.f;
      } else if (a.kept) {
        a.kept[b * a.stride + i] = list[i];
      }
    }
  }
}

}  // namespace

cudaError_t launch_tokens_evict(const dsa_params_t& p, const WsLayout& L, char* ws, const int32_t* budgets, int sinks,
                                int recent, float* mass, int64_t token_stride, const dsa_token_pool_t* pools, int n_pools,
                                int32_t* block_table, int32_t* ctx_lens, int32_t* page_refs, int32_t* kept,
                                cudaStream_t st) {
  TokenPools q = {};
  q.n = n_pools;
  for (int i = 0; i < n_pools; ++i) {
    q.base[i] = static_cast<char*>(pools[i].base);
    q.page_stride[i] = pools[i].page_stride;
    q.layer_stride[i] = pools[i].layer_stride;
    q.layers[i] = pools[i].layers;
    q.fmt[i] = pools[i].fmt;
    q.units += pools[i].layers * (pools[i].fmt >= DSA_TOKEN_LAT_FP8 ? kPage / kLatUnit : 1);
  }
  EvictArgs a = {};
  a.budgets = budgets;
  a.mass = mass;
  a.table = block_table;
  a.ctx = ctx_lens;
  a.refs = page_refs;
  a.kept = kept;
  a.list = reinterpret_cast<int32_t*>(ws + L.ev_list);
  a.head = reinterpret_cast<long long*>(ws + L.ev_head);
  a.item = reinterpret_cast<long long*>(ws + L.ev_req);
  a.plan = reinterpret_cast<int32_t*>(ws + L.ev_req + size_t(8) * p.batch);
  a.fresh = reinterpret_cast<int32_t*>(ws + L.ev_page);
  a.free = reinterpret_cast<int32_t*>(ws + L.ev_free);
  a.err = reinterpret_cast<int*>(ws + L.err);
  a.stride = token_stride;
  a.batch = p.batch;
  a.max_pages = p.max_pages_per_req;
  a.cap = L.cap;
  a.num_pages = p.num_pages;
  a.sinks = sinks;
  a.recent = recent;
  a.units = q.units;
  cudaError_t e = launch_pdl(evict_select_kernel, dim3(kCtas * p.batch), dim3(kThreads), 0, st, a);
  if (e != cudaSuccess) return e;
  e = launch_pdl(evict_plan_kernel, dim3(kCtas), dim3(kThreads), 0, st, a);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(evict_apply_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMoveSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sm_count());
  cfg.blockDim = dim3(32 * kMoveWarps);
  cfg.dynamicSmemBytes = kMoveSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_apply_kernel, a, q);
}

}  // namespace dsa
