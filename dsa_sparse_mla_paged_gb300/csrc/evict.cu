// Eviction of cached tokens by accumulated attention weight: choose the tokens that stay, plan the pages,
// move the rows together.
//
// select: a cluster per request finds the k-th largest weight exactly, by three passes of histograms (11, 11
//   and 10 bits of the order key) over its slices of the weights, summed through distributed shared memory; then
//   one pass writes the kept tokens in order. The weights are read once, their keys stay in shared memory; of a slice of more than
//   45,056 tokens a CTA (long contexts in large batches, one of more than 720,896) what lies behind is read in all five passes.
// plan: one cluster ranks the free pages (if a shared page has to be replaced) and gives every request its fresh pages
//   and its place in the list of moves.
// apply: the moves, then tables, counts, lengths and weights. A page is rewritten in place where nobody else holds
//   it, which needs no free pages, but other CTAs may still have to read its old rows. Token i of the new context is token
//   kept[i] >= i of the old one, and kept rises, so whoever reads a row that unit u of a stream (a request's rows in
//   one layer of a pool) overwrites comes no later than u in that stream. The moves are therefore done in batches, in
//   order: every CTA gathers its units of batch k into shared memory, all CTAs meet, and the units are written, while
//   those of batch k + 1 (which read behind all that batches up to k write) are already on their way into the other half of
//   shared memory. The bytes moved bound it, read once and written once.
//
// Measured (one GB300, in a graph, all three): 48 requests of 12,000 tokens to 8,192, FP8 latents and index keys of four layers,
// 250 us (1.15 GB; the moves take some 215, and 195 without their barriers); one of 524,289 tokens to 131,072 89 us, some 35 of
// them the choice by 16 CTAs; 4 of 4,096 to 2,048 24 us, the latency of the passes and barriers. (The choice with its keys in
// global memory and the move's addresses looked up a batch at a time: 324, 218 and 38 us.)
#include <cooperative_groups.h>

#include "dsa_internal.cuh"
#include "sm103_ptx.cuh"

namespace dsa {

namespace {

constexpr int kCtas = 8;        // of the plan's cluster
constexpr int kMaxCl = 16;        // of the choice's, at most
constexpr int kClTokens = 16384;  // tokens of a CTA's slice, at most, while the GPU has CTAs to give
constexpr int kRound = 4096;      // a slice is a multiple of: 128 tokens a warp
constexpr int kMaxKeys = 45056;   // keys that fit a CTA
static_assert(kMaxKeys % kRound == 0, "whole slices");
constexpr int kPieceTokens = 1536;  // what a CTA finishes at once: tables, weights behind the end, kept tokens
constexpr int kThreads = 1024;
constexpr int kBins = 2048;

// a unit of a move: what one warp gathers at a time
constexpr int kLatUnit = 16;    // tokens: 9,216 B (FP8)
constexpr int kSlot = kLatUnit * kLatRowFp8;
static_assert(kSlot >= kPage * (kIdxDim + 4), "a page of index keys is a unit, too");
constexpr int kMassUnit = 1024; // weights
static_assert(kSlot >= kMassUnit * 4, "weights");
// Warps of a CTA, two CTAs an SM. (One of twelve warps: 256 and 91.9 us in a graph for the first two cases above, two of six 249 and
// 88.5; three or four places a warp in the same room, so that rows are gathered two or three batches ahead: 296 and 345 for 264 call by
// call, as a batch has some 2 us whatever it moves; the moves cut into two parts whose batches do not wait for each other 248.5.)
constexpr int kMoveWarps = 6;
constexpr size_t kMoveSmem = size_t(2) * kMoveWarps * kSlot;
constexpr uint32_t kGridPolls = 1u << 22;  // of a counter in L2, 0.5 us and more each

enum { kPlanNew = 0, kPlanOld = 1, kPlanFirstPage = 2, kPlanNeed = 3, kPlanFresh = 4 };  // int32 [5][batch]
enum { kHeadItems = 0, kHeadArrived = 1, kHeadPieces = 2 };                // int64 [8]

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
  long long* item;   // [batch] first item of a request's moves
  long long* piece;  // [batch] and its first piece of what is finished behind them
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
// A cluster per request, of as many CTAs as its tokens need (1 to 16). A CTA has a slice of the tokens, whose keys
// stay in shared memory (`room` of them; what is behind is read again), a warp a stretch of the slice, so that the order within it
// takes shuffles and no barrier. A lane has four consecutive keys at a time. (Loops are not unrolled: a phase's first
// instructions come slower than its keys.)
__global__ void __launch_bounds__(kThreads) evict_select_kernel(EvictArgs a, int room) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(8) uint32_t hist[3][kBins], s_total[kBins];
  __shared__ uint32_t s_part[kThreads], sums[32], s_gt[32], s_eq[32];
  __shared__ uint32_t s_bin, s_left, s_all[kMaxCl][3], s_shared[kMaxCl], s_mine;
  pdl_wait();
  cg::cluster_group cl = cg::this_cluster();
  const int ctas = int(cl.num_blocks()), me = int(cl.block_rank()), tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / ctas, n = a.ctx[b], budget = a.budgets[b];
  if (budget < 0 || n < 0 || n > a.cap || n <= budget) {  // (the same for the whole cluster)
    if (me == 0 && tid == 0) {
      a.plan[kPlanNew * a.batch + b] = -1;
      a.plan[kPlanOld * a.batch + b] = n < 0 || n > a.cap ? 0 : n;
      a.plan[kPlanNeed * a.batch + b] = 0;
      if (budget >= 0 && (n < 0 || n > a.cap)) atomicOr(a.err, DSA_DEVERR_CTX);
    }
    return;
  }
  ptx::cluster_arrive();
  const int head = min(a.sinks, budget), tail = min(a.recent, budget - head);
  const int mid = n - head - tail;                  // tokens to choose from
  const int per = ((mid + ctas - 1) / ctas + kRound - 1) / kRound * kRound, i0 = min(mid, me * per), len = min(mid, i0 + per) - i0;
  const int seg = per / 32, w0 = min(len, warp * seg), w1 = min(len, w0 + seg);  // (whole 128s before the last)
  const float* mass = a.mass + b * a.stride + head + i0;
  int32_t* list = a.list + size_t(b) * a.cap;
  auto keys4 = [&](int i, uint32_t (&x)[4]) {  // those at and past w1 are anything
    if (i + 3 < room) {
      const uint4 v = *reinterpret_cast<const uint4*>(keys + i);
      x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = i + e < w1 ? mass_key(mass[i + e]) : 0;
    }
  };
  // the ends
  for (int i = me * kThreads + tid; i < head; i += ctas * kThreads) list[i] = i;
  for (int i = me * kThreads + tid; i < tail; i += ctas * kThreads) list[budget - tail + i] = n - tail + i;
  for (int i = tid; i < 3 * kBins; i += kThreads) (&hist[0][0])[i] = 0;
  if (tid == 0) s_mine = 0x7FFFFFFF;
  __syncthreads();
  // Many weights may be alike (those of tokens that nothing looked at): one addition for a warp's four each, if they are.
  auto count = [&](uint32_t* h, const bool (&in)[4], const uint32_t (&bin)[4]) {
    uint32_t one = 0xFFFFFFFFu, n = 0;
#pragma unroll
    for (int e = 3; e >= 0; --e) {
      one = in[e] ? bin[e] : one;
      n += in[e];
    }
    const uint32_t m = __ballot_sync(0xffffffffu, n > 0);
    if (m == 0) return;
    const uint32_t b0 = __shfl_sync(0xffffffffu, one, __ffs(m) - 1);
    bool same = true;
#pragma unroll
    for (int e = 0; e < 4; ++e) same &= !in[e] || bin[e] == b0;
    if (__all_sync(0xffffffffu, same)) {
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane == 0) atomicAdd(h + b0, n);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (in[e]) atomicAdd(h + bin[e], 1u);
    }
  };
  const uint32_t k = uint32_t(budget - head - tail);
  // keys above tau stay, and the first `left` that equal it (no key is 0xFFFFFFFF: a NaN's is 0)
  uint32_t tau = 0xFFFFFFFFu, left = 0;
  // the first pass also fills shared memory, eight loads at a time
  for (int j = w0; j < w1; j += 256) {
    float m[8];
#pragma unroll
    for (int d = 0; d < 8; ++d) m[d] = j + 32 * d + lane < w1 ? mass[j + 32 * d + lane] : 0.f;
#pragma unroll
    for (int d = 0; d < 8; d += 4) {
      bool in[4];
      uint32_t bin[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = j + 32 * (d + e) + lane;
        const uint32_t x = mass_key(m[d + e]);
        if (i < w1 && i < room) keys[i] = x;
        in[e] = i < w1;
        bin[e] = x >> 21;
      }
      count(hist[0], in, bin);
    }
  }
  __syncthreads();
  ptx::cluster_wait();  // every CTA has started: their shared memory can be read
  if (k > 0) {
    tau = 0;
    left = k;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : kBins;
      if (pass > 0) {
        const int above = pass == 1 ? 21 : 10;  // the bits from there on are those of tau
#pragma unroll 1
        for (int j = w0; j < w1; j += 128) {
          const int i = j + 4 * lane;
          uint32_t x[4];
          bool in[4];
          keys4(i, x);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            in[e] = i + e < w1 && (x[e] ^ tau) >> above == 0;
            x[e] = (x[e] >> shift) & (bins - 1);
          }
          count(hist[pass], in, x);
        }
        __syncthreads();
      }
      if (ctas > 1) {
        // every CTA adds up its share of the bins over all of them, and hands the sums out. (Every CTA reading all bins
        // of all took 13,000 cycles for 16 CTAs.)
        cl.sync();
        const int share = bins / ctas, bin = tid % share, step = kThreads / share;
        uint32_t sum = 0;
        for (int r = tid / share; r < ctas; r += step) sum += cl.map_shared_rank(&hist[pass][0], (r + me) % ctas)[me * share + bin];
        if (tid < share) s_part[tid] = 0;
        __syncthreads();
        if (sum) atomicAdd(&s_part[bin], sum);
        __syncthreads();
        for (int r = tid / share; r < ctas; r += step) cl.map_shared_rank(s_total, r)[me * share + bin] = s_part[bin];
        cl.sync();
      }
      // thread t: bins from the top, 2t and 2t + 1 below it
      uint32_t c[2] = {0, 0};
      const int bin = bins - 2 - 2 * tid;
      if (bin >= 0) {
        const uint2 v = *reinterpret_cast<const uint2*>((ctas > 1 ? s_total : hist[pass]) + bin);
        c[0] = v.y;
        c[1] = v.x;
      }
      uint32_t total;
      const uint32_t upto = block_scan<uint32_t>(c[0] + c[1], sums, total), before = upto - c[0] - c[1];
      if (before < left && upto >= left) {
        const int second = before + c[0] < left;
        s_bin = bin + 1 - second;
        s_left = left - before - (second ? c[0] : 0);
      }
      __syncthreads();
      tau |= s_bin << shift;
      left = s_left;
    }
  }
  // how many of each kind the warps and the CTAs hold, and the first token that goes (equal ones go from `left` on)
  uint32_t gt = 0, eq = 0;
#pragma unroll 1
  for (int j = w0; j < w1; j += 128) {
    const int i = j + 4 * lane;
    uint32_t x[4];
    keys4(i, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      gt += i + e < w1 && x[e] > tau;
      eq += i + e < w1 && x[e] == tau;
    }
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
  }
  __syncthreads();
  // (every warp scans the warps' counts)
  uint32_t up_gt = s_gt[lane], up_eq = s_eq[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, up_gt, o), y = __shfl_up_sync(0xffffffffu, up_eq, o);
    if (lane >= o) {
      up_gt += x;
      up_eq += y;
    }
  }
  const uint32_t all_gt = __shfl_sync(0xffffffffu, up_gt, 31), all_eq = __shfl_sync(0xffffffffu, up_eq, 31);
  gt = __shfl_sync(0xffffffffu, up_gt, warp) - gt;
  eq = __shfl_sync(0xffffffffu, up_eq, warp) - eq;
  if (ctas > 1) {
    if (tid < ctas) {
      uint32_t* to = cl.map_shared_rank(&s_all[me][0], tid);
      to[0] = all_gt;
      to[1] = all_eq;
    }
    cl.sync();
    for (int r = 0; r < me; ++r) {
      gt += s_all[r][0];
      eq += s_all[r][1];
    }
  }
  // the kept tokens, in order; a tie's rank decides
  int first = 0x7FFFFFFF;
  uint32_t at = head + gt + min(eq, left);
  const uint32_t below = (1u << lane) - 1;
#pragma unroll 1
  for (int j = w0; j < w1; j += 128) {
    uint32_t x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = j + 32 * e + lane;  // (128 tokens are on one side of `room`)
      x[e] = j < room ? keys[i] : i < w1 ? mass_key(mass[i]) : 0;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = j + 32 * e + lane;
      bool keep = i < w1 && x[e] > tau;
      const uint32_t ties = __ballot_sync(0xffffffffu, i < w1 && x[e] == tau);
      if (ties) {
        keep |= (ties >> lane & 1) && eq + __popc(ties & below) < left;
        eq += __popc(ties);
      }
      const uint32_t kept = __ballot_sync(0xffffffffu, keep);
      if (keep) list[at + __popc(kept & below)] = head + i0 + i;
      else if (i < w1) first = min(first, head + i0 + i);
      at += __popc(kept);
    }
  }
  first = __reduce_min_sync(0xffffffffu, first);
  if (lane == 0 && first != 0x7FFFFFFF) atomicMin(&s_mine, uint32_t(first));
  __syncthreads();
  first = int(s_mine);
  if (ctas > 1) {
    if (tid < ctas) cl.map_shared_rank(&s_all[me][0], tid)[2] = uint32_t(first);
    cl.sync();
    for (int r = 0; r < ctas; ++r) first = min(first, int(s_all[r][2]));
  }
  // the request's pages, a range of them each
  const int used = pages_of(n), want = pages_of(budget), from = first < budget ? first / kPage : want;
  const int per_page = (used + ctas - 1) / ctas, p0 = min(used, me * per_page), p1 = min(used, p0 + per_page);
  const int32_t* row = a.table + size_t(b) * a.max_pages;
  int32_t* fresh = a.fresh + size_t(b) * a.max_pages;
  uint32_t bad = 0, need = 0;
  for (int j0 = p0; j0 < p1; j0 += kThreads) {
    const int j = j0 + tid;
    int shared = 0;
    if (j < p1) {
      const int pg = row[j];
      if (pg < 0 || pg >= a.num_pages) {
        bad |= DSA_DEVERR_BLOCK_TABLE;
      } else {
        const int refs = a.refs[pg];
        if (refs < 1) bad |= DSA_DEVERR_PAGES;
        else shared = j >= from && j < want && refs > 1;
      }
    }
    uint32_t total = 0, up = 0;
    if (__syncthreads_or(shared)) up = block_scan<uint32_t>(shared, sums, total);
    if (j < p1) fresh[j] = shared ? int(need + up - 1) : -1;
    need += total;
  }
  bad = uint32_t(__syncthreads_or(int(bad & DSA_DEVERR_BLOCK_TABLE)) ? DSA_DEVERR_BLOCK_TABLE : 0) |
        uint32_t(__syncthreads_or(int(bad & DSA_DEVERR_PAGES)) ? DSA_DEVERR_PAGES : 0);
  if (ctas > 1) {
    if (tid < ctas) *cl.map_shared_rank(s_shared + me, tid) = need | bad << 24;  // (at most 2^22 pages, bits 0 and 4)
    cl.sync();
    uint32_t before = 0, all = 0;
    for (int r = 0; r < ctas; ++r) {
      const uint32_t v = s_shared[r];
      bad |= v >> 24;
      if (r < me) before += v & 0xFFFFFF;
      all += v & 0xFFFFFF;
    }
    if (before > 0 && need > 0)
      for (int j = p0 + tid; j < p1; j += kThreads)
        if (fresh[j] >= 0) fresh[j] += int(before);
    need = all;
  }
  if (me == 0 && tid == 0) {
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
  long long pages = 0, items = 0, pieces = 0;
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
    const long long rest = b < a.batch && (len >= 0 || a.kept) ? (a.plan[kPlanOld * a.batch + b] + kPieceTokens - 1) / kPieceTokens : 0;
    const long long last = pieces + block_scan<long long>(rest, sums64, total);
    pieces += total;
    if (b < a.batch) {
      a.plan[kPlanFresh * a.batch + b] = int(upto - need);
      a.item[b] = end - mine;
      a.piece[b] = last - rest;
    }
  }
  if (tid == 0) {
    a.head[kHeadItems] = items;
    a.head[kHeadPieces] = pieces;
    a.head[kHeadArrived] = 0;
  }
}

// ---------------------------------------------------------------- apply
// A unit in hand: what to gather (lane i has the addresses of rows i and i + 32; of words, that of the first
// weight's place in the list), and where it goes.
struct Unit {
  const char* src[2];
  const char* scale[2];  // index keys: the tokens' scales
  const int32_t* list;   // weights: which
  char* dst;             // rows, whole 16 B each (null: none)
  char* words;           // index keys' scales, or weights (null: none)
  int n, fmt, width;     // tokens; bytes of a row
};
constexpr int kFmtMass = 4;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)) : "memory");
}

// What a CTA keeps of the requests' plans in shared memory, if there are no more of them.
constexpr int kKept = 192;
struct Plans {
  long long item[kKept];
  int32_t len[kKept], from[kKept], fresh[kKept];
};
static_assert(kMoveSmem + sizeof(Plans) + 1024 + 64 <= 233472 / 2, "two CTAs an SM");

// The last request whose first item (or piece of what follows) is at or before `at`: those without any share their start with the next.
__device__ __forceinline__ int request_of(const long long* first, int batch, long long at) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (first[m] <= at) lo = m;
    else hi = m;
  }
  return lo;
}

// Where item `it` begins and ends. kNear: the plans are in shared memory.
template <bool kNear>
__device__ __forceinline__ Unit look_up(const EvictArgs& a, const TokenPools& pools, const Plans& near, long long it, int lane) {
  const int b = request_of(kNear ? near.item : a.item, a.batch, it), len = kNear ? near.len[b] : a.plan[kPlanNew * a.batch + b];
  const int from = kNear ? near.from[b] : a.plan[kPlanFirstPage * a.batch + b];
  const int first_fresh = kNear ? near.fresh[b] : a.plan[kPlanFresh * a.batch + b];
  const int pages = pages_of(len) - from;
  long long q = it - (kNear ? near.item[b] : a.item[b]);
  const int32_t* list = a.list + size_t(b) * a.cap;
  const int32_t* row = a.table + size_t(b) * a.max_pages;
  Unit u = {};
  if (q >= (long long)pages * a.units) {  // weights
    const int i0 = from * kPage + int(q - (long long)pages * a.units) * kMassUnit;
    u.fmt = kFmtMass;
    u.n = min(kMassUnit, len - i0);
    u.src[0] = reinterpret_cast<const char*>(a.mass + b * a.stride);
    u.list = list + i0;
    u.words = reinterpret_cast<char*>(a.mass + b * a.stride + i0);
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
  u.fmt = pools.fmt[pool];
  const int layer = int(q / ((long long)pages * per)), r = int(q - (long long)layer * pages * per);
  const int j = from + r / per, tokens = kPage / per, slot0 = (r % per) * tokens, i0 = j * kPage + slot0;
  u.n = max(0, min(tokens, len - i0));
  if (u.n == 0) return u;
  u.width = u.fmt == DSA_TOKEN_KEY_FP8 ? 128 : u.fmt == DSA_TOKEN_KEY_MXFP4 ? 64 : u.fmt == DSA_TOKEN_LAT_FP8 ? 576 : 352;
  char* base = pools.base[pool] + layer * pools.layer_stride[pool];
  const int rank = a.fresh[size_t(b) * a.max_pages + j], here = row[j];
  int tok[2], pg[2];
#pragma unroll
  for (int d = 0; d < 2; ++d) tok[d] = list[i0 + min(32 * d + lane, u.n - 1)];
#pragma unroll
  for (int d = 0; d < 2; ++d) pg[d] = row[tok[d] / kPage];
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    const char* page = base + int64_t(pg[d]) * pools.page_stride[pool];
    u.src[d] = page + (tok[d] % kPage) * u.width;
    u.scale[d] = page + kPage * u.width + (tok[d] % kPage) * 4;
  }
  const int to = rank < 0 ? here : a.free[first_fresh + rank];
  char* dst = base + int64_t(to) * pools.page_stride[pool];
  u.dst = dst + slot0 * u.width;
  if (u.fmt <= DSA_TOKEN_KEY_MXFP4) u.words = dst + kPage * u.width;
  return u;
}

// Rows of kChunks 16-B chunks.
template <int kChunks>
__device__ __forceinline__ void gather_rows(uint32_t smem, const Unit& u, int lane) {
  const int n = u.n * kChunks;
#pragma unroll 4
  for (int c0 = 0; c0 < n; c0 += 32) {  // (whole warps: the shuffles)
    const int c = c0 + lane, row = c / kChunks, off = c - row * kChunks;
    const uint64_t lo = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(u.src[0]), row & 31);
    const uint64_t hi = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(u.src[1]), row & 31);
    if (c < n) cp_async16(smem + c * 16, reinterpret_cast<const char*>(row < 32 ? lo : hi) + off * 16);
  }
}

__device__ __forceinline__ void gather(const Unit& u, uint32_t smem, int lane) {
  if (u.n > 0) {
    if (u.fmt == DSA_TOKEN_LAT_FP8) gather_rows<36>(smem, u, lane);
    else if (u.fmt == DSA_TOKEN_LAT_NVFP4) gather_rows<22>(smem, u, lane);
    else if (u.fmt == DSA_TOKEN_KEY_FP8) gather_rows<8>(smem, u, lane);
    else if (u.fmt == DSA_TOKEN_KEY_MXFP4) gather_rows<4>(smem, u, lane);
    else
      for (int i = lane; i < u.n; i += 32) cp_async4(smem + i * 4, u.src[0] + int64_t(u.list[i]) * 4);
    if (u.fmt <= DSA_TOKEN_KEY_MXFP4) {
#pragma unroll
      for (int d = 0; d < 2; ++d)
        if (32 * d + lane < u.n) cp_async4(smem + kPage * u.width + (32 * d + lane) * 4, u.scale[d]);
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

__device__ __forceinline__ void drop_ref(const EvictArgs& a, int pg) {
  if (atomicAdd(a.refs + pg, -1) <= 0) {  // held by fewer than the tables say
    atomicAdd(a.refs + pg, 1);
    atomicOr(a.err, DSA_DEVERR_PAGES);
  }
}

// A cooperative launch (its CTAs meet).
__global__ void __launch_bounds__(32 * kMoveWarps, 2) evict_apply_kernel(const __grid_constant__ EvictArgs a,
                                                                        const __grid_constant__ TokenPools pools) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_ok;
  __shared__ Plans near;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long items = a.head[kHeadItems], per = (long long)gridDim.x * kMoveWarps;
  const long long batches = (items + per - 1) / per;
  unsigned long long* arrived = reinterpret_cast<unsigned long long*>(a.head + kHeadArrived);
  auto slot = [&](long long k) { return smem + (size_t(k & 1) * kMoveWarps + warp) * kSlot; };
  auto unit = [&](long long k) {
    const long long it = k * per + (long long)blockIdx.x * kMoveWarps + warp;
    if (it >= items) return Unit{};
    return a.batch <= kKept ? look_up<true>(a, pools, near, it, lane) : look_up<false>(a, pools, near, it, lane);
  };
  if (a.batch <= kKept) {
    for (int b = threadIdx.x; b < a.batch; b += blockDim.x) {
      near.item[b] = a.item[b];
      near.len[b] = a.plan[kPlanNew * a.batch + b];
      near.from[b] = a.plan[kPlanFirstPage * a.batch + b];
      near.fresh[b] = a.plan[kPlanFresh * a.batch + b];
    }
    __syncthreads();
  }
  // A unit's addresses take a chain of loads, so they are looked up a batch ahead, while rows are under way.
  Unit now = {}, next = {};
  if (batches > 0) {
    now = unit(0);
    gather(now, ptx::smem_u32(slot(0)), lane);
    next = unit(1);
  }
  for (long long k = 0; k < batches; ++k) {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // this CTA has read what it needs of batches up to k
    if (threadIdx.x == 0) {
      __threadfence();
      atomicAdd(arrived, 1ull);
    }
    if (k + 1 < batches) {
      if (lane == 0) ptx::bulk_wait_read();  // the other half was written out from
      __syncwarp();
      gather(next, ptx::smem_u32(slot(k + 1)), lane);
    }
    if (threadIdx.x == 0) {
      const unsigned long long goal = (unsigned long long)(k + 1) * gridDim.x;
      int ok = 0;
      for (uint32_t i = 0; i < kGridPolls && !ok; ++i) {
        unsigned long long v;
        asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(arrived) : "memory");
        ok = v >= goal;
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
    if (now.words) {
      const uint32_t* w = reinterpret_cast<const uint32_t*>(from + (now.dst ? kPage * now.width : 0));
      for (int i = lane; i < now.n; i += 32) reinterpret_cast<uint32_t*>(now.words)[i] = w[i];
    }
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (now.dst) ptx::bulk_store(now.dst, from, uint32_t(now.n * now.width));
      ptx::bulk_commit();
    }
    __syncwarp();
    now = next;
    next = unit(k + 2);
  }
  if (lane == 0) ptx::bulk_wait_read();
  // Every row has been read: tables, counts, lengths, the old indices of what stays, the weights behind the new ends.
  const long long pieces = a.head[kHeadPieces];
  const bool is_near = a.batch <= kKept;
  for (long long q = blockIdx.x; q < pieces; q += gridDim.x) {
    const int b = request_of(a.piece, a.batch, q);
    const int i0 = int(q - a.piece[b]) * kPieceTokens;
    const int len = is_near ? near.len[b] : a.plan[kPlanNew * a.batch + b], old = a.plan[kPlanOld * a.batch + b];
    const int end = min(i0 + kPieceTokens, old);
    const int32_t* list = a.list + size_t(b) * a.cap;
    for (int i = i0 + int(threadIdx.x); i < end; i += blockDim.x) {
      if (len < 0) a.kept[b * a.stride + i] = i;
      else if (i >= len) a.mass[b * a.stride + i] = 0.f;
      else if (a.kept) a.kept[b * a.stride + i] = list[i];
    }
    if (len < 0) continue;
    const int from = is_near ? near.from[b] : a.plan[kPlanFirstPage * a.batch + b], j = i0 / kPage + int(threadIdx.x);
    if (j >= from && j < pages_of(end)) {
      int32_t* row = a.table + size_t(b) * a.max_pages;
      const int pg = row[j], rank = a.fresh[size_t(b) * a.max_pages + j];
      if (j >= pages_of(len)) {
        row[j] = -1;
        drop_ref(a, pg);
      } else if (rank >= 0) {
        const int to = a.free[(is_near ? near.fresh[b] : a.plan[kPlanFresh * a.batch + b]) + rank];
        row[j] = to;
        a.refs[to] = 1;
        drop_ref(a, pg);
      }
    }
    if (i0 == 0 && threadIdx.x == 0) a.ctx[b] = len;
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
  a.piece = a.item + p.batch;
  a.plan = reinterpret_cast<int32_t*>(a.piece + p.batch);
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
  int ctas = 1;
  // (a table may be far wider than its contexts: with 16 CTAs for each of 64 requests of 4,096 tokens in one of 1,048,576
  // a call took 178 us)
  while (ctas < kMaxCl && L.cap > ctas * kClTokens && p.batch * ctas * 2 <= sm_count()) ctas *= 2;
  const int slice = ((L.cap + ctas - 1) / ctas + kRound - 1) / kRound * kRound, room = slice < kMaxKeys ? slice : kMaxKeys;
  static std::atomic<uint64_t> keys_set{0}, cluster_set{0}, slots_set{0};
  cudaError_t e = set_once(keys_set, evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxKeys * 4);
  if (e != cudaSuccess) return e;
  e = set_once(cluster_set, evict_select_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas * p.batch);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = size_t(room) * 4;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    e = cudaLaunchKernelEx(&cfg, evict_select_kernel, a, room);
    if (e != cudaSuccess) return e;
  }
  e = launch_pdl(evict_plan_kernel, dim3(kCtas), dim3(kThreads), 0, st, a);
  if (e != cudaSuccess) return e;
  e = set_once(slots_set, evict_apply_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kMoveSmem));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * sm_count());
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
