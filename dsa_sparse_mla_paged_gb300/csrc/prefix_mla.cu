// Dense attention of a batch that shares a prefix: out = softmax(scale q C^T) C[:, 0:512]
// of every (row, head) over the shared tokens and the request's own ones.
//
// Work is a line of 64-token tiles. First come the prefix jobs: 128 query heads
// (row * 96 + head, so rows pack without padding) against the whole prefix, the
// latents being the same for all of them. Then the private jobs: one row's 96 heads
// against the request's tokens past the prefix that the row may see (a job per row,
// so that a token hidden from a row never enters its products, whatever it holds).
// The line is cut into equal runs, one per CTA pair, and a run into segments at job
// borders; each segment leaves an unnormalised partial output with its softmax
// maximum and sum, and the merge kernel adds up the segments of a row's two jobs.
//
// The products take fp16 operands and fp32 sums. E4M3 and E2M1 x E4M3 values are exact
// in fp16 (one conversion instruction for two values; to bf16 it takes four). The
// query becomes fp16 with a power of two per head, which leaves every value exact
// down to 2^-32 of the head's largest (prefix_query_kernel). Softmax weights are
// scaled to at most 2^7 (2^15 until the running maximum is raised), so that fp16 holds
// them to 11 bits down to 2^-21 of the maximum.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "dsa_internal.cuh"
#include "sm103_ptx.cuh"

namespace dsa {

namespace {

// ---------------------------------------------------------------------------
// A CTA pair works on one tile of 128 query heads. A 128 x 512 fp32 output fills an
// SM's tensor memory, so the pair divides the two products: CTA 0 (scores) multiplies
// S = Q . C^T over all 576 dims and runs the softmax, CTA 1 (output) multiplies
// O += P . V. Per 64-token tile they cost 1,152 and 1,024 tensor-core cycles at full
// rate, and what crosses between them is P alone: 16 KB of fp16, one way. (A
// division by latent dims balances better, 1,088 each, but has to add partial scores,
// 32 KB of fp32 each way per tile; at the 32 B a cycle that an SM takes from
// another's stores that is 1,024 cycles, and it ran at 3,000 cycles a tile.)
//   CTA 0: warps 0..3, 4..7  softmax of the even and of the odd tiles: one query head
//                            per thread; the two groups hand the running maximum on
//          warps 8..15       converters: the page's 64 rows to fp16 (nine 128-B swizzled
//                            K-blocks of 64 dims); at a new job Q to tensor memory
//          warp  16          MMA: Q from tensor memory (288 columns), S in 3 x 64 columns
//   CTA 1: warps 0..3        rescale O where the maximum was raised, write O at a job's end
//          warps 8..15       converters: the 512 value dims, eight K-blocks read MN-major
//          warp  16          MMA: O in all 512 columns, P from shared memory
// A converter thread loads a piece of the next tile as soon as it has stored that
// piece of this one, so that every load has a whole tile's time.
// ---------------------------------------------------------------------------
constexpr int kNT = 64;                      // tokens per tile: one page
constexpr int kBlk = kNT * 128;              // 8,192 B: a K-block, 64 rows of 64 fp16
constexpr int kKBlks = kDQK / 64;            // 9
constexpr int kVBlks = kDNope / 64;          // 8
constexpr int kKBuf = kKBlks * kBlk;         // 73,728
constexpr int kVBuf = kVBlks * kBlk;         // 65,536
constexpr int kKBufs = 2, kVBufs = 3, kSBufs = 3, kPBufs = 2;
// P: 8 chunks of 8 tokens, each 16 B per row in row order (the unswizzled core
// matrices of the MMA, and 512 contiguous bytes for a warp's remote store)
constexpr int kPChunk = 128 * 16;
constexpr int kPBuf = 8 * kPChunk;           // 16,384
constexpr uint32_t kPBytes = kPBuf + 128 * 4;  // P and the rescale factors, per tile
constexpr int kMasks = 8;
constexpr int kThreads = 640;                // five warpgroups; the last holds the MMA warp and three idle ones
constexpr int kMmaWarp = 16;
constexpr uint32_t kSCol = 288;              // S after Q's 9 x 32 columns
constexpr int kNumBars = 36;
constexpr size_t kSmemO = kVBufs * kVBuf + kPBufs * (kPBuf + 512);
constexpr size_t kSmemS = kKBufs * kKBuf + 512 + kMasks * 8;
constexpr size_t kSmem = 1024 + (kSmemO > kSmemS ? kSmemO : kSmemS) + kNumBars * 8 + 16;
static_assert(kSmem + 512 <= 232448, "shared memory of one CTA");
constexpr float kPShift = 7.f;               // weights are 2^(z - max + 7)
constexpr float kLazy = 8.f;                 // the maximum in use is raised when passed by more than 2^8
constexpr int kJobCost = 3;                  // what a job's start and end take, in tiles

struct PfxArgs {
  const uint4* q16;  // [72][rows * 96] chunks of 8 dims: 16 B per head, in head order
  const float* qs;
  const uint8_t* lat;
  const int32_t* prefix_pages;
  const int32_t* table;
  const int32_t* lens;  // [rows] private tokens that a row sees (0: an invalid context length)
  int32_t* plan;  // [jobs][2] first and last CTA pair of a job
  float* ml;      // [slots][2 groups][2][128] softmax maxima (base 2) and sums
  float* part;    // [slots][128][512]
  int* err;
  int64_t stride;
  int prefix, n_q, rows, max_pages, num_pages, tiles;  // tiles: prefix jobs
  float scale_log2, lat_scale;
};

__device__ __forceinline__ int job_tiles(const PfxArgs& a, int job) {
  return job < a.tiles ? a.prefix / kNT : (a.lens[job - a.tiles] + kNT - 1) / kNT;
}

// A CTA pair's run of the line, segment by segment. The line is measured in units: a
// job with n > 0 tiles has kJobCost + n, the tiles at its end.
struct Walk {
  int job, k0, k1, n;  // the current segment: tiles [k0, k1) of a job of n
  int left;            // units of the run after it
  __device__ __forceinline__ bool start(const PfxArgs& a, int job0, int unit, int units) {
    job = job0;
    left = units;
    return take(a, unit) || next(a);
  }
  __device__ __forceinline__ bool take(const PfxArgs& a, int unit) {
    n = job_tiles(a, job);
    if (n == 0) return false;
    const int units = min(kJobCost + n - unit, left);
    left -= units;
    k0 = max(0, unit - kJobCost);
    k1 = max(0, unit + units - kJobCost);
    return k1 > k0;
  }
  __device__ __forceinline__ bool next(const PfxArgs& a) {
    while (left > 0 && ++job < a.tiles + a.rows)
      if (take(a, 0)) return true;
    return false;
  }
};

__device__ __forceinline__ uint32_t half2_from_e4m3x2(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two & 0xFFFFu), __NV_E4M3);
  return uint32_t(h.x) | uint32_t(h.y) << 16;
}

// 16 E4M3 bytes -> 16 fp16, as two 16-B chunks.
__device__ __forceinline__ void expand16(const uint4 w, uint4& lo, uint4& hi) {
  lo.x = half2_from_e4m3x2(w.x); lo.y = half2_from_e4m3x2(w.x >> 16);
  lo.z = half2_from_e4m3x2(w.y); lo.w = half2_from_e4m3x2(w.y >> 16);
  hi.x = half2_from_e4m3x2(w.z); hi.y = half2_from_e4m3x2(w.z >> 16);
  hi.z = half2_from_e4m3x2(w.w); hi.w = half2_from_e4m3x2(w.w >> 16);
}

// 8 E2M1 values times an E4M3 scale (a pair of fp16): 6 significant bits, exact.
__device__ __forceinline__ uint4 expand_e2m1(uint32_t w, __half2 s) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>((w >> (8 * i)) & 0xFFu), __NV_E2M1);
    const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&h), s);
    o[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Two adjacent 16-B chunks of a row of 64 fp16 (128-B swizzle).
__device__ __forceinline__ void put2(uint8_t* blk, int tok, int c, const uint4& lo, const uint4& hi) {
  uint8_t* row = blk + tok * 128;
  *reinterpret_cast<uint4*>(row + ((c ^ (tok & 7)) << 4)) = lo;
  *reinterpret_cast<uint4*>(row + (((c + 1) ^ (tok & 7)) << 4)) = hi;
}

// A converter thread's share of a tile; warp w of 8 has nope K-block w. FP8: eight
// 16-B pieces (8 tokens x 4 pieces a warp load: 64-B runs, and stores without bank
// conflicts). NVFP4: four 16-B units (32 values, two scales). And kRope: one 16-B
// piece of the rope dims. Tokens at or past `valid` are zeros.
template <bool kNv, bool kRope>
struct TileRegs {
  static constexpr int kPieces = kNv ? 4 : 8;
  uint4 v[kPieces];
  uint32_t s[kNv ? 4 : 1];
  uint4 rope;
  __device__ __forceinline__ void load(int u, const uint8_t* page, int valid, int w, int lane) {
    if constexpr (kNv) {
      const int tok = u * 16 + (lane >> 1), unit = 2 * w + (lane & 1);
      const uint8_t* row = page + tok * 352;
      v[u] = tok < valid ? __ldg(reinterpret_cast<const uint4*>(row + 16 * unit)) : make_uint4(0, 0, 0, 0);
      s[u] = tok < valid ? __ldg(reinterpret_cast<const uint16_t*>(row + 256 + 2 * unit)) : 0;
    } else {
      const int tok = u * 8 + (lane >> 2);
      v[u] = tok < valid ? __ldg(reinterpret_cast<const uint4*>(page + tok * 576 + 64 * w + 16 * (lane & 3)))
                         : make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ void load_rope(const uint8_t* page, int valid, int w, int lane) {
    const int ct = w * 32 + lane, tok = ct >> 2;
    rope = tok < valid ? __ldg(reinterpret_cast<const uint4*>(page + tok * (kNv ? 352 : 576) + (kNv ? 288 : 512) + 16 * (ct & 3)))
                       : make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void store(int u, uint8_t* buf, int w, int lane) const {
    uint8_t* blk = buf + w * kBlk;
    if constexpr (kNv) {
      const int tok = u * 16 + (lane >> 1), c0 = (lane & 1) * 4;
      const uint32_t two = half2_from_e4m3x2(s[u]);
      const __half2 h = *reinterpret_cast<const __half2*>(&two);
      const __half2 s0 = __low2half2(h), s1 = __high2half2(h);
      put2(blk, tok, c0, expand_e2m1(v[u].x, s0), expand_e2m1(v[u].y, s0));
      put2(blk, tok, c0 + 2, expand_e2m1(v[u].z, s1), expand_e2m1(v[u].w, s1));
    } else {
      uint4 lo, hi;
      expand16(v[u], lo, hi);
      put2(blk, u * 8 + (lane >> 2), (lane & 3) * 2, lo, hi);
    }
  }
  __device__ __forceinline__ void store_rope(uint8_t* buf, int w, int lane) const {
    const int ct = w * 32 + lane;
    uint4 lo, hi;
    expand16(rope, lo, hi);
    put2(buf + 8 * kBlk, ct >> 2, (ct & 3) * 2, lo, hi);
  }
};

// The converter warps of either CTA (kRope: CTA 0, whose tiles have the rope dims).
// full / free: the buffers' barriers; masks / mask_full: the valid tokens of a tile,
// for the softmax (CTA 0). at_job(g, job): what CTA 0 does after a job's first tile.
template <bool kNv, bool kRope, int kBufs, typename AtJob>
__device__ __forceinline__ bool convert(const PfxArgs& a, Walk wk, int gtot, int job0, int unit, int units, int w,
                                        int lane, uint8_t* bufs, uint32_t full, uint32_t free, unsigned long long* masks,
                                        uint32_t mask_full, AtJob at_job) {
  constexpr int kSize = kRope ? kKBuf : kVBuf;
  TileRegs<kNv, kRope> t;
  const int32_t* pages = nullptr;  // page numbers of the walk's job
  int len = 0, k = 0;              // its tokens, and the next tile's place in it
  auto enter = [&]() {
    if (wk.job < a.tiles) {
      pages = a.prefix_pages;
      len = a.prefix;
    } else {
      const int r = wk.job - a.tiles;
      pages = a.table + size_t(r / a.n_q) * a.max_pages + a.prefix / kNT;
      len = a.lens[r];
    }
    k = wk.k0;
  };
  // the next tile: its page number is loaded a tile ahead of its rows
  int pg = -1, left = 0;
  int begins = -1;                 // the job that the tile begins, -1 none
  auto fetch = [&]() {
    begins = -1;
    if (k >= wk.k1) {
      if (!wk.next(a)) return;
      enter();
      begins = wk.job;
    }
    pg = __ldg(pages + k);
    left = min(kNT, len - k * kNT);
    ++k;
  };
  if (gtot == 0 || !wk.start(a, job0, unit, units)) return true;
  enter();
  fetch();
  int job = wk.job;                // the job that the loaded tile begins
  const uint8_t* page;
  int valid;
  auto resolve = [&]() {
    const bool good = pg >= 0 && pg < a.num_pages;
    if (!good && kRope && w == 0 && lane == 0) atomicOr(a.err, DSA_DEVERR_BLOCK_TABLE);
    valid = good ? left : 0;
    page = a.lat + int64_t(good ? pg : 0) * a.stride;
  };
  resolve();
#pragma unroll
  for (int u = 0; u < t.kPieces; ++u) t.load(u, page, valid, w, lane);
  if constexpr (kRope) t.load_rope(page, valid, w, lane);
  if (gtot > 1) fetch();
#pragma unroll 1
  for (int g = 0; g < gtot; ++g) {
    const int buf = g % kBufs, now_valid = valid;
    const int now_job = job;
    const bool more = g + 1 < gtot;
    if (more) {
      resolve();
      job = begins;
      if (g + 2 < gtot) fetch();
    }
    if (g >= kBufs && !ptx::mbar_wait(free + 8 * (buf), uint32_t(g / kBufs - 1) & 1u)) return false;
    uint8_t* dst = bufs + buf * kSize;
#pragma unroll
    for (int u = 0; u < t.kPieces; ++u) {
      t.store(u, dst, w, lane);
      if (more) t.load(u, page, valid, w, lane);
    }
    if constexpr (kRope) {
      t.store_rope(dst, w, lane);
      if (more) t.load_rope(page, valid, w, lane);
      if (w == 0 && lane == 0) {
        masks[g % kMasks] = now_valid >= 64 ? ~0ull : (1ull << now_valid) - 1;
        ptx::mbar_arrive(mask_full + 8 * (g % kMasks));
      }
    }
    ptx::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(full + 8 * (buf));
    if (now_job >= 0 && !at_job(g, now_job)) return false;
  }
  return true;
}

template <bool kNv>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    prefix_mla_kernel(const __grid_constant__ PfxArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr size_t kData = kSmemO > kSmemS ? kSmemO : kSmemS;
  // the barriers have the same place in both CTAs
  const uint32_t bars = ptx::smem_u32(sm) + uint32_t(kData);
  const uint32_t mma_done = bars + 0 * 8;
  const uint32_t q_full = bars + 1 * 8;
  const uint32_t k_full = bars + 2 * 8;      // [2]
  const uint32_t k_free = bars + 4 * 8;      // [2]  S of the buffer's tile is done
  const uint32_t s_full = bars + 6 * 8;      // [3]
  const uint32_t s_free = bars + 9 * 8;      // [3]  the softmax has read S
  const uint32_t turn = bars + 12 * 8;       // [4]  by softmax warp: the tile's maximum is decided
  const uint32_t p_free = bars + 16 * 8;     // [2]  CTA 1 has multiplied the tile in this half of P
  const uint32_t mask_full = bars + 18 * 8;  // [8]
  const uint32_t v_full = bars + 26 * 8;     // [3]
  const uint32_t v_free = bars + 29 * 8;     // [3]  P . V of the buffer's tile is done
  const uint32_t p_full = bars + 32 * 8;     // [2]  P and the factors have landed
  const uint32_t o_ok = bars + 34 * 8;       // [2]  O is rescaled for the tile
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + kData + kNumBars * 8);
  // CTA 0
  uint8_t* KB = sm;
  float* m_run = reinterpret_cast<float*>(sm + kKBufs * kKBuf);  // [128] the running maximum in use
  unsigned long long* masks = reinterpret_cast<unsigned long long*>(m_run + 128);
  // CTA 1
  uint8_t* VB = sm;
  uint8_t* PB = sm + kVBufs * kVBuf;
  float* factor = reinterpret_cast<float*>(PB + kPBufs * kPBuf);  // [2][128]
  __shared__ long long s_sum[kThreads / 32];
  __shared__ int s_job, s_unit;

  const int half = int(ptx::cluster_ctarank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nclu = int(gridDim.x) >> 1, clu = int(blockIdx.x) >> 1;

  if (threadIdx.x == 0) {
    ptx::mbar_init(mma_done, 1);
    ptx::mbar_init(q_full, 8);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(k_full + 8 * (i), 8);
      ptx::mbar_init(k_free + 8 * (i), 1);
      ptx::mbar_init(p_free + 8 * (i), 1);
      ptx::mbar_init(p_full + 8 * (i), 1);
      ptx::mbar_init(o_ok + 8 * (i), 4);
    }
    for (int i = 0; i < 3; ++i) {
      ptx::mbar_init(s_full + 8 * (i), 1);
      ptx::mbar_init(s_free + 8 * (i), 4);
      ptx::mbar_init(v_full + 8 * (i), 8);
      ptx::mbar_init(v_free + 8 * (i), 1);
    }
    for (int i = 0; i < 4; ++i) ptx::mbar_init(turn + 8 * (i), 1);
    for (int i = 0; i < kMasks; ++i) ptx::mbar_init(mask_full + 8 * (i), 1);
    ptx::fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();

  // ---- the line's length, this pair's run of it, its tiles and the job it starts in
  int units, gtot;
  {
    auto block_sum = [&](long long v) {
#pragma unroll
      for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      __syncthreads();
      if (lane == 0) s_sum[warp] = v;
      __syncthreads();
      long long t = 0;
      for (int i = 0; i < kThreads / 32; ++i) t += s_sum[i];
      return t;
    };
    auto row_units = [&](int r) {
      const int n = job_tiles(a, a.tiles + r);
      return n > 0 ? n + kJobCost : 0;
    };
    long long mine = 0;
    for (int r = threadIdx.x; r < a.rows; r += kThreads) mine += row_units(r);
    const int per = a.tiles ? a.prefix / kNT + kJobCost : 1;  // units of a prefix job
    const int64_t shared = int64_t(a.tiles) * per;
    const int64_t line = shared + block_sum(mine);
    // no pair among those that work goes without a unit: a job's segments are those of
    // consecutive pairs
    const int64_t used = min(int64_t(nclu), line);
    const int64_t lo = clu < used ? line * clu / used : line, hi = clu < used ? line * (clu + 1) / used : line;
    units = int(hi - lo);
    // tiles of the prefix jobs among the line's first x units
    auto prefix_tiles = [&](int64_t x) {
      x = min(x, shared);
      return x / per * (per - kJobCost) + max(int64_t(0), x % per - kJobCost);
    };
    long long tiles = 0;
    if (threadIdx.x == 0) {
      tiles = prefix_tiles(hi) - prefix_tiles(lo);
      if (lo < shared) {
        s_job = int(lo / per);
        s_unit = int(lo % per);
      }
    }
    int64_t base = shared;
    for (int r0 = 0; r0 < a.rows && hi > base; r0 += kThreads) {
      const int r = r0 + int(threadIdx.x);
      const long long n = r < a.rows ? row_units(r) : 0;
      long long up = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += y;
      }
      __syncthreads();
      if (lane == 31) s_sum[warp] = up;
      __syncthreads();
      long long before = base + up - n, all = 0;
      for (int i = 0; i < kThreads / 32; ++i) {
        if (i < warp) before += s_sum[i];
        all += s_sum[i];
      }
      if (n > 0) {
        const long long t0 = before + kJobCost, t1 = before + n;  // its tiles
        tiles += max(0ll, min(t1, (long long)hi) - max(t0, (long long)lo));
        if (lo >= before && lo < t1) {
          s_job = a.tiles + r;
          s_unit = int(lo - before);
        }
      }
      base += all;
    }
    gtot = int(block_sum(tiles));
    // P of the first two tiles may arrive as soon as the pair has synced
    if (half == 1 && threadIdx.x == 0)
      for (int i = 0; i < 2 && i < gtot; ++i) ptx::mbar_arrive_expect_tx(p_full + 8 * (i), kPBytes);
  }
  __syncthreads();
  ptx::cluster_sync();  // the peer's barriers exist before any remote arrive
  const int job0 = s_job;
  const int unit0 = s_unit;
  bool ok = true;
  Walk wk;

  // registers: the five warpgroups start with 96 each (480) and go on with 104, 104, 96, 96 and 80 (480)
  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == kMmaWarp && half == 0) {
      // ---------------------------------------------------------- S = Q . C^T
      const uint32_t id = ptx::idesc(0, 0, 128, kNT);
      const uint32_t kb0 = ptx::smem_u32(KB);
      int g = 0, qn = 0;
      for (bool on = gtot > 0 && wk.start(a, job0, unit0, units); on && ok; on = wk.next(a)) {
        if (!ptx::mbar_wait(q_full, uint32_t(qn++) & 1u)) { ok = false; break; }
        for (int k = wk.k0; k < wk.k1; ++k, ++g) {
          const int buf = g % kKBufs, sb = g % kSBufs;
          if (!ptx::mbar_wait(k_full + 8 * (buf), uint32_t(g / kKBufs) & 1u)) { ok = false; break; }
          if (g >= kSBufs && !ptx::mbar_wait(s_free + 8 * (sb), uint32_t(g / kSBufs - 1) & 1u)) { ok = false; break; }
          ptx::tc_fence_after();
          const uint32_t kb = kb0 + buf * kKBuf, s = tmem + kSCol + sb * kNT;
          if (ptx::elect_one()) {
#pragma unroll 1
            for (int j = 0; j < kKBlks; ++j)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                ptx::mma_f16_tmem_a(s, tmem + j * 32 + kk * 8, ptx::sdesc_sw128(kb + j * kBlk + kk * 32), id,
                                    (j | kk) ? 1u : 0u);
            ptx::mma_commit(k_free + 8 * (buf));
            ptx::mma_commit(s_full + 8 * (sb));
          }
          __syncwarp();
        }
      }
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------- O += P . V
      const uint32_t id = ptx::idesc(0, 0, 128, 256, 0, 1);
      const uint32_t vb0 = ptx::smem_u32(VB), pb0 = ptx::smem_u32(PB);
      int g = 0;
      for (bool on = gtot > 0 && wk.start(a, job0, unit0, units); on && ok; on = wk.next(a)) {
        for (int k = wk.k0; k < wk.k1; ++k, ++g) {
          const int buf = g % kVBufs, pb = g % kPBufs;
          if (!ptx::mbar_wait(v_full + 8 * (buf), uint32_t(g / kVBufs) & 1u)) { ok = false; break; }
          if (!ptx::mbar_wait(o_ok + 8 * (pb), uint32_t(g / kPBufs) & 1u)) { ok = false; break; }
          ptx::tc_fence_after();
          const uint32_t vb = vb0 + buf * kVBuf, p = pb0 + pb * kPBuf;
          if (ptx::elect_one()) {
#pragma unroll 1
            for (int kk = 0; kk < kNT / 16; ++kk)
#pragma unroll
              for (int n = 0; n < 2; ++n)
                ptx::mma_f16(tmem + n * 256, ptx::sdesc_plain(p + kk * 2 * kPChunk, kPChunk, 128),
                             ptx::sdesc_sw128_mn(vb + n * 4 * kBlk + kk * 16 * 128, kBlk, 1024), id,
                             (k > wk.k0 || kk > 0) ? 1u : 0u);
            ptx::mma_commit(v_free + 8 * (buf));
            ptx::mma_commit_to(p_free + 8 * (pb), 1);  // CTA 0's barrier
          }
          __syncwarp();
        }
      }
    }
    if (warp == kMmaWarp) {
      // nothing of this warp's left in flight when the tensor memory is released
      if (ptx::elect_one()) ptx::mma_commit(mma_done);
      __syncwarp();
      ptx::mbar_wait(mma_done, 0);
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ converters
    const int w = warp - 8;
    if (half == 0) {
      // the job's query: each warp 32 heads of five or four K-blocks
      auto load_q = [&](int g, int job) {
        // every product with the old query is done
        if (g >= 1 && !ptx::mbar_wait(k_free + 8 * ((g - 1) % kKBufs), uint32_t((g - 1) / kKBufs) & 1u)) return false;
        const int row = (w & 3) * 32 + lane;
        const int hr = (job < a.tiles ? job * kPfxTileRows : (job - a.tiles) * kHeads) + row;
        const int heads = a.rows * kHeads;
        const bool in = hr < heads;
#pragma unroll 1
        for (int kb = w < 4 ? 0 : 5; kb < (w < 4 ? 5 : kKBlks); ++kb) {
          uint32_t v[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 x = in ? __ldg(a.q16 + size_t(kb * 8 + i) * heads + hr) : make_uint4(0, 0, 0, 0);
            v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
          }
          ptx::tmem_st32_u(tmem + (uint32_t((w & 3) * 32) << 16) + kb * 32, v);
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(q_full);
        return true;
      };
      ok = convert<kNv, true, kKBufs>(a, wk, gtot, job0, unit0, units, w, lane, KB, k_full, k_free, masks, mask_full, load_q);
    } else {
      ok = convert<kNv, false, kVBufs>(a, wk, gtot, job0, unit0, units, w, lane, VB, v_full, v_free, nullptr, 0,
                                       [](int, int) { return true; });
    }
  } else if (half == 0) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    const int group = warp >> 2, w = warp & 3;
    const int row = w * 32 + lane;
    const uint32_t lane_base = uint32_t(w * 32) << 16;
    const uint32_t p_peer = ptx::mapa_shared(ptx::smem_u32(PB) + row * 16, 1);
    const uint32_t f_peer = ptx::mapa_shared(ptx::smem_u32(factor + row), 1);
    const uint32_t bar_peer = ptx::mapa_shared(p_full, 1);
    int g0 = 0;  // the segment's first tile
    for (bool on = gtot > 0 && wk.start(a, job0, unit0, units); on && ok; on = wk.next(a)) {
      const int hr = (wk.job < a.tiles ? wk.job * kPfxTileRows : (wk.job - a.tiles) * kHeads) + row;
      const float cs = fmaxf(hr < a.rows * kHeads ? a.scale_log2 * a.qs[hr] : 1.f, 1.1754944e-38f);
      float m_mine = -INFINITY, l = 0.f;  // the maximum that l is relative to
      const int g1 = g0 + wk.k1 - wk.k0;
      for (int g = g0 + ((g0 ^ group) & 1); g < g1; g += 2) {
        const int sb = g % kSBufs, pb = g % kPBufs;
        if (!ptx::mbar_wait(s_full + 8 * (sb), uint32_t(g / kSBufs) & 1u)) { ok = false; break; }
        ptx::tc_fence_after();
        float sv[64];
        ptx::tmem_ld32_nowait(tmem + lane_base + kSCol + sb * kNT, *reinterpret_cast<float(*)[32]>(&sv[0]));
        ptx::tmem_ld32_nowait(tmem + lane_base + kSCol + sb * kNT + 32, *reinterpret_cast<float(*)[32]>(&sv[32]));
        if (!ptx::mbar_wait(mask_full + 8 * (g % kMasks), uint32_t(g / kMasks) & 1u)) ok = false;
        const unsigned long long vm = masks[g % kMasks];
        ptx::tmem_ld_wait(*reinterpret_cast<float(*)[32]>(&sv[0]));
        ptx::tmem_ld_wait(*reinterpret_cast<float(*)[32]>(&sv[32]));
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(s_free + 8 * (sb));
        if (!ok) break;
        if (vm != ~0ull) {
#pragma unroll
          for (int i = 0; i < 64; ++i) sv[i] = ((vm >> i) & 1ull) ? sv[i] : -INFINITY;
        }
        float t0 = fmaxf(sv[0], sv[1]), t1 = fmaxf(sv[2], sv[3]);
#pragma unroll
        for (int i = 4; i < 64; i += 4) {
          t0 = fmaxf(t0, fmaxf(sv[i], sv[i + 1]));
          t1 = fmaxf(t1, fmaxf(sv[i + 2], sv[i + 3]));
        }
        const float tmax = fmaxf(t0, t1) * cs;
        // the maximum in use passes from tile to tile
        if (g >= 1 && !ptx::mbar_wait(turn + 8 * (w), uint32_t(g - 1) & 1u)) { ok = false; break; }
        const float m_old = g == g0 ? -INFINITY : m_run[row];
        const bool raise = tmax > m_old + kLazy;
        const float m_use = m_old == -INFINITY || raise ? tmax : m_old;
        m_run[row] = m_use;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(turn + 8 * (w));
        const float alpha = raise && m_old != -INFINITY ? ptx::ex2_approx(m_old - m_use) : 1.f;
        if (m_mine != m_use && m_mine != -INFINITY) l *= ptx::ex2_approx(m_mine - m_use);
        m_mine = m_use;
        const float off = m_use == -INFINITY ? 0.f : kPShift - m_use;
        float p0 = 0.f, p1 = 0.f;
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          ptx::fma2(sv[2 * i], sv[2 * i + 1], cs, off);
          const float x = ptx::ex2_approx(sv[2 * i]), y = ptx::ex2_approx(sv[2 * i + 1]);
          ptx::add2(p0, p1, x, y);
          const __half2 h = __floats2half2_rn(x, y);
          pk[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        l += p0 + p1;
        // this half of P is free once P . V of two tiles ago is done
        if (g >= kPBufs && !ptx::mbar_wait_cluster(p_free + 8 * (pb), uint32_t(g / kPBufs - 1) & 1u)) { ok = false; break; }
        const uint32_t dst = p_peer + pb * kPBuf, bar = bar_peer + pb * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          ptx::st_async_f4(dst + i * kPChunk, make_float4(__uint_as_float(pk[4 * i]), __uint_as_float(pk[4 * i + 1]),
                                                          __uint_as_float(pk[4 * i + 2]), __uint_as_float(pk[4 * i + 3])),
                           bar);
        ptx::st_async_f1(f_peer + pb * 512, alpha, bar);
      }
      if (!ok) break;
      g0 = g1;
      float* ml = a.ml + (size_t(wk.job + clu) * 2 + group) * 256 + row;
      ml[0] = m_mine;
      ml[128] = l;
      if (threadIdx.x == 0) {
        if (wk.k0 == 0) a.plan[2 * wk.job] = clu;
        if (wk.k1 == wk.n) a.plan[2 * wk.job + 1] = clu;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    if (warp < 4) {
      // ---------------------------------------------------------- O: rescaling and output
      const int row = warp * 32 + lane;
      const uint32_t lane_base = uint32_t(warp * 32) << 16;
      int g = 0;
      for (bool on = gtot > 0 && wk.start(a, job0, unit0, units); on && ok; on = wk.next(a)) {
        for (int k = wk.k0; k < wk.k1; ++k, ++g) {
          const int pb = g % kPBufs;
          if (!ptx::mbar_wait_cluster(p_full + 8 * (pb), uint32_t(g / kPBufs) & 1u)) { ok = false; break; }
          const float alpha = factor[pb * 128 + row];
          // re-arm for tile g + 2: it is not sent before P . V of this tile, for which every
          // warp here has to arrive below
          if (threadIdx.x == 0 && g + kPBufs < gtot) ptx::mbar_arrive_expect_tx(p_full + 8 * (pb), kPBytes);
          if (k > wk.k0 && __any_sync(0xffffffffu, alpha != 1.f)) {
            if (!ptx::mbar_wait(v_free + 8 * ((g - 1) % kVBufs), uint32_t((g - 1) / kVBufs) & 1u)) { ok = false; break; }
            ptx::tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < kDNope; c += 32) {
              float o[32];
              ptx::tmem_ld32(tmem + lane_base + c, o);
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] *= alpha;
              ptx::tmem_st32(tmem + lane_base + c, o);
            }
          }
          // P came by ordinary (remote) stores; the tensor core reads it through the async proxy
          ptx::fence_proxy_async_smem();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(o_ok + 8 * (pb));
        }
        if (!ok) break;
        if (!ptx::mbar_wait(v_free + 8 * ((g - 1) % kVBufs), uint32_t((g - 1) / kVBufs) & 1u)) { ok = false; break; }
        ptx::tc_fence_after();
        float4* dst = reinterpret_cast<float4*>(a.part + (size_t(wk.job + clu) * kPfxTileRows + row) * kDNope);
        const bool real = wk.job < a.tiles || row < kHeads;
#pragma unroll 1
        for (int c = 0; c < kDNope; c += 32) {
          float o[32];
          ptx::tmem_ld32(tmem + lane_base + c, o);
          if (real) {
#pragma unroll
            for (int j = 0; j < 8; ++j) dst[c / 4 + j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          }
        }
        // the reads of O are ordered before the next job's first P . V (o_ok)
        ptx::tc_fence_before();
      }
    }
  }
  if (!ok) atomicOr(a.err, DSA_DEVERR_TIMEOUT);
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // no remote access to a CTA that has exited
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// The query as fp16: each head's 576 values times a power of two that takes its
// largest into [2^14, 2^15). A bf16 value has 8 significant bits, so what is
// above 2^-32 of the head's largest stays exact (fp16's subnormals are multiples
// of 2^-24). One warp per head. Written in chunks of 8 dims, head by head, so that
// 32 consecutive heads load 512 contiguous bytes into tensor memory wherever a
// tile of heads starts.
// ---------------------------------------------------------------------------
constexpr int kQueryWarps = 8;

__global__ void __launch_bounds__(32 * kQueryWarps)
    prefix_query_kernel(const uint32_t* __restrict__ q, int heads, uint32_t* __restrict__ q16, float* __restrict__ qs,
                        const int32_t* __restrict__ ctx, int32_t* __restrict__ lens, int n_q, int prefix, int cap,
                        int* err) {
  pdl_trigger();
  pdl_wait();
  // the rows' private tokens (a block has fewer rows' heads than threads)
  const int r = blockIdx.x * 32 * kQueryWarps + threadIdx.x;
  if (r < heads / kHeads) {
    const int b = r / n_q, c = ctx[b];
    const bool good = c >= prefix + n_q && c <= cap;
    if (!good) atomicOr(err, DSA_DEVERR_CTX);
    lens[r] = good ? c - n_q + (r - b * n_q) + 1 - prefix : 0;
  }
  const int hr = blockIdx.x * kQueryWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (hr >= heads) return;
  constexpr int kWords = kDQK / 2, kPer = kWords / 32;
  uint32_t w[kPer];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    w[i] = __ldg(q + size_t(hr) * kWords + i * 32 + lane);
    m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  // 2^-e in two factors: e reaches down to -147
  const int e = m > 0.f && m < INFINITY ? ilogbf(m) - 14 : 0;
  const float f0 = scalbnf(1.f, -e / 2), f1 = scalbnf(1.f, -e - (-e / 2));
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const __half2 h = __floats2half2_rn(__uint_as_float(w[i] << 16) * f0 * f1, __uint_as_float(w[i] & 0xFFFF0000u) * f0 * f1);
    const int word = i * 32 + lane;
    q16[(size_t(word >> 2) * heads + hr) * 4 + (word & 3)] = *reinterpret_cast<const uint32_t*>(&h);
  }
  if (lane == 0) qs[hr] = scalbnf(1.f, e);
}

// ---------------------------------------------------------------------------
// Merge of a row's segments, those of its prefix tile and then those of its private
// job: with M the largest maximum, out = lat_scale * sum_i 2^(m_i - M) O_i / L and
// L = sum_i 2^(m_i - M) l_i (a segment's two softmax groups have sums of their own;
// its O is relative to the larger of their maxima). One CTA per (row, 3 heads),
// 128 threads per head, 4 dims each.
// ---------------------------------------------------------------------------
constexpr int kMergeHeads = 3;

__global__ void __launch_bounds__(128 * kMergeHeads) prefix_merge_kernel(PfxArgs a, __nv_bfloat16* __restrict__ out,
                                                                        float* __restrict__ lse) {
  pdl_wait();
  const int r = blockIdx.x, h = blockIdx.y * kMergeHeads + (threadIdx.x >> 7), d4 = threadIdx.x & 127;
  const int hr = r * kHeads + h, job0 = hr / kPfxTileRows, job1 = a.tiles + r;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float L = -INFINITY;
  if (a.lens[r] > 0) {
    const int c0 = a.prefix > 0 ? a.plan[2 * job0] : 0, n0 = a.prefix > 0 ? a.plan[2 * job0 + 1] - c0 + 1 : 0;
    const int c1 = a.plan[2 * job1], n1 = a.plan[2 * job1 + 1] - c1 + 1;
    // segment i's slot and row
    auto slot = [&](int i) { return i < n0 ? job0 + c0 + i : job1 + c1 + i - n0; };
    auto row = [&](int i) { return i < n0 ? hr % kPfxTileRows : h; };
    float m = -INFINITY;
    for (int i = 0; i < n0 + n1; ++i) {
      const float* ml = a.ml + size_t(slot(i)) * 512 + row(i);
      m = fmaxf(m, fmaxf(__ldg(ml), __ldg(ml + 256)));
    }
    const float mm = m == -INFINITY ? 0.f : m;
    float tot = 0.f;
#pragma unroll 4
    for (int i = 0; i < n0 + n1; ++i) {
      const float* ml = a.ml + size_t(slot(i)) * 512 + row(i);
      const float ma = __ldg(ml), mb = __ldg(ml + 256);
      const float w = exp2f(fmaxf(ma, mb) - mm);
      tot = fmaf(exp2f(ma - mm), __ldg(ml + 128), tot);
      tot = fmaf(exp2f(mb - mm), __ldg(ml + 384), tot);
      const float4 v = __ldg(reinterpret_cast<const float4*>(a.part + (size_t(slot(i)) * kPfxTileRows + row(i)) * kDNope) + d4);
      acc.x = fmaf(w, v.x, acc.x); acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z); acc.w = fmaf(w, v.w, acc.w);
    }
    if (tot != 0.f) {  // NaN stays NaN
      const float inv = a.lat_scale / tot;
      acc.x *= inv; acc.y *= inv; acc.z *= inv; acc.w *= inv;
      L = (mm - kPShift + log2f(tot)) * 0.6931471805599453f;
    } else {
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  const __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y), hi = __floats2bfloat162_rn(acc.z, acc.w);
  uint2 pk;
  pk.x = *reinterpret_cast<const uint32_t*>(&lo);
  pk.y = *reinterpret_cast<const uint32_t*>(&hi);
  *reinterpret_cast<uint2*>(out + size_t(hr) * kDNope + 4 * d4) = pk;
  if (lse && d4 == 0) lse[hr] = L;
}

}  // namespace

cudaError_t launch_prefix_mla(const dsa_params_t& p, const WsLayout& L, char* ws, const void* q, const void* lat_pool,
                              const int32_t* prefix_pages, int prefix_len, const int32_t* block_table,
                              const int32_t* ctx_lens, void* out, float* lse, cudaStream_t st) {
  PfxArgs a;
  a.q16 = reinterpret_cast<const uint4*>(ws + L.pfx_q);
  a.qs = reinterpret_cast<const float*>(ws + L.pfx_qs);
  a.lat = static_cast<const uint8_t*>(lat_pool);
  a.prefix_pages = prefix_pages;
  a.table = block_table;
  int32_t* lens = reinterpret_cast<int32_t*>(ws + L.pfx_len);
  a.lens = lens;
  a.plan = reinterpret_cast<int32_t*>(ws + L.pfx_plan);
  a.ml = reinterpret_cast<float*>(ws + L.pfx_ml);
  a.part = reinterpret_cast<float*>(ws + L.pfx_part);
  a.err = reinterpret_cast<int*>(ws + L.err);
  a.stride = p.lat_page_stride;
  a.prefix = prefix_len;
  a.n_q = p.n_q;
  a.rows = L.rows;
  a.max_pages = p.max_pages_per_req;
  a.num_pages = p.num_pages;
  a.tiles = prefix_len > 0 ? L.pfx_tiles : 0;
  a.scale_log2 = p.softmax_scale * p.latent_scale * 1.4426950408889634f;
  a.lat_scale = p.latent_scale;
  const int heads = L.rows * kHeads;
  cudaError_t e = launch_pdl(prefix_query_kernel, dim3((heads + kQueryWarps - 1) / kQueryWarps), dim3(32 * kQueryWarps), 0,
                             st, static_cast<const uint32_t*>(q), heads, reinterpret_cast<uint32_t*>(ws + L.pfx_q),
                             reinterpret_cast<float*>(ws + L.pfx_qs), ctx_lens, lens, int(p.n_q), prefix_len, L.cap, a.err);
  if (e != cudaSuccess) return e;
  auto kern = p.lat_fmt == DSA_LAT_NVFP4_352 ? prefix_mla_kernel<true> : prefix_mla_kernel<false>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
  if (e != cudaSuccess) return e;
  const int clusters = std::max(1, std::min(kPfxMaxClusters, sm_count() / 2));
  e = launch_pdl(kern, dim3(2 * clusters), dim3(kThreads), kSmem, st, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(prefix_merge_kernel, dim3(L.rows, kHeads / kMergeHeads), dim3(128 * kMergeHeads), 0, st, a,
                    static_cast<__nv_bfloat16*>(out), lse);
}

}  // namespace dsa
