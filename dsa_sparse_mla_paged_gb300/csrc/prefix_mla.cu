// Dense attention of a batch that shares a prefix: out = softmax(scale q C^T) C[:, 0:512]
// of every (row, head) over the shared tokens and the request's own ones.
//
// Work is a line of 64-token tiles. First come the prefix jobs: 128 query heads
// (row * 96 + head, so rows pack without padding) against the whole prefix, the
// latents being the same for all of them. Then the private jobs: one row's 96 heads
// against the request's tokens past the prefix that the row may see (a job per row,
// so that a token hidden from a row never enters its products, whatever it holds).
// The line is cut into equal runs, one per CTA pair, and a run into segments at job
// borders; each segment leaves a normalised partial output and its log-sum-exp, and
// the combine kernel merges the segments of a row's two jobs.
//
// The products take fp16 operands and fp32 sums. E4M3 and E2M1 x E4M3 values are exact
// in fp16 (one conversion instruction for two values; to bf16 it takes four). The
// query becomes fp16 with a power of two per head, which leaves every value exact
// down to 2^-32 of the head's largest (query_kernel). Softmax weights are scaled to
// at most 2^7 (2^15 until the running maximum is raised), so that fp16 holds them
// to 11 bits down to 2^-21 of the maximum.
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
// The tile pipeline of a CTA pair. A 128 x 512 fp32 output fills the tensor memory,
// so the pair splits the latent's dims: CTA c owns nope [256c, 256c + 256) (its half
// of the output) and rope [32c, 32c + 32). Each CTA multiplies its own 288 dims,
// S_c = Q[:, own] . C[:, own]^T, sends its partial scores to the peer through
// distributed shared memory, and both add the two parts (the same IEEE sum on
// either side), run the same softmax and finish their halves of O += P . V.
//   warps 0..3   softmax and epilogue, one query head per thread
//   warps 4..7   exchange: read S_c and store it into the peer's shared memory, ahead
//                of the softmax; at a new job load Q
//   warps 8..11  converters: a tile is one page; each CTA expands its dims of the
//                page's 64 rows to fp16 (128-B swizzled K-blocks of 64 dims)
//   warp  12     tensor memory, MMA issue: S of tile g + 1 goes before P . V of tile g
// Tensor memory: O 256 columns, Q's first three K-blocks 96, S 2 x 64, P 32. The
// query's fourth K-block and its rope dims are read from shared memory: keeping
// three in tensor memory saves their 16 KB each of shared-memory reads per tile.
// The latent tile serves as K (K-major) and as V (MN-major) from one copy.
// ---------------------------------------------------------------------------
constexpr int kNT = 64;                      // tokens per tile: one page
constexpr int kLBlk = kNT * 128;             // 8,192 B: 64 rows of 64 fp16
constexpr int kLRope = kNT * 64;             // 4,096 B: 64 rows of 32 fp16
constexpr int kLatBuf = 4 * kLBlk + kLRope;  // 36,864
constexpr int kLatBufs = 3;
constexpr int kQBlk = 128 * 128;             // 16,384 B: the fourth K-block of 128 heads
constexpr int kQRope = 128 * 64;             // 8,192
constexpr int kXRow = 64 * 4 + 16;           // a row of partial scores (+16 B against bank conflicts)
constexpr int kXBuf = 128 * kXRow;           // 34,816
constexpr uint32_t kXBytes = 128 * 64 * 4;   // score bytes the peer sends per tile
constexpr int kStage = 32 * 128;             // one softmax warp's 32 x 32 fp32 output tile
constexpr int kThreads = 416;
constexpr uint32_t kQCol = 256, kSCol = 352, kPCol = 480;
constexpr int kNumBars = 24;
constexpr size_t kSmem = 1024 + kLatBufs * kLatBuf + kQBlk + kQRope + 2 * kXBuf + 4 * kStage + kLatBufs * 8 +
                         kNumBars * 8 + 16;
static_assert(kSmem <= 232448, "shared memory of one CTA");
static_assert(kLatBuf % 1024 == 0 && kXBuf % 1024 == 0, "swizzle atoms stay 1,024-B aligned");
constexpr float kPShift = 7.f;               // weights are 2^(z - max + 7)
constexpr float kLazy = 8.f;                 // the maximum in use is raised when passed by more than 2^8

struct PfxArgs {
  const __half* q16;
  const float* qs;
  const uint8_t* lat;
  const int32_t* prefix_pages;
  const int32_t* table;
  const int32_t* ctx;
  int32_t* plan;    // [jobs][2] first and last CTA pair of a job
  float* part_lse;  // [slots][128]
  int* err;
  int64_t stride;
  int prefix, n_q, rows, max_pages, num_pages, cap, tiles;  // tiles: prefix jobs
  float scale_log2, lat_scale;
};

// Private tokens that row r sees (0 for an invalid context length).
__device__ __forceinline__ int private_len(const PfxArgs& a, int r) {
  const int b = r / a.n_q, t = r - b * a.n_q;
  const int c = a.ctx[b];
  return c < a.prefix + a.n_q || c > a.cap ? 0 : c - a.n_q + t + 1 - a.prefix;
}

__device__ __forceinline__ int job_tiles(const PfxArgs& a, int job) {
  return job < a.tiles ? a.prefix / kNT : (private_len(a, job - a.tiles) + kNT - 1) / kNT;
}

// A CTA pair's run of the line, segment by segment.
struct Walk {
  int job, k0, k1;  // the current segment: tiles [k0, k1) of the job
  int64_t left;     // tiles of the run after it
  __device__ __forceinline__ bool start(const PfxArgs& a, int job0, int first, int64_t n) {
    job = job0;
    k0 = first;
    left = n;
    return n > 0 && take(a);
  }
  __device__ __forceinline__ bool take(const PfxArgs& a) {
    const int len = job_tiles(a, job);
    k1 = int(min(int64_t(len), k0 + left));
    left -= k1 - k0;
    return true;
  }
  __device__ __forceinline__ bool next(const PfxArgs& a) {
    if (left <= 0) return false;
    do {  // left > 0: a job with tiles follows
      if (++job >= a.tiles + a.rows) return false;
    } while (job_tiles(a, job) == 0);
    k0 = 0;
    return take(a);
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

// One converter thread's share of a tile: FP8: eight 16-B pieces of K-block w (8
// tokens x 4 pieces per warp load: 64-B runs, and stores without bank conflicts)
// and one of the rope dims; NVFP4: four 16-B units (32 values, two scales) and the
// rope piece. Tokens at or past `valid` are zeros.
template <bool kNv>
struct TileRegs {
  uint4 v[kNv ? 4 : 8];
  uint32_t s[kNv ? 4 : 1];
  uint4 rope;
  __device__ __forceinline__ void load(const uint8_t* page, int valid, int w, int lane, int half) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const int ct = w * 32 + lane;
    if constexpr (kNv) {
      const int unit = 2 * w + (lane & 1);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int tok = u * 16 + (lane >> 1);
        const uint8_t* row = page + tok * 352;
        v[u] = tok < valid ? __ldg(reinterpret_cast<const uint4*>(row + 128 * half + 16 * unit)) : zero;
        s[u] = tok < valid ? __ldg(reinterpret_cast<const uint16_t*>(row + 256 + 16 * half + 2 * unit)) : 0;
      }
      const int tok = ct >> 1;
      rope = tok < valid ? __ldg(reinterpret_cast<const uint4*>(page + tok * 352 + 288 + 32 * half + 16 * (ct & 1))) : zero;
    } else {
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int tok = u * 8 + (lane >> 2);
        v[u] = tok < valid
                   ? __ldg(reinterpret_cast<const uint4*>(page + tok * 576 + 256 * half + 64 * w + 16 * (lane & 3)))
                   : zero;
      }
      const int tok = ct >> 1;
      rope = tok < valid ? __ldg(reinterpret_cast<const uint4*>(page + tok * 576 + 512 + 32 * half + 16 * (ct & 1))) : zero;
    }
  }
  __device__ __forceinline__ void store(uint8_t* buf, int w, int lane) const {
    uint8_t* blk = buf + w * kLBlk;
    uint4 lo, hi;
    if constexpr (kNv) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int tok = u * 16 + (lane >> 1), c0 = (lane & 1) * 4;
        uint8_t* row = blk + tok * 128;
        const uint32_t two = half2_from_e4m3x2(s[u]);
        const __half2 h = *reinterpret_cast<const __half2*>(&two);
        const __half2 s0 = __low2half2(h), s1 = __high2half2(h);
        *reinterpret_cast<uint4*>(row + (((c0 + 0) ^ (tok & 7)) << 4)) = expand_e2m1(v[u].x, s0);
        *reinterpret_cast<uint4*>(row + (((c0 + 1) ^ (tok & 7)) << 4)) = expand_e2m1(v[u].y, s0);
        *reinterpret_cast<uint4*>(row + (((c0 + 2) ^ (tok & 7)) << 4)) = expand_e2m1(v[u].z, s1);
        *reinterpret_cast<uint4*>(row + (((c0 + 3) ^ (tok & 7)) << 4)) = expand_e2m1(v[u].w, s1);
      }
    } else {
      const int c = (lane & 3) * 2;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int tok = u * 8 + (lane >> 2);
        uint8_t* row = blk + tok * 128;
        expand16(v[u], lo, hi);
        *reinterpret_cast<uint4*>(row + ((c ^ (tok & 7)) << 4)) = lo;
        *reinterpret_cast<uint4*>(row + (((c + 1) ^ (tok & 7)) << 4)) = hi;
      }
    }
    const int ct = w * 32 + lane, tok = ct >> 1, c = (ct & 1) * 2;
    uint8_t* row = buf + 4 * kLBlk + tok * 64;  // 64-B swizzle
    expand16(rope, lo, hi);
    *reinterpret_cast<uint4*>(row + ((c ^ ((tok >> 1) & 3)) << 4)) = lo;
    *reinterpret_cast<uint4*>(row + (((c + 1) ^ ((tok >> 1) & 3)) << 4)) = hi;
  }
};

template <bool kNv>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    prefix_mla_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap rmap,
                      const __grid_constant__ CUtensorMap omap, const __grid_constant__ PfxArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* LAT = sm;
  uint8_t* Qs = LAT + kLatBufs * kLatBuf;
  uint8_t* Qr = Qs + kQBlk;
  uint8_t* X = Qr + kQRope;                            // the peer's partial scores, 2 buffers
  uint8_t* ST = X + 2 * kXBuf;                         // output staging, a tile per softmax warp
  unsigned long long* vmask = reinterpret_cast<unsigned long long*>(ST + 4 * kStage);  // [kLatBufs] valid tokens
  uint64_t* bars = reinterpret_cast<uint64_t*>(vmask + kLatBufs);
  uint64_t* q_full = bars + 0;
  uint64_t* p_full = bars + 1;
  uint64_t* mma_done = bars + 2;
  uint64_t* lat_full = bars + 3;   // [3]
  uint64_t* lat_free = bars + 6;   // [3]  P . V of the buffer's tile is done
  uint64_t* s_full = bars + 9;     // [2]
  uint64_t* s_free = bars + 11;    // [2]  the softmax and the exchange have read S
  uint64_t* x_full = bars + 13;    // [2]  the peer's scores have landed
  uint64_t* x_free = bars + 15;    // [2]  the peer's softmax has read what this CTA sent
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  __shared__ long long s_sum[kThreads / 32];
  __shared__ int s_job, s_first;

  const int half = int(ptx::cluster_ctarank()), peer = half ^ 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nclu = int(gridDim.x) >> 1, clu = int(blockIdx.x) >> 1;

  if (threadIdx.x == 0) {
    ptx::mbar_init(q_full, 5);
    ptx::mbar_init(p_full, 4);
    ptx::mbar_init(mma_done, 1);
    for (int i = 0; i < kLatBufs; ++i) {
      ptx::mbar_init(lat_full + i, 4);
      ptx::mbar_init(lat_free + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(s_full + i, 1);
      ptx::mbar_init(s_free + i, 8);
      ptx::mbar_init(x_full + i, 1);
      ptx::mbar_init(x_free + i, 4);
    }
    ptx::fence_mbar_init();
  }
  if (warp == 12) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait();

  // ---- the line's length, this pair's run of it and the job that the run starts in
  int64_t run, line;
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
    long long mine = 0;
    for (int r = threadIdx.x; r < a.rows; r += kThreads) mine += job_tiles(a, a.tiles + r);
    const int64_t shared = int64_t(a.tiles) * (a.prefix / kNT);
    line = shared + block_sum(mine);
    // no pair between two that work goes without a tile: a job's segments are those
    // of consecutive pairs
    const int64_t used = min(int64_t(nclu), line);
    const int64_t lo = clu < used ? line * clu / used : line;
    run = clu < used ? line * (clu + 1) / used - lo : 0;
    if (lo < shared) {
      if (threadIdx.x == 0) {
        s_job = int(lo / (a.prefix / kNT));
        s_first = int(lo % (a.prefix / kNT));
      }
    } else if (run > 0) {
      int64_t base = shared;
      for (int r0 = 0; r0 < a.rows; r0 += kThreads) {
        const int r = r0 + int(threadIdx.x);
        const long long n = r < a.rows ? job_tiles(a, a.tiles + r) : 0;
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
        if (n > 0 && lo >= before && lo < before + n) {
          s_job = a.tiles + r;
          s_first = int(lo - before);
        }
        base += all;
        if (base > lo) break;
      }
    }
    // the peer's first two score tiles may arrive as soon as the pair has synced
    if (threadIdx.x == 0) {
      if (run > 0) ptx::mbar_arrive_expect_tx(x_full + 0, kXBytes);
      if (run > 1) ptx::mbar_arrive_expect_tx(x_full + 1, kXBytes);
    }
    if (clu == 0 && half == 0)
      for (int b = threadIdx.x; b < a.rows / a.n_q; b += kThreads)
        if (private_len(a, b * a.n_q) == 0) atomicOr(a.err, DSA_DEVERR_CTX);
  }
  __syncthreads();
  ptx::cluster_sync();  // the peer's barriers exist before any remote arrive
  const int gtot = int(run);
  bool ok = true;
  Walk wk;

  if (warp == 12) {
    // ------------------------------------------------------------ MMA issuer
    const uint32_t id_qk = ptx::idesc(0, 0, 128, kNT);
    const uint32_t id_pv = ptx::idesc(0, 0, 128, 256, 0, 1);
    const uint32_t q0 = ptx::smem_u32(Qs), r0 = ptx::smem_u32(Qr), l0 = ptx::smem_u32(LAT);
    int g = 0, qn = 0;
    bool fresh = true;  // the next P . V starts a segment
    auto pv = [&](int j) {
      if (!ok || !ptx::mbar_wait(p_full, uint32_t(j) & 1u)) { ok = false; return; }
      ptx::tc_fence_after();
      const int buf = j % kLatBufs;
      const uint32_t lat = l0 + buf * kLatBuf;
      if (ptx::elect_one()) {
#pragma unroll
        for (int kk = 0; kk < kNT / 16; ++kk)
          ptx::mma_f16_tmem_a(tmem, tmem + kPCol + kk * 8, ptx::sdesc_sw128_mn(lat + kk * 16 * 128, kLBlk, 1024), id_pv,
                              (!fresh || kk > 0) ? 1u : 0u);
        ptx::mma_commit(lat_free + buf);
      }
      __syncwarp();
      fresh = false;
    };
    for (bool on = gtot > 0 && wk.start(a, s_job, s_first, run); on && ok; on = wk.next(a)) {
      for (int k = wk.k0; k < wk.k1 && ok; ++k, ++g) {
        if (k == wk.k0) {
          // the last P . V of the old segment goes before the wait for a new query
          if (g >= 1) pv(g - 1);
          fresh = true;
          if (!ok || !ptx::mbar_wait(q_full, uint32_t(qn++) & 1u)) { ok = false; break; }
        }
        const int buf = g % kLatBufs, sb = g & 1;
        if (!ptx::mbar_wait(lat_full + buf, uint32_t(g / kLatBufs) & 1u)) { ok = false; break; }
        if (g >= 2 && !ptx::mbar_wait(s_free + sb, uint32_t((g >> 1) - 1) & 1u)) { ok = false; break; }
        ptx::tc_fence_after();
        const uint32_t lat = l0 + buf * kLatBuf, s = tmem + kSCol + sb * kNT;
        if (ptx::elect_one()) {
#pragma unroll
          for (int kb = 0; kb < 3; ++kb)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              ptx::mma_f16_tmem_a(s, tmem + kQCol + kb * 32 + kk * 8, ptx::sdesc_sw128(lat + kb * kLBlk + kk * 32), id_qk,
                                  (kb | kk) ? 1u : 0u);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            ptx::mma_f16(s, ptx::sdesc_sw128(q0 + kk * 32), ptx::sdesc_sw128(lat + 3 * kLBlk + kk * 32), id_qk, 1u);
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
            ptx::mma_f16(s, ptx::sdesc_sw64(r0 + kk * 32), ptx::sdesc_sw64(lat + 4 * kLBlk + kk * 32), id_qk, 1u);
          ptx::mma_commit(s_full + sb);
        }
        __syncwarp();
        if (k > wk.k0) pv(g - 1);
      }
    }
    if (ok && g >= 1) pv(g - 1);
    // nothing of this warp's left in flight when the tensor memory is released
    if (ptx::elect_one()) ptx::mma_commit(mma_done);
    __syncwarp();
    ptx::mbar_wait(mma_done, 0);
  } else if (warp >= 8) {
    // ------------------------------------------------------------ converters
    const int w = warp - 8;
    TileRegs<kNv> cur, nxt;
    int g = 0;
    // page of tile k of the walk's job: its address (null for a bad entry) and its visible tokens
    auto tile = [&](const Walk& at, int k, int& valid) -> const uint8_t* {
      int pg;
      if (at.job < a.tiles) {
        pg = __ldg(a.prefix_pages + k);
        valid = kNT;
      } else {
        const int r = at.job - a.tiles;
        pg = __ldg(a.table + size_t(r / a.n_q) * a.max_pages + a.prefix / kNT + k);
        valid = min(kNT, private_len(a, r) - k * kNT);
      }
      if (pg < 0 || pg >= a.num_pages) {
        if (half == 0 && w == 0 && lane == 0) atomicOr(a.err, DSA_DEVERR_BLOCK_TABLE);
        valid = 0;
        return a.lat;
      }
      return a.lat + int64_t(pg) * a.stride;
    };
    if (gtot > 0) {
      wk.start(a, s_job, s_first, run);
      int k = wk.k0, valid, valid_next = 0, valid2 = 0;
      const uint8_t* page = tile(wk, k, valid);
      cur.load(page, valid, w, lane, half);
      // the address of the tile after the next is resolved one tile ahead of its loads
      auto advance = [&]() -> bool {
        if (++k < wk.k1) return true;
        if (!wk.next(a)) return false;
        k = wk.k0;
        return true;
      };
      bool more = advance();
      const uint8_t* page2 = more ? tile(wk, k, valid2) : a.lat;
#pragma unroll 1
      for (; g < gtot && ok; ++g) {
        if (g + 1 < gtot) {
          valid_next = valid2;
          nxt.load(page2, valid_next, w, lane, half);
          more = more && advance();
          if (more) page2 = tile(wk, k, valid2);
        }
        const int buf = g % kLatBufs;
        if (g >= kLatBufs && !ptx::mbar_wait(lat_free + buf, uint32_t(g / kLatBufs - 1) & 1u)) { ok = false; break; }
        cur.store(LAT + buf * kLatBuf, w, lane);
        if (w == 0 && lane == 0) vmask[buf] = valid >= 64 ? ~0ull : (1ull << valid) - 1;
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(lat_full + buf);
        cur = nxt;
        valid = valid_next;
      }
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ exchange and Q
    const int row = (warp - 4) * 32 + lane;
    const uint32_t lane_base = uint32_t((warp - 4) * 32) << 16;
    const uint32_t x_peer = ptx::mapa_shared(ptx::smem_u32(X) + row * kXRow, peer);
    const uint32_t bar_peer = ptx::mapa_shared(ptx::smem_u32(x_full), peer);
    int g = 0, qn = 0;
    for (bool on = gtot > 0 && wk.start(a, s_job, s_first, run); on && ok; on = wk.next(a)) {
      // every product with the old query is done: S of the last tile was complete
      const int hr0 = wk.job < a.tiles ? wk.job * kPfxTileRows : (wk.job - a.tiles) * kHeads;
      if (warp == 4 && lane == 0) {
        ptx::mbar_arrive_expect_tx(q_full, kQBlk + kQRope);
        ptx::tma_load_2d(Qs, &qmap, q_full, 256 * half + 192, hr0);
        ptx::tma_load_2d(Qr, &rmap, q_full, kDNope + 32 * half, hr0);
      }
      __syncwarp();
      {
        const int hr = hr0 + row;
        const uint4* src = reinterpret_cast<const uint4*>(a.q16 + size_t(hr) * kDQK + 256 * half);
        uint32_t v[3][32];
#pragma unroll
        for (int kb = 0; kb < 3; ++kb)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 x = hr < a.rows * kHeads ? src[kb * 8 + i] : make_uint4(0, 0, 0, 0);
            v[kb][4 * i] = x.x; v[kb][4 * i + 1] = x.y; v[kb][4 * i + 2] = x.z; v[kb][4 * i + 3] = x.w;
          }
#pragma unroll
        for (int kb = 0; kb < 3; ++kb) ptx::tmem_st32_u(tmem + lane_base + kQCol + kb * 32, v[kb]);
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(q_full);
        ++qn;
      }
      for (int k = wk.k0; k < wk.k1; ++k, ++g) {
        const int sb = g & 1;
        const uint32_t ph = uint32_t(g >> 1) & 1u;
        if (!ptx::mbar_wait(s_full + sb, ph)) { ok = false; break; }
        ptx::tc_fence_after();
        float sa[32], sc[32];
        ptx::tmem_ld32_nowait(tmem + lane_base + kSCol + sb * kNT, sa);
        ptx::tmem_ld32_nowait(tmem + lane_base + kSCol + sb * kNT + 32, sc);
        ptx::tmem_ld_wait(sa);
        ptx::tmem_ld_wait(sc);
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(s_free + sb);
        if (g >= 2 && !ptx::mbar_wait_cluster(x_free + sb, ph ^ 1u)) { ok = false; break; }
        const uint32_t dst = x_peer + sb * kXBuf, bar = bar_peer + sb * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i)
          ptx::st_async_f4(dst + i * 16, make_float4(sa[4 * i], sa[4 * i + 1], sa[4 * i + 2], sa[4 * i + 3]), bar);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          ptx::st_async_f4(dst + 128 + i * 16, make_float4(sc[4 * i], sc[4 * i + 1], sc[4 * i + 2], sc[4 * i + 3]), bar);
      }
    }
    if (!ok && qn > 0) ptx::mbar_wait(q_full, uint32_t(qn - 1) & 1u);  // no copy left in flight
  } else {
    // ------------------------------------------------------------ softmax and epilogue
    const int row = warp * 32 + lane;
    const uint32_t lane_base = uint32_t(warp * 32) << 16;
    const uint32_t free_peer = ptx::mapa_shared(ptx::smem_u32(x_free), peer);
    uint8_t* stg = ST + warp * kStage;
    int g = 0;
    for (bool on = gtot > 0 && wk.start(a, s_job, s_first, run); on && ok; on = wk.next(a)) {
      const bool shared = wk.job < a.tiles;
      const int hr = (shared ? wk.job * kPfxTileRows : (wk.job - a.tiles) * kHeads) + row;
      const float cs = fmaxf(hr < a.rows * kHeads ? a.scale_log2 * a.qs[hr] : 1.f, 1.1754944e-38f);
      float m_use = -INFINITY, l = 0.f;
      for (int k = wk.k0; k < wk.k1; ++k, ++g) {
        const int sb = g & 1, buf = g % kLatBufs;
        const uint32_t ph = uint32_t(g >> 1) & 1u;
        // lat_full orders the converters' mask before its read
        if (!ptx::mbar_wait(lat_full + buf, uint32_t(g / kLatBufs) & 1u) || !ptx::mbar_wait(s_full + sb, ph)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        float sv[64];
        ptx::tmem_ld32_nowait(tmem + lane_base + kSCol + sb * kNT, *reinterpret_cast<float(*)[32]>(&sv[0]));
        ptx::tmem_ld32_nowait(tmem + lane_base + kSCol + sb * kNT + 32, *reinterpret_cast<float(*)[32]>(&sv[32]));
        ptx::tmem_ld_wait(*reinterpret_cast<float(*)[32]>(&sv[0]));
        ptx::tmem_ld_wait(*reinterpret_cast<float(*)[32]>(&sv[32]));
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(s_free + sb);
        if (!ptx::mbar_wait_cluster(x_full + sb, ph)) { ok = false; break; }
        const float4* xr = reinterpret_cast<const float4*>(X + sb * kXBuf + row * kXRow);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float4 x = xr[i];
          sv[4 * i] += x.x; sv[4 * i + 1] += x.y; sv[4 * i + 2] += x.z; sv[4 * i + 3] += x.w;
        }
        // re-arm for tile g + 2 (its bytes are not sent before all four warps have
        // arrived on the peer's x_free)
        if (warp == 0 && lane == 0 && g + 2 < gtot) ptx::mbar_arrive_expect_tx(x_full + sb, kXBytes);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_remote(free_peer + sb * 8);
        const unsigned long long vm = vmask[buf];
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
        bool raise = false;
        float alpha = 1.f;
        if (m_use == -INFINITY) {
          m_use = tmax;
        } else if (tmax > m_use + kLazy) {
          raise = true;
          alpha = ptx::ex2_approx(m_use - tmax);
          m_use = tmax;
        }
        const float off = m_use == -INFINITY ? 0.f : kPShift - m_use;
        float p0 = 0.f, p1 = 0.f;
        uint32_t pk[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          const float x = ptx::ex2_approx(fmaf(sv[2 * i], cs, off));
          const float y = ptx::ex2_approx(fmaf(sv[2 * i + 1], cs, off));
          p0 += x;
          p1 += y;
          const __half2 h = __floats2half2_rn(x, y);
          pk[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        // P and O are free once the previous tile's P . V is done
        if (g >= 1 && !ptx::mbar_wait(lat_free + (g - 1) % kLatBufs, uint32_t((g - 1) / kLatBufs) & 1u)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        if (__any_sync(0xffffffffu, raise)) {
          l *= alpha;
#pragma unroll 1
          for (int c = 0; c < 256; c += 32) {
            float o[32];
            ptx::tmem_ld32(tmem + lane_base + c, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= alpha;
            ptx::tmem_st32(tmem + lane_base + c, o);
          }
        }
        l += p0 + p1;
        ptx::tmem_st32_u(tmem + lane_base + kPCol, pk);
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(p_full);
      }
      if (!ok) break;
      // ---- the segment's output: O / l of this head's half
      const int gl = g - 1;
      if (!ptx::mbar_wait(lat_free + gl % kLatBufs, uint32_t(gl / kLatBufs) & 1u)) { ok = false; break; }
      ptx::tc_fence_after();
      const int slot = wk.job + clu;
      const float inv = l == 0.f ? 0.f : a.lat_scale / l;  // NaN stays NaN
#pragma unroll 1
      for (int c = 0; c < 256; c += 32) {
        float o[32];
        ptx::tmem_ld32(tmem + lane_base + c, o);
        if (lane == 0) ptx::bulk_wait_read();
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          *reinterpret_cast<float4*>(stg + lane * 128 + ((j ^ (lane & 7)) << 4)) =
              make_float4(o[4 * j] * inv, o[4 * j + 1] * inv, o[4 * j + 2] * inv, o[4 * j + 3] * inv);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          ptx::tma_store_2d(&omap, stg, half * 256 + c, slot * kPfxTileRows + warp * 32);
          ptx::bulk_commit();
        }
      }
      if (half == 0) {
        a.part_lse[size_t(slot) * kPfxTileRows + row] =
            l == 0.f ? -INFINITY : (m_use - kPShift + log2f(l)) * 0.6931471805599453f;
        if (threadIdx.x == 0) {
          if (wk.k0 == 0) a.plan[2 * wk.job] = clu;
          if (wk.k1 == job_tiles(a, wk.job)) a.plan[2 * wk.job + 1] = clu;
        }
      }
      // the reads of O are ordered before the next segment's first P . V (p_full)
      ptx::tc_fence_before();
    }
    if (lane == 0) ptx::bulk_wait_all();
  }
  if (!ok) atomicOr(a.err, DSA_DEVERR_TIMEOUT);
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();  // no remote access to a CTA that has exited
  if (warp == 12) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// The query as fp16: each head's 576 values times a power of two that takes its
// largest into [2^14, 2^15). A bf16 value has 8 significant bits, so what is
// above 2^-32 of the head's largest stays exact (fp16's subnormals are multiples
// of 2^-24). One warp per head.
// ---------------------------------------------------------------------------
constexpr int kQueryWarps = 8;

__global__ void __launch_bounds__(32 * kQueryWarps) prefix_query_kernel(const uint32_t* __restrict__ q, int heads,
                                                                       uint32_t* __restrict__ q16,
                                                                       float* __restrict__ qs) {
  pdl_trigger();
  pdl_wait();
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
    q16[size_t(hr) * kWords + i * 32 + lane] = *reinterpret_cast<const uint32_t*>(&h);
  }
  if (lane == 0) qs[hr] = scalbnf(1.f, e);
}

// ---------------------------------------------------------------------------
// Merge of a row's segments: out = sum_i e^{lse_i - lse} O_i, lse = ln sum_i e^{lse_i},
// over the segments of the row's prefix tile and of its private job, in that order.
// One CTA per (row, 3 heads), 128 threads per head, 4 dims each.
// ---------------------------------------------------------------------------
constexpr int kMergeHeads = 3;

__global__ void __launch_bounds__(128 * kMergeHeads) prefix_merge_kernel(PfxArgs a, const float* __restrict__ part,
                                                                        __nv_bfloat16* __restrict__ out,
                                                                        float* __restrict__ lse) {
  pdl_wait();
  const int r = blockIdx.x, h = blockIdx.y * kMergeHeads + (threadIdx.x >> 7), d4 = threadIdx.x & 127;
  const int hr = r * kHeads + h, job0 = hr / kPfxTileRows, job1 = a.tiles + r;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float L = -INFINITY;
  if (private_len(a, r) > 0) {
    const int c0 = a.prefix > 0 ? a.plan[2 * job0] : 0, n0 = a.prefix > 0 ? a.plan[2 * job0 + 1] - c0 + 1 : 0;
    const int c1 = a.plan[2 * job1], n1 = a.plan[2 * job1 + 1] - c1 + 1;
    // the segment's (slot, row) of the partial arrays
    auto at = [&](int i) {
      return i < n0 ? size_t(job0 + c0 + i) * kPfxTileRows + hr % kPfxTileRows
                    : size_t(job1 + c1 + i - n0) * kPfxTileRows + h;
    };
    float m = -INFINITY;
    bool nan = false;
    for (int i = 0; i < n0 + n1; ++i) {
      const float x = __ldg(a.part_lse + at(i));
      nan |= x != x;
      m = fmaxf(m, x);
    }
    if (m > -INFINITY || nan) {
      float tot = 0.f;
#pragma unroll 4
      for (int i = 0; i < n0 + n1; ++i) {
        const size_t s = at(i);
        const float w = expf(__ldg(a.part_lse + s) - m);
        const float4 v = __ldg(reinterpret_cast<const float4*>(part + s * kDNope) + d4);
        tot += w;
        acc.x = fmaf(w, v.x, acc.x); acc.y = fmaf(w, v.y, acc.y);
        acc.z = fmaf(w, v.z, acc.z); acc.w = fmaf(w, v.w, acc.w);
      }
      const float inv = 1.f / tot;
      acc.x *= inv; acc.y *= inv; acc.z *= inv; acc.w *= inv;
      L = m + logf(tot);
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
  a.q16 = reinterpret_cast<const __half*>(ws + L.pfx_q);
  a.qs = reinterpret_cast<const float*>(ws + L.pfx_qs);
  a.lat = static_cast<const uint8_t*>(lat_pool);
  a.prefix_pages = prefix_pages;
  a.table = block_table;
  a.ctx = ctx_lens;
  a.plan = reinterpret_cast<int32_t*>(ws + L.pfx_plan);
  a.part_lse = reinterpret_cast<float*>(ws + L.pfx_lse);
  a.err = reinterpret_cast<int*>(ws + L.err);
  a.stride = p.lat_page_stride;
  a.prefix = prefix_len;
  a.n_q = p.n_q;
  a.rows = L.rows;
  a.max_pages = p.max_pages_per_req;
  a.num_pages = p.num_pages;
  a.cap = L.cap;
  a.tiles = prefix_len > 0 ? L.pfx_tiles : 0;
  a.scale_log2 = p.softmax_scale * p.latent_scale * 1.4426950408889634f;
  a.lat_scale = p.latent_scale;
  const uint64_t heads = uint64_t(L.rows) * kHeads;
  CUtensorMap qmap, rmap, omap;
  {
    const uint64_t dims[2] = {uint64_t(kDQK), heads}, strides[1] = {uint64_t(kDQK) * 2};
    const uint32_t box[2] = {64, kPfxTileRows};
    if (!encode_map(&qmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.q16, 2, dims, strides, box, true)) return cudaErrorInvalidValue;
  }
  {
    const uint64_t dims[2] = {uint64_t(kDQK), heads}, strides[1] = {uint64_t(kDQK) * 2};
    const uint32_t box[2] = {32, kPfxTileRows};
    if (!encode_map(&rmap, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, a.q16, 2, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
  }
  {
    const uint64_t dims[2] = {uint64_t(kDNope), uint64_t(L.pfx_slots) * kPfxTileRows}, strides[1] = {uint64_t(kDNope) * 4};
    const uint32_t box[2] = {32, 32};
    if (!encode_map(&omap, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, ws + L.pfx_part, 2, dims, strides, box, true))
      return cudaErrorInvalidValue;
  }
  cudaError_t e = launch_pdl(prefix_query_kernel, dim3(unsigned((heads + kQueryWarps - 1) / kQueryWarps)),
                             dim3(32 * kQueryWarps), 0, st, static_cast<const uint32_t*>(q), int(heads),
                             reinterpret_cast<uint32_t*>(ws + L.pfx_q), reinterpret_cast<float*>(ws + L.pfx_qs));
  if (e != cudaSuccess) return e;
  auto kern = p.lat_fmt == DSA_LAT_NVFP4_352 ? prefix_mla_kernel<true> : prefix_mla_kernel<false>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
  if (e != cudaSuccess) return e;
  const int clusters = std::max(1, std::min(kPfxMaxClusters, sm_count() / 2));
  e = launch_pdl(kern, dim3(2 * clusters), dim3(kThreads), kSmem, st, qmap, rmap, omap, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(prefix_merge_kernel, dim3(L.rows, kHeads / kMergeHeads), dim3(128 * kMergeHeads), 0, st, a,
                    reinterpret_cast<const float*>(ws + L.pfx_part), static_cast<__nv_bfloat16*>(out), lse);
}

}  // namespace dsa
