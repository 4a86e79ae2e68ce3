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
// reference and sum, and the merge kernel adds up the segments of a row's two jobs.
//
// Both products take FP8 latents as they lie in the cache, by TMA, and their other operand
// as the sum of two FP8 parts, which costs what one product in fp16 does: the query as
// E4M3 + E5M2, which holds a bf16 value's 8 bits, and a softmax weight as E4M3 + E5M2 too,
// within 2^-8 of it, as bf16 would be, or 2^-10 of the largest in its tile. (With weights and values in fp16 the
// values have to be converted, 96 KB through shared memory per tile beside the 96 KB
// that the product reads: 1.78 k cycles a tile where 1.03 k are the product's.) NVFP4 latents
// have six bits a value, too many for E4M3: they are converted to fp16, which holds
// them exactly, the query and the weights (to 11 bits, or 2^-20 of the tile's largest) too. For that
// the row's reference exponent follows the tiles down as well as up: after one dominant token
// (an attention sink), or among many, the others' weights keep their bits, which
// adds up over the thousands of them. Sums are fp32 throughout.
//
// Measured (one GB300, call after call, where the clock falls under the power limit): 13 x 2 rows
// on 262,144 shared tokens 990 to 1,090 us by the card (1.44 to 1.31 PFLOP/s; 882 us with pauses between
// calls), 64 rows on 32,768 and 1,900 of their own 297 to 317 us (1.52 to 1.43 PFLOP/s; 282 with pauses),
// 24 rows on 8,111 of their own 41.5 us, one row on 4,096 20.4 us; NVFP4, 8 x 6 rows on 16,384 and 700
// of their own 212 us (0.79 PFLOP/s). An FP8 tile takes about
// 1,430 cycles; the scores' products, at 1,165, bound it, and an NVFP4 tile about 2,600: its
// K-blocks' stores and products share CTA 0's shared memory (without the stores 152 us,
// without the arithmetic of the conversion 206). Registers are at their limit of 96: the NVFP4 kernel
// spills 80 bytes a thread, the FP8 one 8.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include <algorithm>
#include <cstring>

#include "dsa_internal.cuh"
#include "sm103_ptx.cuh"

namespace dsa {

namespace {

// ---------------------------------------------------------------------------
// A CTA pair works on one tile of 128 query heads. A 128 x 512 fp32 output fills an
// SM's tensor memory, so the pair divides the two products: CTA 0 (scores) multiplies
// S = Q . C^T over all 576 dims and runs the softmax, CTA 1 (output) multiplies
// O += P . V. Per 64-token tile they cost 1,152 and 1,024 tensor-core cycles at full
// rate, and what crosses between them is P alone: 16 KB, one way. (A
// division by latent dims balances better, 1,088 each, but has to add partial scores,
// 32 KB of fp32 each way per tile; at the 32 B a cycle that an SM takes from
// another's stores that is 1,024 cycles, and it ran at 3,000 cycles a tile.)
//   CTA 0: warps 0..3, 4..7  softmax of the even and of the odd tiles: one query head
//                            per thread; the two groups hand the reference on
//          warps 8..15       at a new job Q to tensor memory; NVFP4: two groups of
//                            converters, the page's 64 rows to fp16 (nine K-blocks)
//          warp  16          MMA of the even tiles: Q from tensor memory (288 columns), S in 3 x 64 columns
//          warp  17          the tiles' pages for the others; FP8: the rows by TMA, as they are
//          warp  18          MMA of the odd tiles
//   CTA 1: warps 0..15       rescale O where the reference has moved, write O at a job's end.
//                            NVFP4: warps 0..3; and 4..15 three groups of converters: the
//                            512 value dims to fp16 (eight K-blocks of 64 dims, read MN-major)
//          warps 16..18      MMA: O in all 512 columns, P from shared memory; the tiles'
//                            pages, FP8: and their 512 value dims by TMA; what the MMA of a
//                            tile waits for
// A converter group issues the loads of its next tile right after it has stored one.
// ---------------------------------------------------------------------------
constexpr int kNT = 64;                      // tokens per tile: one page
constexpr int kBlk = kNT * 128;              // 8,192 B: a K-block, 64 rows of 64 fp16
constexpr int kKBlks = kDQK / 64;            // 9
constexpr int kVBlks = kDNope / 64;          // 8
constexpr int kKBuf = kKBlks * kBlk;         // 73,728 (NVFP4)
constexpr int kKBuf8 = 4 * kBlk + kBlk / 2;  // 36,864 (FP8: 64 rows of 128 E4M3, and of 64 for the rope dims)
constexpr int kVBuf = kVBlks * kBlk;         // 65,536 (NVFP4)
constexpr int kVBuf8 = 4 * kBlk;             // 32,768 (FP8: 64 rows of 128 E4M3)
constexpr int kSBufs = 3;
template <bool kNv>
constexpr int kKBufs = kNv ? 2 : 4;
template <bool kNv>
constexpr int kVBufs = kNv ? 2 : 4;
template <bool kNv>
constexpr int kPBufs = kNv ? 3 : 4;          // (NVFP4: 4 leave the converters' loads less L1: 225 for 199 us)
static_assert(2 * kKBuf == 4 * kKBuf8 && 2 * kVBuf == 4 * kVBuf8, "either kind of buffers");
// P: 8 chunks, of 8 tokens in fp16 or of 16 tokens of the E5M2 (0..3) or the E4M3 part
// (4..7), each 16 B per row in row order (the unswizzled core
// matrices of the MMA, and 512 contiguous bytes for a warp's remote store)
constexpr int kPChunk = 128 * 16;
constexpr int kPBuf = 8 * kPChunk;           // 16,384
constexpr int kPSide = 128 * 4 + 16;         // the rescale factors, and by softmax warp whether one is not 1
constexpr uint32_t kPBytes = kPBuf + kPSide;
constexpr int kThreads = 640;                // five warpgroups; the last holds the warps below and an idle one
constexpr int kMmaWarp = 16, kFeedWarp = 17, kMmaWarp2 = 18, kReadyWarp = 18;
constexpr uint32_t kSCol = 288;              // S after Q's 9 x 32 columns
constexpr int kNumBars = 77;
template <bool kNv>
constexpr size_t kData = 2 * kVBuf + kPBufs<kNv> * (kPBuf + kPSide);  // of CTA 1; CTA 0 needs less
static_assert(kData<true> >= 2 * kKBuf + 1024 && kData<false> >= 2 * kKBuf + 1024, "CTA 0's buffers");
template <bool kNv>
constexpr size_t kSmem = 1024 + kData<kNv> + kNumBars * 8 + 64 + 16;
static_assert(kSmem<true> + 256 <= 232448 && kSmem<false> + 256 <= 232448, "shared memory, with the static variables");
// A weight is 2^(z - ref), with a reference per row that is a whole number, so that rescaling is exact.
// The largest weight of a tile is kept between 2^kLeast and 2^kMost: the segment's first tile puts ref where its
// largest is in [2^kFirst, 2^(kFirst + 1)), a tile above kMost raises ref to bring it to kRaised, and one below kLeast
// lowers ref to bring it to kLowered. Both moves are short, as most tiles of a row are alike, and a move
// by any of a tile's rows costs a rescale of O, about 0.7 us. (FP8, 64 rows on 32,768 tokens with logits of
// a deviation of 1.3, 2.1, 3.1 and 5.2: 282, 292, 348, 516 us, against 275, 301, 410, 440 when ref
// only rose, to 2^6 above 2^12, and the weights after a sink lost their bits. A third E5M2
// part for tiles whose weights are all small, voted on by the four warps: 317, 395, 495, 627.)
// ref is never more than kTopDrop below the segment's highest, which bounds O and the sums.
template <bool kNv>
constexpr float kFirst = kNv ? 7.f : 2.f;
template <bool kNv>
constexpr float kMost = kNv ? 15.f : 12.f;
template <bool kNv>
constexpr float kRaised = kNv ? 12.f : 8.f;
template <bool kNv>
constexpr float kLeast = kNv ? -5.f : -4.f;
template <bool kNv>
constexpr float kLowered = kNv ? 4.f : 0.f;
constexpr float kTopDrop = 40.f;
constexpr float kLarge = 8.f;                // FP8: the order of a row's two parts changes above 2^kLarge
// Poll limit of a wait that may last for a whole run of this many units (for the next rescale or output,
// for the products with a query). A poll that finds nothing sleeps for 3.9 us (measured) and a tile takes
// 0.8 to 1.4 us: one poll a unit is enough, and four leave room for a slow clock. The other waits see a few
// tiles; the default limit gives them 4 s.
constexpr uint32_t kPolls = 1u << 20;
__host__ __device__ constexpr uint32_t run_polls(int units) { return kPolls + 4 * uint32_t(units); }
static_assert(kPolls + 4 * (kPfxMaxTiles / kPfxMaxClusters) < 0xFFFFFFFFll, "the longest run's limit");
constexpr int kMinUnits = 3;
constexpr int kJobCost = 4;                  // what a job's start and end take, in tiles (3: 284 us, 4: 275, 5: 276)

struct PfxArgs {
  const uint4* q;    // [72][rows * 96] 16-B chunks of the prepared query, each head by head
  const float* qs;
  const uint8_t* lat;
  const int32_t* prefix_pages;
  const int32_t* table;
  const int32_t* lens;  // [rows] private tokens that a row sees (0: an invalid context length)
  int32_t* plan;  // [jobs][2] first and last CTA pair of a job
  float* ml;      // [slots][2][2][128] references (base 2) and sums: of the group with the last tile, which O has too; the other's
  float* part;    // [slots][512 / 4][128][4] unnormalised outputs
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
#pragma unroll 1
    while (left > 0 && ++job < a.tiles + a.rows)
      if (take(a, 0)) return true;
    return false;
  }
};

// Four E4M3 bytes -> four fp16. (The header's conversion returns two halves that the
// compiler packs again, which tripled the converters' instructions.)
__device__ __forceinline__ void expand_e4m3(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// 16 E4M3 bytes -> 16 fp16, as two 16-B chunks.
__device__ __forceinline__ void expand16(const uint4 w, uint4& lo, uint4& hi) {
  expand_e4m3(w.x, lo.x, lo.y);
  expand_e4m3(w.y, lo.z, lo.w);
  expand_e4m3(w.z, hi.x, hi.y);
  expand_e4m3(w.w, hi.z, hi.w);
}

// 8 E2M1 values times an E4M3 scale (a pair of fp16): 6 significant bits, exact.
__device__ __forceinline__ uint4 expand_e2m1(uint32_t w, __half2 s) {
  uint32_t o[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&o[i]), s);
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

// A converter thread's share of an NVFP4 tile; warp w of 4 has nope K-blocks 2w and 2w + 1:
// eight 16-B units (32 values, two scales), and for keys (kRope) two 16-B pieces of the
// rope dims. Tokens at or past `valid` are zeros: their weights are 0, but their
// bytes could be NaN.
template <bool kRope>
struct TileRegs {
  uint4 v[2][4];
  uint32_t s[2][4];
  uint4 rope[2];
  __device__ __forceinline__ void load(const uint8_t* page, int valid, int w, int lane) {
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int tok = u * 16 + (lane >> 1), unit = 4 * w + 2 * b + (lane & 1);
        const uint8_t* row = page + tok * 352;
        v[b][u] = tok < valid ? __ldg(reinterpret_cast<const uint4*>(row + 16 * unit)) : zero;
        s[b][u] = tok < valid ? __ldg(reinterpret_cast<const uint16_t*>(row + 256 + 2 * unit)) : 0;
      }
    if constexpr (kRope) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int ct = b * 128 + w * 32 + lane, tok = ct >> 2;
        rope[b] = tok < valid ? __ldg(reinterpret_cast<const uint4*>(page + tok * 352 + 288 + 16 * (ct & 3))) : zero;
      }
    }
  }
  // 16 of the tokens, 16 step and up
  __device__ __forceinline__ void store(int step, uint8_t* buf, int w, int lane) const {
    const int tok = 16 * step + (lane >> 1), c0 = (lane & 1) * 4;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint8_t* blk = buf + (2 * w + b) * kBlk;
      uint32_t two, none;
      expand_e4m3(s[b][step], two, none);
      const __half2 h = *reinterpret_cast<const __half2*>(&two);
      const __half2 s0 = __low2half2(h), s1 = __high2half2(h);
      put2(blk, tok, c0, expand_e2m1(v[b][step].x, s0), expand_e2m1(v[b][step].y, s0));
      put2(blk, tok, c0 + 2, expand_e2m1(v[b][step].z, s1), expand_e2m1(v[b][step].w, s1));
    }
  }
  __device__ __forceinline__ void store_rope(uint8_t* buf, int w, int lane) const {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint4 lo, hi;
      const int ct = b * 128 + w * 32 + lane;
      expand16(rope[b], lo, hi);
      put2(buf + 8 * kBlk, ct >> 2, (ct & 3) * 2, lo, hi);
    }
  }
};

// Four weights as fp16 -> their E4M3 part and the E5M2 part of the rest, for weights up to 2^kLarge. E4M3 is off by half
// of its step, 2^-4 of the weight, which needs three bits, or by 2^-10 of weights under 2^-6: the two parts
// together are within 2^-8 of the weight, or 2^-14.
__device__ __forceinline__ void split_small(uint32_t a, uint32_t b, uint32_t& e5m2, uint32_t& e4m3) {
  asm("{\n\t.reg .b16 x, y;\n\t.reg .b32 u, v;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 x, %2;\n\tcvt.rn.satfinite.e4m3x2.f16x2 y, %3;\n\tmov.b32 %1, {x, y};\n\t"
      "cvt.rn.f16x2.e4m3x2 u, x;\n\tcvt.rn.f16x2.e4m3x2 v, y;\n\t"
      "sub.rn.f16x2 u, %2, u;\n\tsub.rn.f16x2 v, %3, v;\n\t"
      "cvt.rn.satfinite.e5m2x2.f16x2 x, u;\n\tcvt.rn.satfinite.e5m2x2.f16x2 y, v;\n\tmov.b32 %0, {x, y};\n\t}\n"
      : "=r"(e5m2), "=&r"(e4m3)
      : "r"(a), "r"(b));
}
// The other way round, for weights up to 2^kMost: off by 2^-3 of the weight, at most 2^8 (E4M3 ends at 448), and then
// by 2^-8 of it, or 2^-10.
__device__ __forceinline__ void split_large(uint32_t a, uint32_t b, uint32_t& e5m2, uint32_t& e4m3) {
  asm("{\n\t.reg .b16 x, y;\n\t.reg .b32 u, v;\n\t"
      "cvt.rn.satfinite.e5m2x2.f16x2 x, %2;\n\tcvt.rn.satfinite.e5m2x2.f16x2 y, %3;\n\tmov.b32 %0, {x, y};\n\t"
      "cvt.rn.f16x2.e5m2x2 u, x;\n\tcvt.rn.f16x2.e5m2x2 v, y;\n\t"
      "sub.rn.f16x2 u, %2, u;\n\tsub.rn.f16x2 v, %3, v;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 x, u;\n\tcvt.rn.satfinite.e4m3x2.f16x2 y, v;\n\tmov.b32 %1, {x, y};\n}\n"
      : "=&r"(e5m2), "=r"(e4m3)
      : "r"(a), "r"(b));
}

// 2^x of a whole number, exactly; 0 below 2^-126.
__device__ __forceinline__ float pow2_whole(float x) { return __int_as_float((min(max(int(x), -127), 127) + 127) << 23); }

// What the warps of a CTA need to know of a tile, in a ring that one warp fills.
struct Tile {
  int page, valid;  // physical page, and how many of its tokens the job sees (0 for a bad page)
};
constexpr int kRing = 8;

// The ring's producer (one warp): 32 page numbers of the walk's job at a time.
// each(g, tile): what else it does for a tile (lane 0 has just published it).
template <typename Each>
__device__ __forceinline__ bool feed(const PfxArgs& a, int gtot, int job0, int unit, int units, int lane, bool report,
                                     Tile* ring, uint32_t full, uint32_t free, Each each) {
  Walk wk;
  int g = 0;
#pragma unroll 1
  for (bool on = gtot > 0 && wk.start(a, job0, unit, units); on; on = wk.next(a)) {
    const int32_t* list = a.prefix_pages;
    int len = a.prefix;
    if (wk.job >= a.tiles) {
      const int r = wk.job - a.tiles;
      list = a.table + size_t(r / a.n_q) * a.max_pages + a.prefix / kNT;
      len = a.lens[r];
    }
    int mine = 0;
#pragma unroll 1
    for (int k = wk.k0; k < wk.k1; ++k, ++g) {
      const int i = (k - wk.k0) & 31;
      if (i == 0) mine = k + lane < wk.k1 ? __ldg(list + k + lane) : 0;
      const int pg = __shfl_sync(0xffffffffu, mine, i);
      const bool good = pg >= 0 && pg < a.num_pages;
      const Tile t{good ? pg : 0, good ? min(kNT, len - k * kNT) : 0};
      const int slot = g % kRing;
      if (g >= kRing && !ptx::mbar_wait(free + 8 * slot, uint32_t(g / kRing - 1) & 1u)) return false;
      if (lane == 0) {
        if (!good && report) atomicOr(a.err, DSA_DEVERR_BLOCK_TABLE);
        ring[slot] = t;
        ptx::mbar_arrive(full + 8 * slot);
      }
      if (!each(g, t)) return false;
    }
  }
  return true;
}

// One of the kGroups converter groups (4 warps; tiles in turn) of either CTA (NVFP4).
// kKeys (CTA 0): all 576 dims, else (CTA 1) the 512 values, in two halves of 32 tokens. ring and
// its barriers as in feed; full / free: the buffers' (or halves') barriers; turn: the groups take buffers in the order of their
// tiles (a group that came early could take a buffer's barrier for one a round older,
// which has the same parity); after(g): called once tile g is stored.
template <bool kKeys, int kGroups, typename After>
__device__ __forceinline__ bool convert(const PfxArgs& a, int gtot, int group, int w, int lane, const Tile* ring,
                                        uint32_t ring_full, uint32_t ring_free, uint8_t* bufs, uint32_t full,
                                        uint32_t free, uint32_t turn, After after) {
  TileRegs<kKeys> t;
  auto load = [&](int g) {
    const int slot = g % kRing;
    if (!ptx::mbar_wait(ring_full + 8 * slot, uint32_t(g / kRing) & 1u)) return false;
    const Tile tile = ring[slot];
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(ring_free + 8 * slot);
    t.load(a.lat + int64_t(tile.page) * a.stride, tile.valid, w, lane);
    return true;
  };
  if (group < gtot && !load(group)) return false;
#pragma unroll 1
  for (int g = group; g < gtot; g += kGroups) {
    if constexpr (kKeys) {
      constexpr int kBufs = kKBufs<true>;
      const int buf = g % kBufs;
      if (g >= kBufs && !ptx::mbar_wait(free + 8 * buf, uint32_t(g / kBufs - 1) & 1u)) return false;
      uint8_t* dst = bufs + buf * kKBuf;
#pragma unroll
      for (int i = 0; i < 4; ++i) t.store(i, dst, w, lane);
      t.store_rope(dst, w, lane);
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(full + 8 * buf);
    } else {
      const int buf = g % kVBufs<true>;
      if (g > 0 && !ptx::mbar_wait(turn + 8 * ((g - 1) % kGroups), uint32_t((g - 1) / kGroups) & 1u)) return false;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (g >= kVBufs<true> && !ptx::mbar_wait(free + 8 * (2 * buf + i), uint32_t(g / kVBufs<true> - 1) & 1u)) return false;
        if (i == 1 && lane == 0) ptx::mbar_arrive(turn + 8 * group);
        t.store(2 * i, bufs + buf * kVBuf, w, lane);
        t.store(2 * i + 1, bufs + buf * kVBuf, w, lane);
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(full + 8 * (2 * buf + i));
      }
    }
    if (!after(g)) return false;
    if (g + kGroups < gtot && !load(g + kGroups)) return false;
  }
  return true;
}

template <bool kNv>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    prefix_mla_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap rmap,
                      const __grid_constant__ PfxArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  // the barriers have the same place in both CTAs
  const uint32_t bars = ptx::smem_u32(sm) + uint32_t(kData<kNv>);
  const uint32_t mma_done = bars + 0 * 8;
  const uint32_t q_full = bars + 1 * 8;      // a later job's query is there
  const uint32_t q_first = bars + 76 * 8;    // the first job's
  const uint32_t q_free = bars + 2 * 8;      // every product with the job's query is done
  const uint32_t k_full = bars + 3 * 8;      // [kKBufs]
  const uint32_t k_free = bars + 7 * 8;      // [kKBufs]  S of the buffer's tile is done
  const uint32_t s_full = bars + 11 * 8;     // [kSBufs]
  const uint32_t s_free = bars + 70 * 8;     // [2 kSBufs]  the softmax has read S of a tile (modulo 6)
  const uint32_t turn = bars + 17 * 8;       // [4]  by softmax warp: the tile's reference is decided
  const uint32_t ring_full = bars + 21 * 8;  // [kRing]
  const uint32_t ring_free = bars + 29 * 8;  // [kRing]
  const uint32_t p_free = bars + 37 * 8;     // [kPBufs]  P . V of the tile in this slot of P is done (CTA 0; NVFP4: both)
  const uint32_t p_full = bars + 41 * 8;     // [kPBufs]  P and the factors have landed
  const uint32_t go = bars + 45 * 8;         // [kPBufs]  P and O are ready for P . V
  const uint32_t v_full = bars + 49 * 8;     // [4] NVFP4: by half tile
  const uint32_t v_free = bars + 54 * 8;     // [4]  its P . V is done
  const uint32_t v_turn = bars + 60 * 8;     // [3]  by group: the tile's buffer is the group's
  const uint32_t ask = bars + 67 * 8;        // O is to be rescaled, or written
  const uint32_t o_ok = bars + 68 * 8;       // and it is
  Tile* ring = reinterpret_cast<Tile*>(sm + kData<kNv> + kNumBars * 8);  // [8]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(ring + kRing);
  // CTA 0
  uint8_t* KB = sm;
  float* m_run = reinterpret_cast<float*>(sm + 2 * kKBuf);  // [128] the reference in use
  float* m_top = m_run + 128;                               // [128] the highest of the segment
  // CTA 1
  uint8_t* VB = sm;
  uint8_t* PB = sm + 2 * kVBuf;
  uint8_t* side = PB + kPBufs<kNv> * kPBuf;  // [kPBufs] factors and flags
  __shared__ long long s_sum[kThreads / 32];
  __shared__ int s_job, s_unit, s_tiles, s_ask;  // s_ask: the tile that wants O rescaled, -1 at a job's end

  const int half = int(ptx::cluster_ctarank());
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nclu = int(gridDim.x) >> 1, clu = int(blockIdx.x) >> 1;

  if (threadIdx.x == 0) {
    s_tiles = 0;
    ptx::mbar_init(mma_done, half == 0 ? 2 : 1);
    ptx::mbar_init(q_full, 8);
    ptx::mbar_init(q_first, 16);
    ptx::mbar_init(q_free, 2);
    ptx::mbar_init(ask, 1);
    for (int i = 0; i < 3; ++i) ptx::mbar_init(v_turn + 8 * i, 4);
    ptx::mbar_init(o_ok, kNv ? 4 : 16);
    for (int i = 0; i < kPBufs<kNv>; ++i) {
      ptx::mbar_init(p_free + 8 * i, 1);
      ptx::mbar_init(p_full + 8 * i, 1);
      ptx::mbar_init(go + 8 * i, 1);
    }
    for (int i = 0; i < kSBufs; ++i) {
      ptx::mbar_init(s_full + 8 * i, 1);
    }
    for (int i = 0; i < 2 * kSBufs; ++i) ptx::mbar_init(s_free + 8 * i, 4);
    for (int i = 0; i < 4; ++i) {
      ptx::mbar_init(v_full + 8 * i, kNv ? 4 : 1);
      ptx::mbar_init(v_free + 8 * i, 1);
    }
    for (int i = 0; i < 4; ++i) {
      ptx::mbar_init(turn + 8 * i, 1);
      ptx::mbar_init(k_full + 8 * i, kNv ? 4 : 1);
      ptx::mbar_init(k_free + 8 * i, 1);
    }
    for (int i = 0; i < kRing; ++i) {
      ptx::mbar_init(ring_full + 8 * i, 1);
      // who reads it: a softmax and a converter group, or one of them, or the warp that readies tiles
      ptx::mbar_init(ring_free + 8 * i, kNv ? (half == 0 ? 8 : 4) : (half == 0 ? 4 : 1));
    }
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
    auto row_units = [&](int r) {
      const int n = r < a.rows ? job_tiles(a, a.tiles + r) : 0;
      return n > 0 ? (long long)(n + kJobCost) : 0ll;
    };
    auto warp_scan = [&](long long v) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += y;
      }
      return v;
    };
    // rows in chunks of a thread each: a chunk's units before this thread's row, and in all
    constexpr int kWarps = kThreads / 32;
    auto chunk_scan = [&](long long n, long long& before, long long& all) {
      const long long up = warp_scan(n);
      if (lane == 31) s_sum[warp] = up;
      __syncthreads();
      const long long sums = warp_scan(lane < kWarps ? s_sum[lane] : 0ll);
      before = up - n + (warp ? __shfl_sync(0xffffffffu, sums, warp - 1) : 0ll);
      all = __shfl_sync(0xffffffffu, sums, kWarps - 1);
    };
    long long n = row_units(threadIdx.x), before, all;
    chunk_scan(n, before, all);
    int64_t line = all;
    for (int r0 = kThreads; r0 < a.rows; r0 += kThreads) {
      long long b, more;
      __syncthreads();
      chunk_scan(row_units(r0 + int(threadIdx.x)), b, more);
      line += more;
    }
    const int per = a.tiles ? a.prefix / kNT + kJobCost : 1;  // units of a prefix job
    const int64_t shared = int64_t(a.tiles) * per;
    line += shared;
    // A pair has at least kMinUnits, so that a short line leaves the merge less (one request
    // of 4,096 tokens: 23.5 us, 24.4 with at least two, 26.0 with one, 25.5 with four),
    // and no pair among those that work goes without: a job's segments are those of
    // consecutive pairs.
    const int64_t used = min(int64_t(nclu), (line + kMinUnits - 1) / kMinUnits);
    const int64_t lo = clu < used ? line * clu / used : line, hi = clu < used ? line * (clu + 1) / used : line;
    units = int(hi - lo);
    // tiles of the prefix jobs among the line's first x units
    auto prefix_tiles = [&](int64_t x) {
      x = min(x, shared);
      return x / per * (per - kJobCost) + max(int64_t(0), x % per - kJobCost);
    };
    if (threadIdx.x == 0) {
      const int t = int(prefix_tiles(hi) - prefix_tiles(lo));
      if (t) atomicAdd(&s_tiles, t);
      if (lo < shared) {
        s_job = int(lo / per);
        s_unit = int(lo % per);
      }
    }
    int64_t base = shared;
    for (int r0 = 0;;) {
      if (n > 0) {
        const int64_t first = base + before, t0 = first + kJobCost, t1 = first + n;  // its tiles
        const int t = int(max(int64_t(0), min(t1, hi) - max(t0, lo)));
        if (t) atomicAdd(&s_tiles, t);
        if (lo >= first && lo < t1) {
          s_job = a.tiles + r0 + int(threadIdx.x);
          s_unit = int(lo - first);
        }
      }
      base += all;
      r0 += kThreads;
      if (r0 >= a.rows || hi <= base) break;
      n = row_units(r0 + int(threadIdx.x));
      __syncthreads();
      chunk_scan(n, before, all);
    }
    __syncthreads();
    gtot = s_tiles;
    // P of the first tiles may arrive as soon as the pair has synced
    if (half == 1 && threadIdx.x == 0)
      for (int i = 0; i < kPBufs<kNv> && i < gtot; ++i) ptx::mbar_arrive_expect_tx(p_full + 8 * (i), kPBytes);
  }
  ptx::cluster_sync();  // the peer's barriers exist before any remote arrive
  const int job0 = s_job;
  const int unit0 = s_unit;
  bool ok = true;
  Walk wk;

  // CTA 1: rescaling and writing columns [c0, c1) of O, one warp of four a quarter of the rows
  auto output = [&](int c0, int c1) {
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_base = uint32_t((warp & 3) * 32) << 16;
    int asked = 0;
#pragma unroll 1
    for (bool on = gtot > 0 && wk.start(a, job0, unit0, units); on; on = wk.next(a)) {
#pragma unroll 1
      for (;;) {
        if (!ptx::mbar_wait(ask, uint32_t(asked++) & 1u, run_polls(units))) return false;
        const int what = s_ask;
        // O is up to date, and still, once P . V of the tile before g is done
        const int g = what < 0 ? -1 - what : what;
        // (FP8: by the barrier of its values, which comes sooner than the one that both CTAs
        // get; it is at most a phase back, as the tile's values came before it was asked for.
        // NVFP4's could be two back.)
        const uint32_t done = kNv ? p_free : v_free, of = kNv ? kPBufs<kNv> : kVBufs<kNv>, t = uint32_t(g - 1);
        if (!ptx::mbar_wait(done + 8 * (t % of), (t / of) & 1u)) return false;
        ptx::tc_fence_after();
        if (what < 0) break;
        const float alpha = reinterpret_cast<const float*>(side + (g % kPBufs<kNv>) * kPSide)[row];
        if (__any_sync(0xffffffffu, alpha != 1.f)) {
#pragma unroll 1
          for (int c = c0; c < c1; c += 32) {
            float o[32];
            ptx::tmem_ld32(tmem + lane_base + c, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= alpha;
            ptx::tmem_st32(tmem + lane_base + c, o);
          }
        }
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(o_ok);
      }
      // (four dims of all rows together, so that a warp's stores are whole lines)
      float4* dst = reinterpret_cast<float4*>(a.part) + size_t(wk.job + clu) * kPfxTileRows * (kDNope / 4) + row;
      const bool real = wk.job < a.tiles ? wk.job * kPfxTileRows + row < a.rows * kHeads : row < kHeads;
#pragma unroll 1
      for (int c = c0; c < c1; c += 32) {
        float o[32];
        ptx::tmem_ld32(tmem + lane_base + c, o);
        if (real) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            dst[(c / 4 + j) * kPfxTileRows] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
        }
      }
      // the reads of O are ordered before the next job's first P . V
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(o_ok);
    }
    return true;
  };

  // CTA 1, NVFP4, warps 4..15
  auto values = [&]() {
    return convert<false, 3>(a, gtot, (warp >> 2) - 1, warp & 3, lane, ring, ring_full, ring_free, VB, v_full, v_free, v_turn,
                             [](int) { return true; });
  };

  // CTA 0: 32 heads of a job's query, `blocks` times 32 columns from block kb0, to tensor memory
  auto query_blocks = [&](int job, int kb0, auto blocks, uint32_t bar, auto until) {
    const int row = (warp & 3) * 32 + lane;
    const int hr = (job < a.tiles ? job * kPfxTileRows : (job - a.tiles) * kHeads) + row;
    const int heads = a.rows * kHeads;
    // (a private job's last 32 rows are zeros: the next row's heads would ask for rescales, too. Not for NVFP4, whose
    // converters have no registers to spare: 214.7 for 212.8 us)
    const bool in = kNv || job < a.tiles ? hr < heads : row < kHeads;
    auto load = [&](int kb, uint32_t (&v)[32]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint4 x = in ? __ldg(a.q + size_t(kb * 8 + i) * heads + hr) : make_uint4(0, 0, 0, 0);
        v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
      }
    };
    // blocks are loaded ahead, the first before the old query is let go: one at a time
    // after that took 4.3 us a job. (NVFP4: one ahead, as the converters' registers allow.)
    constexpr int kBlocks = decltype(blocks)::value, kAhead = kNv ? 1 : 2;
    uint32_t v[kAhead][32];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(kb0 + i, v[i]);
    if (!until()) return false;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      ptx::tmem_st32_u(tmem + (uint32_t((warp & 3) * 32) << 16) + (kb0 + i) * 32, v[i % kAhead]);
      if (i + kAhead < kBlocks) load(kb0 + i + kAhead, v[i % kAhead]);
    }
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar);
    return true;
  };
  constexpr std::integral_constant<int, 2> two{};
  constexpr std::integral_constant<int, 3> three{};
  constexpr std::integral_constant<int, 4> four{};
  constexpr std::integral_constant<int, 5> five{};
  // the first query, when nothing else is to be done: the nine blocks by four groups of warps
  auto first_query = [&](int job) {
    auto now = [] { return true; };
    const int quarter = warp >> 2;
    return quarter == 0 ? query_blocks(job, 0, three, q_first, now) : query_blocks(job, 1 + 2 * quarter, two, q_first, now);
  };

  // registers: the five warpgroups start with 96 each (480) and go on with 104, 104, 96, 96 and 80 (480)
  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if ((warp == kMmaWarp || warp == kMmaWarp2) && half == 0) {
      // ---------------------------------------------------------- S = Q . C^T
      // (the even and the odd tiles by a warp each: a wait takes its turn behind the products
      // that its warp has issued, and while one waits the other's keep the tensor core busy)
      const uint32_t kb0 = ptx::smem_u32(KB);
      int g = 0, qn = 0;
#pragma unroll 1
      for (bool on = gtot > 0 && wk.start(a, job0, unit0, units); on && ok; on = wk.next(a)) {
        if (!(qn == 0 ? ptx::mbar_wait(q_first, 0) : ptx::mbar_wait(q_full, uint32_t(qn - 1) & 1u))) { ok = false; break; }
        ++qn;
#pragma unroll 1
        for (int k = wk.k0; k < wk.k1; ++k, ++g) {
          if ((g & 1) != (warp == kMmaWarp2)) continue;
          const int buf = g % kKBufs<kNv>, sb = g % kSBufs;
          if (!ptx::mbar_wait(k_full + 8 * buf, uint32_t(g / kKBufs<kNv>) & 1u)) { ok = false; break; }
          // S of the tile three before has been read. (It has a barrier that only tiles of its
          // own kind, odd or even, use: they are read in order, so the barrier is at most a
          // round back. One for all tiles in this place could be two rounds back, which
          // has the same parity.)
          if (g >= kSBufs) {
            const int t = g - kSBufs;
            if (!ptx::mbar_wait(s_free + 8 * (t % (2 * kSBufs)), uint32_t(t / (2 * kSBufs)) & 1u)) { ok = false; break; }
          }
          ptx::tc_fence_after();
          const uint32_t kb = kb0 + buf * (kNv ? kKBuf : kKBuf8), s = tmem + kSCol + sb * kNT;
          if (ptx::elect_one()) {
            if constexpr (kNv) {
              const uint32_t id = ptx::idesc(0, 0, 128, kNT);
#pragma unroll 1
              for (int j = 0; j < kKBlks; ++j)
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  ptx::mma_f16_tmem_a(s, tmem + j * 32 + kk * 8, ptx::sdesc_sw128(kb + j * kBlk + kk * 32), id,
                                      (j | kk) ? 1u : 0u);
            } else {
#pragma unroll
              for (int part = 0; part < 2; ++part) {  // the query's E4M3, then its E5M2 part
                const uint32_t id = ptx::idesc(part, 0, 128, kNT), q = tmem + part * 144;
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                  for (int kk = 0; kk < 4; ++kk)
                    ptx::mma_f8_tmem_a(s, q + j * 32 + kk * 8, ptx::sdesc_sw128(kb + j * kBlk + kk * 32), id,
                                       (part | j | kk) ? 1u : 0u);
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
                  ptx::mma_f8_tmem_a(s, q + 128 + kk * 8, ptx::sdesc_sw64(kb + 4 * kBlk + kk * 32), id, 1u);
              }
            }
            ptx::mma_commit(s_full + 8 * sb);
            ptx::mma_commit(k_free + 8 * buf);
          }
          __syncwarp();
        }
        if (ok && ptx::elect_one()) ptx::mma_commit(q_free);
        __syncwarp();
      }
    } else if (warp == kFeedWarp) {
      // ---------------------------------------------------------- tiles; FP8 rows by TMA
      const uint32_t dst0 = ptx::smem_u32(sm), full = half == 0 ? k_full : v_full, free = half == 0 ? k_free : v_free;
      const uint32_t bytes = half == 0 ? kKBuf8 : kVBuf8;
      constexpr int kBufs = 4;
      static_assert(kNv || (kKBufs<kNv> == kBufs && kVBufs<kNv> == kBufs), "FP8 buffers");
      ok = feed(a, gtot, job0, unit0, units, lane, half == 0, ring, ring_full, ring_free, [&](int g, const Tile& t) {
        if (kNv) return true;
        const int buf = g % kBufs;
        if (g >= kBufs && !ptx::mbar_wait(free + 8 * buf, uint32_t(g / kBufs - 1) & 1u)) return false;
        if (lane == 0) {
          const uint32_t dst = dst0 + buf * bytes, bar = full + 8 * buf;
          ptx::mbar_arrive_expect_tx(bar, bytes);
#pragma unroll
          for (int j = 0; j < 4; ++j) ptx::tma_load_3d(dst + j * kBlk, &kmap, bar, j * 128, 0, t.page);
          if (half == 0) ptx::tma_load_3d(dst + 4 * kBlk, &rmap, bar, kDNope, 0, t.page);
        }
        __syncwarp();
        return true;
      });
      // no copy left in flight
      if (!ok && !kNv)
        for (int i = 0; i < 2 * kBufs; ++i) ptx::mbar_wait(full + 8 * (i >> 1), uint32_t(i & 1), 1 << 8);
    } else if (warp == kMmaWarp) {
      // ---------------------------------------------------------- O += P . V
      const uint32_t vb0 = ptx::smem_u32(VB), pb0 = ptx::smem_u32(PB);
      int g = 0;
#pragma unroll 1
      for (bool on = gtot > 0 && wk.start(a, job0, unit0, units); on && ok; on = wk.next(a)) {
#pragma unroll 1
        for (int k = wk.k0; k < wk.k1 && ok; ++k, ++g) {
          const int buf = g % kVBufs<kNv>, pb = g % kPBufs<kNv>;
          const uint32_t vpar = uint32_t(g / kVBufs<kNv>) & 1u, p0 = pb0 + pb * kPBuf;
          if (!ptx::mbar_wait(go + 8 * pb, uint32_t(g / kPBufs<kNv>) & 1u)) { ok = false; break; }
          if constexpr (kNv) {
            const uint32_t id = ptx::idesc(0, 0, 128, 256, 0, 1);
#pragma unroll 1
            for (int i = 0; i < 2; ++i) {  // 32 tokens of the tile
              if (!ptx::mbar_wait(v_full + 8 * (2 * buf + i), vpar)) { ok = false; break; }
              ptx::tc_fence_after();
              const uint32_t vb = vb0 + buf * kVBuf + i * 32 * 128, p = p0 + i * 4 * kPChunk;
              if (ptx::elect_one()) {
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                  for (int n = 0; n < 2; ++n)
                    ptx::mma_f16(tmem + n * 256, ptx::sdesc_plain(p + kk * 2 * kPChunk, kPChunk, 128),
                                 ptx::sdesc_sw128_mn(vb + n * 4 * kBlk + kk * 16 * 128, kBlk, 1024), id,
                                 (k > wk.k0 || i > 0 || kk > 0) ? 1u : 0u);
                ptx::mma_commit(v_free + 8 * (2 * buf + i));
                if (i) ptx::mma_commit_to(p_free + 8 * pb, 3);  // in both CTAs
              }
              __syncwarp();
            }
          } else {
            if (!ptx::mbar_wait(v_full + 8 * buf, vpar)) { ok = false; break; }
            ptx::tc_fence_after();
            const uint32_t vb = vb0 + buf * kVBuf8;
            if (ptx::elect_one()) {
#pragma unroll
              for (int part = 0; part < 2; ++part)  // the weights' E5M2, then their E4M3 part
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                  for (int n = 0; n < 2; ++n)
                    ptx::mma_f8f6f4(tmem + n * 256, ptx::sdesc_plain(p0 + (part * 4 + kk * 2) * kPChunk, kPChunk, 128),
                                    ptx::sdesc_sw128_mn(vb + n * 2 * kBlk + kk * 32 * 128, kBlk, 1024),
                                    ptx::idesc(1 - part, 0, 128, 256, 0, 1), (k > wk.k0 || part > 0 || kk > 0) ? 1u : 0u);
              ptx::mma_commit(v_free + 8 * buf);
              ptx::mma_commit_to(p_free + 8 * pb, 1);
            }
            __syncwarp();
          }
        }
      }
    } else if (warp == kReadyWarp && half == 1) {
      // ---------------------------------------------------------- what P . V waits for
      // (in a warp of its own, a tile ahead: the MMA warp issues at the rate of the
      // products, and each of these steps of its own would leave the tensor core idle)
      int g = 0, asked = 0, answered = 0;
      auto request = [&](int what) {
        if (lane == 0) {
          s_ask = what;
          ptx::mbar_arrive(ask);
        }
        __syncwarp();
        ++asked;
      };
      auto settled = [&]() {
        while (answered < asked)
          if (!ptx::mbar_wait(o_ok, uint32_t(answered++) & 1u)) return false;
        return true;
      };
#pragma unroll 1
      for (bool on = gtot > 0 && wk.start(a, job0, unit0, units); on && ok; on = wk.next(a)) {
#pragma unroll 1
        for (int k = wk.k0; k < wk.k1; ++k, ++g) {
          const int pb = g % kPBufs<kNv>;
          if (!ptx::mbar_wait_cluster(p_full + 8 * pb, uint32_t(g / kPBufs<kNv>) & 1u)) { ok = false; break; }
          if constexpr (!kNv) {
            // The tile's values, and zeros for rows that the job does not see: their weights
            // are 0, but their bytes could be NaN. (This tile's P was sent after the product
            // kPBufs tiles ago, so its buffer's barrier is at most a phase back.)
            static_assert(kPBufs<kNv> <= kVBufs<kNv>, "the buffer's last product is done");
            const int slot = g % kRing, buf = g % kVBufs<kNv>;
            if (!ptx::mbar_wait(ring_full + 8 * slot, uint32_t(g / kRing) & 1u)) { ok = false; break; }
            const int valid = ring[slot].valid;
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(ring_free + 8 * slot);
            if (!ptx::mbar_wait(v_full + 8 * buf, uint32_t(g / kVBufs<kNv>) & 1u)) { ok = false; break; }
            if (valid < kNT) {
              uint8_t* v = VB + buf * kVBuf8 + (lane >> 3) * kBlk + (lane & 7) * 16;
              for (int t = valid; t < kNT; ++t) *reinterpret_cast<uint4*>(v + t * 128) = make_uint4(0, 0, 0, 0);
            }
          }
          const uint4 flags = *reinterpret_cast<const uint4*>(side + pb * kPSide + 512);
          // re-arm for the next tile in this slot: it is not sent before this one's P . V is done
          if (lane == 0 && g + kPBufs<kNv> < gtot) ptx::mbar_arrive_expect_tx(p_full + 8 * pb, kPBytes);
          if (k > wk.k0 && (flags.x | flags.y | flags.z | flags.w)) request(g);
          if (!settled()) { ok = false; break; }  // (at a job's first tile: the old output is written)
          // P came by ordinary (remote) stores; the tensor core reads it through the async proxy
          ptx::fence_proxy_async_smem();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(go + 8 * pb);
        }
        if (ok) request(-1 - g);
      }
      if (ok) ok = settled();
    }
    if (warp == kMmaWarp || (warp == kMmaWarp2 && half == 0)) {
      // nothing of these warps' left in flight when the tensor memory is released
      if (ptx::elect_one()) ptx::mma_commit(mma_done);
      __syncwarp();
      ptx::mbar_wait(mma_done, 0);
      // nor of the other CTA's arrivals here, when this one exits
      if (half == 0 && warp == kMmaWarp && ok)
        for (int g = max(0, gtot - kPBufs<kNv>); g < gtot && ok; ++g)
          ok = ptx::mbar_wait_cluster(p_free + 8 * (g % kPBufs<kNv>), uint32_t(g / kPBufs<kNv>) & 1u);
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------ converters, query
    const int w = warp & 3, group = (warp - 8) >> 2;
    if (half == 0) {
      int jobs = 0;
      auto load_q = [&](int job) {
        if (jobs++ == 0) return first_query(job);
        auto until = [&] { return ptx::mbar_wait(q_free, uint32_t(jobs - 2) & 1u, run_polls(units)); };
        return group == 0 ? query_blocks(job, 0, five, q_full, until) : query_blocks(job, 5, four, q_full, until);
      };
      bool on = gtot > 0 && wk.start(a, job0, unit0, units);
      if constexpr (kNv) {
        // between a group's tiles, when none is in its registers: the queries of the jobs
        // that begin before its next one
        int begin = 0;
        auto queries = [&](int g) {
#pragma unroll 1
          while (on && begin <= g + 2) {
            if (!load_q(wk.job)) return false;
            begin += wk.k1 - wk.k0;
            on = wk.next(a);
          }
          return true;
        };
        ok = queries(-2) && convert<true, 2>(a, gtot, group, w, lane, ring, ring_full, ring_free, KB, k_full, k_free, 0,
                                                   queries);
      } else {
#pragma unroll 1
        for (; on && ok; on = wk.next(a)) ok = load_q(wk.job);
      }
    } else {
      if constexpr (kNv)
        ok = values();
      else
        ok = output((warp >> 2) * 128, (warp >> 2) * 128 + 128);
    }
  } else if (half == 0) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    const int group = warp >> 2, w = warp & 3;
    const int row = w * 32 + lane;
    const uint32_t lane_base = uint32_t(w * 32) << 16;
    const uint32_t p_peer = ptx::mapa_shared(ptx::smem_u32(PB) + row * 16, 1);
    const uint32_t f_peer = ptx::mapa_shared(ptx::smem_u32(side), 1);
    const uint32_t bar_peer = ptx::mapa_shared(p_full, 1);
    int g0 = 0;  // the segment's first tile
#pragma unroll 1
    for (bool on = gtot > 0 && wk.start(a, job0, unit0, units); on && ok; on = wk.next(a)) {
      const int hr = (wk.job < a.tiles ? wk.job * kPfxTileRows : (wk.job - a.tiles) * kHeads) + row;
      const float cs = fmaxf(hr < a.rows * kHeads ? a.scale_log2 * a.qs[hr] : 1.f, 1.1754944e-38f);
      if (g0 == 0) first_query(wk.job);
      float m_mine = -INFINITY, l = 0.f;  // the reference that l is relative to
      const int g1 = g0 + wk.k1 - wk.k0;
#pragma unroll 1
      for (int g = g0 + ((g0 ^ group) & 1); g < g1; g += 2) {
        const int sb = g % kSBufs, pb = g % kPBufs<kNv>;
        if (!ptx::mbar_wait(s_full + 8 * (sb), uint32_t(g / kSBufs) & 1u)) { ok = false; break; }
        ptx::tc_fence_after();
        float sv[64];
        ptx::tmem_ld32_nowait(tmem + lane_base + kSCol + sb * kNT, *reinterpret_cast<float(*)[32]>(&sv[0]));
        ptx::tmem_ld32_nowait(tmem + lane_base + kSCol + sb * kNT + 32, *reinterpret_cast<float(*)[32]>(&sv[32]));
        if (!ptx::mbar_wait(ring_full + 8 * (g % kRing), uint32_t(g / kRing) & 1u)) ok = false;
        const int valid = ring[g % kRing].valid;
        ptx::tmem_ld_wait(*reinterpret_cast<float(*)[32]>(&sv[0]));
        ptx::tmem_ld_wait(*reinterpret_cast<float(*)[32]>(&sv[32]));
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          ptx::mbar_arrive(s_free + 8 * (g % (2 * kSBufs)));
          ptx::mbar_arrive(ring_free + 8 * (g % kRing));
        }
        if (!ok) break;
        if (valid < kNT) {
#pragma unroll
          for (int i = 0; i < kNT; ++i) sv[i] = i < valid ? sv[i] : -INFINITY;
        }
        float t0 = fmaxf(sv[0], sv[1]), t1 = fmaxf(sv[2], sv[3]);
#pragma unroll
        for (int i = 4; i < 64; i += 4) {
          t0 = fmaxf(t0, fmaxf(sv[i], sv[i + 1]));
          t1 = fmaxf(t1, fmaxf(sv[i + 2], sv[i + 3]));
        }
        const float tmax = fmaxf(t0, t1) * cs;
        // the reference in use passes from tile to tile
        if (g >= 1 && !ptx::mbar_wait(turn + 8 * (w), uint32_t(g - 1) & 1u)) { ok = false; break; }
        const float m_old = g == g0 ? -INFINITY : m_run[row];
        float m_use = m_old, alpha = 1.f;
        bool moved = false;
        if (__any_sync(0xffffffffu, !(tmax - m_old <= kMost<kNv> && tmax - m_old >= kLeast<kNv>))) {
          const bool first = m_old == -INFINITY;
          const float top = first ? -INFINITY : m_top[row];
          if (first) m_use = floorf(tmax) - kFirst<kNv>;
          else if (tmax - m_old > kMost<kNv>) m_use = floorf(tmax) - kRaised<kNv>;
          else if (tmax - m_old < kLeast<kNv> && tmax != -INFINITY) m_use = fmaxf(floorf(tmax) - kLowered<kNv>, top - kTopDrop);
          m_run[row] = m_use;
          m_top[row] = fmaxf(top, m_use);
          if (!first) alpha = pow2_whole(m_old - m_use);
          moved = __any_sync(0xffffffffu, alpha != 1.f);
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(turn + 8 * (w));
        if (m_mine != m_use && m_mine != -INFINITY) l *= pow2_whole(m_mine - m_use);
        m_mine = m_use;
        const float off = m_use == -INFINITY ? 0.f : -m_use;
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
        if constexpr (!kNv) {
          if (tmax - m_use > kLarge) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) split_large(pk[i], pk[i + 1], pk[i], pk[i + 1]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; i += 2) split_small(pk[i], pk[i + 1], pk[i], pk[i + 1]);
          }
        }
        l += p0 + p1;
        // this slot of P is free once P . V of the tile before in it is done
        if (g >= kPBufs<kNv> && !ptx::mbar_wait_cluster(p_free + 8 * (pb), uint32_t(g / kPBufs<kNv> - 1) & 1u)) { ok = false; break; }
        const uint32_t dst = p_peer + pb * kPBuf, bar = bar_peer + pb * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // (FP8: the words of the two parts alternate; chunks 0..3 are the E5M2 part's)
          const int at = kNv ? 4 * i : 8 * (i & 3) + (i >> 2), by = kNv ? 1 : 2;
          ptx::st_async_f4(dst + i * kPChunk, make_float4(__uint_as_float(pk[at]), __uint_as_float(pk[at + by]),
                                                          __uint_as_float(pk[at + 2 * by]), __uint_as_float(pk[at + 3 * by])),
                           bar);
        }
        ptx::st_async_f1(f_peer + pb * kPSide + row * 4, alpha, bar);
        if (lane == 0) ptx::st_async_f1(f_peer + pb * kPSide + 512 + w * 4, __uint_as_float(moved ? 1u : 0u), bar);
      }
      if (!ok) break;
      g0 = g1;
      // (the reference of the segment's last tile is O's)
      float* ml = a.ml + (size_t(wk.job + clu) * 2 + ((group ^ (g1 - 1)) & 1)) * 256 + row;
      ml[0] = m_mine;
      ml[128] = l;
      if (threadIdx.x == 0) {
        if (wk.k0 == 0) a.plan[2 * wk.job] = clu;
        if (wk.k1 == wk.n) a.plan[2 * wk.job + 1] = clu;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;");
    if constexpr (kNv)
      ok = warp >= 4 ? values() : output(0, kDNope);
    else
      ok = output((warp >> 2) * 128, (warp >> 2) * 128 + 128);
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
// The query, each head's 576 values times a power of two, one warp per head. For NVFP4
// latents as fp16, the largest in [2^14, 2^15): a bf16 value has 8 significant bits,
// so what is above 2^-32 of the largest stays exact (fp16's subnormals are multiples
// of 2^-24). For FP8 latents as x = hi + lo, hi = E4M3(x) and lo = E5M2(x - hi), the
// largest in [2^7, 2^8): hi has 4 bits of x, and the rest is at most 8 units of x's
// last bit, which three bits hold, so the sum is exact where hi is not subnormal,
// that is above 2^-13 of the largest; below, x - hi <= 2^-10 is off by at most 2^-13,
// 2^-20 of the largest. Written in 16-B chunks, each head by head, so that
// 32 consecutive heads load 512 contiguous bytes into tensor memory wherever a tile
// of heads starts; a block's eight heads go through shared memory and out as whole
// lines (64 rows: 4.8 us, 5.9 written word by word with scalar conversions).
// ---------------------------------------------------------------------------
constexpr int kQueryWarps = 8;
static_assert(kHeads % kQueryWarps == 0, "whole blocks");

// Two values' E4M3 parts and the E5M2 parts of the rests, a's in the low byte.
__device__ __forceinline__ void split_query(float a, float b, uint32_t& hi, uint32_t& lo) {
  asm("{\n\t.reg .b16 h, l, p, q;\n\t.reg .b32 u;\n\t.reg .f32 x, y;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %3, %2;\n\tcvt.rn.f16x2.e4m3x2 u, h;\n\tmov.b32 {p, q}, u;\n\t"
      "cvt.f32.f16 x, p;\n\tcvt.f32.f16 y, q;\n\tsub.rn.f32 x, %2, x;\n\tsub.rn.f32 y, %3, y;\n\t"
      "cvt.rn.satfinite.e5m2x2.f32 l, y, x;\n\tcvt.u32.u16 %0, h;\n\tcvt.u32.u16 %1, l;\n}\n"
      : "=&r"(hi), "=r"(lo)
      : "f"(a), "f"(b));
}

template <bool kNv>
__global__ void __launch_bounds__(32 * kQueryWarps)
    prefix_query_kernel(const uint32_t* __restrict__ q, int heads, uint32_t* __restrict__ prepared, float* __restrict__ qs,
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
  constexpr int kChunks = 2 * kDQK / 16, kPitch = 4 * kQueryWarps + 4;  // words of a chunk of all heads, padded
  __shared__ __align__(16) uint32_t s_out[kChunks * kPitch];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, hr = blockIdx.x * kQueryWarps + warp;
  auto put = [&](int chunk0, int i, uint32_t v) { s_out[(chunk0 + (i >> 2)) * kPitch + warp * 4 + (i & 3)] = v; };
  // nine words (two values each) per lane; FP8 needs them in pairs (four values to a word)
  constexpr int kWords = kDQK / 2, kPer = kWords / 32;
  uint32_t w[kPer + 1];
  auto word = [&](int i) { return kNv ? i * 32 + lane : (i >> 1) * 64 + 2 * lane + (i & 1); };
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < kPer + 1; ++i) {
    w[i] = word(i) < kWords && i < (kNv ? kPer : kPer + 1) ? __ldg(q + size_t(hr) * kWords + word(i)) : 0u;
    m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  // 2^-e in two factors: e reaches down to -147
  const int e = m > 0.f && m < INFINITY ? ilogbf(m) - (kNv ? 14 : 7) : 0;
  // An infinity makes each logit infinite or NaN, and the softmax NaN: the whole head is NaN
  // (a saturating conversion would make it finite).
  const float f0 = m < INFINITY ? scalbnf(1.f, -e / 2) : __uint_as_float(0x7FC00000u), f1 = scalbnf(1.f, -e - (-e / 2));
  if constexpr (kNv) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const __half2 h = __floats2half2_rn(__uint_as_float(w[i] << 16) * f0 * f1, __uint_as_float(w[i] & 0xFFFF0000u) * f0 * f1);
      put(0, word(i), *reinterpret_cast<const uint32_t*>(&h));
    }
  } else {
#pragma unroll
    for (int i = 0; i < kPer + 1; i += 2) {
      if (word(i) >= kWords) continue;
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int d = 0; d < 2; ++d)
        split_query(__uint_as_float(w[i + d] << 16) * f0 * f1, __uint_as_float(w[i + d] & 0xFFFF0000u) * f0 * f1, hi[d],
                    lo[d]);
      const int out = word(i) >> 1;  // the word of four dims: 16 dims a chunk
      put(0, out, hi[0] | hi[1] << 16);
      put(kChunks / 2, out, lo[0] | lo[1] << 16);
    }
  }
  if (lane == 0) qs[hr] = scalbnf(1.f, e);
  __syncthreads();
  for (int i = threadIdx.x; i < kChunks * kQueryWarps; i += 32 * kQueryWarps) {
    const int chunk = i / kQueryWarps, h = i % kQueryWarps;
    reinterpret_cast<uint4*>(prepared)[size_t(chunk) * heads + blockIdx.x * kQueryWarps + h] =
        *reinterpret_cast<const uint4*>(s_out + chunk * kPitch + h * 4);
  }
}

// ---------------------------------------------------------------------------
// Merge of a row's segments, those of its prefix tile and then those of its private
// job: with M the largest reference, out = lat_scale * sum_i 2^(m_i - M) O_i / L and
// L = sum_i 2^(m_i - M) l_i (a segment's two softmax groups have sums and references m of their
// own; its O has the first one's). A warp has 32 heads, a lane each, 16
// dims of them and every kSplit-th segment: a row alone has a segment from nearly
// every pair, many rows have few each. The partial outputs' bytes bound it: 64 rows, 33 MB, 8.1 us;
// 252 rows, 99 MB, 24 us.
// ---------------------------------------------------------------------------
constexpr int kMergeWarps = 8;

template <int kSplit>
__global__ void __launch_bounds__(32 * kMergeWarps) prefix_merge_kernel(PfxArgs a, __nv_bfloat16* __restrict__ out,
                                                                       float* __restrict__ lse) {
  constexpr int kParts = kMergeWarps / kSplit;  // warps with dims of their own
  constexpr int kChunks = 4 * kParts;           // of four dims, of the CTA
  constexpr int kPitch = kChunks + 1;
  __shared__ float4 s_acc[kSplit > 1 ? kMergeWarps : 1][4][32];
  __shared__ float2 s_ml[kSplit > 1 ? kMergeWarps : 1][32];
  __shared__ uint2 s_out[32][kPitch];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % kSplit;
  const int r = blockIdx.x, h = blockIdx.y * 32 + lane, c0 = blockIdx.z * kChunks + warp / kSplit * 4;
  const int hr = r * kHeads + h, job0 = hr / kPfxTileRows, job1 = a.tiles + r;
  float4 acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, tot = 0.f;
  auto add = [&](int j, float w, const float4& v) {
    acc[j].x = fmaf(w, v.x, acc[j].x); acc[j].y = fmaf(w, v.y, acc[j].y);
    acc[j].z = fmaf(w, v.z, acc[j].z); acc[j].w = fmaf(w, v.w, acc[j].w);
  };
  if (a.lens[r] > 0) {
    const int f0 = a.prefix > 0 ? a.plan[2 * job0] : 0, n0 = a.prefix > 0 ? a.plan[2 * job0 + 1] - f0 + 1 : 0;
    const int f1 = a.plan[2 * job1], n1 = a.plan[2 * job1 + 1] - f1 + 1;
    // segment i's slot and row
    auto slot = [&](int i) { return i < n0 ? job0 + f0 + i : job1 + f1 + i - n0; };
    auto row = [&](int i) { return i < n0 ? hr % kPfxTileRows : h; };
#pragma unroll 2
    for (int i = part; i < n0 + n1; i += kSplit) {
      const float* ml = a.ml + size_t(slot(i)) * 512 + row(i);
      const float4* o = reinterpret_cast<const float4*>(a.part) + size_t(slot(i)) * kPfxTileRows * (kDNope / 4) +
                        c0 * kPfxTileRows + row(i);
      float4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = __ldg(o + j * kPfxTileRows);
      const float ma = __ldg(ml), mb = __ldg(ml + 256), la = __ldg(ml + 128), lb = __ldg(ml + 384);
      const float old = m;
      m = fmaxf(m, fmaxf(ma, mb));
      const float mm = m == -INFINITY ? 0.f : m;
      const float keep = exp2f(old - mm), w = exp2f(ma - mm);
      tot = fmaf(exp2f(ma - mm), la, fmaf(exp2f(mb - mm), lb, tot * keep));
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[j].x *= keep; acc[j].y *= keep; acc[j].z *= keep; acc[j].w *= keep;
        add(j, w, v[j]);
      }
    }
  }
  if constexpr (kSplit > 1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) s_acc[warp][j][lane] = acc[j];
    s_ml[warp][lane] = make_float2(m, tot);
    __syncthreads();
    if (part == 0) {
      for (int i = 1; i < kSplit; ++i) m = fmaxf(m, s_ml[warp + i][lane].x);
      const float mm = m == -INFINITY ? 0.f : m;
      tot = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i = 0; i < kSplit; ++i) {
        const float2 ml = s_ml[warp + i][lane];
        const float w = exp2f(ml.x - mm);  // a warp without a segment has m = -infinity and weight 0
        tot = fmaf(w, ml.y, tot);
#pragma unroll
        for (int j = 0; j < 4; ++j) add(j, w, s_acc[warp + i][j][lane]);
      }
    }
  }
  if (part == 0) {
    const float inv = tot != 0.f ? a.lat_scale / tot : 0.f;  // NaN stays NaN
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float4 v = tot != 0.f ? make_float4(acc[j].x * inv, acc[j].y * inv, acc[j].z * inv, acc[j].w * inv)
                                  : make_float4(0.f, 0.f, 0.f, 0.f);
      const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
      s_out[lane][warp / kSplit * 4 + j] =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    }
    const float mm = m == -INFINITY ? 0.f : m;
    if (lse && c0 == 0) lse[hr] = tot != 0.f ? (mm + log2f(tot)) * 0.6931471805599453f : -INFINITY;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * kChunks; i += 32 * kMergeWarps) {
    const int row = i / kChunks, c = i % kChunks;
    reinterpret_cast<uint2*>(out + size_t(r * kHeads + blockIdx.y * 32 + row) * kDNope)[blockIdx.z * kChunks + c] =
        s_out[row][c];
  }
}

}  // namespace

cudaError_t launch_prefix_mla(const dsa_params_t& p, const WsLayout& L, char* ws, const void* q, const void* lat_pool,
                              const int32_t* prefix_pages, int prefix_len, const int32_t* block_table,
                              const int32_t* ctx_lens, void* out, float* lse, cudaStream_t st) {
  PfxArgs a;
  a.q = reinterpret_cast<const uint4*>(ws + L.pfx_q);
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
  const bool nv = p.lat_fmt == DSA_LAT_NVFP4_352;
  a.lat_scale = p.latent_scale;
  CUtensorMap kmap, rmap;
  std::memset(&kmap, 0, sizeof(kmap));  // NVFP4 rows go through the converters
  std::memset(&rmap, 0, sizeof(rmap));
  if (!nv) {
    // [num_pages][64][576] bytes: 128 dims of a page's rows at a time, and the 64 rope dims
    const uint64_t dims[3] = {uint64_t(kDQK), uint64_t(kPage), uint64_t(p.num_pages)};
    const uint64_t strides[2] = {uint64_t(kDQK), uint64_t(p.lat_page_stride)};
    const uint32_t box[3] = {128, kPage, 1}, rbox[3] = {64, kPage, 1};
    if (!encode_map(&kmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, lat_pool, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_map(&rmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, lat_pool, 3, dims, strides, rbox, CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
  }
  const int heads = L.rows * kHeads;
  cudaError_t e = launch_pdl(nv ? prefix_query_kernel<true> : prefix_query_kernel<false>,
                             dim3((heads + kQueryWarps - 1) / kQueryWarps), dim3(32 * kQueryWarps), 0, st,
                             static_cast<const uint32_t*>(q), heads, reinterpret_cast<uint32_t*>(ws + L.pfx_q),
                             reinterpret_cast<float*>(ws + L.pfx_qs), ctx_lens, lens, int(p.n_q), prefix_len, L.cap, a.err);
  if (e != cudaSuccess) return e;
  const size_t smem = nv ? kSmem<true> : kSmem<false>;
  auto kern = nv ? prefix_mla_kernel<true> : prefix_mla_kernel<false>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  const int clusters = std::max(1, std::min(kPfxMaxClusters, sm_count() / 2));
  e = launch_pdl(kern, dim3(2 * clusters), dim3(kThreads), smem, st, kmap, rmap, a);
  if (e != cudaSuccess) return e;
  // a row has a little more than clusters / rows segments (one row of 65: 20.5 us shared by
  // eight warps, 26.5 not; 24 rows of five: 42.3 and 39.7)
  const bool split = L.rows * 4 <= clusters;
  return launch_pdl(split ? prefix_merge_kernel<kMergeWarps> : prefix_merge_kernel<1>,
                    dim3(L.rows, kHeads / 32, kDNope / 4 / (split ? 4 : 4 * kMergeWarps)), dim3(32 * kMergeWarps), 0, st,
                    a, static_cast<__nv_bfloat16*>(out), lse);
}

}  // namespace dsa
