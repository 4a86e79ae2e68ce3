// Accumulated attention weight of every cached token: mass[s] += sum over rows t and heads h of
// exp(scale q_th . c_s - lse_th), for the tokens that the rows see.
//
// It is the dense attention's first product without its second, and its sum runs over the heads, not the tokens. So a
// token is a row of the product here: S = C . Q^T with 128 tokens (two pages) against a query row's 96 heads,
// one accumulator lane per token; a thread has one token, and its sum over the heads is its own: no shuffle, no
// atomic, the same bits in any batch. The query is prepared as for the dense attention (FP8 latents: two FP8 parts, here both
// E4M3, the second times 2^5, multiplied with the latents as TMA brings them in one product of 192 columns, so that the latents
// are read from shared memory once: with a product for each part 60.8 us for 40 requests; NVFP4 ones: fp16) and stays in
// shared memory (110 KB) while tiles of tokens stream past it. NVFP4 latents are converted to fp16 and multiplied from tensor
// memory: through shared memory, which the products read 28 KB of per K-block, their 16 KB took 226 us for the 48 rows.
//
// The tiles of all requests are a line that is cut into equal runs, one per CTA, and a run into chunks of at most 16
// tiles of one request. A chunk is gone through once per row (its latents come from L2 after the first), its sums
// wait in shared memory, and are added to the weights once. The next row's query arrives block by block behind the
// last tile that uses the old one.
//
// Measured (one GB300; these are "the 40 requests" and "the 48 rows" of this file): 40 requests of up to 16,384 FP8 tokens 57.5 us in
// a graph, of which the query's preparation and the start are some 8 (292 MB of latents and weights, 5.1 TB/s; 15.8 ms with plain
// loops), bound by the bytes, then by the issue of the products; 6 requests of 8 rows on 20,001 NVFP4 tokens 92.5 us (1.11 PFLOP/s),
// bound by the converters, which go through a tile once per row, and by shared memory; one row on 4,100 tokens 8.6 us.
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include <cstring>

#include "dsa_internal.cuh"
#include "sm103_ptx.cuh"

namespace dsa {

namespace {

constexpr int kTok = 128;                     // tokens of a tile
// A tile comes in three parts. FP8: 192 dims of its rows, 128 rows of 128 B and 128 of 64 B, in four stages. NVFP4: 128 B of its
// rows as they lie, in six. (The issuing warp's wait for a part costs some 95 cycles behind its products, which it blocks on:
// parts of 128 dims took 62.6 us for the 40 requests, these 60.8.)
constexpr int kParts = 3;
template <bool kNv>
constexpr int kStage = kNv ? kTok * 128 : kTok * 192;  // 16,384 or 24,576 B
template <bool kNv>
constexpr int kStages = kNv ? 6 : 4;
constexpr int kRingBytes = 6 * 16384;
static_assert(kStage<true> * kStages<true> == kRingBytes && kStage<false> * kStages<false> == kRingBytes, "either ring");
constexpr int kQBlk = kHeads * 128;           // 12,288 B: 128 B of each head
// of a row's heads: pieces of the dims (FP8: [4][part], and [part] of 64 rotary bytes)
constexpr int kQBytes = 9 * kQBlk;
constexpr int kChunk = 16;                    // tiles of a chunk
// tensor memory: two accumulators of 96 columns, FP8: of 192, for the two parts of the query; NVFP4: and a tile's values in three
// stages of 96 columns (192 dims: with a stage for each of the nine K-blocks the wait and the fence of every four products took
// 116 us for the 48 rows, this 102)
constexpr int kDBufs = 2;
template <bool kNv>
constexpr int kDCols = kNv ? 96 : 192;
constexpr int kACol = 192;
static_assert(kACol + kDQK / 2 <= 512, "tensor memory");
template <bool kNv>
constexpr int kThreads = kNv ? 512 : 256;
// warps: 0..3 sums, 4 products, 5 latents, 6 query, 7 the heads' constants, 8..15 converters (NVFP4)
constexpr int kMmaWarp = 4, kTileWarp = 5, kQueryWarp = 6, kHeadWarp = 7;
constexpr int kNumBars = 2 * 6 + 2 * kParts + 2 * 4 + 4 + 2 * kParts + 1;
constexpr size_t kSmem = 1024 + kRingBytes + kQBytes + kChunk * kTok * 4 + 2 * 2 * kHeads * 4 + kNumBars * 8 + 64;
static_assert(kSmem <= 232448 - 512, "shared memory, with the static variables");
constexpr uint32_t kPolls = 1u << 20;  // 4 s

struct MassArgs {
  const float* qs;    // [rows * 96] the prepared query's scales
  const float* lse;   // [rows * 96]
  const int32_t* table;
  const int32_t* ctx;
  float* mass;
  int* err;
  int64_t mass_stride;
  int batch, n_q, max_pages, cap, num_pages, sinks, window, fresh;
  float scale_log2;
};

__device__ __forceinline__ int pages_of(int n) { return (n + kPage - 1) / kPage; }

// The pages that some row of a request with n tokens sees: those of its sinks and those from its first row's window on.
struct Span {
  int n, n_head, p0, pages;
  __device__ __forceinline__ Span(const MassArgs& a, int ctx) {
    n = ctx >= a.n_q && ctx <= a.cap ? ctx : 0;
    const int first = max(0, n - a.n_q + 1 - a.window), head = first <= a.sinks ? 0 : a.sinks;
    n_head = pages_of(head);
    p0 = head == 0 && first <= a.sinks ? 0 : max(first / kPage, n_head);
    pages = n > 0 ? n_head + pages_of(n) - p0 : 0;
  }
  __device__ __forceinline__ int tiles() const { return (pages + 1) / 2; }
  __device__ __forceinline__ int page(int i) const { return i < n_head ? i : p0 + i - n_head; }
};

// A CTA's run of the line, chunk by chunk, and the rows that a chunk is gone through for.
struct Walk {
  int b, t0, nt, left;  // tiles [t0, t0 + nt) of request b
  int r0, r1;           // rows [r0, r1] of it see some of them
  __device__ __forceinline__ void set(const MassArgs& a, const Span& s) {
    nt = min(min(kChunk, left), s.tiles() - t0);
    const int lo = s.page(2 * t0) * kPage, hi = min(s.n - 1, s.page(min(2 * (t0 + nt), s.pages) - 1) * kPage + kPage - 1);
    const int base = s.n - a.n_q;  // row t sees base + t + 1 tokens
    r0 = max(0, lo - base);
    r1 = lo < a.sinks ? a.n_q - 1 : min(a.n_q - 1, hi + a.window - base - 1);
    left -= nt;
  }
  __device__ __forceinline__ bool start(const MassArgs& a, int b0, int tile, int tiles) {
    b = b0;
    t0 = tile;
    left = tiles;
    if (left <= 0) return false;
    set(a, Span(a, a.ctx[b]));
    return true;
  }
  __device__ __forceinline__ bool next(const MassArgs& a) {
    if (left <= 0) return false;
    t0 += nt;
    if (t0 >= Span(a, a.ctx[b]).tiles()) {
      t0 = 0;
      do ++b;
      while (Span(a, a.ctx[b]).tiles() == 0);
    }
    set(a, Span(a, a.ctx[b]));
    return true;
  }
};

// Four E4M3 bytes -> four fp16.
__device__ __forceinline__ void expand_e4m3(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
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

template <bool kNv>
__global__ void __launch_bounds__(kThreads<kNv>, 1)
    mass_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap rmap,
                const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap qrmap,
                const __grid_constant__ MassArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* qbuf = ring + kRingBytes;
  float* acc = reinterpret_cast<float*>(qbuf + kQBytes);   // [kChunk][128]
  float* heads = acc + kChunk * kTok;                      // [2][2][96] factors and offsets
  const uint32_t bars = ptx::smem_u32(heads + 2 * 2 * kHeads);
  const uint32_t full = bars, free = full + 8 * 6;                        // [kStages]
  const uint32_t q_full = free + 8 * 6, q_free = q_full + 8 * kParts;     // the query's blocks that a part needs first
  const uint32_t d_full = q_free + 8 * kParts, d_free = d_full + 8 * 4;   // [kDBufs]
  const uint32_t h_full = d_free + 8 * 4, h_free = h_full + 16;           // [2]
  const uint32_t a_full = h_free + 16, a_free = a_full + 8 * kParts;      // NVFP4: a part's values in tensor memory
  const uint32_t mma_done = a_free + 8 * kParts;
  __shared__ uint32_t tmem_slot;
  __shared__ int s_sum[32], s_b, s_tile, s_bad[2];
  constexpr int kD = kDBufs, kSt = kStages<kNv>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSt; ++i) {
      ptx::mbar_init(full + 8 * i, 1);
      ptx::mbar_init(free + 8 * i, kNv ? 8 : 1);
    }
    for (int i = 0; i < kParts; ++i) {
      ptx::mbar_init(a_full + 8 * i, 8);
      ptx::mbar_init(a_free + 8 * i, 1);
      ptx::mbar_init(q_full + 8 * i, 1);
      ptx::mbar_init(q_free + 8 * i, 1);
    }
    for (int i = 0; i < kDBufs; ++i) {
      ptx::mbar_init(d_full + 8 * i, 1);
      ptx::mbar_init(d_free + 8 * i, 4);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(h_full + 8 * i, 1);
      ptx::mbar_init(h_free + 8 * i, 4);
    }
    ptx::mbar_init(mma_done, 1);
    ptx::fence_mbar_init();
    s_b = s_tile = 0;
  }
  if (warp == kMmaWarp) {
    ptx::tmem_alloc(&tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_wait();

  // ---- this CTA's run of the line
  auto scan = [&](int n, int& before, int& all) {
    int v = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += y;
    }
    __syncthreads();
    if (lane == 31) s_sum[warp] = v;
    __syncthreads();
    before = v - n;
    all = 0;
    for (int i = 0; i < kThreads<kNv> / 32; ++i) {
      if (i < warp) before += s_sum[i];
      all += s_sum[i];
    }
  };
  auto tiles_of = [&](int b) { return b < a.batch ? Span(a, a.ctx[b]).tiles() : 0; };
  long long line = 0;
  int before, all;
  for (int b0 = 0; b0 < a.batch; b0 += kThreads<kNv>) {
    scan(tiles_of(b0 + int(threadIdx.x)), before, all);
    line += all;
  }
  const long long lo = line * blockIdx.x / gridDim.x, hi = line * (blockIdx.x + 1) / gridDim.x;
  const int run = int(hi - lo);
  long long base = 0;
  for (int b0 = 0; b0 < a.batch && base <= lo; b0 += kThreads<kNv>) {
    const int b = b0 + int(threadIdx.x), n = tiles_of(b);
    scan(n, before, all);
    const long long first = base + before;
    if (lo >= first && lo < first + n) {
      s_b = b;
      s_tile = int(lo - first);
    }
    base += all;
  }
  __syncthreads();
  const int b0 = s_b, tile0 = s_tile;
  bool ok = true;
  Walk wk;

  if (warp < 4) {
    // ------------------------------------------------------------ sums
    const int tok = threadIdx.x;
    const uint32_t lanes = uint32_t(warp * 32) << 16;
    int g = 0, hn = 0;
#pragma unroll 1
    for (bool on = wk.start(a, b0, tile0, run); on && ok; on = wk.next(a)) {
      const Span s(a, a.ctx[wk.b]);
#pragma unroll 1
      for (int r = wk.r0; r <= wk.r1 && ok; ++r, ++hn) {
        const int hb = hn & 1, seen = s.n - a.n_q + r + 1;
        if (!ptx::mbar_wait(h_full + 8 * hb, uint32_t(hn >> 1) & 1u, kPolls)) { ok = false; break; }
        const float4* cs = reinterpret_cast<const float4*>(heads + hb * 2 * kHeads);
        const float4* co = cs + kHeads / 4;
        const bool bad = s_bad[hb] != 0;
#pragma unroll 1
        for (int k = 0; k < wk.nt; ++k, ++g) {
          // the token, and at the last row what its weight was
          const int i = 2 * (wk.t0 + k) + (tok >> 6);
          const int at = i < s.pages ? s.page(i) * kPage + (tok & 63) : s.n;
          bool put = r == wk.r1 && at < s.n && (at < a.sinks || at + a.window >= s.n - a.n_q + 1);
          float old = 0.f;
          float* dst = a.mass + wk.b * a.mass_stride + at;
          if (put) {
            const int pg = __ldg(a.table + size_t(wk.b) * a.max_pages + at / kPage);
            put = pg >= 0 && pg < a.num_pages;
            if (at < s.n - a.fresh) old = *dst;
          }
          const int buf = g % kD;
          if (!ptx::mbar_wait(d_full + 8 * buf, uint32_t(g / kD) & 1u, kPolls)) { ok = false; break; }
          ptx::tc_fence_after();
          float w0 = 0.f, w1 = 0.f, w2 = 0.f, w3 = 0.f;
          float z[2][32];  // NVFP4: a piece of 32 heads and the next; FP8: both parts of one
          const uint32_t d = tmem + lanes + buf * kDCols<kNv>;
          ptx::tmem_ld32_nowait(d, z[0]);
#pragma unroll
          for (int c = 0; c < 3; ++c) {
            float(&x)[32] = z[kNv ? c & 1 : 0];
            if constexpr (kNv) {
              ptx::tmem_ld_wait(x);
              if (c < 2) ptx::tmem_ld32_nowait(d + 32 * (c + 1), z[(c + 1) & 1]);
            } else {
              ptx::tmem_ld32_nowait(d + kHeads + 32 * c, z[1]);
              ptx::tmem_ld_wait(x);
              ptx::tmem_ld_wait(z[1]);
#pragma unroll
              for (int h = 0; h < 32; ++h) x[h] = fmaf(z[1][h], 0.03125f, x[h]);  // 2^-5
            }
#pragma unroll
            for (int h = 0; h < 32; h += 4) {
              const float4 f = cs[8 * c + h / 4], o = co[8 * c + h / 4];
              float y[4] = {fmaf(x[h], f.x, o.x), fmaf(x[h + 1], f.y, o.y), fmaf(x[h + 2], f.z, o.z), fmaf(x[h + 3], f.w, o.w)};
              if (bad) {  // heads without a finite lse, whatever their products are
                y[0] = o.x == -INFINITY ? o.x : y[0];
                y[1] = o.y == -INFINITY ? o.y : y[1];
                y[2] = o.z == -INFINITY ? o.z : y[2];
                y[3] = o.w == -INFINITY ? o.w : y[3];
              }
              ptx::add2(w0, w1, ptx::ex2_approx(y[0]), ptx::ex2_approx(y[1]));
              ptx::add2(w2, w3, ptx::ex2_approx(y[2]), ptx::ex2_approx(y[3]));
            }
            if (!kNv && c < 2) ptx::tmem_ld32_nowait(d + 32 * (c + 1), z[0]);
          }
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(d_free + 8 * buf);
          const bool sees = at < seen && (at < a.sinks || at >= seen - a.window);
          float w = sees ? (w0 + w1) + (w2 + w3) : 0.f;
          if (r > wk.r0) w += acc[k * kTok + tok];
          if (r < wk.r1) acc[k * kTok + tok] = w;
          else if (put) *dst = old + w;
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(h_free + 8 * hb);
      }
    }
  } else if (warp == kMmaWarp) {
    // ------------------------------------------------------------ S = C . Q^T
    const uint32_t r0 = ptx::smem_u32(ring), q0 = ptx::smem_u32(qbuf);
    int g = 0, st = 0, qn = -1, row_in = -1;  // tiles, the K-block's place in its ring, queries so far; the row in shared memory
    uint32_t par = 0;
    bool on = wk.start(a, b0, tile0, run);
#pragma unroll 1
    while (on && ok) {
      const int first = wk.b * a.n_q + wk.r0, last = wk.b * a.n_q + wk.r1, nt = wk.nt;
      on = wk.next(a);
      const int then = on ? wk.b * a.n_q + wk.r0 : -1;
#pragma unroll 1
      for (int row = first; row <= last && ok; ++row) {
        const bool fresh_q = row != row_in;
        if (fresh_q) ++qn;
        row_in = row;
        const bool leaves = (row < last ? row + 1 : then) != row;
#pragma unroll 1
        for (int k = 0; k < nt && ok; ++k, ++g) {
          const int buf = g % kD;
          if (g >= kD && !ptx::mbar_wait(d_free + 8 * buf, uint32_t(g / kD - 1) & 1u, kPolls)) { ok = false; break; }
          ptx::tc_fence_after();
          const uint32_t d = tmem + buf * kDCols<kNv>;
#pragma unroll
          for (int i = 0; i < kParts; ++i) {
            if (fresh_q && k == 0 && !ptx::mbar_wait(q_full + 8 * i, uint32_t(qn) & 1u, kPolls)) { ok = false; break; }
            if (!ptx::mbar_wait(kNv ? a_full + 8 * i : full + 8 * st, kNv ? uint32_t(g) & 1u : par, kPolls)) { ok = false; break; }
            // (TMA's writes need no fence; the converters' in tensor memory do)
            if (kNv) ptx::tc_fence_after();
            const uint32_t in = r0 + st * kStage<kNv>;
            if (ptx::elect_one()) {
              if constexpr (kNv) {
#pragma unroll
                for (int kk = 0; kk < 12; ++kk) {
                  const int n = 12 * i + kk;  // 16 dims of the tile's 576
                  ptx::mma_f16_tmem_a(d, tmem + kACol + n * 8, ptx::sdesc_sw128(q0 + n / 4 * kQBlk + n % 4 * 32),
                                      ptx::idesc(0, 0, kTok, kHeads), n ? 1u : 0u);
                }
                ptx::mma_commit(a_free + 8 * i);
              } else {
#pragma unroll
                for (int kk = 0; kk < 6; ++kk) {
                  const int n = 6 * i + kk;  // 32 dims of the tile's 576, against both parts of the query
                  ptx::mma_f8f6f4(d, kk < 4 ? ptx::sdesc_sw128(in + kk * 32) : ptx::sdesc_sw64(in + kTok * 128 + (kk - 4) * 32),
                                  n < 16 ? ptx::sdesc_sw128(q0 + n / 4 * 2 * kQBlk + n % 4 * 32) : ptx::sdesc_sw64(q0 + 8 * kQBlk + n % 2 * 32),
                                  ptx::idesc(0, 0, kTok, 2 * kHeads), n ? 1u : 0u);
                }
                ptx::mma_commit(free + 8 * st);
              }
              if (k == nt - 1 && leaves) {  // (FP8: the first part's blocks are used by the second, too)
                if (kNv || i == 2) ptx::mma_commit(q_free + 8 * i);
                if (!kNv && i == 1) {
                  ptx::mma_commit(q_free);
                  ptx::mma_commit(q_free + 8);
                }
              }
              if (i == kParts - 1) ptx::mma_commit(d_full + 8 * buf);
            }
            __syncwarp();
            if (!kNv && ++st == kSt) {
              st = 0;
              par ^= 1;
            }
          }
        }
      }
    }
    // nothing of this warp's left in flight when the tensor memory is released
    if (ptx::elect_one()) ptx::mma_commit(mma_done);
    __syncwarp();
    ptx::mbar_wait(mma_done, 0, kPolls);
  } else if (warp == kQueryWarp) {
    // ------------------------------------------------------------ the rows' queries
    const uint32_t q0 = ptx::smem_u32(qbuf);
    int qn = 0, row_in = -1;
#pragma unroll 1
    for (bool on = wk.start(a, b0, tile0, run); on && ok; on = wk.next(a)) {
#pragma unroll 1
      for (int row = wk.b * a.n_q + wk.r0; row <= wk.b * a.n_q + wk.r1 && ok; ++row) {
        if (row == row_in) continue;
        row_in = row;
#pragma unroll 1
        for (int i = 0; i < kParts; ++i) {
          if (qn > 0 && !ptx::mbar_wait(q_free + 8 * i, uint32_t(qn - 1) & 1u, kPolls)) { ok = false; break; }
          if (lane == 0) {
            const uint32_t bar = q_full + 8 * i;
            auto block = [&](int at, int piece) { ptx::tma_load_3d(q0 + at * kQBlk, &qmap, bar, 128 * piece, 0, row); };
            if constexpr (kNv) {
              ptx::mbar_arrive_expect_tx(bar, 3 * kQBlk);
              for (int j = 3 * i; j < 3 * i + 3; ++j) block(j, j);
            } else {  // both parts of 128-dim pieces: 0 and 1, 2, 3 and the rotary dims
              ptx::mbar_arrive_expect_tx(bar, (i == 0 ? 4 : i == 1 ? 2 : 3) * kQBlk);
              for (int j = i == 0 ? 0 : i + 1; j < i + 2; ++j)
                for (int part = 0; part < 2; ++part) block(2 * j + part, 4 * part + j);
              if (i == 2)
                for (int part = 0; part < 2; ++part)
                  ptx::tma_load_3d(q0 + 8 * kQBlk + part * kQBlk / 2, &qrmap, bar, 1024 + 64 * part, 0, row);
            }
          }
          __syncwarp();
        }
        ++qn;
      }
    }
    // no copy left in flight
    if (!ok)
      for (int i = 0; i < 2 * kParts; ++i) ptx::mbar_wait(q_full + 8 * (i >> 1), uint32_t(i & 1), 1 << 8);
  } else if (warp == kHeadWarp) {
    // ------------------------------------------------------------ the heads' factors and offsets
    int hn = 0;
#pragma unroll 1
    for (bool on = wk.start(a, b0, tile0, run); on && ok; on = wk.next(a)) {
#pragma unroll 1
      for (int r = wk.r0; r <= wk.r1; ++r, ++hn) {
        const int hb = hn & 1;
        float f[3], o[3];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          const int64_t hr = int64_t(wk.b * a.n_q + r) * kHeads + 32 * i + lane;
          f[i] = a.scale_log2 * __ldg(a.qs + hr);
          const float lse = __ldg(a.lse + hr);
          const bool good = lse - lse == 0.f;  // finite
          o[i] = good ? lse * -1.4426950408889634f : -INFINITY;
          bad |= !good;
        }
        if (hn >= 2 && !ptx::mbar_wait(h_free + 8 * hb, uint32_t(hn / 2 - 1) & 1u, kPolls)) { ok = false; break; }
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          heads[hb * 2 * kHeads + 32 * i + lane] = f[i];
          heads[hb * 2 * kHeads + kHeads + 32 * i + lane] = o[i];
        }
        const int any = __any_sync(0xffffffffu, bad);
        if (lane == 0) s_bad[hb] = any;
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(h_full + 8 * hb);
      }
    }
  } else if (warp == kTileWarp) {
    // ------------------------------------------------------------ latents by TMA, page by page
    const uint32_t r0 = ptx::smem_u32(ring);
    int c = 0;
#pragma unroll 1
    for (bool on = wk.start(a, b0, tile0, run); on && ok; on = wk.next(a)) {
      const Span s(a, a.ctx[wk.b]);
      const int i0 = 2 * wk.t0 + lane;  // a chunk's pages: a lane each
      int mine = -1;
      if (lane < 2 * wk.nt && i0 < s.pages) {
        mine = __ldg(a.table + size_t(wk.b) * a.max_pages + s.page(i0));
        if (mine < 0 || mine >= a.num_pages) {
          atomicOr(a.err, DSA_DEVERR_BLOCK_TABLE);
          mine = -1;
        }
      }
#pragma unroll 1
      for (int r = wk.r0; r <= wk.r1 && ok; ++r) {
#pragma unroll 1
        for (int k = 0; k < wk.nt && ok; ++k) {
          const int p0 = __shfl_sync(0xffffffffu, mine, 2 * k), p1 = __shfl_sync(0xffffffffu, mine, 2 * k + 1);
#pragma unroll 1
          for (int i = 0; i < kParts; ++i, ++c) {
            const int st = c % kSt, j = kNv ? (i + 2) % 3 : i;  // (NVFP4: the last 128 B, with the scales, first)
            if (c >= kSt && !ptx::mbar_wait(free + 8 * st, uint32_t(c / kSt - 1) & 1u, kPolls)) { ok = false; break; }
            if (lane == 0) {
              const uint32_t dst = r0 + st * kStage<kNv>, bar = full + 8 * st;
              // (a page that is missing leaves what lay there: its tokens' sums are not used)
              const uint32_t bytes = ((p0 >= 0) + (p1 >= 0)) * (kStage<kNv> / 2);
              if (bytes) ptx::mbar_arrive_expect_tx(bar, bytes);
              else ptx::mbar_arrive(bar);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int pg = h ? p1 : p0;
                if (pg < 0) continue;
                ptx::tma_load_3d(dst + h * 8192, &kmap, bar, kNv ? 32 * j : 192 * j, 0, pg);
                if (!kNv) ptx::tma_load_3d(dst + kTok * 128 + h * 4096, &rmap, bar, 192 * j + 128, 0, pg);
              }
            }
            __syncwarp();
          }
        }
      }
    }
    if (!ok)
      for (int i = 0; i < 2 * kSt; ++i) ptx::mbar_wait(full + 8 * (i >> 1), uint32_t(i & 1), 1 << 8);
  } else if (kNv && warp >= 8) {
    // ------------------------------------------------------------ NVFP4 latents to fp16, two threads a token (a warp of
    // each group): 32 values are 16 columns of the token's lane of tensor memory, so they cost shared memory nothing
    const int group = (warp - 8) >> 2, tok = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + (uint32_t((warp & 3) * 32) << 16) + kACol;
    const uint8_t* mine = ring + tok * 128;
    auto piece = [&](int slot, int i) {  // 16 B of the token's 128 in a stage (128-B swizzle)
      return *reinterpret_cast<const uint4*>(mine + slot * kStage<kNv> + ((i ^ (tok & 7)) << 4));
    };
    int g = 0;
#pragma unroll 1
    for (bool on = wk.start(a, b0, tile0, run); on && ok; on = wk.next(a)) {
#pragma unroll 1
      for (int n = wk.nt * (wk.r1 - wk.r0 + 1); n > 0 && ok; --n, ++g) {
        const int s0 = g % 2 * 3;
        const uint32_t par = uint32_t(g / 2) & 1u;
        auto take = [&](int slot) {  // a stage has been read
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(free + 8 * (s0 + slot));
        };
        if (!ptx::mbar_wait(full + 8 * s0, par, kPolls)) { ok = false; break; }
        const uint4 sc[2] = {piece(s0, 0), piece(s0, 1)};
        uint4 rope[4];
        if (group == 1) {
#pragma unroll
          for (int i = 0; i < 4; ++i) rope[i] = piece(s0, 2 + i);
        }
        take(0);
        if (!ptx::mbar_wait(full + 8 * (s0 + 1), par, kPolls)) { ok = false; break; }
#pragma unroll
        for (int i = 0; i < kParts; ++i) {
          // the group's three of the tile's 18 pieces of 32 dims, of which the last two are rotary
          if (i == 1 && !ptx::mbar_wait(full + 8 * (s0 + 2), par, kPolls)) ok = false;
          uint32_t f[3][16];
          auto convert = [&](int p, uint32_t (&o)[16]) {
            if (p < 16) {
              const uint4 v = piece(s0 + 1 + p / 8, p % 8);
              const uint4& q = sc[p / 8];
              const uint32_t four = p / 2 % 4 == 0 ? q.x : p / 2 % 4 == 1 ? q.y : p / 2 % 4 == 2 ? q.z : q.w;
              uint32_t two, none;
              expand_e4m3(p % 2 ? four >> 16 : four, two, none);
              const __half2 h = *reinterpret_cast<const __half2*>(&two);
              const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint4 x = expand_e2m1(w[e], e < 2 ? __low2half2(h) : __high2half2(h));
                o[4 * e] = x.x; o[4 * e + 1] = x.y; o[4 * e + 2] = x.z; o[4 * e + 3] = x.w;
              }
            } else {
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const uint4& x = rope[2 * (p - 16) + e];
                expand_e4m3(x.x, o[8 * e], o[8 * e + 1]);
                expand_e4m3(x.y, o[8 * e + 2], o[8 * e + 3]);
                expand_e4m3(x.z, o[8 * e + 4], o[8 * e + 5]);
                expand_e4m3(x.w, o[8 * e + 6], o[8 * e + 7]);
              }
            }
          };
          if (group == 0) {
#pragma unroll
            for (int e = 0; e < 3; ++e) convert(6 * i + e, f[e]);
          } else {
#pragma unroll
            for (int e = 0; e < 3; ++e) convert(6 * i + 3 + e, f[e]);
          }
          if (i == 1) take(1);
          if (i == 2) take(2);
          if (!ok || (g > 0 && !ptx::mbar_wait(a_free + 8 * i, uint32_t(g - 1) & 1u, kPolls))) { ok = false; break; }
          ptx::tc_fence_after();
#pragma unroll
          for (int e = 0; e < 3; ++e) ptx::tmem_st16_nowait(lanes + 96 * i + 48 * group + 16 * e, f[e]);
          ptx::tmem_st_wait();
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(a_full + 8 * i);
        }
      }
    }
  }
  if (!ok) atomicOr(a.err, DSA_DEVERR_TIMEOUT);
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_attention_mass(const dsa_params_t& p, const WsLayout& L, char* ws, const void* q, const void* lat_pool,
                                  int sinks, int window, const int32_t* block_table, const int32_t* ctx_lens,
                                  const float* lse, int fresh, float* mass, int64_t mass_stride, cudaStream_t st) {
  MassArgs a = {};
  a.qs = reinterpret_cast<const float*>(ws + L.pfx_qs);
  a.lse = lse;
  a.table = block_table;
  a.ctx = ctx_lens;
  a.mass = mass;
  a.err = reinterpret_cast<int*>(ws + L.err);
  a.mass_stride = mass_stride;
  a.batch = p.batch;
  a.n_q = p.n_q;
  a.max_pages = p.max_pages_per_req;
  a.cap = L.cap;
  a.num_pages = p.num_pages;
  a.sinks = sinks < L.cap ? sinks : L.cap;
  a.window = window < L.cap ? window : L.cap;
  a.fresh = fresh;
  a.scale_log2 = p.softmax_scale * p.latent_scale * 1.4426950408889634f;
  const bool nv = p.lat_fmt == DSA_LAT_NVFP4_352;
  CUtensorMap kmap, rmap;
  std::memset(&rmap, 0, sizeof(rmap));
  if (nv) {
    // [num_pages][64][88] words, 32 of them at a time (the last 8 of 96 are past the row, and read as 0)
    const uint64_t dims[3] = {88, uint64_t(kPage), uint64_t(p.num_pages)};
    const uint64_t strides[2] = {352, uint64_t(p.lat_page_stride)};
    const uint32_t box[3] = {32, kPage, 1};
    if (!encode_map(&kmap, CU_TENSOR_MAP_DATA_TYPE_UINT32, lat_pool, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
  } else {
    // [num_pages][64][576] bytes: 128 dims of a page's rows at a time, and 64
    const uint64_t dims[3] = {uint64_t(kDQK), uint64_t(kPage), uint64_t(p.num_pages)};
    const uint64_t strides[2] = {uint64_t(kDQK), uint64_t(p.lat_page_stride)};
    const uint32_t box[3] = {128, kPage, 1}, rbox[3] = {64, kPage, 1};
    if (!encode_map(&kmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, lat_pool, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !encode_map(&rmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, lat_pool, 3, dims, strides, rbox, CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
  }
  CUtensorMap qmap, qrmap;
  std::memset(&qrmap, 0, sizeof(qrmap));
  {
    const uint64_t dims[3] = {1152, uint64_t(kHeads), uint64_t(L.rows)}, strides[2] = {1152, uint64_t(1152) * kHeads};
    const uint32_t box[3] = {128, kHeads, 1}, rbox[3] = {64, kHeads, 1};
    if (!encode_map(&qmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, ws + L.pfx_q, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return cudaErrorInvalidValue;
    if (!nv && !encode_map(&qrmap, CU_TENSOR_MAP_DATA_TYPE_UINT8, ws + L.pfx_q, 3, dims, strides, rbox, CU_TENSOR_MAP_SWIZZLE_64B))
      return cudaErrorInvalidValue;
  }
  cudaError_t e = launch_prefix_query(p, L, ws, q, ctx_lens, 0, true, st);
  if (e != cudaSuccess) return e;
  auto kern = nv ? mass_kernel<true> : mass_kernel<false>;
  static std::atomic<uint64_t> smem_set[2];
  e = set_once(smem_set[nv], kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kSmem));
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(sm_count()), dim3(nv ? kThreads<true> : kThreads<false>), kSmem, st, kmap, rmap,
                    qmap, qrmap, a);
}

}  // namespace dsa
