// The attention's front end: per query head and per new latent the RMS norm of 512 values and the
// rotation of 64 in one pass, and the latent's row, quantised, written into the paged cache.
//
// A row moves 220 KB of query through (96 heads of 576 bf16 values, read once and written once) for
// about 120,000 multiplications: bytes bound it, and a small call its launch. One warp has a head: 64
// 16-B chunks of the normed part, two a lane, so that the sum of squares is 16 values a lane and five
// shuffles; two heads at a time, whose 2 x 8 chunks of the rotary part are then one for every other lane.
// The angles of a row are worked out once per block, in fp64 (a product of a 31-bit position and a 24-bit
// frequency does not fit fp32), 32 lanes a frequency each.
//
// Measured (one GB300): 8,194 rows, FP8 latents, 296 us (1.83 GB, 6.2 TB/s: 0.92 of a plain copy); 384 rows,
// NVFP4, 18.0 us in a graph (86 MB, within L2); one row 4.2 us, which is a launch and a chain of two loads.
#include <cuda_bf16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "dsa_internal.cuh"
#include "sm103_ptx.cuh"

namespace dsa {

namespace {

constexpr int kWarps = 8;
// Heads of a warp at a time, and how often; blocks a row. (With normalised heads, 1, 64, 384 and 8,194 rows: 4.8, 7.6, 18.1 and
// 298 us; one block a row 7.3, 7.6, 18.5, 300; four heads at a time in three blocks 4.9, 8.5, 21.3, 371 at two blocks an SM and
// 4.7, 8.3, 18.8, 312 at three; twelve blocks of a head a warp 4.8, 8.6, 26.2, 506.)
constexpr int kPer = 2, kLoops = 3, kSplits = 2;
static_assert(kWarps * kPer * kLoops * kSplits == kHeads, "a row's heads");

// cos and sin of p * f, each rounded once from fp64 (in all but about one in 2^13): the angle reduced to
// [-pi/4, pi/4] by whole quarter turns (pi/2 as the sum of two doubles, Cody and Waite's reduction), then the
// Taylor series, which end there below 2^-45.
__device__ __forceinline__ void cos_sin(int p, float f, float& c, float& s) {
  const double a = double(p) * double(f);
  const double k = rint(a * 0.63661977236758134);  // 2 / pi
  double x = fma(-k, 1.5707963267948966, a);
  x = fma(-k, 6.1232339957367660e-17, x);
  const double z = x * x;
  double u = fma(z, 1.0 / 6227020800.0, -1.0 / 39916800.0);
  u = fma(z, u, 1.0 / 362880.0);
  u = fma(z, u, -1.0 / 5040.0);
  u = fma(z, u, 1.0 / 120.0);
  u = fma(z, u, -1.0 / 6.0);
  const double sn = fma(x * z, u, x);
  double v = fma(z, -1.0 / 87178291200.0, 1.0 / 479001600.0);
  v = fma(z, v, -1.0 / 3628800.0);
  v = fma(z, v, 1.0 / 40320.0);
  v = fma(z, v, -1.0 / 720.0);
  v = fma(z, v, 1.0 / 24.0);
  v = fma(z, v, -0.5);
  const double cn = fma(z, v, 1.0);
  const int q = int(static_cast<long long>(k) & 3);  // quarter turns
  const double cc = (q & 1) ? sn : cn, ss = (q & 1) ? cn : sn;
  c = float(q == 1 || q == 2 ? -cc : cc);
  s = float(q >= 2 ? -ss : ss);
}

// Eight bf16 values of a 16-B chunk in fp32, and back.
__device__ __forceinline__ void unpack8(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(u[i] << 16);
    x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    u[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

// Rotates chunk j (dims 8j .. 8j + 7 of 64) held by this lane; the chunks of a head are in eight consecutive lanes.
// cs(i): cosine and sine of angle i. Each product and sum is rounded by itself, as the definition says.
template <bool kInterleaved, typename CosSin>
__device__ __forceinline__ void rotate8(float (&x)[8], int j, CosSin cs) {
  if constexpr (kInterleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 a = cs(4 * j + i);
      const float x0 = x[2 * i], x1 = x[2 * i + 1];
      x[2 * i] = __fsub_rn(__fmul_rn(x0, a.x), __fmul_rn(x1, a.y));
      x[2 * i + 1] = __fadd_rn(__fmul_rn(x1, a.x), __fmul_rn(x0, a.y));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = __shfl_xor_sync(0xffffffffu, x[i], 4);  // chunk j +- 4: 32 dims away
      const float2 a = cs(8 * (j & 3) + i);
      const float m = __fmul_rn(other, a.y), own = __fmul_rn(x[i], a.x);
      x[i] = j < 4 ? __fsub_rn(own, m) : __fadd_rn(own, m);
    }
  }
}

// (a length may be anything: without positions it is checked, and the sum of a bad one wraps)
__device__ __forceinline__ int row_position(const LatentIn& in, int row, int b, int n_q) {
  return in.positions ? in.positions[row] : int(uint32_t(in.ctx_lens[b]) - uint32_t(n_q) + uint32_t(row - b * n_q));
}

// Blocks [0, lat_blocks): a warp per row's latent. The others: kSplits a row, a warp has kPer heads at a time, kLoops times.
template <bool kInterleaved, bool kNv>
__global__ void __launch_bounds__(32 * kWarps, 4)
    latent_frontend_kernel(const __grid_constant__ LatentIn in, int rows, int n_q, int max_pages, int cap, int num_pages,
                           int64_t stride, float inv_scale, int lat_blocks, int* err) {
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (int(blockIdx.x) < lat_blocks) {
    // ------------------------------------------------------------ latents
    const int row = blockIdx.x * kWarps + warp;
    if (row >= rows) return;
    const int b = row / n_q, t = row - b * n_q, ctx = in.ctx_lens[b];
    const uint4* c = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(in.c_kv) + row * in.c_kv_row);
    const uint4* g = static_cast<const uint4*>(in.gamma_kv);
    const uint4 w[2] = {__ldg(c + lane), __ldg(c + 32 + lane)}, gw[2] = {__ldg(g + lane), __ldg(g + 32 + lane)};
    uint4 rw = make_uint4(0, 0, 0, 0);
    if (lane < 8)
      rw = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(in.k_rope) + row * in.k_rope_row) + lane);
    float co, si;
    cos_sin(row_position(in, row, b, n_q), __ldg(in.inv_freq + lane), co, si);
    int page = -1, slot = 0;
    if (ctx < n_q || ctx > cap) {
      if (lane == 0) atomicOr(err, DSA_DEVERR_CTX);
    } else {
      slot = ctx - n_q + t;
      page = in.block_table[size_t(b) * max_pages + slot / kPage];
      if (page < 0 || page >= num_pages) {
        if (lane == 0) atomicOr(err, DSA_DEVERR_BLOCK_TABLE);
        page = -1;
      }
    }
    float x[2][8], gm[2][8];
    double sum = 0.;  // a code next to a border goes by the sum's last bits
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      unpack8(w[d], x[d]);
      unpack8(gw[d], gm[d]);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum = fma(double(x[d][i]), double(x[d][i]), sum);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float r = float(1.0 / sqrt(sum / kDNope + double(in.eps)));
#pragma unroll
    for (int d = 0; d < 2; ++d)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[d][i] = __fmul_rn(__fmul_rn(__fmul_rn(x[d][i], r), gm[d][i]), inv_scale);
    float rope[8];
    unpack8(rw, rope);
    rotate8<kInterleaved>(rope, lane & 7, [&](int i) {
      return make_float2(__shfl_sync(0xffffffffu, co, i), __shfl_sync(0xffffffffu, si, i));
    });
    auto e4m3x4 = [](float a0, float a1, float a2, float a3) {
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a0, a1), __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(a2, a3), __NV_SATFINITE, __NV_E4M3);
      return lo | hi << 16;
    };
    uint2 rc;
    rc.x = e4m3x4(__fmul_rn(rope[0], inv_scale), __fmul_rn(rope[1], inv_scale), __fmul_rn(rope[2], inv_scale),
                  __fmul_rn(rope[3], inv_scale));
    rc.y = e4m3x4(__fmul_rn(rope[4], inv_scale), __fmul_rn(rope[5], inv_scale), __fmul_rn(rope[6], inv_scale),
                  __fmul_rn(rope[7], inv_scale));
    uint8_t* dst = static_cast<uint8_t*>(in.lat_pool) + int64_t(page) * stride + (slot % kPage) * (kNv ? 352 : kLatRowFp8);
    if constexpr (!kNv) {
      if (page < 0) return;
#pragma unroll
      for (int d = 0; d < 2; ++d)
        reinterpret_cast<uint2*>(dst)[32 * d + lane] =
            make_uint2(e4m3x4(x[d][0], x[d][1], x[d][2], x[d][3]), e4m3x4(x[d][4], x[d][5], x[d][6], x[d][7]));
      if (lane < 8) reinterpret_cast<uint2*>(dst + kDNope)[lane] = rc;
    } else {
#pragma unroll
      for (int d = 0; d < 2; ++d) {
        // a block of 16: two lanes (a NaN passes the maximum by, so it is looked for by itself)
        float m = 0.f;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          m = fmaxf(m, fabsf(x[d][i]));
          bad |= x[d][i] != x[d][i];
        }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        bad |= __shfl_xor_sync(0xffffffffu, int(bad), 1) != 0;
        const uint32_t code = bad ? 0x7Fu : uint32_t(__nv_cvt_float_to_fp8(__fdiv_rn(m, 6.f), __NV_SATFINITE, __NV_E4M3));
        const float s = __half2float(__half(__nv_cvt_fp8_to_halfraw(__nv_fp8_storage_t(code), __NV_E4M3)));
        uint32_t out = 0;
        if (s > 0.f) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            out |= uint32_t(__nv_cvt_float2_to_fp4x2(make_float2(__fdiv_rn(x[d][2 * i], s), __fdiv_rn(x[d][2 * i + 1], s)),
                                                     __NV_E2M1, cudaRoundNearest))
                   << (8 * i);
        }
        if (page >= 0) {
          reinterpret_cast<uint32_t*>(dst)[32 * d + lane] = out;
          if (!(lane & 1)) dst[256 + 16 * d + (lane >> 1)] = uint8_t(code);
        }
      }
      if (page >= 0 && lane < 8) reinterpret_cast<uint2*>(dst + 288)[lane] = rc;
    }
    return;
  }
  // -------------------------------------------------------------- query heads
  __shared__ float2 s_cs[32];
  const int item = int(blockIdx.x) - lat_blocks, row = item / kSplits, part = item - row * kSplits;
  const int b = row / n_q;
  const __nv_bfloat16* nope = static_cast<const __nv_bfloat16*>(in.q_nope) + row * in.q_nope_row;
  const __nv_bfloat16* rope = static_cast<const __nv_bfloat16*>(in.q_rope) + row * in.q_rope_row;
  uint4* out = static_cast<uint4*>(in.q_out) + size_t(row) * kHeads * (kDQK / 8);
  const int h0 = (part * kWarps + warp) * kPer * kLoops;
  const int rh = lane >> 3, rj = lane & 7;  // the rotary chunk of this lane
  uint4 w[kPer][2], rw;
  auto load = [&](int h) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const uint4* p = reinterpret_cast<const uint4*>(nope + (h + i) * in.q_nope_head);
      w[i][0] = p[lane];
      w[i][1] = p[32 + lane];
    }
    rw = make_uint4(0, 0, 0, 0);
    if (rh < kPer) rw = reinterpret_cast<const uint4*>(rope + (h + rh) * in.q_rope_head)[rj];
  };
  load(h0);
  if (warp == 0) {
    float c, s;
    cos_sin(row_position(in, row, b, n_q), __ldg(in.inv_freq + lane), c, s);
    s_cs[lane] = make_float2(c, s);
    if (lat_blocks == 0 && !in.positions && part == 0 && lane == 0) {  // no latent's warp looks at the length
      const int ctx = in.ctx_lens[b];
      if (ctx < n_q || ctx > cap) atomicOr(err, DSA_DEVERR_CTX);
    }
  }
  float gm[2][8];
  const bool norm = in.gamma_q != nullptr;
  if (norm) {
    const uint4* g = static_cast<const uint4*>(in.gamma_q);
    unpack8(__ldg(g + lane), gm[0]);
    unpack8(__ldg(g + 32 + lane), gm[1]);
  }
  __syncthreads();
#pragma unroll 1
  for (int l = 0; l < kLoops; ++l) {
    const int h = h0 + l * kPer;
    if (norm) {
      float x[8], sum[kPer];
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        sum[i] = 0.f;
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          unpack8(w[i][d], x);
#pragma unroll
          for (int e = 0; e < 8; ++e) sum[i] = fmaf(x[e], x[e], sum[i]);
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1)
#pragma unroll
        for (int i = 0; i < kPer; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float r = rsqrtf(sum[i] * (1.f / kDNope) + in.eps);
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          unpack8(w[i][d], x);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = x[e] * r * gm[d][e];
          w[i][d] = pack8(x);
        }
      }
    }
    float y[8];
    unpack8(rw, y);
    rotate8<kInterleaved>(y, rj, [&](int i) { return s_cs[i]; });
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      uint4* o = out + (h + i) * (kDQK / 8);
      o[lane] = w[i][0];
      o[32 + lane] = w[i][1];
    }
    if (rh < kPer) out[(h + rh) * (kDQK / 8) + kDNope / 8 + rj] = pack8(y);
    if (l + 1 < kLoops) load(h + kPer);
  }
}

}  // namespace

cudaError_t launch_latent_frontend(const dsa_params_t& p, int* err, const LatentIn& in, bool interleaved, cudaStream_t st) {
  const int rows = p.batch * p.n_q, cap = p.max_pages_per_req * p.page_size;
  const int lat_blocks = in.c_kv ? (rows + kWarps - 1) / kWarps : 0;
  const int blocks = lat_blocks + (in.q_out ? rows * kSplits : 0);
  const bool nv = p.lat_fmt == DSA_LAT_NVFP4_352;
  auto kern = interleaved ? (nv ? latent_frontend_kernel<true, true> : latent_frontend_kernel<true, false>)
                          : (nv ? latent_frontend_kernel<false, true> : latent_frontend_kernel<false, false>);
  return launch_pdl(kern, dim3(blocks), dim3(32 * kWarps), 0, st, in, rows, int(p.n_q), int(p.max_pages_per_req), cap,
                    int(p.num_pages), int64_t(p.lat_page_stride), 1.f / p.latent_scale, lat_blocks, err);
}

}  // namespace dsa
