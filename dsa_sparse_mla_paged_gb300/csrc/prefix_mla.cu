// Dense attention of a batch that shares a prefix.
#include <cuda_bf16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "dsa_internal.cuh"
#include "sm103_ptx.cuh"

namespace dsa {

namespace {

struct PfxArgs {
  const __nv_bfloat16* q;
  const uint8_t* lat;
  const int32_t* prefix_pages;
  const int32_t* table;
  const int32_t* ctx;
  __nv_bfloat16* out;
  float* lse;
  int* err;
  int64_t stride;
  int prefix, n_q, max_pages, num_pages, cap, nvfp4;
  float scale, lat_scale;
};

constexpr int kSimpleHeads = 8, kSimpleTok = 32, kSimplePitch = kDQK + 1;

__device__ __forceinline__ float latent_value(const uint8_t* row, int d, int nvfp4) {
  auto e4m3 = [](uint8_t c) {
    const __half_raw h = __nv_cvt_fp8_to_halfraw(c, __NV_E4M3);
    return __half2float(*reinterpret_cast<const __half*>(&h));
  };
  if (!nvfp4) return e4m3(row[d]);
  if (d >= kDNope) return e4m3(row[288 + d - kDNope]);
  const __half_raw h = __nv_cvt_fp4_to_halfraw((row[d >> 1] >> (4 * (d & 1))) & 15, __NV_E2M1);
  return __half2float(*reinterpret_cast<const __half*>(&h)) * e4m3(row[256 + (d >> 4)]);
}

// One CTA per (row, 8 heads), a warp per head: 32 tokens at a time through shared memory.
__global__ void __launch_bounds__(256) prefix_mla_simple_kernel(PfxArgs a) {
  extern __shared__ float sm[];
  pdl_wait();
  float* C = sm;                              // [32][577]
  float* Q = sm + kSimpleTok * kSimplePitch;  // [8][576]
  __shared__ int s_ok[kSimpleTok];
  const int r = blockIdx.x, b = r / a.n_q, t = r - b * a.n_q;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y * kSimpleHeads + warp;
  const int c = a.ctx[b];
  const bool valid = c >= a.prefix + a.n_q && c <= a.cap;
  if (!valid && t == 0 && threadIdx.x == 0) atomicOr(a.err, DSA_DEVERR_CTX);
  const int L = valid ? c - a.n_q + t + 1 : 0;
  const __nv_bfloat16* q = a.q + (size_t(r) * kHeads + h) * kDQK;
  for (int d = lane; d < kDQK; d += 32) Q[warp * kDQK + d] = __bfloat162float(q[d]);
  float m = -INFINITY, l = 0.f, o[16];
  for (int i = 0; i < 16; ++i) o[i] = 0.f;
  const int row_bytes = a.nvfp4 ? 352 : 576;
  for (int s0 = 0; s0 < L; s0 += kSimpleTok) {
    __syncthreads();
    const int pi = s0 / kPage;
    const int pg = s0 < a.prefix ? a.prefix_pages[pi] : a.table[size_t(b) * a.max_pages + pi];
    const bool page_ok = pg >= 0 && pg < a.num_pages;
    if (!page_ok && threadIdx.x == 0) atomicOr(a.err, DSA_DEVERR_BLOCK_TABLE);
    if (threadIdx.x < kSimpleTok) s_ok[threadIdx.x] = page_ok && s0 + int(threadIdx.x) < L;
    for (int i = threadIdx.x; i < kSimpleTok * kDQK; i += 256) {
      const int j = i / kDQK, d = i - j * kDQK;
      float v = 0.f;
      if (page_ok && s0 + j < L)
        v = latent_value(a.lat + size_t(pg) * a.stride + size_t(s0 % kPage + j) * row_bytes, d, a.nvfp4) * a.lat_scale;
      C[j * kSimplePitch + d] = v;
    }
    __syncthreads();
    float z = 0.f;
    for (int d = 0; d < kDQK; ++d) z = fmaf(Q[warp * kDQK + d], C[lane * kSimplePitch + d], z);
    z = s_ok[lane] ? z * a.scale : -INFINITY;
    float mt = z;
    for (int k = 16; k; k >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, k));
    const float mn = fmaxf(m, mt);
    if (mn == -INFINITY) continue;
    const float al = expf(m - mn), p = expf(z - mn);
    float ps = p;
    for (int k = 16; k; k >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, k);
    l = l * al + ps;
    m = mn;
    for (int i = 0; i < 16; ++i) o[i] *= al;
    for (int j = 0; j < kSimpleTok; ++j) {
      const float pj = __shfl_sync(0xffffffffu, p, j);
      for (int i = 0; i < 16; ++i) o[i] = fmaf(pj, C[j * kSimplePitch + lane + 32 * i], o[i]);
    }
  }
  __nv_bfloat16* out = a.out + (size_t(r) * kHeads + h) * kDNope;
  for (int i = 0; i < 16; ++i) out[lane + 32 * i] = __float2bfloat16_rn(l > 0.f ? o[i] / l : 0.f);
  if (a.lse && lane == 0) a.lse[size_t(r) * kHeads + h] = l > 0.f ? m + logf(l) : -INFINITY;
}

}  // namespace

cudaError_t launch_prefix_mla(const dsa_params_t& p, const WsLayout& L, char* ws, const void* q, const void* lat_pool,
                              const int32_t* prefix_pages, int prefix_len, const int32_t* block_table,
                              const int32_t* ctx_lens, void* out, float* lse, cudaStream_t st) {
  PfxArgs a;
  a.q = static_cast<const __nv_bfloat16*>(q);
  a.lat = static_cast<const uint8_t*>(lat_pool);
  a.prefix_pages = prefix_pages;
  a.table = block_table;
  a.ctx = ctx_lens;
  a.out = static_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  a.err = reinterpret_cast<int*>(ws + L.err);
  a.stride = p.lat_page_stride;
  a.prefix = prefix_len;
  a.n_q = p.n_q;
  a.max_pages = p.max_pages_per_req;
  a.num_pages = p.num_pages;
  a.cap = L.cap;
  a.nvfp4 = p.lat_fmt == DSA_LAT_NVFP4_352;
  a.scale = p.softmax_scale;
  a.lat_scale = p.latent_scale;
  const size_t smem = (kSimpleTok * kSimplePitch + kSimpleHeads * kDQK) * 4;
  cudaError_t e = cudaFuncSetAttribute(prefix_mla_simple_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  return launch_pdl(prefix_mla_simple_kernel, dim3(L.rows, kHeads / kSimpleHeads), dim3(256), smem, st, a);
}

}  // namespace dsa
