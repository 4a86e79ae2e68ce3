// Accumulated attention weight of every cached token: mass[s] += sum over rows and heads of
// exp(scale q_h . c_s - lse_h). The simple form: a block per page, its latents in fp32 in shared
// memory, a thread per token and 24 heads.
#include <cuda_bf16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "dsa_internal.cuh"

namespace dsa {

namespace {

constexpr int kPitch = kDQK + 1;

struct MassArgs {
  const __nv_bfloat16* q;
  const uint8_t* lat;
  const int32_t* table;
  const int32_t* ctx;
  const float* lse;
  float* mass;
  int* err;
  int64_t stride, mass_stride;
  int n_q, max_pages, cap, num_pages, sinks, window, fresh, nv;
  float scale;
};

__device__ __forceinline__ float e4m3(uint8_t v) { return __half2float(__half(__nv_cvt_fp8_to_halfraw(v, __NV_E4M3))); }

__global__ void __launch_bounds__(256) mass_kernel(MassArgs a) {
  extern __shared__ float lat[];  // [64][kPitch]
  __shared__ float part[4][kPage];
  pdl_wait();
  const int b = blockIdx.y, n = a.ctx[b];
  if (n < a.n_q || n > a.cap) {
    if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(a.err, DSA_DEVERR_CTX);
    return;
  }
  const int tok = threadIdx.x & 63, grp = threadIdx.x >> 6;
  for (int j = blockIdx.x; j * kPage < n; j += gridDim.x) {
    const int oldest = max(0, n - a.n_q + 1 - a.window);  // first token of the first row's window
    if (j * kPage >= a.sinks && (j + 1) * kPage <= oldest) continue;
    const int pg = a.table[size_t(b) * a.max_pages + j];
    if (pg < 0 || pg >= a.num_pages) {
      if (threadIdx.x == 0) atomicOr(a.err, DSA_DEVERR_BLOCK_TABLE);
      continue;
    }
    __syncthreads();
    const uint8_t* page = a.lat + int64_t(pg) * a.stride;
    for (int i = threadIdx.x; i < kPage * kDQK; i += 256) {
      const int s = i / kDQK, d = i - s * kDQK;
      float v;
      if (!a.nv) {
        v = e4m3(page[s * kDQK + d]);
      } else if (d < kDNope) {
        const uint8_t* row = page + s * 352;
        const __half2_raw pair = __nv_cvt_fp4x2_to_halfraw2(row[d / 2], __NV_E2M1);
        v = __half2float(__half(__half_raw{(d & 1) ? pair.y : pair.x})) * e4m3(row[256 + d / 16]);
      } else {
        v = e4m3(page[s * 352 + 288 + d - kDNope]);
      }
      lat[s * kPitch + d] = v;
    }
    __syncthreads();
    const int s = j * kPage + tok;
    float sum = 0.f;
    bool seen = false;
    for (int t = 0; t < a.n_q; ++t) {
      const int L = n - a.n_q + t + 1;
      const bool sees = s < L && (s < a.sinks || s >= L - a.window);
      seen |= sees;
      float w = 0.f;
      for (int h = grp * 24; h < grp * 24 + 24; ++h) {
        const size_t hr = size_t(b * a.n_q + t) * kHeads + h;
        const float lse = a.lse[hr];
        if (!isfinite(lse)) continue;
        const __nv_bfloat16* q = a.q + hr * kDQK;
        float z = 0.f;
        for (int d = 0; d < kDQK; ++d) z = fmaf(__bfloat162float(q[d]), lat[tok * kPitch + d], z);
        w += expf(z * a.scale - lse);
      }
      part[grp][tok] = w;
      __syncthreads();
      if (sees) sum += part[0][tok] + part[1][tok] + part[2][tok] + part[3][tok];
      __syncthreads();
    }
    if (grp == 0 && seen) {
      float* m = a.mass + b * a.mass_stride + s;
      *m = s >= n - a.fresh ? sum : *m + sum;
    }
  }
}

}  // namespace

cudaError_t launch_attention_mass(const dsa_params_t& p, const WsLayout& L, char* ws, const void* q, const void* lat_pool,
                                  int sinks, int window, const int32_t* block_table, const int32_t* ctx_lens,
                                  const float* lse, int fresh, float* mass, int64_t mass_stride, cudaStream_t st) {
  MassArgs a = {static_cast<const __nv_bfloat16*>(q), static_cast<const uint8_t*>(lat_pool), block_table, ctx_lens, lse, mass,
                reinterpret_cast<int*>(ws + L.err), p.lat_page_stride, mass_stride, p.n_q, p.max_pages_per_req, L.cap,
                p.num_pages, sinks, window, fresh, p.lat_fmt == DSA_LAT_NVFP4_352, p.softmax_scale * p.latent_scale};
  const size_t smem = size_t(kPage) * kPitch * 4;
  cudaError_t e = cudaFuncSetAttribute(mass_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  return launch_pdl(mass_kernel, dim3(p.max_pages_per_req < 1024 ? p.max_pages_per_req : 1024, p.batch), dim3(256), smem, st, a);
}

}  // namespace dsa
