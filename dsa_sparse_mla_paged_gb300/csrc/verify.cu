// Verification of drafted tokens: each request's drafts are tested against the
// target's probabilities, and the next token is drawn from what the target has
// beyond the draft (rejection sampling, so that the tokens follow the target).
//
// One cluster of up to 8 CTAs per request. Every CTA runs the few draft tests
// (one lane per draft, exact in fp64), then reads its slice of the one row of p
// (and of q after a rejection) that the draw needs, each element once. A
// warp owns a contiguous run of the vocabulary and sums its weights; the CTAs'
// sums meet in distributed shared memory, and the CTA that holds the threshold
// goes over the one warp's run again to find the token. The two rows' bytes bound
// a large batch, the chain of dependent loads (token -> probabilities ->
// row) a small one.
//
// Weights are 64-bit integers (multiples of 2^-60): integer sums are exact in any
// order, so the token does not depend on how the vocabulary is cut, and no
// probability mass is lost over a long row.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "dsa_internal.cuh"
#include "sm103_ptx.cuh"

namespace dsa {

namespace {

constexpr int kVThreads = 512;
constexpr int kVWarps = kVThreads / 32;
constexpr int kVMaxCluster = 8;
constexpr int kVUnroll = 8;
constexpr int kVMinRun = 32 * kVUnroll;  // a warp's shortest run of the vocabulary worth a warp

typedef unsigned long long u64;

// A row's weights sum to about 1. Sums stop at kTooMuch, far from where the
// integers wrap, and a sum above kMostMass draws no token.
constexpr u64 kMostMass = 4ull << 60, kTooMuch = 5ull << 60;

__device__ __forceinline__ float as_float(float x) { return x; }
__device__ __forceinline__ float as_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float as_float(__half x) { return __half2float(x); }

// x in [0, 1] as a multiple of 2^-60, rounded down; anything else is 0 and bad.
__device__ __forceinline__ u64 fixed(float x, bool& bad) {
  const bool ok = x >= 0.f && x <= 1.f;
  bad |= !ok;
  return ok ? __float2ull_rz(x * 1152921504606846976.f) : 0ull;
}

struct VerifyArgs {
  VerifyIn in;
  int n_q;
  int run;  // elements of a warp's run
  int* err;
};

// The weight of element v: max(p - q, 0). `one_hot`: the draft has all its mass on token x.
template <typename T>
__device__ __forceinline__ u64 weight(T pv, T qv, bool has_q, bool one_hot, int v, int x, bool& bad) {
  const u64 p = fixed(as_float(pv), bad);
  if (one_hot) return v == x ? 0ull : p;
  if (!has_q) return p;
  const u64 q = fixed(as_float(qv), bad);
  return p > q ? p - q : 0ull;
}

__device__ __forceinline__ u64 capped(u64 v) { return v < kTooMuch ? v : kTooMuch; }

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ u64 warp_scan(u64 v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kVThreads) verify_kernel(const __grid_constant__ VerifyArgs a) {
  namespace cg = cooperative_groups;
  pdl_wait();
  cg::cluster_group cl = cg::this_cluster();
  __shared__ int s_acc, s_count, s_flags;
  __shared__ u64 s_warp[kVWarps], s_cta[2][kVMaxCluster];
  __shared__ u64 s_scan[kVWarps];
  const VerifyIn& in = a.in;
  const int cta = int(cl.block_rank()), ctas = int(cl.num_blocks());
  const int b = int(blockIdx.x) / ctas;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* P = static_cast<const T*>(in.p);
  const T* Q = static_cast<const T*>(in.q);
  const int most = a.n_q - 1, V = in.vocab;

  // ---- the draft tests
  if (warp == 0) {
    int flags = 0;
    int k = in.n_draft ? in.n_draft[b] : most;
    if (k < 0 || k > most) {
      flags |= DSA_DEVERR_DRAFT;
      k = k < 0 ? 0 : most;
    }
    int acc = k;
    for (int i0 = 0; i0 < k && acc == k; i0 += 32) {
      const int i = i0 + lane;
      bool pass = true;
      if (i < k) {
        const int x = in.tokens[size_t(b) * most + i];
        if (x < 0 || x >= V) {
          flags |= DSA_DEVERR_DRAFT;
          pass = false;
        } else {
          const float p = as_float(P[(size_t(b) * a.n_q + i) * in.p_stride + x]);
          const float q = Q ? as_float(Q[(size_t(b) * most + i) * in.q_stride + x]) : 1.f;
          pass = double(in.uniforms[size_t(b) * a.n_q + i]) * double(q) < double(p);
        }
      }
      const unsigned no = __ballot_sync(0xffffffffu, !pass);
      if (no) acc = i0 + __ffs(no) - 1;
    }
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (lane == 0) {
      s_acc = acc;
      s_count = k;
      s_flags = flags;
    }
  }
  __syncthreads();
  const int acc = s_acc;
  const bool rejected = acc < s_count;
  const T* prow = P + (size_t(b) * a.n_q + acc) * in.p_stride;
  const T* qrow = rejected && Q ? Q + (size_t(b) * most + acc) * in.q_stride : nullptr;
  const int x = rejected ? in.tokens[size_t(b) * most + acc] : -1;
  const float u = in.uniforms[size_t(b) * a.n_q + most];
  const float uc = u >= 0.f ? fminf(u, 0.99999994f) : 0.f;
  const u64 u64th = __float2ull_rz(uc * 18446744073709551616.f);

  // ---- sums over the warp runs; a second round with p alone if p - q has no mass
  const int64_t v0 = (int64_t(cta) * kVWarps + warp) * a.run;
  const int lo = int(v0 < V ? v0 : V), hi = int(v0 + a.run < V ? v0 + a.run : V);
  bool has_q = qrow != nullptr, one_hot = rejected && !Q, bad = false;
  u64 sum = 0, total = 0, before = 0;
  for (int round = 0; round < 2; ++round) {
    uint32_t coarse = 0;  // the sum in units of 2^-16: the integers of 2^-60 wrap at 16
    sum = 0;
    for (int v = lo + lane; v < hi; v += 32 * kVUnroll) {
      T pv[kVUnroll], qv[kVUnroll];
#pragma unroll
      for (int j = 0; j < kVUnroll; ++j) {
        const bool in_run = v + 32 * j < hi;
        pv[j] = in_run ? prow[v + 32 * j] : T(0.f);
        qv[j] = in_run && has_q ? qrow[v + 32 * j] : T(0.f);
      }
#pragma unroll
      for (int j = 0; j < kVUnroll; ++j) {
        const u64 w = weight<T>(pv[j], qv[j], has_q, one_hot, v + 32 * j, x, bad);
        sum += w;
        coarse += uint32_t(w >> 44);
      }
    }
    sum = warp_sum(sum);
    if (warp_sum(coarse) > (4u << 16)) sum = kTooMuch;
    if (lane == 0) s_warp[warp] = sum;
    __syncthreads();
    if (threadIdx.x < ctas) {
      u64 t = 0;
      for (int i = 0; i < kVWarps; ++i) t = capped(t + s_warp[i]);
      *cl.map_shared_rank(&s_cta[round][cta], threadIdx.x) = t;
    }
    cl.sync();
    total = 0;
    for (int i = 0; i < ctas; ++i) {
      if (i == cta) before = total;
      total = capped(total + s_cta[round][i]);
    }
    if (total != 0 || (!has_q && !one_hot)) break;  // the same for every CTA of the cluster
    has_q = one_hot = false;
  }
  const bool drawn = total != 0 && total <= kMostMass;
  if (bad || !drawn) atomicOr(a.err, DSA_DEVERR_PROB);

  // ---- what does not depend on the draw
  int32_t* out = in.out_tokens + size_t(b) * a.n_q;
  if (cta == 0) {
    if (threadIdx.x == 0) {
      in.n_accepted[b] = acc;
      if (s_flags) atomicOr(a.err, s_flags);
      if (in.new_lens) {
        const int ctx = in.ctx_lens[b];
        if (ctx < a.n_q) atomicOr(a.err, DSA_DEVERR_CTX);
        in.new_lens[b] = ctx < a.n_q ? -1 : ctx - a.n_q + 1 + acc;
      }
    }
    for (int i = threadIdx.x; i < a.n_q; i += kVThreads)
      if (i != acc) out[i] = i < acc ? in.tokens[size_t(b) * most + i] : -1;
    if (!drawn && threadIdx.x == 0) out[acc] = -1;
  }
  // ---- the CTA that holds the threshold looks for the token
  const u64 thr = __umul64hi(u64th, total);
  if (!drawn || thr < before) return;
  u64 at = before;
  int w = 0;
  for (; w < kVWarps && at + s_warp[w] <= thr; ++w) at += s_warp[w];
  if (w == kVWarps) return;
  const int64_t r0 = (int64_t(cta) * kVWarps + w) * a.run;
  const int end = int(r0 + a.run < V ? r0 + a.run : V);
  for (int c0 = int(r0); c0 < end; c0 += kVThreads) {
    const int v = c0 + int(threadIdx.x);
    u64 own = 0;
    if (v < end) own = weight<T>(prow[v], has_q ? qrow[v] : T(0.f), has_q, one_hot, v, x, bad);
    const u64 inc = warp_scan(own);
    __syncthreads();
    if (lane == 31) s_scan[warp] = inc;
    __syncthreads();
    u64 pre = at, all = 0;
    for (int i = 0; i < kVWarps; ++i) {
      if (i < warp) pre += s_scan[i];
      all += s_scan[i];
    }
    // exactly one element has the threshold inside its weight
    if (own && pre + inc > thr && pre + inc - own <= thr) out[acc] = v;
    at += all;
    if (at > thr) break;
  }
}

}  // namespace

cudaError_t launch_verify_draft(const dsa_params_t& p, const WsLayout& L, char* ws, const VerifyIn& in, cudaStream_t st) {
  VerifyArgs a;
  a.in = in;
  a.n_q = p.n_q;
  a.err = reinterpret_cast<int*>(ws + L.err);
  int ctas = 1;
  while (ctas < kVMaxCluster && int64_t(ctas) * kVWarps * kVMinRun < in.vocab) ctas *= 2;
  const int per = (in.vocab + ctas * kVWarps - 1) / (ctas * kVWarps);
  a.run = (per + 31) / 32 * 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(p.batch) * ctas);
  cfg.blockDim = dim3(kVThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(ctas);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  switch (in.dtype) {
    case DSA_PROB_F32: return cudaLaunchKernelEx(&cfg, verify_kernel<float>, a);
    case DSA_PROB_BF16: return cudaLaunchKernelEx(&cfg, verify_kernel<__nv_bfloat16>, a);
    default: return cudaLaunchKernelEx(&cfg, verify_kernel<__half>, a);
  }
}

}  // namespace dsa
