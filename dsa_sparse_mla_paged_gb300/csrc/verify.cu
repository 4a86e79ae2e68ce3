// Verification of drafted tokens: each request's drafts are tested against the
// target's probabilities, and the next token is drawn from what the target has
// beyond the draft (rejection sampling, so that the tokens follow the target).
//
// One cluster of up to 8 CTAs per request. Every CTA runs the few draft tests
// (one lane per draft, exact in fp64), then reads its slice of the one row of p
// (and of q after a rejection) that the draw needs, each element once. A
// warp owns a contiguous run of the vocabulary in two parts and sums their weights; the
// CTAs' sums meet in distributed shared memory, and the CTA that holds the threshold
// goes over the one part again to find the token.
//
// Bounds: the chain of dependent loads (token -> probabilities -> row -> sums -> threshold), 6.7
// us for one request of 32,000 values; and for a large batch, after that, each warp's turns of
// loads and of arithmetic (about 17 instructions per pair of values; a third of the issue
// slots are used): 64 requests of 131,072 fp32 values, 67 MB, take 16.7 us (4.0 TB/s), 256 of
// 100,003 bf16 values, rows on any boundary, 102 MB, 32.2 us (3.2 TB/s). Loading a step ahead
// of the sums made it slower (38 us), and so did more CTAs than run at once (37).
//
// Weights are 64-bit integers (multiples of 2^-60): integer sums are exact in any
// order, so the token does not depend on how the vocabulary is cut, and no
// probability mass is lost over a long row.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "dsa_internal.cuh"
#include "sm103_ptx.cuh"

namespace dsa {

namespace {

constexpr int kVThreads = 256;
constexpr int kVWarps = kVThreads / 32;
constexpr int kVMaxCluster = 8;
constexpr int kVPerSM = 4;     // resident CTAs
constexpr int kVUnit = 256;    // a part of a warp's run is a multiple: 32 lanes x 16 B of 16-bit values
// Parts of a warp's run with sums of their own: the search for the token goes over one again
// (256 requests of 100,003 bf16 values: one part 35.9 us, two 32.2, four 33.0).
constexpr int kVParts = 2;

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

// Two values in [0, 1], each in three integers of a register, x = h 2^-22 + m 2^-44 +
// l 2^-60, from the mantissas of sums rounded towards zero (2 + x has steps of 2^-22,
// and so on), two at a time: a conversion to 64 bits takes several times as long.
// Only differences of two values' integers are used, which drops the sums' exponents.
struct Pieces {
  float2 h, m, l;
};
__device__ __forceinline__ Pieces pieces(float2 x) {
  constexpr float kMid = 1.f / (1 << 21), kLow = kMid / (1 << 16);
  Pieces o;
  o.h = ptx::add2_rz(x, make_float2(2.f, 2.f));
  const float2 r = ptx::sub2(x, ptx::sub2(o.h, make_float2(2.f, 2.f)));
  o.m = ptx::add2_rz(r, make_float2(kMid, kMid));
  o.l = ptx::add2_rz(ptx::sub2(r, ptx::sub2(o.m, make_float2(kMid, kMid))), make_float2(kLow, kLow));
  return o;
}
__device__ __forceinline__ uint32_t bits(float x) { return __float_as_uint(x); }

struct VerifyArgs {
  VerifyIn in;
  int n_q;
  int run, part;  // elements of a warp's run, and of a part of it
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

// The weights of a lane's elements: `sum` in units of 2^-60 modulo 2^64, and `coarse`
// in units of 2^-22 (rounded either way, and held at its top), which tells whether
// `sum` has wrapped. kFast: for values in [0, 1]; `top` tells whether all were.
template <bool kFast>
struct Mass {
  u64 sum = 0;
  uint32_t coarse = 0, top = 0;
  uint32_t h = 0, m = 0, l = 0;
  bool bad = false;
  __device__ __forceinline__ void add(float p, float q) {
    if constexpr (kFast) {
      top = max(top, max(bits(p), bits(q)));
      const Pieces a = pieces(make_float2(p, q));
      if (p > q) {
        h += bits(a.h.x) - bits(a.h.y);
        m += bits(a.m.x) - bits(a.m.y);
        l += bits(a.l.x) - bits(a.l.y);
      }
    } else {
      const u64 a = fixed(p, bad), b = fixed(q, bad);
      if (a > b) {
        sum += a - b;
        h += uint32_t((a - b) >> 38);
      }
    }
  }
  // two elements without a q
  __device__ __forceinline__ void add_two(float p0, float p1) {
    if constexpr (kFast) {
      top = max(top, max(bits(p0), bits(p1)));
      const Pieces a = pieces(make_float2(p0, p1));
      h += bits(a.h.x) - bits(2.f) + (bits(a.h.y) - bits(2.f));
      m += bits(a.m.x) - kMidBits + (bits(a.m.y) - kMidBits);
      l += bits(a.l.x) - kLowBits + (bits(a.l.y) - kLowBits);
    } else {
      add(p0, 0.f);
      add(p1, 0.f);
    }
  }
  // after at most 256 elements
  __device__ __forceinline__ void flush() {
    if constexpr (kFast) sum += (u64(h) << 38) + (u64(int64_t(int32_t(m))) << 16) + u64(int64_t(int32_t(l)));
    coarse = min(coarse + h, 1u << 31);
    h = m = l = 0;
  }
  static constexpr uint32_t kMidBits = uint32_t(127 - 21) << 23, kLowBits = uint32_t(127 - 37) << 23;
};

template <typename T>
struct Vec {
  static constexpr int kN = 16 / int(sizeof(T));
  union {
    uint4 u;
    T e[kN];
  };
  __device__ __forceinline__ Vec() {}
};

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

// The kN elements that begin `s` elements into the two vectors.
template <typename T>
__device__ __forceinline__ Vec<T> shifted(const Vec<T>& a, const Vec<T>& b, int s) {
  uint32_t w[8] = {a.u.x, a.u.y, a.u.z, a.u.w, b.u.x, b.u.y, b.u.z, b.u.w};
  constexpr int kPerWord = 4 / int(sizeof(T));
  auto drop = [&](bool on, int n) {
#pragma unroll
    for (int i = 0; i < 8 - n; ++i) w[i] = on ? w[i + n] : w[i];
  };
  drop((s & (2 * kPerWord)) != 0, 2);
  drop((s & kPerWord) != 0, 1);
  if constexpr (kPerWord == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16 * (s & 1));
  }
  Vec<T> r;
  r.u = make_uint4(w[0], w[1], w[2], w[3]);
  return r;
}

// Where a row begins within its 16 bytes, in elements.
template <typename T>
__device__ __forceinline__ int place(const T* p) {
  return int(reinterpret_cast<uintptr_t>(p) / sizeof(T)) & (Vec<T>::kN - 1);
}

// Elements [lo, hi) of rows of V, 16 B of p at a time where the row allows it: rows of an odd
// number of elements lie on any boundary, so the ends go one by one, and q's
// vectors, which p's do not match, are put together from two (never beyond its row).
template <typename T, bool kQ, bool kFast>
__device__ __forceinline__ void gather(Mass<kFast>& acc, const T* __restrict__ prow, const T* __restrict__ qrow, int lo,
                                       int hi, int V, int lane) {
  constexpr int kN = Vec<T>::kN, kStep = 32 * kN;
  auto singles = [&](int from, int to) {
#pragma unroll 1
    for (int v = from + lane; v < to; v += 32) acc.add(as_float(prow[v]), kQ ? as_float(qrow[v]) : 0.f);
    acc.flush();
  };
  if constexpr (!kFast) {  // (rarely taken)
    for (int v = lo; v < hi; v += 1024) singles(v, min(v + 1024, hi));
    return;
  }
  int v = lo + (-(place(prow) + lo) & (kN - 1)), end = hi, s = 0;
  if constexpr (kQ) {
    s = (place(qrow) - place(prow)) & (kN - 1);
    if (s) {
      if (v < s) v += kN;
      end = min(end, V - kN);
    }
  }
  auto vectors = [&](auto unroll, auto apart) {
    constexpr int kU = decltype(unroll)::value;
#pragma unroll 1
    for (; v + kStep * kU <= end; v += kStep * kU) {
      Vec<T> p[kU], q[kQ ? kU : 1];
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        p[u].u = __ldg(reinterpret_cast<const uint4*>(prow + v) + 32 * u + lane);
        if constexpr (kQ) {
          const uint4* from = reinterpret_cast<const uint4*>(qrow + v - s) + 32 * u + lane;
          q[u].u = __ldg(from);
          if constexpr (decltype(apart)::value) {
            Vec<T> next;
            next.u = __ldg(from + 1);
            q[u] = shifted(q[u], next, s);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int j = 0; j < kN; j += kQ ? 1 : 2) {
          if constexpr (kQ) acc.add(as_float(p[u].e[j]), as_float(q[u].e[j]));
          else acc.add_two(as_float(p[u].e[j]), as_float(p[u].e[j + 1]));
        }
      acc.flush();
    }
  };
  singles(lo, min(v, hi));
  if (s) {
    vectors(std::integral_constant<int, 2>(), std::true_type());
    vectors(std::integral_constant<int, 1>(), std::true_type());
  } else {
    vectors(std::integral_constant<int, kQ ? 2 : 4>(), std::false_type());
    vectors(std::integral_constant<int, 1>(), std::false_type());
  }
  singles(min(v, hi), hi);
}

// A warp's elements [lo, hi): the sum in every lane, kTooMuch where it has wrapped.
template <typename T, bool kFast>
__device__ __forceinline__ u64 warp_mass(const T* prow, const T* qrow, int lo, int hi, int V, int x, bool& bad) {
  const int lane = threadIdx.x & 31;
  Mass<kFast> acc;
  if (qrow) gather<T, true>(acc, prow, qrow, lo, hi, V, lane);
  else gather<T, false>(acc, prow, qrow, lo, hi, V, lane);
  if constexpr (kFast) {
    // a value above 1, a NaN or a sign (-0's too): value by value
    if (__any_sync(0xffffffffu, acc.top > bits(1.f))) return warp_mass<T, false>(prow, qrow, lo, hi, V, x, bad);
  }
  bad |= acc.bad;
  if (lane == 0 && x >= lo && x < hi) {  // the token that has no weight
    const u64 own = fixed(as_float(prow[x]), bad);
    acc.sum -= own;
    acc.coarse -= min(acc.coarse, uint32_t(own >> 38));
  }
  const u64 sum = warp_sum(acc.sum);
  return warp_sum(acc.coarse) > (5ull << 22) ? kTooMuch : sum;
}

template <typename T>
__global__ void __launch_bounds__(kVThreads, kVPerSM) verify_kernel(const __grid_constant__ VerifyArgs a) {
  namespace cg = cooperative_groups;
  ptx::cluster_arrive();
  pdl_wait();
  cg::cluster_group cl = cg::this_cluster();
  __shared__ int s_acc, s_count, s_flags;
  __shared__ u64 s_part[kVWarps * kVParts], s_cta[2][kVMaxCluster];
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
          float p = as_float(P[(size_t(b) * a.n_q + i) * in.p_stride + x]);
          float q = Q ? as_float(Q[(size_t(b) * most + i) * in.q_stride + x]) : 1.f;
          if (!(p >= 0.f && p <= 1.f)) flags |= DSA_DEVERR_PROB, p = 0.f;
          if (!(q >= 0.f && q <= 1.f)) flags |= DSA_DEVERR_PROB, q = 0.f;
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
  // (cut at p's 16-B boundaries)
  const int part = a.part, run = a.run, head = -place(prow) & (Vec<T>::kN - 1);
  auto cut = [&](int64_t at) { return at > 0 ? int(min(at + head, int64_t(V))) : 0; };
  auto part_begin = [&](int w) {
    return cut((int64_t(cta) * kVWarps + w / kVParts) * run + min(w % kVParts * part, run));
  };
  auto part_end = [&](int w) {
    return cut((int64_t(cta) * kVWarps + w / kVParts) * run + min((w % kVParts + 1) * part, run));
  };
  bool has_q = qrow != nullptr, one_hot = rejected && !Q, bad = false;
  u64 total = 0, before = 0;
  for (int round = 0; round < 2; ++round) {
    const T* q = has_q ? qrow : nullptr;
    for (int i = 0; i < kVParts; ++i) {
      const int w = warp * kVParts + i;
      const u64 sum = warp_mass<T, true>(prow, q, part_begin(w), part_end(w), V, one_hot ? x : -1, bad);
      if (lane == 0) s_part[w] = sum;
    }
    __syncthreads();
    if (round == 0) ptx::cluster_wait();  // every CTA has started: their shared memory can be written
    if (threadIdx.x < ctas) {
      u64 t = 0;
      for (int i = 0; i < kVWarps * kVParts; ++i) t = capped(t + s_part[i]);
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
  for (; w < kVWarps * kVParts && at + s_part[w] <= thr; ++w) at += s_part[w];
  if (w == kVWarps * kVParts) return;
  // (a thread has a piece of that part, and the one with the threshold walks its own)
  const int r0 = part_begin(w), end = part_end(w);
  const int piece = (end - r0 + kVThreads - 1) / kVThreads;
  const int mine = r0 + piece * int(threadIdx.x);
  const int v0t = min(mine, end), v1t = min(mine + piece, end);
  u64 own = 0;
#pragma unroll 4
  for (int v = v0t; v < v1t; ++v) own += weight<T>(prow[v], has_q ? qrow[v] : T(0.f), has_q, one_hot, v, x, bad);
  const u64 inc = warp_scan(own);
  if (lane == 31) s_scan[warp] = inc;
  __syncthreads();
  u64 pre = at + inc - own;
  for (int i = 0; i < warp; ++i) pre += s_scan[i];
  // exactly one thread, and one of its elements, has the threshold inside its weight
  if (own && pre + own > thr && pre <= thr) {
#pragma unroll 1
    for (int v = v0t; v < v1t; ++v) {
      pre += weight<T>(prow[v], has_q ? qrow[v] : T(0.f), has_q, one_hot, v, x, bad);
      if (pre > thr) {
        out[acc] = v;
        break;
      }
    }
  }
}

}  // namespace

cudaError_t launch_verify_draft(const dsa_params_t& p, const WsLayout& L, char* ws, const VerifyIn& in, cudaStream_t st) {
  VerifyArgs a;
  a.in = in;
  a.n_q = p.n_q;
  a.err = reinterpret_cast<int*>(ws + L.err);
  // as many CTAs to a request as are worth it and as run at once (the integers do not
  // depend on the cut): past one wave, each CTA's chain of loads before its row is paid again
  const int slots = sm_count() * kVPerSM;
  int ctas = 1;
  while (ctas < kVMaxCluster && int64_t(ctas) * kVWarps * kVUnit < in.vocab && 2 * ctas * int64_t(p.batch) <= slots)
    ctas *= 2;
  auto units = [](int n, int by) { return (n + by * kVUnit - 1) / (by * kVUnit); };
  a.run = units(in.vocab, ctas * kVWarps) * kVUnit;
  a.part = units(a.run, kVParts) * kVUnit;
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
