// libdsa C ABI: host-side validation, workspace carving and stage launches.
#include <algorithm>
#include <cstdint>
#include <cstring>
#include <initializer_list>

#include "dsa_internal.cuh"

using namespace dsa;

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

dsa_status_t check_params(const dsa_params_t* p) {
  if (!p) return DSA_ERR_INVALID;
  if (p->batch < 1 || p->n_q < 1 || p->max_pages_per_req < 1 || p->num_pages < 1) return DSA_ERR_INVALID;
  if (p->topk < 1) return DSA_ERR_INVALID;
  if (p->topk > kMaxTopK) return DSA_ERR_UNSUPPORTED;
  if (p->page_size != kPage || p->idx_heads != kIdxHeads || p->idx_dim != kIdxDim ||
      p->heads != kHeads || p->d_nope != kDNope || p->d_rope != kDRope)
    return DSA_ERR_UNSUPPORTED;
  if (p->key_fmt != DSA_KEY_FP8_132 && p->key_fmt != DSA_KEY_MXFP4_68) return DSA_ERR_INVALID;
  if (p->lat_fmt != DSA_LAT_FP8_576 && p->lat_fmt != DSA_LAT_NVFP4_352) return DSA_ERR_INVALID;
  const int64_t key_row = p->key_fmt == DSA_KEY_FP8_132 ? p->idx_dim + 4 : p->idx_dim / 2 + p->idx_dim / 32;
  const int64_t lat_row = p->lat_fmt == DSA_LAT_FP8_576 ? p->d_nope + p->d_rope
                                                        : p->d_nope / 2 + p->d_nope / 16 + p->d_rope;
  const int64_t key_page = int64_t(p->page_size) * key_row;
  const int64_t lat_page = int64_t(p->page_size) * lat_row;
  if (p->key_page_stride < key_page || (p->key_page_stride & 15)) return DSA_ERR_INVALID;
  if (p->lat_page_stride < lat_page || (p->lat_page_stride & 15)) return DSA_ERR_INVALID;
  if (!(p->softmax_scale > 0.f) || !(p->latent_scale > 0.f)) return DSA_ERR_INVALID;
  if (p->flags & ~int32_t(DSA_EMIT_PHYS_ROWS | DSA_Q_PREPARED)) return DSA_ERR_INVALID;
  // keep every index of the kernels inside int32 / the grid limits
  if (int64_t(p->max_pages_per_req) * p->page_size > (int64_t(1) << 28)) return DSA_ERR_UNSUPPORTED;
  if (int64_t(p->batch) * p->n_q > 65535) return DSA_ERR_UNSUPPORTED;
  return DSA_OK;
}

dsa_status_t check_ws(const dsa_params_t* p, void* ws, size_t ws_bytes, WsLayout* L) {
  if (!ws || !aligned16(ws)) return DSA_ERR_INVALID;
  *L = ws_layout(*p);
  if (ws_bytes < L->total) return DSA_ERR_WORKSPACE;
  return DSA_OK;
}

dsa_status_t cuda_status(cudaError_t e) { return e == cudaSuccess ? DSA_OK : DSA_ERR_CUDA; }

dsa_status_t check_indexer_args(const dsa_params_t* p, const void* q_idx, const float* w,
                                const void* key_pool, const int32_t* bt, const int32_t* ctx) {
  if (!key_pool || !bt || !ctx || !aligned16(key_pool)) return DSA_ERR_INVALID;
  if (p->flags & DSA_Q_PREPARED)  // the query is already in the workspace (decode rows only)
    return p->n_q > kMaxNQ ? DSA_ERR_UNSUPPORTED : DSA_OK;
  if (!q_idx || !w) return DSA_ERR_INVALID;
  if (!aligned16(q_idx) || !aligned16(key_pool) || (reinterpret_cast<uintptr_t>(w) & 3)) return DSA_ERR_INVALID;
  return DSA_OK;
}

dsa_status_t check_mla_args(const void* q, const void* lat_pool, const int32_t* bt, const int32_t* ctx,
                            void* out) {
  if (!q || !lat_pool || !bt || !ctx || !out) return DSA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(lat_pool) || !aligned16(out)) return DSA_ERR_INVALID;
  return DSA_OK;
}

// The page operations' loops over the pages count in 32 bits, past the end by a block's stride.
dsa_status_t check_page_count(const dsa_params_t* p) {
  return p->num_pages > (1 << 30) ? DSA_ERR_UNSUPPORTED : DSA_OK;
}

dsa_status_t check_pools(const dsa_page_pool_t* pools, int32_t n_pools) {
  if (n_pools < 0 || (n_pools > 0 && !pools)) return DSA_ERR_INVALID;
  if (n_pools > kMaxPools) return DSA_ERR_UNSUPPORTED;
  for (int i = 0; i < n_pools; ++i) {
    const dsa_page_pool_t& q = pools[i];
    if (!q.base || !aligned16(q.base) || q.page_bytes < 16 || (q.page_bytes & 15) || q.page_stride < q.page_bytes ||
        (q.page_stride & 15))
      return DSA_ERR_INVALID;
    if (q.page_bytes > (int64_t(1) << 32)) return DSA_ERR_UNSUPPORTED;
  }
  return DSA_OK;
}

// (sizes of a page in a token pool, by dsa_token_fmt_t)
constexpr int64_t kTokenPage[4] = {kPage * 132, kPage * 68, kPage * 576, kPage * 352};

dsa_status_t check_token_pools(const dsa_params_t* p, const dsa_token_pool_t* pools, int32_t n_pools) {
  if (n_pools < 0 || (n_pools > 0 && !pools)) return DSA_ERR_INVALID;
  if (n_pools > kMaxPools) return DSA_ERR_UNSUPPORTED;
  for (int i = 0; i < n_pools; ++i) {
    const dsa_token_pool_t& q = pools[i];
    for (int j = 0; j < i; ++j)  // a pool's tokens move once
      if (pools[j].base == q.base) return DSA_ERR_INVALID;
    if (!q.base || !aligned16(q.base) || q.fmt < DSA_TOKEN_KEY_FP8 || q.fmt > DSA_TOKEN_LAT_NVFP4 || q.layers < 1)
      return DSA_ERR_INVALID;
    if (q.layers > 4096) return DSA_ERR_UNSUPPORTED;
    const int64_t page = kTokenPage[q.fmt];
    if (q.page_stride < page || (q.page_stride & 15)) return DSA_ERR_INVALID;
    // (2^50 B: what the sums below, and the kernels' offsets, hold)
    if (q.page_stride > std::min(int64_t(1) << 40, (int64_t(1) << 50) / p->num_pages) || q.layer_stride > (int64_t(1) << 50))
      return DSA_ERR_UNSUPPORTED;
    if (q.layers == 1) continue;
    if (q.layer_stride < page || (q.layer_stride & 15)) return DSA_ERR_INVALID;
    // layers inside a page's row, or pages inside a layer
    if (q.page_stride < (q.layers - 1) * q.layer_stride + page &&
        q.layer_stride < (int64_t(p->num_pages) - 1) * q.page_stride + page)
      return DSA_ERR_INVALID;
  }
  return DSA_OK;
}

}  // namespace

extern "C" {

dsa_status_t dsa_workspace_size(const dsa_params_t* params, size_t* bytes) {
  dsa_status_t s = check_params(params);
  if (s != DSA_OK) return s;
  if (!bytes) return DSA_ERR_INVALID;
  *bytes = ws_layout(*params).total;
  return DSA_OK;
}

dsa_status_t dsa_indexer_scores(const dsa_params_t* params, const void* q_idx, const float* w,
                                const void* key_pool, const int32_t* block_table,
                                const int32_t* ctx_lens, float* scores, int64_t score_stride,
                                void* ws, size_t ws_bytes, cudaStream_t stream) {
  dsa_status_t s = check_params(params);
  if (s != DSA_OK) return s;
  if ((s = check_indexer_args(params, q_idx, w, key_pool, block_table, ctx_lens)) != DSA_OK) return s;
  if (!scores || !aligned16(scores) || score_stride < 1 || (score_stride & 3)) return DSA_ERR_INVALID;
  WsLayout L;
  if ((s = check_ws(params, ws, ws_bytes, &L)) != DSA_OK) return s;
  char* w8 = static_cast<char*>(ws);
  cudaError_t e = (params->flags & DSA_Q_PREPARED) ? cudaSuccess
                                                   : launch_idx_q_quant(*params, L, w8, q_idx, w, ctx_lens, stream);
  if (e == cudaSuccess)
    e = launch_indexer(*params, L, w8, key_pool, block_table, ctx_lens, scores, score_stride, stream);
  return cuda_status(e);
}

dsa_status_t dsa_indexer_prefill_scores(const dsa_params_t* params, int32_t world, int32_t rank, const void* q_idx,
                                        const float* w, const void* key_pool, const int32_t* block_table,
                                        const int32_t* ctx_lens, float* scores, int64_t score_stride, void* ws,
                                        size_t ws_bytes, cudaStream_t stream) {
  dsa_status_t s = check_params(params);
  if (s != DSA_OK) return s;
  if (world < 1 || rank < 0 || rank >= world) return DSA_ERR_INVALID;
  if (world > 1 && params->n_q % (2 * world * kMaxNQ)) return DSA_ERR_INVALID;
  if (params->flags & DSA_Q_PREPARED) return DSA_ERR_INVALID;
  if ((s = check_indexer_args(params, q_idx, w, key_pool, block_table, ctx_lens)) != DSA_OK) return s;
  if (!scores || !aligned16(scores) || score_stride < 1 || (score_stride & 3)) return DSA_ERR_INVALID;
  WsLayout L;
  if ((s = check_ws(params, ws, ws_bytes, &L)) != DSA_OK) return s;
  char* w8 = static_cast<char*>(ws);
  cudaError_t e = launch_idx_q_quant(*params, L, w8, q_idx, w, ctx_lens, stream, world, rank);
  if (e == cudaSuccess)
    e = launch_indexer(*params, L, w8, key_pool, block_table, ctx_lens, scores, score_stride, stream, world, rank);
  return cuda_status(e);
}

dsa_status_t dsa_topk(const dsa_params_t* params, const float* scores, int64_t score_stride,
                      const int32_t* ctx_lens, const int32_t* block_table, int32_t* topk_idx,
                      int32_t* phys_rows, void* ws, size_t ws_bytes, cudaStream_t stream) {
  dsa_status_t s = check_params(params);
  if (s != DSA_OK) return s;
  if (!scores || !aligned16(scores) || score_stride < 1 || (score_stride & 3)) return DSA_ERR_INVALID;
  if (!ctx_lens || !topk_idx) return DSA_ERR_INVALID;
  if (phys_rows && (!(params->flags & DSA_EMIT_PHYS_ROWS) || !block_table)) return DSA_ERR_INVALID;
  WsLayout L;
  if ((s = check_ws(params, ws, ws_bytes, &L)) != DSA_OK) return s;
  return cuda_status(launch_topk(*params, L, static_cast<char*>(ws), scores, score_stride, ctx_lens,
                                 block_table, topk_idx, phys_rows, stream, false));
}

dsa_status_t dsa_indexer_frontend(const dsa_params_t* params, const dsa_frontend_dims_t* dims, const void* c_q,
                                  const void* gamma_q, const void* w_q, const float* w, const void* x,
                                  const void* w_k, void* key_pool, const int32_t* block_table,
                                  const int32_t* ctx_lens, void* q8_out, float* w_out, void* ws, size_t ws_bytes,
                                  cudaStream_t stream) {
  dsa_status_t s = check_params(params);
  if (s != DSA_OK) return s;
  if (!dims) return DSA_ERR_INVALID;
  for (int d : {dims->d_c, dims->d_model})
    if (d < 256 || d > 8192 || (d % 256)) return DSA_ERR_UNSUPPORTED;
  if (!(dims->eps >= 0.f) || !(dims->eps < 1e30f)) return DSA_ERR_INVALID;
  if (int64_t(params->batch) * params->n_q > kFeMaxRows || params->n_q > kMaxNQ) return DSA_ERR_UNSUPPORTED;
  for (const void* ptr : {c_q, gamma_q, w_q, x, w_k, static_cast<const void*>(key_pool)})
    if (!ptr || !aligned16(ptr)) return DSA_ERR_INVALID;
  if (!w || (reinterpret_cast<uintptr_t>(w) & 3) || !block_table || !ctx_lens) return DSA_ERR_INVALID;
  if ((reinterpret_cast<uintptr_t>(q8_out) & 3) || (reinterpret_cast<uintptr_t>(w_out) & 3)) return DSA_ERR_INVALID;
  WsLayout L;
  if ((s = check_ws(params, ws, ws_bytes, &L)) != DSA_OK) return s;
  FrontendIn in{c_q, gamma_q, w_q, w, x, w_k, key_pool, block_table, ctx_lens, q8_out, w_out,
                dims->d_c, dims->d_model, dims->eps};
  return cuda_status(launch_idx_frontend(*params, L, static_cast<char*>(ws), in, stream));
}

dsa_status_t dsa_dcp_topk_merge(const dsa_params_t* params, const float* scores, int64_t score_stride,
                                const int32_t* ctx_lens, int32_t world, int32_t* topk_idx, int32_t* stats,
                                void* ws, size_t ws_bytes, cudaStream_t stream) {
  dsa_status_t s = check_params(params);
  if (s != DSA_OK) return s;
  if (!scores || !aligned16(scores) || score_stride < 1 || (score_stride & 3)) return DSA_ERR_INVALID;
  if (!ctx_lens || !topk_idx) return DSA_ERR_INVALID;
  if (world < 1 || world > dsa::kDcpMaxWorld) return DSA_ERR_INVALID;
  WsLayout L;
  if ((s = check_ws(params, ws, ws_bytes, &L)) != DSA_OK) return s;
  return cuda_status(launch_dcp_merge(*params, L, static_cast<char*>(ws), scores, score_stride, ctx_lens, world,
                                      topk_idx, stats, stream));
}

dsa_status_t dsa_lse_combine(const dsa_params_t* params, int32_t parts, const void* part_out,
                             const float* part_lse, void* out, float* lse, cudaStream_t stream) {
  dsa_status_t s = check_params(params);
  if (s != DSA_OK) return s;
  if (parts < 1 || parts > dsa::kDcpMaxWorld) return DSA_ERR_INVALID;
  if (!part_out || !part_lse || !out || !aligned16(part_out) || !aligned16(out)) return DSA_ERR_INVALID;
  return cuda_status(
      launch_dcp_lse_combine(params->batch * params->n_q, parts, part_out, part_lse, out, lse, stream));
}

dsa_status_t dsa_sparse_mla_decode(const dsa_params_t* params, const void* q, const void* lat_pool,
                                   const int32_t* block_table, const int32_t* ctx_lens,
                                   const int32_t* topk_idx, void* out, float* lse, void* ws,
                                   size_t ws_bytes, cudaStream_t stream) {
  dsa_status_t s = check_params(params);
  if (s != DSA_OK) return s;
  if ((s = check_mla_args(q, lat_pool, block_table, ctx_lens, out)) != DSA_OK) return s;
  if (!topk_idx) return DSA_ERR_INVALID;
  WsLayout L;
  if ((s = check_ws(params, ws, ws_bytes, &L)) != DSA_OK) return s;
  return cuda_status(launch_sparse_mla(*params, L, static_cast<char*>(ws), q, lat_pool, block_table,
                                       ctx_lens, topk_idx, out, lse, stream));
}

dsa_status_t dsa_decode(const dsa_params_t* params, const void* q_idx, const float* w,
                        const void* key_pool, const void* q, const void* lat_pool,
                        const int32_t* block_table, const int32_t* ctx_lens, void* out, float* lse,
                        int32_t* topk_idx_out, void* ws, size_t ws_bytes, cudaStream_t stream) {
  dsa_status_t s = check_params(params);
  if (s != DSA_OK) return s;
  if ((s = check_indexer_args(params, q_idx, w, key_pool, block_table, ctx_lens)) != DSA_OK) return s;
  if ((s = check_mla_args(q, lat_pool, block_table, ctx_lens, out)) != DSA_OK) return s;
  WsLayout L;
  if ((s = check_ws(params, ws, ws_bytes, &L)) != DSA_OK) return s;
  char* w8 = static_cast<char*>(ws);
  if (!topk_idx_out) topk_idx_out = reinterpret_cast<int32_t*>(w8 + L.topk);
  float* scores = reinterpret_cast<float*>(w8 + L.scores);
  cudaError_t e = (params->flags & DSA_Q_PREPARED) ? cudaSuccess
                                                   : launch_idx_q_quant(*params, L, w8, q_idx, w, ctx_lens, stream);
  if (e == cudaSuccess)
    e = launch_indexer(*params, L, w8, key_pool, block_table, ctx_lens, scores, L.cap, stream, 1, 0, true);
  if (e == cudaSuccess)
    e = launch_topk(*params, L, w8, scores, L.cap, ctx_lens, block_table, topk_idx_out, nullptr, stream, true,
                    lat_pool);
  if (e == cudaSuccess)
    e = launch_sparse_mla(*params, L, w8, q, lat_pool, block_table, ctx_lens, topk_idx_out, out, lse,
                          stream, true);
  return cuda_status(e);
}

dsa_status_t dsa_prefix_mla_decode(const dsa_params_t* params, const void* q, const void* lat_pool,
                                   const int32_t* prefix_pages, int32_t prefix_len, const int32_t* block_table,
                                   const int32_t* ctx_lens, void* out, float* lse, void* ws, size_t ws_bytes,
                                   cudaStream_t stream) {
  dsa_status_t s = check_params(params);
  if (s != DSA_OK) return s;
  if ((s = check_mla_args(q, lat_pool, block_table, ctx_lens, out)) != DSA_OK) return s;
  if (prefix_len < 0 || prefix_len % params->page_size || (prefix_len > 0 && !prefix_pages)) return DSA_ERR_INVALID;
  if (int64_t(prefix_len) + params->n_q > int64_t(params->max_pages_per_req) * params->page_size)
    return DSA_ERR_INVALID;
  if (int64_t(params->batch) * params->n_q * params->max_pages_per_req > kPfxMaxTiles) return DSA_ERR_UNSUPPORTED;
  WsLayout L;
  if ((s = check_ws(params, ws, ws_bytes, &L)) != DSA_OK) return s;
  return cuda_status(launch_prefix_mla(*params, L, static_cast<char*>(ws), q, lat_pool, prefix_pages, prefix_len,
                                       block_table, ctx_lens, out, lse, stream));
}

dsa_status_t dsa_pages_resize(const dsa_params_t* params, const int32_t* new_lens, const dsa_page_pool_t* pools,
                              int32_t n_pools, int32_t* block_table, int32_t* ctx_lens, int32_t* page_refs, void* ws,
                              size_t ws_bytes, cudaStream_t stream) {
  dsa_status_t s = check_params(params);
  if (s != DSA_OK) return s;
  if (!new_lens || !block_table || !ctx_lens || !page_refs) return DSA_ERR_INVALID;
  if ((s = check_page_count(params)) != DSA_OK) return s;
  if ((s = check_pools(pools, n_pools)) != DSA_OK) return s;
  WsLayout L;
  if ((s = check_ws(params, ws, ws_bytes, &L)) != DSA_OK) return s;
  return cuda_status(launch_pages_resize(*params, L, static_cast<char*>(ws), new_lens, pools, n_pools, block_table,
                                         ctx_lens, page_refs, stream));
}

dsa_status_t dsa_pages_fork(const dsa_params_t* params, int32_t n, const int32_t* src, const int32_t* dst,
                            int32_t* block_table, int32_t* ctx_lens, int32_t* page_refs, void* ws, size_t ws_bytes,
                            cudaStream_t stream) {
  dsa_status_t s = check_params(params);
  if (s != DSA_OK) return s;
  if (n < 0 || n > params->batch || (n > 0 && (!src || !dst))) return DSA_ERR_INVALID;
  if (!block_table || !ctx_lens || !page_refs) return DSA_ERR_INVALID;
  if ((s = check_page_count(params)) != DSA_OK) return s;
  WsLayout L;
  if ((s = check_ws(params, ws, ws_bytes, &L)) != DSA_OK) return s;
  if (n == 0) return DSA_OK;
  return cuda_status(launch_pages_fork(*params, L, static_cast<char*>(ws), n, src, dst, block_table, ctx_lens,
                                       page_refs, stream));
}

dsa_status_t dsa_pages_compact(const dsa_params_t* params, const dsa_page_pool_t* pools, int32_t n_pools,
                               int32_t* block_table, const int32_t* ctx_lens, int32_t* page_refs, int32_t* page_map,
                               int32_t* live, void* ws, size_t ws_bytes, cudaStream_t stream) {
  dsa_status_t s = check_params(params);
  if (s != DSA_OK) return s;
  if (!block_table || !ctx_lens || !page_refs) return DSA_ERR_INVALID;
  if ((s = check_page_count(params)) != DSA_OK) return s;
  if ((s = check_pools(pools, n_pools)) != DSA_OK) return s;
  WsLayout L;
  if ((s = check_ws(params, ws, ws_bytes, &L)) != DSA_OK) return s;
  return cuda_status(launch_pages_compact(*params, L, static_cast<char*>(ws), pools, n_pools, block_table, ctx_lens,
                                          page_refs, page_map, live, stream));
}

dsa_status_t dsa_latent_frontend(const dsa_params_t* params, const dsa_latent_dims_t* dims, const void* q_nope,
                                 const void* q_rope, const void* gamma_q, const void* c_kv, const void* k_rope,
                                 const void* gamma_kv, const float* inv_freq, const int32_t* positions,
                                 void* lat_pool, const int32_t* block_table, const int32_t* ctx_lens, void* q_out,
                                 void* ws, size_t ws_bytes, cudaStream_t stream) {
  dsa_status_t s = check_params(params);
  if (s != DSA_OK) return s;
  if (!dims || !(dims->eps >= 1e-30f) || !(dims->eps <= 1e30f) || (dims->interleaved != 0 && dims->interleaved != 1))
    return DSA_ERR_INVALID;
  if ((!q_out && !c_kv) || !inv_freq || !ctx_lens) return DSA_ERR_INVALID;
  if (!aligned16(inv_freq) || (reinterpret_cast<uintptr_t>(positions) & 3)) return DSA_ERR_INVALID;
  auto input = [](const void* x, std::initializer_list<int64_t> strides, int64_t least) {
    if (!x || !aligned16(x)) return false;
    for (int64_t d : strides)
      if (d < least || (d & 7) || d > (int64_t(1) << 40)) return false;
    return true;
  };
  if (q_out) {
    // (rows of heads, or heads of rows)
    if (!input(q_nope, {dims->q_nope_row, dims->q_nope_head}, kDNope) ||
        !input(q_rope, {dims->q_rope_row, dims->q_rope_head}, kDRope) || !aligned16(q_out) || !aligned16(gamma_q))
      return DSA_ERR_INVALID;
  }
  if (c_kv) {
    if (!input(c_kv, {dims->c_kv_row}, kDNope) || !input(k_rope, {dims->k_rope_row}, kDRope) || !input(gamma_kv, {}, 0) ||
        !input(lat_pool, {}, 0) || !block_table)
      return DSA_ERR_INVALID;
  }
  const WsLayout L = ws_layout(*params);
  if (!ws || !aligned16(ws)) return DSA_ERR_INVALID;
  if (ws_bytes < L.q8) return DSA_ERR_WORKSPACE;  // the error word is all it uses
  const LatentIn in{q_nope, q_rope, gamma_q, c_kv, k_rope, gamma_kv, inv_freq, positions, lat_pool, block_table, ctx_lens,
                    q_out, dims->q_nope_row, dims->q_nope_head, dims->q_rope_row, dims->q_rope_head, dims->c_kv_row,
                    dims->k_rope_row, dims->eps};
  return cuda_status(launch_latent_frontend(*params, reinterpret_cast<int*>(static_cast<char*>(ws) + L.err), in,
                                            dims->interleaved == 1, stream));
}

dsa_status_t dsa_window_mla_decode(const dsa_params_t* params, const void* q, const void* lat_pool, int32_t sinks,
                                   int32_t window, const int32_t* block_table, const int32_t* ctx_lens, void* out,
                                   float* lse, void* ws, size_t ws_bytes, cudaStream_t stream) {
  dsa_status_t s = check_params(params);
  if (s != DSA_OK) return s;
  if ((s = check_mla_args(q, lat_pool, block_table, ctx_lens, out)) != DSA_OK) return s;
  if (sinks < 0 || window < 1 || (reinterpret_cast<uintptr_t>(lse) & 3)) return DSA_ERR_INVALID;
  if (int64_t(params->batch) * params->n_q * params->max_pages_per_req > kPfxMaxTiles / 2) return DSA_ERR_UNSUPPORTED;
  WsLayout L;
  if ((s = check_ws(params, ws, ws_bytes, &L)) != DSA_OK) return s;
  return cuda_status(launch_window_mla(*params, L, static_cast<char*>(ws), q, lat_pool, sinks, window, block_table, ctx_lens,
                                       out, lse, stream));
}

dsa_status_t dsa_attention_mass(const dsa_params_t* params, const void* q, const void* lat_pool, int32_t sinks,
                                int32_t window, const int32_t* block_table, const int32_t* ctx_lens,
                                const float* lse, int32_t fresh, float* mass, int64_t mass_stride, void* ws,
                                size_t ws_bytes, cudaStream_t stream) {
  dsa_status_t s = check_params(params);
  if (s != DSA_OK) return s;
  if (!q || !lat_pool || !block_table || !ctx_lens || !mass) return DSA_ERR_INVALID;
  if (!aligned16(q) || !aligned16(lat_pool) || (reinterpret_cast<uintptr_t>(mass) & 3)) return DSA_ERR_INVALID;
  if (sinks < 0 || window < 1 || fresh < 0 || !lse || (reinterpret_cast<uintptr_t>(lse) & 3)) return DSA_ERR_INVALID;
  if (mass_stride < int64_t(params->max_pages_per_req) * params->page_size) return DSA_ERR_INVALID;
  if (int64_t(params->batch) * params->n_q * params->max_pages_per_req > kPfxMaxTiles / 2) return DSA_ERR_UNSUPPORTED;
  WsLayout L;
  if ((s = check_ws(params, ws, ws_bytes, &L)) != DSA_OK) return s;
  return cuda_status(launch_attention_mass(*params, L, static_cast<char*>(ws), q, lat_pool, sinks, window, block_table,
                                           ctx_lens, lse, fresh, mass, mass_stride, stream));
}

dsa_status_t dsa_tokens_evict(const dsa_params_t* params, const int32_t* budgets, int32_t sinks, int32_t recent,
                              float* mass, int64_t token_stride, const dsa_token_pool_t* pools, int32_t n_pools,
                              int32_t* block_table, int32_t* ctx_lens, int32_t* page_refs, int32_t* kept, void* ws,
                              size_t ws_bytes, cudaStream_t stream) {
  dsa_status_t s = check_params(params);
  if (s != DSA_OK) return s;
  if (!budgets || !mass || !block_table || !ctx_lens || !page_refs || sinks < 0 || recent < 0) return DSA_ERR_INVALID;
  if ((reinterpret_cast<uintptr_t>(mass) & 3) || (reinterpret_cast<uintptr_t>(kept) & 3)) return DSA_ERR_INVALID;
  if (token_stride < int64_t(params->max_pages_per_req) * params->page_size) return DSA_ERR_INVALID;
  if ((s = check_page_count(params)) != DSA_OK) return s;
  if ((s = check_token_pools(params, pools, n_pools)) != DSA_OK) return s;
  WsLayout L;
  if ((s = check_ws(params, ws, ws_bytes, &L)) != DSA_OK) return s;
  return cuda_status(launch_tokens_evict(*params, L, static_cast<char*>(ws), budgets, sinks, recent, mass, token_stride, pools,
                                         n_pools, block_table, ctx_lens, page_refs, kept, stream));
}

dsa_status_t dsa_verify_draft(const dsa_params_t* params, int32_t vocab, int32_t dtype, const void* p_target,
                              int64_t p_stride, const void* p_draft, int64_t q_stride, const int32_t* draft_tokens,
                              const int32_t* n_draft, const float* uniforms, const int32_t* ctx_lens,
                              int32_t* n_accepted, int32_t* out_tokens, int32_t* new_lens, void* ws, size_t ws_bytes,
                              cudaStream_t stream) {
  dsa_status_t s = check_params(params);
  if (s != DSA_OK) return s;
  if (vocab < 1 || dtype < DSA_PROB_F32 || dtype > DSA_PROB_F16) return DSA_ERR_INVALID;
  if (vocab > (1 << 24)) return DSA_ERR_UNSUPPORTED;
  const uintptr_t mis = dtype == DSA_PROB_F32 ? 3 : 1;  // elements are aligned to their size
  if (!p_target || (reinterpret_cast<uintptr_t>(p_target) & mis) || p_stride < vocab) return DSA_ERR_INVALID;
  if (p_draft && ((reinterpret_cast<uintptr_t>(p_draft) & mis) || q_stride < vocab)) return DSA_ERR_INVALID;
  if (params->n_q > 1 && !draft_tokens) return DSA_ERR_INVALID;
  if (!uniforms || !n_accepted || !out_tokens || (new_lens && !ctx_lens)) return DSA_ERR_INVALID;
  const WsLayout L = ws_layout(*params);
  if (!ws || !aligned16(ws)) return DSA_ERR_INVALID;
  if (ws_bytes < L.q8) return DSA_ERR_WORKSPACE;  // the error word is all it uses
  const VerifyIn in{p_target, p_draft, p_stride, q_stride, draft_tokens, n_draft, uniforms, ctx_lens,
                    n_accepted, out_tokens, new_lens, vocab, dtype};
  return cuda_status(launch_verify_draft(*params, L, static_cast<char*>(ws), in, stream));
}

dsa_status_t dsa_get_device_error(void* ws, cudaStream_t stream, int32_t* code) {
  if (!ws || !code) return DSA_ERR_INVALID;
  int32_t v = 0;
  cudaError_t e = cudaMemcpyAsync(&v, ws, sizeof(int32_t), cudaMemcpyDeviceToHost, stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e == cudaSuccess) e = cudaMemsetAsync(ws, 0, sizeof(int32_t), stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return DSA_ERR_CUDA;
  *code = v;
  return (v & DSA_DEVERR_TIMEOUT) ? DSA_ERR_TIMEOUT : DSA_OK;
}

const char* dsa_status_string(dsa_status_t status) {
  switch (status) {
    case DSA_OK: return "DSA_OK";
    case DSA_ERR_INVALID: return "DSA_ERR_INVALID: invalid argument";
    case DSA_ERR_UNSUPPORTED: return "DSA_ERR_UNSUPPORTED: size or format not implemented";
    case DSA_ERR_WORKSPACE: return "DSA_ERR_WORKSPACE: workspace too small";
    case DSA_ERR_CUDA: return "DSA_ERR_CUDA: CUDA launch or runtime error";
    case DSA_ERR_TIMEOUT: return "DSA_ERR_TIMEOUT: device wait gave up";
  }
  return "unknown dsa_status_t";
}

}  // extern "C"
