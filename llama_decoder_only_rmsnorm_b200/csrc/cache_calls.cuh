// cache_calls.cuh -- host side of the cache operators (tree attention, observed
// attention, eviction, acceptance).  Included at the end of llama3.cu, whose
// launch and argument helpers it uses.
#pragma once

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct TreeWorkspace {
  size_t total;
};
TreeWorkspace tree_layout(const llama3_config*, int, int, int) {
  TreeWorkspace w;
  w.total = 0;
  return w;
}

struct ObserveWorkspace {
  size_t lse, total;
};
ObserveWorkspace observe_layout(const llama3_config* c, int batch, int seq, int max_len) {
  ObserveWorkspace w;
  (void)max_len;
  size_t off = 0;
  w.lse = off; off += up256((size_t)batch * c->n_heads * seq * 4);
  w.total = off;
  return w;
}

int check_tree_shape(const llama3_config* c, int batch, int nodes, int max_len) {
  L3_TRY(check_config(c));
  if (batch < 1 || nodes < 1 || nodes > kMaxTreeNodes || max_len < 0) return LLAMA3_ERR_ARG;
  return LLAMA3_OK;
}

template <typename T>
int run_tree_simt(const llama3_config* c, const void* q, const void* kc, const void* vc, int cap, const int32_t* lens,
                  int max_len, const void* kn, const void* vn, const int32_t* parents, int B, int nodes, void* out,
                  cudaStream_t st) {
  const long long warps = (long long)B * nodes * c->n_heads;
  L3_LAUNCH(LLAMA3_KERNEL_TREE_ATTENTION, st,
            launch_k((tree_attention_simt_kernel<T>), blocks_for(warps * 32, 256), 256, 0, st, (const T*)q,
                     (const T*)kc, (const T*)vc, (const T*)kn, (const T*)vn, lens, parents, (T*)out, B, nodes,
                     c->n_heads, c->n_kv_heads, c->head_dim, cap, max_len, (float)(1.0 / sqrt((double)c->head_dim))));
  return launch_check();
}

template <typename T>
int run_observe_simt(const llama3_config* c, const void* q, const void* kc, const void* vc, int cap, int B, int S,
                     const int32_t* lens, const int32_t* seq_lens, int max_len, void* out, const float* win,
                     float* wout, const int32_t* positions, int32_t* slot_pos, float* lse, cudaStream_t st) {
  const float scale = (float)(1.0 / sqrt((double)c->head_dim));
  const int H = c->n_heads, KV = c->n_kv_heads, hd = c->head_dim;
  L3_LAUNCH(LLAMA3_KERNEL_OBSERVED_ATTENTION, st,
            launch_k((observed_attention_simt_kernel<T>), blocks_for((long long)B * S * H * 32, 256), 256, 0, st,
                     (const T*)q, (const T*)kc, (const T*)vc, lens, seq_lens, (T*)out, lse, B, S, H, KV, hd, cap,
                     max_len, scale));
  L3_TRY(launch_check());
  L3_LAUNCH(LLAMA3_KERNEL_OBSERVED_ATTENTION, st,
            launch_k((observed_weights_simt_kernel<T>), blocks_for((long long)B * KV * (max_len + S) * 32, 256), 256,
                     0, st, (const T*)q, (const T*)kc, lens, seq_lens, (const float*)lse, win, wout, positions,
                     slot_pos, B, S, H, KV, hd, cap, max_len, scale));
  return launch_check();
}

}  // namespace

extern "C" {

int llama3_tree_workspace_size(const llama3_config* cfg, int batch, int n_nodes, int max_len, size_t* bytes) {
  L3_TRY(check_tree_shape(cfg, batch, n_nodes, max_len));
  if (!bytes) return LLAMA3_ERR_ARG;
  *bytes = tree_layout(cfg, batch, n_nodes, max_len).total;
  return LLAMA3_OK;
}

int llama3_attention_tree(const llama3_config* cfg, const void* q, const void* k_cache, const void* v_cache,
                          int cache_cap, const int32_t* kv_lens, int max_len, const void* k_nodes, const void* v_nodes,
                          const int32_t* parents, int batch, int n_nodes, void* out, void* ws, size_t ws_bytes,
                          llama3_stream_t stream) {
  L3_TRY(check_tree_shape(cfg, batch, n_nodes, max_len));
  if (!q || !k_cache || !v_cache || !kv_lens || !k_nodes || !v_nodes || !parents || !out) return LLAMA3_ERR_ARG;
  if (cache_cap < 1 || max_len > cache_cap) return LLAMA3_ERR_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_nodes) || !aligned16(v_nodes) ||
      !aligned16(out) || !aligned4(kv_lens) || !aligned4(parents))
    return LLAMA3_ERR_ALIGN;
  const TreeWorkspace L = tree_layout(cfg, batch, n_nodes, max_len);
  if (L.total && (!ws || ws_bytes < L.total)) return LLAMA3_ERR_WORKSPACE;
  if (!aligned16(ws)) return LLAMA3_ERR_ALIGN;
  cudaStream_t st = (cudaStream_t)stream;
  return cfg->dtype == LLAMA3_DTYPE_F32
             ? run_tree_simt<float>(cfg, q, k_cache, v_cache, cache_cap, kv_lens, max_len, k_nodes, v_nodes, parents,
                                    batch, n_nodes, out, st)
             : run_tree_simt<bf16>(cfg, q, k_cache, v_cache, cache_cap, kv_lens, max_len, k_nodes, v_nodes, parents,
                                   batch, n_nodes, out, st);
}

int llama3_observe_workspace_size(const llama3_config* cfg, int batch, int seq, int max_len, size_t* bytes) {
  L3_TRY(check_config(cfg));
  if (!bytes || batch < 1 || seq < 1 || max_len < 0) return LLAMA3_ERR_ARG;
  *bytes = observe_layout(cfg, batch, seq, max_len).total;
  return LLAMA3_OK;
}

int llama3_attention_observed(const llama3_config* cfg, const void* q, const void* k_cache, const void* v_cache,
                              int cache_cap, int batch, int seq, const int32_t* kv_lens, const int32_t* seq_lens,
                              int max_len, void* out, const float* weights_in, float* weights,
                              const int32_t* positions, int32_t* slot_pos, void* ws, size_t ws_bytes,
                              llama3_stream_t stream) {
  L3_TRY(check_config(cfg));
  if (!q || !k_cache || !v_cache || !out || !weights || batch < 1 || seq < 1 || max_len < 0) return LLAMA3_ERR_ARG;
  if ((long long)max_len + seq > cache_cap) return LLAMA3_ERR_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned4(kv_lens) ||
      !aligned4(seq_lens) || !aligned4(weights_in) || !aligned4(weights) || !aligned4(positions) ||
      !aligned4(slot_pos))
    return LLAMA3_ERR_ALIGN;
  const ObserveWorkspace L = observe_layout(cfg, batch, seq, max_len);
  if (!ws || ws_bytes < L.total) return LLAMA3_ERR_WORKSPACE;
  if (!aligned16(ws)) return LLAMA3_ERR_ALIGN;
  cudaStream_t st = (cudaStream_t)stream;
  float* lse = ws_at<float>(ws, L.lse);
  return cfg->dtype == LLAMA3_DTYPE_F32
             ? run_observe_simt<float>(cfg, q, k_cache, v_cache, cache_cap, batch, seq, kv_lens, seq_lens, max_len,
                                       out, weights_in, weights, positions, slot_pos, lse, st)
             : run_observe_simt<bf16>(cfg, q, k_cache, v_cache, cache_cap, batch, seq, kv_lens, seq_lens, max_len,
                                      out, weights_in, weights, positions, slot_pos, lse, st);
}

int llama3_evict_workspace_size(const llama3_config* cfg, int n_layers, int batch, int max_len, int budget,
                                size_t* bytes) {
  L3_TRY(check_config(cfg));
  if (!bytes || n_layers < 1 || batch < 1 || max_len < 0 || budget < 1) return LLAMA3_ERR_ARG;
  *bytes = up256((size_t)n_layers * batch * cfg->n_kv_heads * (size_t)evict_row_words(max_len, budget) * 4);
  return LLAMA3_OK;
}

int llama3_cache_evict(const llama3_config* cfg, const llama3_bounded_cache* src, int src_cap,
                       const llama3_bounded_cache* dst, int dst_cap, int n_layers, int batch, const int32_t* kv_lens,
                       int max_len, int budget, int recent, const int32_t* positions, int32_t* kv_lens_out, void* ws,
                       size_t ws_bytes, llama3_stream_t stream) {
  L3_TRY(check_config(cfg));
  if (!src || !kv_lens || !positions || !kv_lens_out || n_layers < 1 || batch < 1) return LLAMA3_ERR_ARG;
  if (src_cap < 1 || max_len < 0 || max_len > src_cap || budget < 1 || recent < 0 || recent > budget)
    return LLAMA3_ERR_ARG;
  // what stays is at most min(max_len, budget) slots
  if (dst && (dst_cap < 1 || dst_cap < std::min(max_len, budget))) return LLAMA3_ERR_ARG;
  for (int i = 0; i < n_layers; ++i) {
    for (const llama3_bounded_cache* c : {src + i, dst ? dst + i : src + i}) {
      if (!c->k || !c->v || !c->weights || !c->slot_pos) return LLAMA3_ERR_ARG;
      if (!aligned16(c->k) || !aligned16(c->v) || !aligned4(c->weights) || !aligned4(c->slot_pos))
        return LLAMA3_ERR_ALIGN;
    }
    // one layer's buffers are all its own or all the source's
    if (dst && (dst[i].k == src[i].k || dst[i].v == src[i].v || dst[i].weights == src[i].weights ||
                dst[i].slot_pos == src[i].slot_pos))
      return LLAMA3_ERR_ARG;
  }
  if (!aligned4(kv_lens) || !aligned4(positions) || !aligned4(kv_lens_out)) return LLAMA3_ERR_ALIGN;
  size_t need = 0;
  L3_TRY(llama3_evict_workspace_size(cfg, n_layers, batch, max_len, budget, &need));
  if (!ws || ws_bytes < need) return LLAMA3_ERR_WORKSPACE;
  if (!aligned16(ws)) return LLAMA3_ERR_ALIGN;
  if ((long long)std::min(n_layers, kEvictLayers) * batch * cfg->n_kv_heads > INT_MAX) return LLAMA3_ERR_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  const long long words = evict_row_words(max_len, budget);
  EvictParams p;
  memset(&p, 0, sizeof(p));
  p.kv_lens = kv_lens;
  p.positions = positions;
  p.B = batch; p.KV = cfg->n_kv_heads; p.row16 = (int)(cfg->head_dim * esize(cfg) / 16);
  p.cap = src_cap; p.dst_cap = dst ? dst_cap : src_cap;
  p.max_len = max_len; p.budget = budget; p.recent = recent; p.in_place = dst ? 0 : 1;
  p.ws_row = words;
  for (int l0 = 0; l0 < n_layers; l0 += kEvictLayers) {
    const int nl = std::min(kEvictLayers, n_layers - l0);
    for (int i = 0; i < nl; ++i) {
      const llama3_bounded_cache& s = src[l0 + i];
      const llama3_bounded_cache& d = dst ? dst[l0 + i] : s;
      p.layer[i] = {(const uint4*)s.k, (const uint4*)s.v, s.weights, s.slot_pos,
                    (uint4*)d.k, (uint4*)d.v, d.weights, d.slot_pos};
    }
    p.ws = (int32_t*)ws + (size_t)l0 * batch * cfg->n_kv_heads * words;
    const int rows = nl * batch * cfg->n_kv_heads;
    L3_LAUNCH(LLAMA3_KERNEL_EVICT, st, launch_k(evict_select_kernel, rows, kEvictThreads, 0, st, p));
    L3_TRY(launch_check());
    const long long pieces = (long long)std::min(max_len, budget) * p.row16;
    const int parts = (int)std::max(1LL, std::min((pieces + 2047) / 2048, 64LL));
    L3_LAUNCH(LLAMA3_KERNEL_EVICT, st, launch_k(evict_move_kernel, dim3(rows, parts), 256, 0, st, p));
    L3_TRY(launch_check());
  }
  L3_LAUNCH(LLAMA3_KERNEL_EVICT, st,
            launch_k(evict_lens_kernel, blocks_for(batch, 256), 256, 0, st, kv_lens, kv_lens_out, batch, max_len,
                     budget));
  return launch_check();
}

int llama3_tree_accept(const int32_t* draft_ids, const int32_t* target_ids, const int32_t* parents, int batch,
                       int n_nodes, const int32_t* kv_lens, int32_t* path, int32_t* n_accepted, int32_t* next_ids,
                       int32_t* kv_lens_out, const int32_t* positions, int32_t* positions_out,
                       llama3_stream_t stream) {
  if (!draft_ids || !target_ids || !parents || !kv_lens || !path || !n_accepted || !next_ids || !kv_lens_out)
    return LLAMA3_ERR_ARG;
  if (batch < 1 || n_nodes < 1 || n_nodes > kMaxTreeNodes || (positions_out && !positions)) return LLAMA3_ERR_ARG;
  for (const void* p : {(const void*)draft_ids, (const void*)target_ids, (const void*)parents, (const void*)kv_lens,
                        (const void*)path, (const void*)n_accepted, (const void*)next_ids, (const void*)kv_lens_out,
                        (const void*)positions, (const void*)positions_out})
    if (!aligned4(p)) return LLAMA3_ERR_ALIGN;
  cudaStream_t st = (cudaStream_t)stream;
  L3_LAUNCH(LLAMA3_KERNEL_ACCEPT, st,
            launch_k(tree_accept_kernel, batch, kMaxTreeNodes, 0, st, draft_ids, target_ids, parents, n_nodes, kv_lens,
                     path, n_accepted, next_ids, kv_lens_out, positions, positions_out));
  return launch_check();
}

int llama3_tree_commit(const llama3_config* cfg, const llama3_bounded_cache* nodes, const llama3_bounded_cache* caches,
                       int cache_cap, int n_layers, int batch, int n_nodes, const int32_t* path,
                       const int32_t* n_accepted, const int32_t* kv_lens, const int32_t* positions,
                       llama3_stream_t stream) {
  L3_TRY(check_config(cfg));
  if (!nodes || !caches || !path || !n_accepted || !kv_lens) return LLAMA3_ERR_ARG;
  if (n_layers < 1 || batch < 1 || n_nodes < 1 || n_nodes > kMaxTreeNodes || cache_cap < 1) return LLAMA3_ERR_ARG;
  for (int i = 0; i < n_layers; ++i) {
    if (!nodes[i].k || !nodes[i].v || !caches[i].k || !caches[i].v) return LLAMA3_ERR_ARG;
    if (!aligned16(nodes[i].k) || !aligned16(nodes[i].v) || !aligned16(caches[i].k) || !aligned16(caches[i].v) ||
        !aligned4(caches[i].weights) || !aligned4(caches[i].slot_pos))
      return LLAMA3_ERR_ALIGN;
  }
  if (!aligned4(path) || !aligned4(n_accepted) || !aligned4(kv_lens) || !aligned4(positions)) return LLAMA3_ERR_ALIGN;
  cudaStream_t st = (cudaStream_t)stream;
  CommitParams p;
  memset(&p, 0, sizeof(p));
  p.path = path; p.accepted = n_accepted; p.kv_lens = kv_lens; p.positions = positions;
  p.nodes = n_nodes; p.KV = cfg->n_kv_heads;
  p.row16 = (int)((size_t)cfg->n_kv_heads * cfg->head_dim * esize(cfg) / 16);
  p.cap = cache_cap;
  constexpr int kLayers = sizeof(p.layer) / sizeof(p.layer[0]);
  for (int l0 = 0; l0 < n_layers; l0 += kLayers) {
    const int nl = std::min(kLayers, n_layers - l0);
    for (int i = 0; i < nl; ++i)
      p.layer[i] = {(const uint4*)nodes[l0 + i].k, (const uint4*)nodes[l0 + i].v, (uint4*)caches[l0 + i].k,
                    (uint4*)caches[l0 + i].v, caches[l0 + i].weights, caches[l0 + i].slot_pos};
    L3_LAUNCH(LLAMA3_KERNEL_ACCEPT, st, launch_k(tree_commit_kernel, dim3(batch, nl), 256, 0, st, p));
    L3_TRY(launch_check());
  }
  return LLAMA3_OK;
}

}  // extern "C"
