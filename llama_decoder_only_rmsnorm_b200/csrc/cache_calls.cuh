// cache_calls.cuh -- host side of the cache operators (tree attention, observed
// attention, eviction, acceptance).  Included at the end of llama3.cu, whose
// launch and argument helpers it uses.
#pragma once

namespace {

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// The tensor-core kernels take bf16 heads of 32 and more, up to 128 query heads per
// KV head; fp32, head_dim 16 and the plain kernel path go to the CUDA cores, which
// take up to 64.  Larger groups are refused.
bool rows_on_tc(const llama3_config* c) {
  return c->dtype == LLAMA3_DTYPE_BF16 && g_kernel_path != 1 && c->head_dim >= 32 && c->n_heads / c->n_kv_heads <= 128;
}
bool rows_supported(const llama3_config* c) { return rows_on_tc(c) || c->n_heads / c->n_kv_heads <= kSimtTile; }

// How T query positions per sequence over at most max_keys cached rows are laid
// out, and what the launch needs of the workspace.
struct RowsPlan {
  RowsShape rs;
  bool tc, pair;
  bool fits;       // the plans' units stay below 2^30
  size_t cuts, ml, o, nlse, sums, scores, total;
  bool scored;     // observed: the weights come from kept scores
};
RowsPlan plan_rows(const llama3_config* c, bool tree, int B, int T, int max_len) {
  RowsPlan p;
  memset(&p, 0, sizeof(p));
  RowsShape& rs = p.rs;
  p.tc = rows_on_tc(c);
  rs.B = B; rs.T = T; rs.H = c->n_heads; rs.KV = c->n_kv_heads; rs.rep = c->n_heads / c->n_kv_heads;
  rs.tile_rows = p.tc ? 128 : kSimtTile;
  rs.qpt = std::max(1, rs.tile_rows / rs.rep);
  rs.tiles = (T + rs.qpt - 1) / rs.qpt;
  const long long keys = (long long)max_len + (tree ? 0 : T);
  // Two row tiles per CTA share every K/V tile.  Out of little work, one row tile at
  // a time makes longer runs of keys, and so fewer records to write and join: 28 us
  // against 31 for a tree of 64 nodes over 8192 rows of the 8B heads, 20 against
  // 22.5 over 2000, 49 alike over 30000.  Not for a chunk, which writes whole
  // segments without records (8 x 517 rows: 51 us against 47).
  const long long steps = (long long)B * rs.KV * rs.tiles * ((keys + 127) / 128);
  p.pair = p.tc && rs.tiles > 1 && (!tree || steps > 16LL * num_sms());
  rs.slots = p.pair ? 2 : 1;
  rs.groups = (rs.tiles + rs.slots - 1) / rs.slots;
  rs.key_shift = p.tc ? 7 : 6;
  rs.max_len = max_len;
  rs.scale_log2 = (float)(1.4426950408889634 / sqrt((double)c->head_dim));
  // One CTA per SM for the tensor-core kernels, two of the others (of head_dim 128 an
  // SM holds one at a time, 119 KB each, and takes the second after it); no more than
  // there is work for.  (Four tiles at least per CTA, for fewer pieces to join:
  // 34 us against 27 for 4 sequences of 1000 fp32 keys.)
  const long long work = (long long)B * rs.groups * rs.KV * ((keys + (1 << rs.key_shift) - 1) >> rs.key_shift);
  rs.G = (int)std::min((long long)num_sms() * (p.tc ? 1 : 2), work);
  const long long units = (long long)B * rs.KV * rs.groups * (((keys + 63) >> rs.key_shift) + kFlatLead + 1);
  const long long sums = tree ? 0 : (long long)B * rs.KV * ((keys >> (p.tc ? 8 : 6)) + 1) * (rs.tiles + kFlatLead);
  p.fits = units < (1LL << 30) && sums < (1LL << 30);
  // More than 64 pieces of a segment, if all segments are of one length, are joined by
  // a launch of their own: 37 us against 60 with 148 pieces a row (one observed step
  // over 60000 rows of one KV head of 128), 50 against 43 with 37 (four heads of 64).
  // One long sequence among short ones counts by the average, and may so be joined by
  // one warp per row although it has as many pieces: the host does not know the lengths.
  rs.folded = rs.G / ((long long)B * rs.groups * rs.KV) > 64;
  const size_t records = tree ? (size_t)B * rs.groups * rs.KV + rs.G : (size_t)2 * rs.G;
  const size_t rows = records * rs.slots * rs.tile_rows;
  size_t off = 0;
  p.cuts = off; off += up256((size_t)2 * num_sms() * sizeof(FlatCut));
  p.ml = off; off += up256(rows * 2 * 4);
  p.o = off; off += up256(rows * c->head_dim * 4);
  if (!tree) {
    p.nlse = off; off += up256((size_t)B * rs.KV * rs.tiles * rs.tile_rows * 4);
    p.sums = off; off += up256((size_t)2 * num_sms() * 2 * 256 * 4);
    // Scores kept in fp32 cost 8 bytes per row and slot (written, read), a second
    // pass over K 2 hd bytes per slot: up to hd / 4 rows the scores are less.
    p.scored = p.tc && (long long)T * rs.rep <= c->head_dim / 4 && (long long)B * rs.KV <= 65535;
    p.scores = off;
    if (p.scored) off += up256((size_t)B * rs.H * T * (((size_t)keys + 127) / 128 * 128) * 4);
  }
  p.total = rs.G > 0 ? off : 0;
  return p;
}

// q as 128-row tiles of 128 / rep positions x rep heads: {hd, rep, KV, T, B}.
int make_map_rows(CUtensorMap* m, const void* q, const llama3_config* c, const RowsShape& rs) {
  EncodeTiledFn enc;
  L3_TRY(encode_fn(&enc));
  const cuuint64_t hd = c->head_dim;
  cuuint64_t dims[5] = {hd, (cuuint64_t)rs.rep, (cuuint64_t)rs.KV, (cuuint64_t)rs.T, (cuuint64_t)rs.B};
  cuuint64_t strides[4] = {hd * 2, rs.rep * hd * 2, rs.H * hd * 2, rs.T * (rs.H * hd * 2)};
  cuuint32_t box[5] = {64u, (cuuint32_t)rs.rep, 1u, (cuuint32_t)rs.qpt, 1u};
  cuuint32_t es[5] = {1u, 1u, 1u, 1u, 1u};
  CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, const_cast<void*>(q), dims, strides, box, es,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) {
    t_last_cuda = (int)r;
    return LLAMA3_ERR_CUDA;
  }
  return LLAMA3_OK;
}

template <typename K>
int opt_in_smem(K kern, int bytes, bool* done) {
  int dev = 0;
  L3_TRY(current_device(&dev));
  if (!done[dev]) {
    L3_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    done[dev] = true;
  }
  return LLAMA3_OK;
}

template <int HD, bool TREE, bool PAIR>
int run_rows_tc_t(const llama3_config* c, const RowsPlan& p, const void* q, const void* kc, const void* vc, int cap,
                  cudaStream_t st) {
  const RowsShape& rs = p.rs;
  const long long e = 2, keys = (long long)rs.max_len + (TREE ? 0 : rs.T);
  CUtensorMap mq, mk, mv;
  L3_TRY(make_map_rows(&mq, q, c, rs));
  L3_TRY(make_map_4d(&mk, kc, HD, rs.KV, keys, rs.B, HD * e, rs.KV * HD * e, (long long)cap * rs.KV * HD * e));
  L3_TRY(make_map_4d(&mv, vc, HD, rs.KV, keys, rs.B, HD * e, rs.KV * HD * e, (long long)cap * rs.KV * HD * e));
  auto kern = rows_attention_kernel<HD, TREE, PAIR>;
  constexpr int smem = RowsCfg<HD, PAIR>::SMEM_BYTES;
  int dev = 0;
  L3_TRY(current_device(&dev));
  static bool attr_done[kMaxDevices], regs_ok[kMaxDevices];
  if (!attr_done[dev]) {
    L3_CUDA(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
    // the warpgroups' register shares have to fit the block's (see run_flash_attention_t)
    cudaFuncAttributes fa;
    L3_CUDA(cudaFuncGetAttributes(&fa, kern));
    regs_ok[dev] = (long long)fa.numRegs * kFlashThreads >= 128LL * kFlashLowRegs + 256LL * kFlashHighRegs;
    attr_done[dev] = true;
  }
  if (!regs_ok[dev]) return LLAMA3_ERR_UNSUPPORTED;
  L3_LAUNCH(TREE ? LLAMA3_KERNEL_TREE_ATTENTION : LLAMA3_KERNEL_OBSERVED_ATTENTION, st,
            launch_k(kern, rs.G, kFlashThreads, smem, st, mq, mk, mv, rs, wait_ns()));
  return launch_check();
}

template <typename T, int HD, bool TREE>
int run_rows_simt_t(const RowsPlan& p, const void* q, const void* kc, const void* vc, int cap, cudaStream_t st) {
  auto kern = rows_simt_kernel<T, HD, TREE>;
  static bool done[kMaxDevices];
  L3_TRY(opt_in_smem(kern, SimtCfg<HD>::ATT_BYTES, done));
  L3_LAUNCH(TREE ? LLAMA3_KERNEL_TREE_ATTENTION : LLAMA3_KERNEL_OBSERVED_ATTENTION, st,
            launch_k(kern, p.rs.G, 256, SimtCfg<HD>::ATT_BYTES, st, p.rs, (const T*)q, (const T*)kc, (const T*)vc, cap));
  return launch_check();
}

// The main pass over the cache for T = float or bf16.
template <typename T, int HD, bool TREE>
int run_rows_main(const llama3_config* c, const RowsPlan& p, const void* q, const void* kc, const void* vc, int cap,
             cudaStream_t st) {
  if constexpr (std::is_same<T, bf16>::value && HD >= 32) {
    if (p.tc)
      return p.pair ? run_rows_tc_t<HD, TREE, true>(c, p, q, kc, vc, cap, st)
                    : run_rows_tc_t<HD, TREE, false>(c, p, q, kc, vc, cap, st);
  }
  return run_rows_simt_t<T, HD, TREE>(p, q, kc, vc, cap, st);
}

template <typename T, int HD, bool TREE>
int run_rows(const llama3_config* c, const RowsPlan& p, const void* q, const void* kc, const void* vc, int cap,
             cudaStream_t st) {
  L3_TRY((run_rows_main<T, HD, TREE>(c, p, q, kc, vc, cap, st)));
  if (!p.rs.folded) return LLAMA3_OK;
  const int rows = std::min(p.rs.slots * p.rs.tile_rows, std::min(p.rs.T, p.rs.qpt * p.rs.slots) * p.rs.rep);
  L3_LAUNCH(TREE ? LLAMA3_KERNEL_TREE_ATTENTION : LLAMA3_KERNEL_OBSERVED_ATTENTION, st,
            launch_k((fold_pieces_kernel<HD, TREE>), dim3(p.rs.G - 1, rows), 32 * kFoldWarps, 0, st, p.rs));
  return launch_check();
}

struct TreeArgs {
  const void *q, *kc, *vc, *kn, *vn;
  const int32_t *kv_lens, *parents;
  int cap;
  void *out, *ws;
};
template <typename T, int HD>
int run_tree(const llama3_config* c, RowsPlan& p, const TreeArgs& a, cudaStream_t st) {
  RowsShape& rs = p.rs;
  rs.kv_lens = a.kv_lens;
  rs.out = a.out;
  rs.cuts = ws_at<FlatCut>(a.ws, p.cuts);
  rs.part_ml = ws_at<float>(a.ws, p.ml);
  rs.part_o = ws_at<float>(a.ws, p.o);
  if (rs.G > 0) L3_TRY((run_rows<T, HD, true>(c, p, a.q, a.kc, a.vc, a.cap, st)));
  // Query heads of a node per warp: up to four of those that share its KV head,
  // once there are rows enough to fill the GPU with such warps (8B batch, 16384 rows: 18 us
  // against 30 with one; 8B single, 2048 rows: 20 against 13).
  const long long rows = (long long)rs.B * rs.T * rs.H;
  const int nr = rs.rep % 4 == 0 && rows >= 64LL * num_sms() ? 4 : rs.rep % 2 == 0 && rows >= 32LL * num_sms() ? 2 : 1;
  auto join = nr == 4 ? tree_join_kernel<T, HD, 4> : nr == 2 ? tree_join_kernel<T, HD, 2> : tree_join_kernel<T, HD, 1>;
  L3_LAUNCH(LLAMA3_KERNEL_TREE_ATTENTION, st,
            launch_k(join, dim3(rs.B * rs.KV, (rs.T * rs.rep / nr + kJoinWarps - 1) / kJoinWarps), 32 * kJoinWarps, 0,
                     st, rs, (const T*)a.q, (const T*)a.kn, (const T*)a.vn, a.parents));
  return launch_check();
}

struct ObserveArgs {
  const void *q, *kc, *vc;
  const int32_t *kv_lens, *seq_lens, *positions;
  const float* win;
  float* wout;
  int32_t* slot_pos;
  int cap;
  void *out, *ws;
};
template <typename T, int HD>
int run_observe(const llama3_config* c, RowsPlan& p, const ObserveArgs& a, cudaStream_t st) {
  RowsShape& rs = p.rs;
  rs.kv_lens = a.kv_lens;
  rs.seq_lens = a.seq_lens;
  rs.out = a.out;
  rs.cuts = ws_at<FlatCut>(a.ws, p.cuts);
  rs.part_ml = ws_at<float>(a.ws, p.ml);
  rs.part_o = ws_at<float>(a.ws, p.o);
  rs.nlse = ws_at<float>(a.ws, p.nlse);
  rs.scores = p.scored ? ws_at<float>(a.ws, p.scores) : nullptr;
  L3_TRY((run_rows<T, HD, false>(c, p, a.q, a.kc, a.vc, a.cap, st)));
  if (rs.G > 1) {
    L3_LAUNCH(LLAMA3_KERNEL_OBSERVED_ATTENTION, st,
              launch_k((causal_join_kernel<T, HD>), dim3(rs.G - 1, (rs.slots * rs.tile_rows + CausalJoin<HD>::ROWS - 1) / CausalJoin<HD>::ROWS),
                       CausalJoin<HD>::THREADS, 0, st, rs));
    L3_TRY(launch_check());
  }
  WeightShape w;
  memset(&w, 0, sizeof(w));
  w.B = rs.B; w.S = rs.T; w.KV = rs.KV; w.rep = rs.rep; w.qpt = rs.qpt; w.tiles = rs.tiles; w.tile_rows = rs.tile_rows;
  w.key_shift = p.tc ? 8 : 6;
  w.key_tiles = (rs.max_len + rs.T + (1 << w.key_shift) - 1) >> w.key_shift;
  w.max_len = rs.max_len; w.cap = a.cap; w.scale_log2 = rs.scale_log2;
  w.kv_lens = a.kv_lens; w.seq_lens = a.seq_lens; w.positions = a.positions;
  w.nlse = rs.nlse; w.win = a.win; w.wout = a.wout; w.slot_pos = a.slot_pos;
  w.part = ws_at<float>(a.ws, p.sums);
  w.scores = rs.scores;
  w.cuts = rs.cuts;   // the attention's cuts have been joined when the weights' are written
  if (p.scored) {
    L3_LAUNCH(LLAMA3_KERNEL_OBSERVED_ATTENTION, st,
              launch_k(scored_weights_kernel, dim3((rs.max_len + rs.T - 1) / (256 * kScoredSlots) + 1, rs.B * rs.KV), 256, 0, st, w));
    return launch_check();
  }
  const long long most = (long long)w.B * w.key_tiles * w.KV * w.tiles;
  w.G = (int)std::min((long long)num_sms() * (p.tc ? 1 : 2), most);
  bool launched = false;
  if constexpr (std::is_same<T, bf16>::value && HD >= 32) {
    if (p.tc) {
      CUtensorMap mq, mk;
      L3_TRY(make_map_rows(&mq, a.q, c, rs));
      L3_TRY(make_map_4d(&mk, a.kc, HD, rs.KV, (long long)rs.max_len + rs.T, rs.B, HD * 2, rs.KV * HD * 2,
                         (long long)a.cap * rs.KV * HD * 2));
      auto kern = slot_weights_kernel<HD>;
      static bool done[kMaxDevices];
      L3_TRY(opt_in_smem(kern, WeightCfg<HD>::SMEM_BYTES, done));
      L3_LAUNCH(LLAMA3_KERNEL_OBSERVED_ATTENTION, st,
                launch_k(kern, w.G, kWeightThreads, WeightCfg<HD>::SMEM_BYTES, st, mq, mk, w, wait_ns()));
      L3_TRY(launch_check());
      launched = true;
    }
  }
  if (!launched) {
    auto kern = slot_weights_simt_kernel<T, HD>;
    static bool done[kMaxDevices];
    L3_TRY(opt_in_smem(kern, SimtCfg<HD>::WGT_BYTES, done));
    L3_LAUNCH(LLAMA3_KERNEL_OBSERVED_ATTENTION, st,
              launch_k(kern, w.G, 256, SimtCfg<HD>::WGT_BYTES, st, w, (const T*)a.q, (const T*)a.kc, rs.H));
    L3_TRY(launch_check());
  }
  L3_LAUNCH(LLAMA3_KERNEL_OBSERVED_ATTENTION, st,
            launch_k(slot_weights_join_kernel, w.G - 1 + w.B, 256, 0, st, w));
  return launch_check();
}

#define L3_FOR_HEADS(c, CALL)                                          \
  ((c)->dtype == LLAMA3_DTYPE_F32                                      \
       ? ((c)->head_dim == 16   ? CALL(float, 16)                      \
          : (c)->head_dim == 32 ? CALL(float, 32)                      \
          : (c)->head_dim == 64 ? CALL(float, 64)                      \
          : (c)->head_dim == 96 ? CALL(float, 96)                      \
                                : CALL(float, 128))                    \
       : ((c)->head_dim == 16   ? CALL(bf16, 16)                       \
          : (c)->head_dim == 32 ? CALL(bf16, 32)                       \
          : (c)->head_dim == 64 ? CALL(bf16, 64)                       \
          : (c)->head_dim == 96 ? CALL(bf16, 96)                       \
                                : CALL(bf16, 128)))

// Sizes that the kernels' 32-bit indexes hold.
bool rows_in_range(const llama3_config* c, int batch, int rows, long long keys) {
  const long long lim = 1LL << 30;
  return keys < lim && (long long)batch * rows < lim && (long long)batch * rows * c->n_heads < lim &&
         (long long)batch * c->n_kv_heads * ((keys + 63) / 64) < lim &&
         (long long)rows * (c->n_heads / c->n_kv_heads) / kJoinWarps < 65535;
}

int check_tree_shape(const llama3_config* c, int batch, int nodes, int max_len) {
  L3_TRY(check_config(c));
  if (batch < 1 || nodes < 1 || nodes > kMaxTreeNodes || max_len < 0) return LLAMA3_ERR_ARG;
  if (!rows_in_range(c, batch, nodes, max_len)) return LLAMA3_ERR_ARG;
  return rows_supported(c) ? LLAMA3_OK : LLAMA3_ERR_UNSUPPORTED;
}
int check_observe_shape(const llama3_config* c, int batch, int seq, int max_len) {
  L3_TRY(check_config(c));
  if (batch < 1 || seq < 1 || max_len < 0) return LLAMA3_ERR_ARG;
  const long long lim = 1LL << 30, keys = (long long)max_len + seq;
  if (keys >= lim || (long long)batch * seq >= lim || (long long)batch * seq * c->n_heads >= lim ||
      (long long)batch * c->n_kv_heads * ((keys + 63) / 64) >= lim)
    return LLAMA3_ERR_ARG;
  return rows_supported(c) ? LLAMA3_OK : LLAMA3_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

int llama3_tree_workspace_size(const llama3_config* cfg, int batch, int n_nodes, int max_len, size_t* bytes) {
  L3_TRY(check_tree_shape(cfg, batch, n_nodes, max_len));
  if (!bytes) return LLAMA3_ERR_ARG;
  const RowsPlan p = plan_rows(cfg, true, batch, n_nodes, max_len);
  if (!p.fits) return LLAMA3_ERR_UNSUPPORTED;
  *bytes = p.total;
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
  RowsPlan p = plan_rows(cfg, true, batch, n_nodes, max_len);
  if (!p.fits) return LLAMA3_ERR_UNSUPPORTED;
  if (p.total && (!ws || ws_bytes < p.total)) return LLAMA3_ERR_WORKSPACE;
  if (!aligned16(ws)) return LLAMA3_ERR_ALIGN;
  const TreeArgs a = {q, k_cache, v_cache, k_nodes, v_nodes, kv_lens, parents, cache_cap, out, ws};
  cudaStream_t st = (cudaStream_t)stream;
#define L3_TREE(T, HD) run_tree<T, HD>(cfg, p, a, st)
  return L3_FOR_HEADS(cfg, L3_TREE);
#undef L3_TREE
}

int llama3_observe_workspace_size(const llama3_config* cfg, int batch, int seq, int max_len, size_t* bytes) {
  L3_TRY(check_observe_shape(cfg, batch, seq, max_len));
  if (!bytes) return LLAMA3_ERR_ARG;
  const RowsPlan p = plan_rows(cfg, false, batch, seq, max_len);
  if (!p.fits) return LLAMA3_ERR_UNSUPPORTED;
  *bytes = p.total;
  return LLAMA3_OK;
}

int llama3_attention_observed(const llama3_config* cfg, const void* q, const void* k_cache, const void* v_cache,
                              int cache_cap, int batch, int seq, const int32_t* kv_lens, const int32_t* seq_lens,
                              int max_len, void* out, const float* weights_in, float* weights,
                              const int32_t* positions, int32_t* slot_pos, void* ws, size_t ws_bytes,
                              llama3_stream_t stream) {
  L3_TRY(check_observe_shape(cfg, batch, seq, max_len));
  if (!q || !k_cache || !v_cache || !out || !weights) return LLAMA3_ERR_ARG;
  if ((long long)max_len + seq > cache_cap) return LLAMA3_ERR_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) || !aligned4(kv_lens) ||
      !aligned4(seq_lens) || !aligned4(weights_in) || !aligned4(weights) || !aligned4(positions) ||
      !aligned4(slot_pos))
    return LLAMA3_ERR_ALIGN;
  RowsPlan p = plan_rows(cfg, false, batch, seq, max_len);
  if (!p.fits) return LLAMA3_ERR_UNSUPPORTED;
  if (!ws || ws_bytes < p.total) return LLAMA3_ERR_WORKSPACE;
  if (!aligned16(ws)) return LLAMA3_ERR_ALIGN;
  const ObserveArgs a = {q,          k_cache, v_cache,  kv_lens,   seq_lens, positions,
                         weights_in, weights, slot_pos, cache_cap, out,      ws};
  cudaStream_t st = (cudaStream_t)stream;
#define L3_OBSERVE(T, HD) run_observe<T, HD>(cfg, p, a, st)
  return L3_FOR_HEADS(cfg, L3_OBSERVE);
#undef L3_OBSERVE
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
  // the kernels count the rows of one launch, and the 16-byte pieces that stay of one layer's sequence, in 32 bits
  if ((long long)std::min(n_layers, kEvictLayers) * batch * cfg->n_kv_heads > INT_MAX ||
      (long long)std::min(max_len, budget) * cfg->n_kv_heads * (long long)(cfg->head_dim * esize(cfg) / 16) > INT_MAX / 2)
    return LLAMA3_ERR_UNSUPPORTED;
  cudaStream_t st = (cudaStream_t)stream;
  const long long words = evict_row_words(max_len, budget);
  EvictParams p;
  memset(&p, 0, sizeof(p));
  p.kv_lens = kv_lens;
  p.positions = positions;
  p.B = batch; p.KV = cfg->n_kv_heads;
  p.row16.set((uint32_t)(cfg->head_dim * esize(cfg) / 16));
  p.slot16.set(p.row16.d * cfg->n_kv_heads);
  p.cap = src_cap; p.dst_cap = dst ? dst_cap : src_cap;
  p.max_len = max_len; p.budget = budget; p.recent = recent; p.in_place = dst ? 0 : 1;
  p.from_words = evict_kept(max_len, budget);
  p.move_words = evict_moves(max_len, budget);
  p.ws_row = words;
  const bool many = (long long)std::min(n_layers, kEvictLayers) * batch * cfg->n_kv_heads >= 2LL * num_sms() &&
                    max_len <= EvictCfg<true>::THREADS * EvictCfg<true>::OWN;
  const bool stored = max_len <= kEvictKeys;
  // many rows are stored ones: their slots fit the registers of 256 threads
  static_assert(EvictCfg<true>::THREADS * EvictCfg<true>::OWN <= kEvictKeys, "eviction variants");
  auto select = many ? evict_select_kernel<true, true>
                     : stored ? evict_select_kernel<true, false> : evict_select_kernel<false, false>;
  // four slots per thread, up to the kernel's threads
  const int most_threads = many ? EvictCfg<true>::THREADS : EvictCfg<false>::THREADS;
  const int threads = std::max(64, std::min(most_threads, (int)(((long long)max_len / 4 + 31) / 32 * 32)));
  const int smem = stored ? max_len * 4 : 0;
  static bool done[2][kMaxDevices];
  if (stored) L3_TRY(opt_in_smem(select, kEvictKeys * 4, done[many]));
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
    p.lens_out = l0 + nl == n_layers ? kv_lens_out : nullptr;
    L3_LAUNCH(LLAMA3_KERNEL_EVICT, st,
              launch_k(select, rows, threads, smem, st, p));
    L3_TRY(launch_check());
    const long long pieces = (long long)(dst ? p.from_words : p.move_words) * p.slot16.d;
    const int parts = (int)std::max(1LL, std::min((pieces + 255) / 256, 65535LL));
    L3_LAUNCH(LLAMA3_KERNEL_EVICT, st, launch_k(evict_move_kernel, dim3(nl * batch, parts), 256, 0, st, p));
    L3_TRY(launch_check());
  }
  return LLAMA3_OK;
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
    // enough parts for a path of 16 nodes at one piece per thread; longer ones loop
    const int parts = std::min(std::max(1, (int)(std::min(n_nodes, 16) * (long long)p.row16 / 256)), 64);
    L3_LAUNCH(LLAMA3_KERNEL_ACCEPT, st, launch_k(tree_commit_kernel, dim3(batch, nl, parts), 256, 0, st, p));
    L3_TRY(launch_check());
  }
  return LLAMA3_OK;
}

}  // extern "C"
