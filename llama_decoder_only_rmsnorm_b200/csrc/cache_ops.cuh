// cache_ops.cuh -- operators around the K/V cache for drafted (speculative)
// and bounded decoding, in their plain CUDA-core form: any head size, fp32 and
// bf16.  Sums, softmax statistics and accumulated weights are fp32.
//
//   tree attention      node t of a drafted tree sees the cached rows
//                       0..kv_len-1, its ancestors in the tree and itself
//   observed attention  causal attention that also adds up, per cache slot and
//                       KV head, the softmax weight the slot received
//   eviction            the kept slots of a bounded cache, selected by
//                       recency and accumulated weight
//   acceptance          the path of the tree that the target's tokens confirm,
//                       and the copy of its rows into the caches
#pragma once
#include <limits.h>

#include "common.cuh"

namespace l3 {

constexpr int kMaxTreeNodes = 256;

// Cached length of a sequence: lens[b] (or max_len where lens is NULL), clamped into
// [0, max_len]; a length outside is reported through the status word.
__device__ __forceinline__ int cached_len(const int32_t* lens, int b, int max_len) {
  if (!lens) return max_len;
  const int n = lens[b];
  if (n < 0 || n > max_len) record_error(LLAMA3_ERR_ARG);
  return max(0, min(n, max_len));
}

// ---- eviction ---------------------------------------------------------------
struct EvictLayer {
  const uint4 *k, *v;
  const float* w;
  const int32_t* pos;
  uint4 *dk, *dv;
  float* dw;
  int32_t* dpos;
};
constexpr int kEvictLayers = 32;   // layers of one launch (the structs travel as a kernel parameter)
struct EvictParams {
  EvictLayer layer[kEvictLayers];
  const int32_t *kv_lens, *positions;
  int32_t* ws;
  int B, KV, row16, cap, dst_cap, max_len, budget, recent, in_place;
  long long ws_row;    // words of scratch per row (evict_row_words)
};

// Words of scratch per (layer, sequence, KV head): the number of moves, the
// holes below the budget, and where each kept slot comes from.
__host__ __device__ inline long long evict_row_words(int max_len, int budget) {
  const long long moves = budget < max_len - budget ? budget : (max_len > budget ? max_len - budget : 0);
  return 4 + moves + budget;
}

// Order key of a slot: larger is kept first.  Recent slots come before all
// others, a NaN weight before every number; -0 equals +0.
__device__ __forceinline__ uint32_t evict_key(float w, int32_t pos, long long floor_pos) {
  if (pos >= floor_pos) return 0xffffffffu;
  if (w != w) return 0xfffffffeu;
  return float_order_key(w == 0.f ? 0.f : w);
}

// Exclusive prefix sum over a block of 1024 threads of a 0/1 flag; total to all.
__device__ __forceinline__ int block_rank(bool f, int* warp_tot, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t m = __ballot_sync(0xffffffffu, f);
  __syncthreads();
  if (lane == 0) warp_tot[warp] = __popc(m);
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < 32; ++i) {
    const int c = warp_tot[i];
    before += i < warp ? c : 0;
    all += c;
  }
  total = all;
  return before + __popc(m & ((1u << lane) - 1u));
}

constexpr int kEvictThreads = 1024;

// One block per (layer, sequence, KV head): the budget-th largest key by four
// passes of an 8-bit radix select, then the kept slots in order.
__global__ void __launch_bounds__(kEvictThreads) evict_select_kernel(const __grid_constant__ EvictParams p) {
  griddep_wait_and_release();
  __shared__ int hist[256], warp_tot[32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int row = blockIdx.x, g = row % p.KV, b = (row / p.KV) % p.B, layer = row / (p.KV * p.B);
  const int n = cached_len(p.kv_lens, b, p.max_len), left = min(n, p.budget);
  const size_t base = ((size_t)b * p.KV + g) * p.cap;
  const float* w = p.layer[layer].w + base;
  const int32_t* pos = p.layer[layer].pos + base;
  const long long floor_pos = (long long)p.positions[b] - p.recent;
  int32_t* ws = p.ws + (size_t)row * p.ws_row;
  int32_t* from = ws + 4;                  // source of every kept slot
  int32_t* holes = ws + 4 + p.budget;
  if (n <= p.budget) {
    if (threadIdx.x == 0) ws[0] = 0;
    for (int i = threadIdx.x; i < left; i += kEvictThreads) from[i] = i;
    return;
  }
  if (threadIdx.x == 0) { s_prefix = 0; s_need = p.budget; }
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (threadIdx.x < 256) hist[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix, mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
    for (int j = threadIdx.x; j < n; j += kEvictThreads) {
      const uint32_t key = evict_key(w[j], pos[j], floor_pos);
      if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & 255], 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int need = s_need, d = 255;
      while (d > 0 && hist[d] < need) need -= hist[d--];
      s_prefix = prefix | ((uint32_t)d << shift);
      s_need = need;
    }
    __syncthreads();
  }
  const uint32_t cut = s_prefix;
  const int ties = s_need;     // slots at the cut that are kept: the lowest ones
  int seen_ties = 0, n_holes = 0, n_fill = 0;
  for (int j0 = 0; j0 < n; j0 += kEvictThreads) {
    const int j = j0 + threadIdx.x;
    const bool in = j < n;
    const uint32_t key = in ? evict_key(w[j], pos[j], floor_pos) : 0u;
    int tot;
    const int rank = seen_ties + block_rank(in && key == cut, warp_tot, tot);
    seen_ties += tot;
    const bool keep = in && (key > cut || (key == cut && rank < ties));
    const bool hole = in && j < p.budget && !keep, fill = keep && j >= p.budget;
    const int hr = n_holes + block_rank(hole, warp_tot, tot);
    n_holes += tot;
    const int fr = n_fill + block_rank(fill, warp_tot, tot);
    n_fill += tot;
    if (in && j < p.budget && keep) from[j] = j;
    if (hole) holes[hr] = j;
    __syncthreads();          // the r-th kept slot behind the budget fills the r-th hole
    if (fill) from[holes[fr]] = j;
  }
  if (threadIdx.x == 0) ws[0] = n_holes;
}

// Copies the kept slots: blockIdx.x = row, blockIdx.y = part of the row's slots.
__global__ void __launch_bounds__(256) evict_move_kernel(const __grid_constant__ EvictParams p) {
  griddep_wait_and_release();
  const int row = blockIdx.x, g = row % p.KV, b = (row / p.KV) % p.B, layer = row / (p.KV * p.B);
  const EvictLayer& L = p.layer[layer];
  const int left = min(cached_len(p.kv_lens, b, p.max_len), p.budget);
  const int32_t* ws = p.ws + (size_t)row * p.ws_row;
  const int32_t* from = ws + 4;
  const int32_t* holes = ws + 4 + p.budget;
  const int moves = p.in_place ? ws[0] : left;
  const size_t sbase = ((size_t)b * p.KV + g) * p.cap, dbase = ((size_t)b * p.KV + g) * p.dst_cap;
  for (long long i = (long long)blockIdx.y * 256 + threadIdx.x; i < (long long)moves * p.row16; i += 256LL * gridDim.y) {
    const int m = (int)(i / p.row16), c = (int)(i % p.row16);
    const int to = p.in_place ? holes[m] : m, fr = from[to];
    const size_t s = (((size_t)b * p.cap + fr) * p.KV + g) * p.row16 + c;
    const size_t d = (((size_t)b * p.dst_cap + to) * p.KV + g) * p.row16 + c;
    L.dk[d] = L.k[s];
    L.dv[d] = L.v[s];
    if (c == 0) {
      L.dw[dbase + to] = L.w[sbase + fr];
      L.dpos[dbase + to] = L.pos[sbase + fr];
    }
  }
}

__global__ void evict_lens_kernel(const int32_t* kv_lens, int32_t* lens_out, int B, int max_len, int budget) {
  griddep_wait_and_release();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b < B) lens_out[b] = min(cached_len(kv_lens, b, max_len), budget);
}

// ---- acceptance -------------------------------------------------------------
// One block per sequence: the lowest child of every node whose drafted token is
// the node's target token, for all nodes at once, then the walk from node 0.
__global__ void __launch_bounds__(kMaxTreeNodes) tree_accept_kernel(
    const int32_t* __restrict__ draft, const int32_t* __restrict__ target, const int32_t* __restrict__ parents,
    int nodes, const int32_t* kv_lens, int32_t* __restrict__ path, int32_t* __restrict__ accepted,
    int32_t* __restrict__ next_ids, int32_t* lens_out, const int32_t* positions, int32_t* positions_out) {
  griddep_wait_and_release();
  __shared__ int32_t next[kMaxTreeNodes];
  const int b = blockIdx.x, t = threadIdx.x;
  const size_t at = (size_t)b * nodes;
  next[t] = INT_MAX;
  __syncthreads();
  if (t < nodes) {
    const int p = parents[at + t];
    if (p >= t) {
      record_error(LLAMA3_ERR_ARG);
    } else if (p >= 0 && draft[at + t] == target[at + p]) {
      atomicMin(&next[p], t);
    }
    path[at + t] = -1;
  }
  __syncthreads();
  if (t == 0) {
    int n = 0, last = -1;
    for (int c = parents[at] == -1 ? 0 : INT_MAX; c != INT_MAX; c = next[c]) {
      path[at + n++] = c;
      last = c;
    }
    accepted[b] = n;
    next_ids[b] = last < 0 ? -1 : target[at + last];
    lens_out[b] = kv_lens[b] + n;
    if (positions_out) positions_out[b] = positions[b] + n;
  }
}

struct CommitLayer {
  const uint4 *kn, *vn;
  uint4 *k, *v;
  float* w;
  int32_t* pos;
};
struct CommitParams {
  CommitLayer layer[64];
  const int32_t *path, *accepted, *kv_lens, *positions;
  int nodes, KV, row16, cap;   // row16: 16-byte pieces of one token's row (all KV heads)
};
// blockIdx.x = sequence, blockIdx.y = layer.
__global__ void __launch_bounds__(256) tree_commit_kernel(const __grid_constant__ CommitParams p) {
  griddep_wait_and_release();
  const int b = blockIdx.x;
  const CommitLayer& L = p.layer[blockIdx.y];
  const int n = p.accepted[b], base = p.kv_lens[b] - n;
  const int32_t* path = p.path + (size_t)b * p.nodes;
  if (n < 0 || n > p.nodes || base < 0 || base > p.cap - n) {
    if (threadIdx.x == 0) record_error(LLAMA3_ERR_ARG);
    return;
  }
  for (int i = threadIdx.x; i < n * p.row16; i += 256) {
    const int m = i / p.row16, c = i % p.row16, from = path[m];
    if (from < 0 || from >= p.nodes) {
      record_error(LLAMA3_ERR_ARG);
      continue;
    }
    const size_t s = ((size_t)b * p.nodes + from) * p.row16 + c, d = ((size_t)b * p.cap + base + m) * p.row16 + c;
    L.k[d] = L.kn[s];
    L.v[d] = L.vn[s];
  }
  for (int i = threadIdx.x; i < n * p.KV; i += 256) {
    const size_t at = ((size_t)b * p.KV + i / n) * p.cap + base + i % n;
    if (L.w) L.w[at] = 0.f;
    if (L.pos) L.pos[at] = (p.positions ? p.positions[b] - n : base) + i % n;
  }
}

}  // namespace l3
