// cache_ops.cuh -- operators on the rows of the K/V cache for drafted
// (speculative) and bounded decoding; they move rows and decide which, and
// compute nothing on them.
//
//   eviction    the kept slots of a bounded cache, selected by recency and
//               accumulated weight
//   acceptance  the path of a drafted tree that the target's tokens confirm,
//               and the copy of its rows into the caches
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
// Division of n < 2^31 by a fixed d >= 1 (Granlund and Montgomery, "Division by
// invariant integers using multiplication"): l = ceil(log2 d), m = floor(2^32 (2^l - d) / d) + 1.
struct FastDiv {
  uint32_t d, m;
  int s1, s2;
  __host__ void set(uint32_t d_) {
    d = d_;
    int l = 0;
    while (l < 32 && (1ull << l) < d) ++l;
    m = (uint32_t)(((1ull << 32) * ((1ull << l) - d)) / d + 1);
    s1 = l < 1 ? l : 1;
    s2 = l < 1 ? 0 : l - 1;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    const uint32_t t = __umulhi(m, n);
    return (t + ((n - t) >> s1)) >> s2;
  }
};

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
  int32_t *ws, *lens_out;
  FastDiv row16, slot16;   // 16-byte pieces of a slot's row of one KV head, and of all
  int B, KV, cap, dst_cap, max_len, budget, recent, in_place;
  int from_words, move_words;
  long long ws_row;    // words of scratch per row: 4, the sources, the holes and the slots that fill them
};

// Kept slots of a row at most, and moves of one at most.
inline int evict_kept(int max_len, int budget) { return budget < max_len ? budget : max_len; }
inline int evict_moves(int max_len, int budget) {
  const int out = max_len > budget ? max_len - budget : 0;
  return out < budget ? out : budget;
}
inline long long evict_row_words(int max_len, int budget) {
  return 4LL + evict_kept(max_len, budget) + 2LL * evict_moves(max_len, budget);
}

// Order key of a slot: larger is kept first.  Recent slots come before all
// others, a NaN weight before every number; -0 equals +0.
__device__ __forceinline__ uint32_t evict_key(float w, int32_t pos, int32_t floor_pos) {
  if (pos >= floor_pos) return 0xffffffffu;
  if (w != w) return 0xfffffffeu;
  return float_order_key(w == 0.f ? 0.f : w);
}

// Exclusive prefix sums over the block of two counts at once; totals to all.
// s: 2 * 32 ints.  Every thread of the block.
__device__ __forceinline__ void block_scan2(int& x, int& y, int& tx, int& ty, int* s) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int ix = x, iy = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int ux = __shfl_up_sync(0xffffffffu, ix, o), uy = __shfl_up_sync(0xffffffffu, iy, o);
    if (lane >= o) { ix += ux; iy += uy; }
  }
  __syncthreads();
  if (lane == 31) { s[warp] = ix; s[32 + warp] = iy; }
  __syncthreads();
  const int wx = lane < warps ? s[lane] : 0, wy = lane < warps ? s[32 + lane] : 0;
  x = ix - x + __reduce_add_sync(0xffffffffu, lane < warp ? wx : 0);
  y = iy - y + __reduce_add_sync(0xffffffffu, lane < warp ? wy : 0);
  tx = __reduce_add_sync(0xffffffffu, wx);
  ty = __reduce_add_sync(0xffffffffu, wy);
}

// Order keys of a row that a block keeps in shared memory (128 KB); longer rows
// compute them anew at every look, each thread along its own run of slots (16 rows
// of 60000 slots, moves included: 286 us).
constexpr int kEvictKeys = 32768;
// Threads of a block at most, and the keys of each that stay in registers.  Many
// rows: 256 threads of 32 keys, four blocks on an SM (512 rows are then one wave).
// Fewer rows than two per SM, or more slots than that: 1024 threads of 16 keys
// (eviction in place to an eighth, moves included, of one row of 16384 slots: 30 us
// against 49; of 512 of them with 128-wide heads: 314 against 380).
template <bool MANY>
struct EvictCfg {
  static constexpr int THREADS = MANY ? 256 : 1024, OWN = MANY ? 32 : 16, BLOCKS = MANY ? 4 : 1;
};
// Keys that one warp searches alone.
constexpr int kEvictShort = 256;

// One block per (layer, sequence, KV head).  Thread i owns the slots [i * per, (i +
// 1) * per), so ranks by slot are prefix sums over the threads.  The cut -- the
// budget-th largest key -- is found two bits at a time by counting: three
// thresholds per look, counts added up by redux and once through shared memory.
// What bounds it is the number of instructions (all 16 looks by the whole block
// over 8192 keys: 49 us for 512 rows, 37 as it is), so once at most 256 keys are
// left in the interval the search goes on among those, in one warp and without
// barriers.  A look whose
// count is the budget itself ends the search.
template <bool STORED, bool MANY>
__global__ void __launch_bounds__(EvictCfg<MANY>::THREADS, EvictCfg<MANY>::BLOCKS) evict_select_kernel(const __grid_constant__ EvictParams p) {
  constexpr int kEvictOwn = EvictCfg<MANY>::OWN;
  extern __shared__ uint32_t evict_keys[];
  __shared__ int scan[64], counts[2][3][EvictCfg<MANY>::THREADS / 32], short_n;
  __shared__ uint32_t short_keys[kEvictShort], short_cut;
  griddep_wait_and_release();
  const int row = blockIdx.x, g = row % p.KV, b = (row / p.KV) % p.B, layer = row / (p.KV * p.B);
  const int NT = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = NT >> 5;
  const int n = cached_len(p.kv_lens, b, p.max_len), left = min(n, p.budget);
  const size_t base = ((size_t)b * p.KV + g) * p.cap;
  const float* w = p.layer[layer].w + base;
  const int32_t* pos = p.layer[layer].pos + base;
  const int32_t floor_pos = (int32_t)max((long long)p.positions[b] - p.recent, (long long)INT_MIN);
  int32_t* ws = p.ws + (size_t)row * p.ws_row;
  int32_t* from = ws + 4;                  // source of every kept slot
  int32_t* holes = ws + 4 + p.from_words;
  if (n <= p.budget) {
    if (threadIdx.x == 0) ws[0] = 0;
    for (int i = threadIdx.x; i < left; i += NT) from[i] = i;
    return;
  }
  // Counting needs no order: a thread keeps its keys in registers for it.
  uint32_t own[kEvictOwn];
  const bool in_regs = STORED && n <= kEvictOwn * NT;
  if (in_regs) {
#pragma unroll
    for (int u8 = 0; u8 < kEvictOwn; u8 += 16) {       // sixteen slots' loads in flight
      if (u8 * NT >= n) {
#pragma unroll
        for (int u = 0; u < 16; ++u) own[u8 + u] = 0u;
        continue;
      }
      float wv[16];
      int32_t pv[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const int j = threadIdx.x + (u8 + u) * NT;
        wv[u] = j < n ? w[j] : 0.f;
        pv[u] = j < n ? pos[j] : 0;
      }
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const int j = threadIdx.x + (u8 + u) * NT;
        own[u8 + u] = j < n ? evict_key(wv[u], pv[u], floor_pos) : 0u;   // 0 is below every threshold
        if (j < n) evict_keys[j] = own[u8 + u];
      }
    }
    __syncthreads();
  } else if (STORED) {
    for (int j = threadIdx.x; j < n; j += NT) evict_keys[j] = evict_key(w[j], pos[j], floor_pos);
    __syncthreads();
  }
  // an odd stride: 32 threads at the same place of their runs read 32 banks
  const int per = ((n + NT - 1) / NT) | 1;
  const int j0 = min(n, (int)threadIdx.x * per), j1 = min(n, j0 + per);
  auto key_at = [&](int j) { return STORED ? evict_keys[j] : evict_key(w[j], pos[j], floor_pos); };
  const int used = in_regs ? (n + NT - 1) / NT : 0;
  uint32_t cut = 0;              // at_least >= budget keys are >= cut,
  int at_least = n, over = 0;    // over < budget of them lie behind the open interval [cut, cut + 2^open)
  int open = 32;
  bool exact = false;
  for (int look = 0; open > 0 && !exact && at_least - over > kEvictShort; look ^= 1) {
    open -= 2;
    const uint32_t t1 = cut | (1u << open), t2 = cut | (2u << open), t3 = cut | (3u << open);
    int c1 = 0, c2 = 0, c3 = 0;
    if (in_regs) {
#pragma unroll
      for (int u4 = 0; u4 < kEvictOwn; u4 += 4) {
        if (u4 >= used) break;
#pragma unroll
        for (int u = u4; u < u4 + 4; ++u) {
          c1 += own[u] >= t1;
          c2 += own[u] >= t2;
          c3 += own[u] >= t3;
        }
      }
    } else {
      for (int j = j0; j < j1; ++j) {
        const uint32_t k = key_at(j);
        c1 += k >= t1;
        c2 += k >= t2;
        c3 += k >= t3;
      }
    }
    c1 = __reduce_add_sync(0xffffffffu, c1);
    c2 = __reduce_add_sync(0xffffffffu, c2);
    c3 = __reduce_add_sync(0xffffffffu, c3);
    if (lane == 0) { counts[look][0][warp] = c1; counts[look][1][warp] = c2; counts[look][2][warp] = c3; }
    __syncthreads();     // the next look but one writes here again, behind the next look's barrier
    c1 = __reduce_add_sync(0xffffffffu, lane < warps ? counts[look][0][lane] : 0);
    c2 = __reduce_add_sync(0xffffffffu, lane < warps ? counts[look][1][lane] : 0);
    c3 = __reduce_add_sync(0xffffffffu, lane < warps ? counts[look][2][lane] : 0);
    if (c3 >= p.budget) { cut = t3; at_least = c3; }
    else if (c2 >= p.budget) { cut = t2; at_least = c2; over = c3; }
    else if (c1 >= p.budget) { cut = t1; at_least = c1; over = c2; }
    else over = c1;
    exact = at_least == p.budget;
  }
  if (open > 0 && !exact) {
    // few keys are left in the interval: one warp goes through them, without barriers
    if (threadIdx.x == 0) short_n = 0;
    __syncthreads();
    const uint32_t span = open < 32 ? (1u << open) - 1u : 0xffffffffu;
    if (in_regs) {
#pragma unroll
      for (int u = 0; u < kEvictOwn; ++u)
        if (threadIdx.x + u * NT < n && own[u] - cut <= span) short_keys[atomicAdd(&short_n, 1)] = own[u];
    } else {
      for (int j = j0; j < j1; ++j) {
        const uint32_t k = key_at(j);
        if (k - cut <= span) short_keys[atomicAdd(&short_n, 1)] = k;
      }
    }
    __syncthreads();
    if (warp == 0) {
      const int m = short_n, need = p.budget - over;
      uint32_t mine[kEvictShort / 32];
#pragma unroll
      for (int i = 0; i < kEvictShort / 32; ++i) mine[i] = lane + 32 * i < m ? short_keys[lane + 32 * i] : 0u;
      while (open > 0) {
        open -= 2;
        const uint32_t t1 = cut | (1u << open), t2 = cut | (2u << open), t3 = cut | (3u << open);
        int c1 = 0, c2 = 0, c3 = 0;
#pragma unroll
        for (int i = 0; i < kEvictShort / 32; ++i) {
          c1 += mine[i] >= t1;
          c2 += mine[i] >= t2;
          c3 += mine[i] >= t3;
        }
        c1 = __reduce_add_sync(0xffffffffu, c1);
        c2 = __reduce_add_sync(0xffffffffu, c2);
        c3 = __reduce_add_sync(0xffffffffu, c3);
        int got = 0;
        if (c3 >= need) { cut = t3; got = c3; }
        else if (c2 >= need) { cut = t2; got = c2; }
        else if (c1 >= need) { cut = t1; got = c1; }
        if (got == need) break;
      }
      if (lane == 0) short_cut = cut;
    }
    __syncthreads();
    cut = short_cut;
  }
  // Of the slots at the cut the lowest are kept, as many as the budget leaves.
  int above = 0, equal = 0, all_above, all_equal;
  for (int j = j0; j < j1; ++j) {
    const uint32_t k = key_at(j);
    above += k > cut;
    equal += k == cut;
  }
  const int my_equal = equal;
  block_scan2(above, equal, all_above, all_equal, scan);
  const int room = p.budget - all_above;       // for keys equal to the cut
  const int taken = min(max(room - equal, 0), my_equal);
  // The kept ones of up to 32 slots from j on, as bits; eq: how many at the cut are still to be kept.
  auto kept_bits = [&](int j, int cnt, int& eq) {
    uint32_t m = 0;
    for (int i = 0; i < cnt; ++i) {
      const uint32_t k = key_at(j + i);
      bool keep = k > cut;
      if (k == cut && eq > 0) { --eq; keep = true; }
      m |= (uint32_t)keep << i;
    }
    return m;
  };
  auto low_bits = [](int cnt) { return cnt <= 0 ? 0u : cnt >= 32 ? 0xffffffffu : (1u << cnt) - 1u; };
  // the evicted slots below the budget and the kept ones behind it
  int n_holes = 0, n_spare = 0, all_holes, all_spare;
  uint32_t bits[2] = {0, 0};       // of the first 64 slots; longer runs look at their keys again
  for (int j = j0, eq = taken; j < j1; j += 32) {
    const int cnt = min(32, j1 - j);
    const uint32_t m = kept_bits(j, cnt, eq), front = low_bits(min(cnt, p.budget - j));
    n_holes += __popc(~m & front);
    n_spare += __popc(m & ~front);
    if (j == j0) bits[0] = m;
    if (j == j0 + 32) bits[1] = m;
  }
  block_scan2(n_holes, n_spare, all_holes, all_spare, scan);
  int32_t* spare = holes + p.move_words;
  for (int j = j0, eq = taken; j < j1; j += 32) {
    const int cnt = min(32, j1 - j);
    const uint32_t front = low_bits(min(cnt, p.budget - j));
    const uint32_t m = per > 64 ? kept_bits(j, cnt, eq) : j == j0 ? bits[0] : bits[1];
    for (uint32_t x = m & front; x; x &= x - 1) from[j + __ffs(x) - 1] = j + __ffs(x) - 1;
    for (uint32_t x = ~m & front; x; x &= x - 1) holes[n_holes++] = j + __ffs(x) - 1;
    for (uint32_t x = m & ~front; x; x &= x - 1) spare[n_spare++] = j + __ffs(x) - 1;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < all_holes; i += NT) from[holes[i]] = spare[i];
  if (threadIdx.x == 0) ws[0] = all_holes;
}

// Copies the kept slots: blockIdx.x = (layer, sequence), blockIdx.y = part of its
// slots.  The KV heads' pieces of one slot lie side by side, so a block takes all
// heads of its slots and the stores are contiguous although every head keeps other
// slots.  One 16-byte piece of K and of V per thread and eight blocks on an SM: a
// copy wants loads in flight, and threads that wait for the look-up of their
// piece's source stand in each other's way the less, the more there are (8B
// prompts, 537 MB moved: 145 us with four pieces of each per thread, 120 with two,
// 109 with one, 145 with one of K or of V).  The last launch of a call also writes
// the lengths: kv_lens_out may be kv_lens, whose shortened values give every
// block here the same `left`.
__global__ void __launch_bounds__(256, 8) evict_move_kernel(const __grid_constant__ EvictParams p) {
  griddep_wait_and_release();
  const int b = blockIdx.x % p.B, layer = blockIdx.x / p.B;
  const EvictLayer& L = p.layer[layer];
  const int left = min(cached_len(p.kv_lens, b, p.max_len), p.budget);
  if (p.lens_out && layer == 0 && blockIdx.y + threadIdx.x == 0) p.lens_out[b] = left;
  const int32_t* ws0 = p.ws + (size_t)blockIdx.x * p.KV * p.ws_row;
  // In place each head has its own number of moves, at most move_words: a bound
  // from the lengths would change under the blocks once they are shortened.
  const int most = p.in_place ? min(p.move_words, left) : left;
  const uint32_t slot16 = p.slot16.d, total = (uint32_t)most * slot16, step = 256 * gridDim.y;
  for (uint32_t i = blockIdx.y * 256 + threadIdx.x; i < total; i += step) {
    const uint32_t m = p.slot16.div(i), c = i - m * slot16, g = p.row16.div(c);
    const int32_t* ws = ws0 + g * p.ws_row;
    int to = m;
    if (p.in_place) {
      if ((int)m >= __ldg(ws)) continue;
      to = __ldg(ws + 4 + p.from_words + m);
    }
    const int fr = __ldg(ws + 4 + to);
    const size_t s = ((size_t)b * p.cap + fr) * slot16 + c, d = ((size_t)b * p.dst_cap + to) * slot16 + c;
    const uint4 k = __ldcs(L.k + s), v = __ldcs(L.v + s);
    __stcs(L.dk + d, k);
    __stcs(L.dv + d, v);
    if (c == g * p.row16.d) {
      const size_t head = (size_t)b * p.KV + g;
      L.dw[head * p.dst_cap + to] = L.w[head * p.cap + fr];
      L.dpos[head * p.dst_cap + to] = L.pos[head * p.cap + fr];
    }
  }
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
// blockIdx.x = sequence, blockIdx.y = layer, blockIdx.z = part of the path's rows:
// one 16-byte piece of K and of V per thread, so that a path costs one round
// trip however long it is (8B, 32 layers of 8 drafts: 5.3 us, with one block per
// path 9.1).
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
  const int row = blockIdx.z * 256 + threadIdx.x, step = 256 * gridDim.z;
  for (long long i = row; i < (long long)n * p.row16; i += step) {
    const int m = (int)(i / p.row16), c = (int)(i - (long long)m * p.row16), from = path[m];
    if (from < 0 || from >= p.nodes) {
      record_error(LLAMA3_ERR_ARG);
      continue;
    }
    const size_t s = ((size_t)b * p.nodes + from) * p.row16 + c, d = ((size_t)b * p.cap + base + m) * p.row16 + c;
    const uint4 k = L.kn[s], v = L.vn[s];
    L.k[d] = k;
    L.v[d] = v;
  }
  if (!L.w && !L.pos) return;
  for (int i = row; i < n * p.KV; i += step) {
    const size_t at = ((size_t)b * p.KV + i / n) * p.cap + base + i % n;
    if (L.w) L.w[at] = 0.f;
    if (L.pos) L.pos[at] = (p.positions ? p.positions[b] - n : base) + i % n;
  }
}

}  // namespace l3
