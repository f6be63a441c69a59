// slot_weights.cuh -- the softmax weight that every cache slot received, once
// the rows' log-sum-exp is known (observed attention, second pass):
//   sum[b, g, j] = sum over rows (t, head) of 2^(s[t, head, j] log2(e)/sqrt(hd) - lse2[t, head]).
//
// On tcgen05 the product is taken the other way round than in the attention:
// S^T = K Q^T with the 128 keys of a tile on the accumulator's lanes and 128
// packed rows (position x head, as in rows_attention.cuh) on its columns.  A
// thread owns one slot and adds up its columns in registers: no shuffle, no
// atomic, one order for every run.  A segment is two key tiles, and two threads
// per slot share its columns; the keys stay in shared memory while the query
// tiles stream past, each read once for both tiles (one key tile per query tile
// asks the L2 for 64 bytes per cycle and SM: 421 us on the 8B prompt of 8192).
// Of the exponentials, 16 per cycle and SM, a quarter goes to the FMA pipe by the
// fine polynomial, since the sums are fp32 results (8B prompt: 327 us; with an
// eighth 340, three eighths 349, none 380).  No pipe is full: under the profiler
// the exponentials' one is busy 57 % of the cycles, the tensor core 36 %, and 59 %
// issue an instruction.  A thread waits for all of its 64 columns before the first
// exponential, and 640 threads of 96 registers leave no room to hold two loads (24
// bytes of the plan spill as it is).
//
// A few rows over a long cache (a decode step) leave their scores in the
// workspace instead, and scored_weights_kernel below adds them up: K is then
// not read a second time.
#pragma once
#include "rows_attention.cuh"

namespace l3 {

struct WeightShape {
  int B, S, KV, rep, qpt, tiles, tile_rows;
  int key_tiles, key_shift;   // segments per (sequence, KV head), log2 of their slots (8 or 6)
  int G, max_len, cap;
  float scale_log2;
  const int32_t *kv_lens, *seq_lens, *positions;
  const float *nlse, *scores;
  const float* win;
  float* wout;
  int32_t* slot_pos;
  FlatCut* cuts;        // [G]
  float* part;          // [2 G][slots of a segment]: sums of cut segments
};

// Query tiles that see key tile i % key_tiles of sequence i / key_tiles.
struct WeightTiles {
  const WeightShape& ws;
  __device__ __forceinline__ int first(int i) const {
    const int b = i / ws.key_tiles, key0 = (i % ws.key_tiles) << ws.key_shift;
    return max(0, key0 - cached_len(ws.kv_lens, b, ws.max_len)) / ws.qpt;
  }
  __device__ __forceinline__ int operator()(int i) const {
    const int b = i / ws.key_tiles, key0 = (i % ws.key_tiles) << ws.key_shift;
    const int len = cached_len(ws.kv_lens, b, ws.max_len), live = cached_len(ws.seq_lens, b, ws.S);
    if (live == 0 || key0 >= len + live) return 0;
    return (live + ws.qpt - 1) / ws.qpt - max(0, key0 - len) / ws.qpt;
  }
  __device__ __forceinline__ int items() const { return ws.B * ws.key_tiles; }
  __device__ __forceinline__ int record(const FlatSeg& s, int c, int a) const {
    return 2 * c + (s.s0 < a ? 0 : 1);
  }
};

// The finished sum of slot `key`: into the weights, with the slot's position if it is new.
__device__ __forceinline__ void put_weight(const WeightShape& ws, int b, int g, int key, int len, int live, float sum) {
  if (key >= len + live) return;
  const size_t at = ((size_t)b * ws.KV + g) * ws.cap + key;
  ws.wout[at] = (ws.win && key < len ? ws.win[at] : 0.f) + sum;
  if (ws.slot_pos && key >= len) ws.slot_pos[at] = (ws.positions ? ws.positions[b] : len) + key - len;
}

template <int HD>
struct WeightCfg {
  static constexpr int CHUNKS = (HD + 63) / 64;
  static constexpr int TILE = 128 * 128;
  static constexpr int K_BYTES = CHUNKS * TILE;
  static constexpr int KRING = 3;                        // a segment's two key tiles and the next one's first
  static constexpr int Q_STAGE = CHUNKS * TILE + 1024;   // 128 rows of q and their 128 log-sum-exps
  static constexpr int RING0 = (232448 - 1024 - 4096 - 1024 - KRING * K_BYTES) / Q_STAGE;
  static constexpr int RING = RING0 > 6 ? 6 : RING0;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_Q = KRING * K_BYTES;
  static constexpr int OFF_SUM = OFF_Q + RING * Q_STAGE;   // [2][key tile][128] sums of the right columns
  static constexpr int OFF_BOX = OFF_SUM + 2048;           // the summing warps' plans, 128 bytes each
  static constexpr int OFF_BAR = OFF_BOX + 16 * 128;
  static constexpr int N_BARS = 2 * KRING + 2 * RING + 8 + 2;
  static constexpr int SMEM_BYTES = 1024 + OFF_BAR + N_BARS * 8 + 16;
  static_assert(SMEM_BYTES <= 232448 && RING >= 3, "shared memory");
};

// 32 columns of a slot's scores: p = 2^(s scl + nlse[c]) where lo <= c < hi, added to sum.
template <bool MASKED>
__device__ __forceinline__ void weight_add(uint32_t (&r)[32], const float* nlse, int c0, int lo, int hi, float scl,
                                           float& sa, float& sb) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 n = *reinterpret_cast<const float4*>(nlse + c0 + 4 * i);
    float x[4], p[4];
    fma2(x[0], x[1], __uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]), scl, scl, n.x, n.y);
    fma2(x[2], x[3], __uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]), scl, scl, n.z, n.w);
    p[0] = ex2_approx(x[0]);
    p[1] = ex2_approx(x[1]);
    if (!MASKED && i % 2 == 0) {
      // a quarter of the exponentials
      exp2_poly2_huge(x[2], x[3], p[2], p[3]);
    } else {
      p[2] = ex2_approx(x[2]);
      p[3] = ex2_approx(x[3]);
    }
    if (MASKED) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = c0 + 4 * i + k;
        if (c < lo || c >= hi) p[k] = 0.f;
      }
    }
    add2(sa, sb, p[0], p[1]);
    add2(sa, sb, p[2], p[3]);
  }
}

constexpr int kWeightThreads = 128 + 512;
template <int HD>
__global__ void __launch_bounds__(kWeightThreads, 1)
    slot_weights_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                        const __grid_constant__ WeightShape ws, const unsigned long long wait_ns) {
  using C = WeightCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* k_empty = k_full + C::KRING;
  uint64_t* q_full = k_empty + C::KRING;
  uint64_t* q_empty = q_full + C::RING;
  uint64_t* s_full = q_empty + C::RING;    // [key tile][2]
  uint64_t* s_empty = s_full + 4;
  uint64_t* meet = s_empty + 4;            // [key tile]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(meet + 2);
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::KRING; ++i) { mbar_init(&k_full[i], 1); mbar_init(&k_empty[i], 1); }
    for (int i = 0; i < C::RING; ++i) { mbar_init(&q_full[i], 1); mbar_init(&q_empty[i], 1 + 16); }
    for (int i = 0; i < 4; ++i) { mbar_init(&s_full[i], 1); mbar_init(&s_empty[i], 8); }
    for (int i = 0; i < 2; ++i) mbar_init(&meet[i], 256);
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) { prefetch_tensormap(&mapQ); prefetch_tensormap(&mapK); }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  griddep_wait_and_release();
  const WeightTiles tiles_of{ws};
  FlatRun<WeightTiles> run;
  FlatSeg seg;
  int w0, w1;
  if (warp == 0) {
    // ---------------------------------------------------------------- producer
    run.start(tiles_of.items(), ws.KV, tiles_of, blockIdx.x, gridDim.x);
    if (lane == 0) {
      run.leave(ws.cuts, blockIdx.x);
      int st = 0, ks = 0;
      uint32_t ph = 0, kph = 0, iss = 0, par = 0, kiss = 0, kpar = 0;
      bool ok = true;
      const uint32_t bytes = (uint32_t)(ws.rep * ws.qpt * 128 * C::CHUNKS + 512);
      while (ok && run.next(tiles_of, seg, w0, w1)) {
        const int b = seg.item / ws.key_tiles, key0 = (seg.item % ws.key_tiles) * 256, g = seg.sub;
        const int rt0 = tiles_of.first(seg.item);
        for (int h = 0; h < 2 && ok; ++h) {
          if (!mbar_wait(&k_empty[ks], kph ^ 1u, wait_ns)) { ok = false; break; }
          mbar_arrive_expect_tx(&k_full[ks], C::K_BYTES);
          for (int c = 0; c < C::CHUNKS; ++c)
            tma_load_4d(smem + C::OFF_K + ks * C::K_BYTES + c * C::TILE, &mapK, &k_full[ks], c * 64, g,
                        key0 + h * 128, b);
          kiss |= 1u << ks; kpar = (kpar & ~(1u << ks)) | (kph << ks);
          if (++ks == C::KRING) { ks = 0; kph ^= 1u; }
        }
        for (int w = w0; w < w1 && ok; ++w) {
          if (!mbar_wait(&q_empty[st], ph ^ 1u, wait_ns)) { ok = false; break; }
          uint8_t* q = smem + C::OFF_Q + st * C::Q_STAGE;
          mbar_arrive_expect_tx(&q_full[st], bytes);
          for (int c = 0; c < C::CHUNKS; ++c)
            tma_load_5d(q + c * C::TILE, &mapQ, &q_full[st], c * 64, 0, g, (rt0 + w) * ws.qpt, b);
          bulk_load(q + C::CHUNKS * C::TILE, ws.nlse + ((size_t)(b * ws.KV + g) * ws.tiles + rt0 + w) * 128,
                    &q_full[st], 512);
          iss |= 1u << st; par = (par & ~(1u << st)) | (ph << st);
          if (++st == C::RING) { st = 0; ph ^= 1u; }
        }
      }
      for (int s = 0; s < C::KRING; ++s)
        if (kiss & (1u << s)) mbar_wait(&k_full[s], (kpar >> s) & 1u, wait_ns);
      for (int s = 0; s < C::RING; ++s)
        if (iss & (1u << s)) mbar_wait(&q_full[s], (par >> s) & 1u, wait_ns);
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    constexpr uint32_t IDESC = idesc_bf16_f32(128, 128, 0, 0);
    run.start(tiles_of.items(), ws.KV, tiles_of, blockIdx.x, gridDim.x);
    const bool leader = elect_one_sync();
    int st = 0, ks = 0;
    uint32_t ph = 0, kph = 0, i = 0;   // i: query tiles so far; buffer i & 1 of each warpgroup
    bool ok = true;
    while (ok && run.next_uniform(tiles_of, seg, w0, w1)) {
      int kst[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!mbar_wait_warp(&k_full[ks], kph, wait_ns)) ok = false;
        kst[h] = ks;
        if (++ks == C::KRING) { ks = 0; kph ^= 1u; }
      }
      for (int w = w0; w < w1 && ok; ++w, ++i) {
        if (!mbar_wait_warp(&q_full[st], ph, wait_ns)) { ok = false; break; }
        const uint32_t qa = smem_u32(smem + C::OFF_Q + st * C::Q_STAGE);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int buf = h * 2 + (i & 1);
          if (!mbar_wait_warp(&s_empty[buf], ((i >> 1) & 1u) ^ 1u, wait_ns)) { ok = false; break; }
          tc_fence_after();
          const uint32_t ka = smem_u32(smem + C::OFF_K + kst[h] * C::K_BYTES);
          if (leader) {
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) {
              const uint32_t off = (k >> 2) * C::TILE + (k & 3) * 32;
              tc_mma_f16_ss(tmem_base + buf * 128, sw128_desc(ka + off, 1024, 16), sw128_desc(qa + off, 1024, 16),
                            IDESC, k > 0);
            }
            tc_commit(&s_full[buf]);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (leader) tc_commit(&q_empty[st]);
        __syncwarp();
        if (++st == C::RING) { st = 0; ph ^= 1u; }
      }
      if (!ok) break;
      if (leader) {
        tc_commit(&k_empty[kst[0]]);
        tc_commit(&k_empty[kst[1]]);
      }
      __syncwarp();
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- sums (two threads per slot)
    const int kt = (warp - 4) >> 3, half = ((warp - 4) >> 2) & 1;   // key tile, half of the columns
    const int quarter = warp & 3, row = quarter * 32 + lane;
    const uint32_t s_base = tmem_base + ((uint32_t)(quarter * 32) << 16) + kt * 256 + half * 64;
    float* right = reinterpret_cast<float*>(smem + C::OFF_SUM) + kt * 128 + row;
    typedef FlatBox<WeightTiles> Box;
    static_assert(sizeof(Box) <= 128, "plan");
    Box* box = reinterpret_cast<Box*>(smem + C::OFF_BOX + (warp - 4) * 128);
    box->start(tiles_of.items(), ws.KV, tiles_of, blockIdx.x, gridDim.x);
    int st = 0;
    uint32_t i = 0, ph = 0, pieces = 0;
    bool ok = true;
    while (ok && box->next(tiles_of)) {
      // what the tile loop needs: the first tile's position, and from there what each key sees
      int b = box->seg.item / ws.key_tiles;
      const int key0 = (box->seg.item % ws.key_tiles) * 256 + kt * 128;
      const int len = cached_len(ws.kv_lens, b, ws.max_len), live = cached_len(ws.seq_lens, b, ws.S);
      int left = warp_uniform(box->w1 - box->w0), t0 = (tiles_of.first(box->seg.item) + box->w0) * ws.qpt;
      float sum = 0.f;
      for (; left > 0; --left, ++i, t0 += ws.qpt) {
        const int buf = kt * 2 + (i & 1);
        if (!mbar_wait_warp(&q_full[st], ph, wait_ns) || !mbar_wait_warp(&s_full[buf], (i >> 1) & 1u, wait_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        uint32_t ra[32], rb[32];
        tmem_ld32(s_base + (i & 1) * 128, ra);
        tmem_ld32(s_base + (i & 1) * 128 + 32, rb);
        tc_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[buf]);
        const float* nlse = reinterpret_cast<const float*>(smem + C::OFF_Q + st * C::Q_STAGE + C::CHUNKS * C::TILE);
        float a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
        const int hi = min(ws.qpt, live - t0) * ws.rep;
        if (hi < 128 || key0 + 127 > len + t0) {
          const int lo = max(0, key0 + row - len - t0) * ws.rep;
          weight_add<true>(ra, nlse, half * 64, lo, hi, ws.scale_log2, a0, a1);
          weight_add<true>(rb, nlse, half * 64 + 32, lo, hi, ws.scale_log2, a2, a3);
        } else {
          weight_add<false>(ra, nlse, half * 64, 0, 128, ws.scale_log2, a0, a1);
          weight_add<false>(rb, nlse, half * 64 + 32, 0, 128, ws.scale_log2, a2, a3);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_empty[st]);
        if (++st == C::RING) { st = 0; ph ^= 1u; }
        sum += (a0 + a1) + (a2 + a3);    // tile by tile: two short sums instead of one long one
      }
      if (!ok) break;
      // The right columns' sums join the left ones'.  The buffer is used again two
      // pieces on, behind a meeting that the left threads come to after reading it.
      if (half) right[(pieces & 1u) * 256] = sum;
      mbar_arrive(&meet[kt]);
      if (!mbar_wait_warp(&meet[kt], pieces & 1u, wait_ns)) break;
      if (!half) {
        sum += right[(pieces & 1u) * 256];
        // No slot receives more than a weight of 1 per row: beyond that lies what the
        // polynomial makes of a row that is not a number (keeping its NaN there costs
        // 20 us on the 8B prompt of 8192).
        if (sum > 1e30f) sum = NAN;
        seg = box->seg;
        b = seg.item / ws.key_tiles;
        if (box->w0 == 0 && box->w1 == seg.n)
          put_weight(ws, b, seg.sub, key0 + row, len, live, sum);
        else
          ws.part[(size_t)tiles_of.record(seg, blockIdx.x, box->run.a) * 256 + kt * 128 + row] = sum;
      }
      ++pieces;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// The weights from scores that the attention kernel left in the workspace (few
// rows): four slots per thread, over the sequence's rows and the group's heads.
// A block's loads are contiguous, and 16 of a thread's are in flight (8B decode
// step: 22 us with one slot per thread, 14 with two, 13 with four, 20 with eight).
constexpr int kScoredSlots = 4;
__global__ void __launch_bounds__(256) scored_weights_kernel(const __grid_constant__ WeightShape ws) {
  griddep_wait_and_release();
  const int b = blockIdx.y / ws.KV, g = blockIdx.y % ws.KV, key = blockIdx.x * (256 * kScoredSlots) + threadIdx.x;
  const int len = cached_len(ws.kv_lens, b, ws.max_len), live = cached_len(ws.seq_lens, b, ws.S);
  if (key >= len + live) return;
  const int ld = (ws.max_len + ws.S + 127) / 128 * 128;
  const float* sc = ws.scores + (size_t)blockIdx.y * ws.rep * ws.S * ld + key;
  const float* nlse = ws.nlse + (size_t)blockIdx.y * ws.tile_rows;
  const int rows = live * ws.rep;       // the packed rows of live positions come first
  float sum[kScoredSlots] = {};
#pragma unroll 4
  for (int r = 0; r < rows; ++r) {
    const float n = nlse[r];
#pragma unroll
    for (int u = 0; u < kScoredSlots; ++u)
      if (key + 256 * u < len + live) sum[u] += exp2f(sc[(size_t)r * ld + 256 * u] + n);
  }
#pragma unroll
  for (int u = 0; u < kScoredSlots; ++u) put_weight(ws, b, g, key + 256 * u, len, live, sum[u]);
}

// The slots of cut segments: block i < G - 1 takes the one that CTA i + 1's border
// cuts, adding its pieces in order.  Block G - 1 + b
// carries sequence b's weights over where it has no row in this call.
__global__ void __launch_bounds__(256) slot_weights_join_kernel(const __grid_constant__ WeightShape ws) {
  griddep_wait_and_release();
  const WeightTiles tiles_of{ws};
  if ((int)blockIdx.x >= ws.G - 1) {
    const int b = blockIdx.x - (ws.G - 1);
    const int len = cached_len(ws.kv_lens, b, ws.max_len);
    if (cached_len(ws.seq_lens, b, ws.S) > 0) return;
    for (int g = 0; g < ws.KV; ++g)
      for (int key = threadIdx.x; key < len; key += 256) put_weight(ws, b, g, key, len, 0, 0.f);
    return;
  }
  const int KT = 1 << ws.key_shift;
  int per;
  const FlatSeg seg = flat_cut(ws.cuts, blockIdx.x + 1, per);
  if (seg.n == 0) return;
  const int b = seg.item / ws.key_tiles, key0 = (seg.item % ws.key_tiles) << ws.key_shift;
  const int len = cached_len(ws.kv_lens, b, ws.max_len), live = cached_len(ws.seq_lens, b, ws.S);
  if ((int)threadIdx.x >= KT) return;
  float sum = 0.f;
  for (int c = (int)(seg.s0 / per); c <= (int)((seg.end() - 1) / per); ++c) {
    int w0, w1;
    if (!seg.cut(c * per, (c + 1) * per, w0, w1)) continue;
    if (w0 == 0 && w1 == seg.n) return;
    sum += ws.part[(size_t)tiles_of.record(seg, c, c * per) * KT + threadIdx.x];
  }
  put_weight(ws, b, seg.sub, key0 + threadIdx.x, len, live, sum);
}

}  // namespace l3
