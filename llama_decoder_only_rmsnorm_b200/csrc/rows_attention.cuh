// rows_attention.cuh -- attention of several query rows per sequence over a
// ragged cache, on tcgen05: the main kernel of tree attention (a drafted tree's
// nodes over the cached rows) and of observed attention (a chunk's rows,
// causal, leaving each row's log-sum-exp).
//
//  * The rows of one KV head are its sequence's query positions times the rep =
//    H / KV query heads that share the head: row t * rep + j is position t,
//    head g * rep + j.  A 128-row tile holds 128 / rep whole positions (one 5-D
//    TMA box of q), so GQA heads fill the tensor core's rows even for a few
//    positions, and every K/V tile is read once for up to 256 rows.
//  * PAIR = true: a CTA works on two row tiles (slots) at once, each with its
//    own softmax warpgroup; both use the same K/V tile.  PAIR = false, for at
//    most 128 rows per KV head: the two warpgroups take alternate key tiles of
//    the one row tile, so one's softmax hides behind the other's products, and
//    join their (m, l, O) at the end of the piece through TMEM, in which both can
//    read the same lanes.
//  * Work is cut into equal shares over the CTAs by flat_plan.cuh: a long cache
//    of one sequence spreads over the whole GPU, ragged batches stay balanced.
//    A cut piece leaves a record (m, l, O) per row for the kernels below.
//  * Within a tile: S = Q K^T (M = 128 rows, N = 128 keys) and O += P V with P
//    in TMEM, one softmax thread per row, lazy rescaling, P handed over in two
//    halves: the same scheme and register split as flash_attention.cuh.
//  * The probabilities go to the tensor core in bf16, as its product with bf16 values
//    wants them: each is off by 2^-8 at most, like the output's own rounding
//    (relative error of the outputs against 64 bits 2.0e-3 to 2.3e-3; 1.7e-3 for fp32
//    rounded once).  Their sum l takes them in fp32, before that rounding.
//  * What bounds it: the DRAM for a few rows over long caches (8B decode step,
//    32 x 8192 keys: 1.07 GB in 167 us, 6.4 TB/s; 8B batch of 16-node trees:
//    0.69 GB in 120 us), the tensor core and the exponentials for many rows (8B
//    prompt of 8192: 483 us, 1139 TFLOP/s; flash_attention.cuh, which need not
//    leave a sum that fp32 weights can be divided by, 440 us beside it).
//  * V rows behind the sequence are zeroed in shared memory before the product
//    (their probability is 0, but 0 x NaN is NaN), so the cache may hold
//    anything there.
#pragma once
#include "cache_ops.cuh"
#include "flash_attention.cuh"
#include "flat_plan.cuh"

namespace l3 {

__device__ __forceinline__ void tma_load_5d(void* smem_dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t c0, int32_t c1, int32_t c2, int32_t c3, int32_t c4) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4)
      : "memory");
}
// L2 policy for data that is read once: first to go when room is needed.
__device__ __forceinline__ uint64_t policy_evict_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void tma_load_4d_once(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int32_t c0,
                                                 int32_t c1, int32_t c2, int32_t c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
      : "memory");
}
// Untiled copy of `bytes` (a multiple of 16, both addresses 16-byte aligned).
__device__ __forceinline__ void bulk_load(void* smem_dst, const void* src, uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(smem_dst)),
      "l"(__cvta_generic_to_global(src)), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// The row and key tiles of a launch, for the main kernels and for those that join
// their records.
struct RowsShape {
  int B, T, H, KV, rep;              // T query positions per sequence
  int qpt, tiles, tile_rows;         // positions per row tile, row tiles, rows of a tile (128 or 64)
  int slots, groups;                 // row tiles that a CTA works on together, and groups of them
  int key_shift;                     // log2 of a key tile (7 or 6)
  int G, max_len;                    // CTAs of the main kernel
  int folded;                        // fold_pieces_kernel ran: a segment's first record stands for all
  float scale_log2;                  // log2(e) / sqrt(hd)
  const int32_t *kv_lens, *seq_lens;
  FlatCut* cuts;                     // [G] the plan, for the kernels that join
  float *part_ml, *part_o;           // records: [id][row][2] and [id][hd/4][row][4], slots * tile_rows rows
  float* scores;                     // observed, few rows: [B][H * T][key tiles * 128] in the log2 domain, or NULL
  float* nlse;                       // observed: minus the rows' log-sum-exp (log2), [B * KV][tiles][tile_rows]
  void* out;
};

// Key tiles of an item.  Tree: item = sequence.  Causal: item = sequence and group.
template <bool TREE>
struct RowsTiles {
  const RowsShape& rs;
  __device__ __forceinline__ int operator()(int i) const {
    const int up = (1 << rs.key_shift) - 1;
    if (TREE) return (cached_len(rs.kv_lens, i, rs.max_len) + up) >> rs.key_shift;
    const int b = i / rs.groups, t0 = (i % rs.groups) * rs.qpt * rs.slots;
    const int live = cached_len(rs.seq_lens, b, rs.T);
    if (t0 >= live) return 0;
    return (cached_len(rs.kv_lens, b, rs.max_len) + min(live, t0 + rs.qpt * rs.slots) + up) >> rs.key_shift;
  }
  __device__ __forceinline__ int items() const { return TREE ? rs.B : rs.B * rs.groups; }
  __device__ __forceinline__ int mult() const { return TREE ? rs.KV * rs.groups : rs.KV; }
  __device__ __forceinline__ void where(const FlatSeg& s, int& b, int& grp, int& g) const {
    b = TREE ? s.item : s.item / rs.groups;
    grp = TREE ? s.sub / rs.KV : s.item % rs.groups;
    g = s.sub % rs.KV;
  }
  // Record of the piece of segment s that the CTA c, whose run begins at unit a,
  // works on.  Tree: every piece has one, and the segment's number plus the
  // CTA's is another for each.  Causal: only the pieces of cut segments, which
  // lie at the ends of a CTA's run.
  __device__ __forceinline__ int record(const FlatSeg& s, int c, int a) const {
    return TREE ? s.item * mult() + s.sub + c : 2 * c + (s.s0 < a ? 0 : 1);
  }
};

template <int HD, bool PAIR>
struct RowsCfg {
  static constexpr int CHUNKS = (HD + 63) / 64;
  static constexpr int TILE = 128 * 128;               // 128 rows of 64 bf16
  static constexpr int Q_BYTES = CHUNKS * TILE, KV_BYTES = CHUNKS * TILE;
  static constexpr int NQ = PAIR ? 2 : 1;
  static constexpr int RING0 = (232448 - 1024 - 1024 - 2048 - 8 * 2048 - NQ * Q_BYTES) / KV_BYTES;
  static constexpr int RING = RING0 > 8 ? 8 : RING0;   // K and V tiles in flight
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_RING = NQ * Q_BYTES;
  static constexpr int OFF_STAGE = OFF_RING + RING * KV_BYTES;   // 2 KB per softmax warp
  static constexpr int OFF_ML = OFF_STAGE + 8 * 2048;            // [slot][128] x (m, l)
  static constexpr int OFF_BAR = OFF_ML + 2048;
  static constexpr int N_BARS = 4 + 2 * RING + 8 + 2;
  static constexpr int SMEM_BYTES = 1024 + OFF_BAR + N_BARS * 8 + 16;
  static_assert(SMEM_BYTES <= 232448 && RING >= 4, "shared memory");
  static_assert(HD % 32 == 0 && HD <= 128, "head_dim");
};

__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// max(x, floor), NaN where x is one (fmaxf gives the floor)
__device__ __forceinline__ float max_or_nan(float x, float floor) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(floor));
  return y;
}

// 2^x = p * 2^n for two x <= 0 by the range reduction of exp2_poly2, with a
// polynomial of degree 5 (this project's own fit, max relative error 2.4e-7): the
// accumulated weights and the row sums that they are divided by are fp32 results.
// `shift` is 1.5 * 2^23 plus a small integer k, and t's low bits hold n + k.  Where
// x is a NaN, p and t are the canonical one.
__device__ __forceinline__ void exp2_poly2_fine(float shift, float x0, float x1, uint64_t& p, float& t0, float& t1) {
  const uint64_t x = f2_pack(max_or_nan(x0, -126.0f), max_or_nan(x1, -126.0f));
  const uint64_t t = f2_add(x, f2_pack(shift, shift));
  const uint64_t f = f2_fma(f2_add(t, f2_pack(-shift, -shift)), f2_pack(-1.0f, -1.0f), x);
  p = f2_pack(0.001327647129073739f, 0.001327647129073739f);
  p = f2_fma(p, f, f2_pack(0.009675541892647743f, 0.009675541892647743f));
  p = f2_fma(p, f, f2_pack(0.05550713092088699f, 0.05550713092088699f));
  p = f2_fma(p, f, f2_pack(0.24022120237350464f, 0.24022120237350464f));
  p = f2_fma(p, f, f2_pack(0.6931469440460205f, 0.6931469440460205f));
  p = f2_fma(p, f, f2_pack(1.0000001192092896f, 1.0000001192092896f));
  f2_unpack(t, t0, t1);
}
// 2^x, NaN where x is one: 2^n is a factor, as adding n to the exponent of a NaN
// makes a number of it.
__device__ __forceinline__ void exp2_poly2_nan(float x0, float x1, float& y0, float& y1) {
  uint64_t p;
  float t0, t1;
  exp2_poly2_fine(12583039.0f, x0, x1, p, t0, t1);   // k = 127: the low bits are the exponent field of 2^n
  f2_unpack(f2_mul(p, f2_pack(__int_as_float(__float_as_int(t0) << 23), __int_as_float(__float_as_int(t1) << 23))), y0,
            y1);
}
// 2^x, the largest finite number where x is a NaN (0x7fffffff plus the same moved up
// by 23 bits): one instruction less per number.
__device__ __forceinline__ void exp2_poly2_huge(float x0, float x1, float& y0, float& y1) {
  uint64_t p;
  float p0, p1, t0, t1;
  exp2_poly2_fine(12582912.0f, x0, x1, p, t0, t1);
  f2_unpack(p, p0, p1);
  y0 = __int_as_float(__float_as_int(p0) + (__float_as_int(t0) << 23));
  y1 = __int_as_float(__float_as_int(p1) + (__float_as_int(t1) << 23));
}

// p = 2^(s * scl - m) for 32 scores in place and their sum; the FMA pipe takes
// 2 of 16 pairs of an unmasked row (8B prompt: 832 k cycles against 872 k with 4
// and 839 k with none; trees of 128 nodes over 8 x 8000 rows of 64: 59 us, 58 with 4
// pairs by the cubic, which has no place for a NaN, and over 4 x 8000 rows of 128:
// 65.4 against 66.0).
template <bool MASKED>
__device__ __forceinline__ void rows_exp(uint32_t (&r)[32], float scl, float neg_m, float& sa, float& sb) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float x0, x1, p0, p1;
    fma2(x0, x1, __uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]), scl, scl, neg_m, neg_m);
    if (!MASKED && (i & 7) < 1) {
      exp2_poly2_nan(x0, x1, p0, p1);
    } else {
      p0 = ex2_approx(x0);
      p1 = ex2_approx(x1);
    }
    add2(sa, sb, p0, p1);
    r[2 * i] = __float_as_uint(p0);
    r[2 * i + 1] = __float_as_uint(p1);
  }
}
template <bool MASKED>
__device__ __forceinline__ float rows_exp_half(uint32_t (&ra)[32], uint32_t (&rb)[32], float scl, float neg_m,
                                               uint32_t taddr) {
  float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
  rows_exp<MASKED>(ra, scl, neg_m, s0, s1);
  rows_exp<MASKED>(rb, scl, neg_m, s2, s3);
  flash_pack_store(ra, taddr);
  flash_pack_store(rb, taddr + 16);
  return (s0 + s1) + (s2 + s3);
}

__device__ __forceinline__ void rows_put_scores(const uint32_t (&r)[32], float* s, float scl) {
#pragma unroll
  for (int i = 0; i < 32; i += 4)
    *reinterpret_cast<float4*>(s + i) = make_float4(__uint_as_float(r[i]) * scl, __uint_as_float(r[i + 1]) * scl,
                                                    __uint_as_float(r[i + 2]) * scl, __uint_as_float(r[i + 3]) * scl);
}

struct RowsBars {
  uint64_t *q_full, *q_empty, *full, *empty, *s_full, *p_half, *p_full, *o_done, *merge;
};

// The order in which a piece of n key tiles uses its K and V tiles, which is the
// order of their loads: f(is_v, tile).
//   PAIR:  K0 V0 K1 V1 ...       (V_j is released before K_j+1)
//   else:  K0 K1 V0 K2 V1 K3 ... (the warpgroups are one tile apart)
template <bool PAIR, class F>
__device__ __forceinline__ bool rows_ring_order(int n, const F& f) {
  if (!f(false, 0)) return false;
  if (!PAIR && n > 1 && !f(false, 1)) return false;
  constexpr int ahead = PAIR ? 1 : 2;
  for (int j = 0; j < n; ++j) {
    if (!f(true, j)) return false;
    if (j + ahead < n && !f(false, j + ahead)) return false;
  }
  return true;
}

template <int HD, bool TREE, bool PAIR>
__global__ void __launch_bounds__(kFlashThreads, 1)
    rows_attention_kernel(const __grid_constant__ CUtensorMap mapQ, const __grid_constant__ CUtensorMap mapK,
                          const __grid_constant__ CUtensorMap mapV, const __grid_constant__ RowsShape rs,
                          const unsigned long long wait_ns) {
  using C = RowsCfg<HD, PAIR>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  RowsBars bars;
  bars.q_full = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  bars.q_empty = bars.q_full + 2;
  bars.full = bars.q_empty + 2;
  bars.empty = bars.full + C::RING;
  bars.s_full = bars.empty + C::RING;
  bars.p_half = bars.s_full + 2;
  bars.p_full = bars.p_half + 2;
  bars.o_done = bars.p_full + 2;
  bars.merge = bars.o_done + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars.merge + 2);

  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.q_full[s], 1); mbar_init(&bars.q_empty[s], 1);
      mbar_init(&bars.s_full[s], 1); mbar_init(&bars.o_done[s], 1);
      mbar_init(&bars.p_half[s], 128); mbar_init(&bars.p_full[s], 128);
      mbar_init(&bars.merge[s], 256);
    }
    for (int s = 0; s < C::RING; ++s) { mbar_init(&bars.full[s], 1); mbar_init(&bars.empty[s], 1); }
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&mapQ); prefetch_tensormap(&mapK); prefetch_tensormap(&mapV);
  }
  if (warp == 1) tmem_alloc(tmem_slot, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const RowsTiles<TREE> tiles_of{rs};
  FlatRun<RowsTiles<TREE>> run;
  FlatSeg seg;
  int w0, w1, b, grp, g;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kFlashLowRegs));
    griddep_wait_and_release();
    if (warp == 0) {
      // -------------------------------------------------------------- producer
      run.start(tiles_of.items(), tiles_of.mult(), tiles_of, blockIdx.x, gridDim.x);
      if (lane == 0) {
        run.leave(rs.cuts, blockIdx.x);
        int st = 0;
        uint32_t ph = 0, qph = 0, iss = 0, par = 0, qiss = 0, qpar = 0;
        bool ok = true;
        const uint32_t q_bytes = (uint32_t)(rs.rep * rs.qpt * 128 * C::CHUNKS);
        const uint64_t once = policy_evict_first();
        while (ok && run.next(tiles_of, seg, w0, w1)) {
          tiles_of.where(seg, b, grp, g);
          for (int s = 0; s < C::NQ; ++s) {
            const int rt = grp * C::NQ + s;
            if (rt >= rs.tiles) break;
            if (!mbar_wait(&bars.q_empty[s], ((qph >> s) & 1u) ^ 1u, wait_ns)) { ok = false; break; }
            mbar_arrive_expect_tx(&bars.q_full[s], q_bytes);
            for (int c = 0; c < C::CHUNKS; ++c)
              tma_load_5d(smem + C::OFF_Q + s * C::Q_BYTES + c * C::TILE, &mapQ, &bars.q_full[s], c * 64, 0, g,
                          rt * rs.qpt, b);
            qiss |= 1u << s; qpar = (qpar & ~(1u << s)) | (qph & (1u << s));
            qph ^= 1u << s;
          }
          if (!ok) break;
          ok = rows_ring_order<PAIR>(w1 - w0, [&](bool is_v, int j) {
            if (!mbar_wait(&bars.empty[st], ph ^ 1u, wait_ns)) return false;
            mbar_arrive_expect_tx(&bars.full[st], C::KV_BYTES);
            for (int c = 0; c < C::CHUNKS; ++c)
              // No other CTA of this launch reads this tile: the L2 is for records and scores
              // (8B decode step observed 203 -> 189 us, 8B batch of trees 127 -> 120).  Observed
              // rows whose scores are not kept do read K again, in the launch of the weights.
              if (rs.groups == 1)
                tma_load_4d_once(smem + C::OFF_RING + st * C::KV_BYTES + c * C::TILE, is_v ? &mapV : &mapK,
                                 &bars.full[st], c * 64, g, (w0 + j) * 128, b, once);
              else
                tma_load_4d(smem + C::OFF_RING + st * C::KV_BYTES + c * C::TILE, is_v ? &mapV : &mapK, &bars.full[st],
                            c * 64, g, (w0 + j) * 128, b);
            iss |= 1u << st; par = (par & ~(1u << st)) | (ph << st);
            if (++st == C::RING) { st = 0; ph ^= 1u; }
            return true;
          });
        }
        for (int s = 0; s < 2; ++s)
          if (qiss & (1u << s)) mbar_wait(&bars.q_full[s], (qpar >> s) & 1u, wait_ns);
        for (int s = 0; s < C::RING; ++s)
          if (iss & (1u << s)) mbar_wait(&bars.full[s], (par >> s) & 1u, wait_ns);
      }
    } else if (warp == 1) {
      // -------------------------------------------------------------- MMA issuer
      constexpr uint32_t IDESC_S = idesc_bf16_f32(128, 128, 0, 0);
      constexpr uint32_t IDESC_O = idesc_bf16_f32(128, HD, 0, 1);   // A = P (TMEM), B = V MN-major
      run.start(tiles_of.items(), tiles_of.mult(), tiles_of, blockIdx.x, gridDim.x);
      const bool leader = elect_one_sync();
      const uint32_t q_addr = smem_u32(smem + C::OFF_Q), ring_addr = smem_u32(smem + C::OFF_RING);
      int st = 0;
      uint32_t ph = 0, qph = 0, pph = 0;
      bool ok = true;
      // PAIR calls name their slot by a literal: addresses and descriptors of the
      // two slots are then constants of the code, and the next S is ready 1100
      // cycles after a row's last P instead of 1390 (8B prompt of 8192).
      // the next tile of the ring, once it has landed; -1 if the wait gave up
      auto take = [&]() -> int {
        if (!mbar_wait_warp(&bars.full[st], ph, wait_ns)) return -1;
        const int got = st;
        if (++st == C::RING) { st = 0; ph ^= 1u; }
        tc_fence_after();
        return got;
      };
      auto issue_s = [&](int s, int kst) {
        const uint32_t qa = q_addr + (PAIR ? s * C::Q_BYTES : 0), ka = ring_addr + kst * C::KV_BYTES;
        if (leader) {
#pragma unroll
          for (int k = 0; k < HD / 16; ++k) {
            const uint32_t off = (k >> 2) * C::TILE + (k & 3) * 32;
            tc_mma_f16_ss(tmem_base + s * 256, sw128_desc(qa + off, 1024, 16), sw128_desc(ka + off, 1024, 16), IDESC_S,
                          k > 0);
          }
          tc_commit(&bars.s_full[s]);
        }
        __syncwarp();
      };
      // waits for the halves of slot s's P and adds P V; false if a wait gave up
      auto issue_pv = [&](int s, int vst, bool accumulate) -> bool {
        const uint32_t va = ring_addr + vst * C::KV_BYTES;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!mbar_wait_warp(half ? &bars.p_full[s] : &bars.p_half[s], (pph >> s) & 1u, wait_ns)) return false;
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int kk = half * 4 + k;
              tc_mma_f16_ts(tmem_base + s * 256 + 128, tmem_base + s * 256 + kk * 8,
                            sw128_desc(va + kk * 2048, 1024, C::TILE), IDESC_O, (accumulate || kk > 0) ? 1u : 0u);
            }
            if (half) tc_commit(&bars.o_done[s]);
          }
          __syncwarp();
        }
        pph ^= 1u << s;
        return true;
      };
      // V rows from `valid` on become zero
      auto clear_tail = [&](int vst, int valid) {
        uint8_t* v = smem + C::OFF_RING + vst * C::KV_BYTES;
        for (int c = 0; c < C::CHUNKS; ++c)
          for (int i = valid * 8 + lane; i < 128 * 8; i += 32)
            *reinterpret_cast<uint4*>(v + c * C::TILE + i * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
      };
      while (ok && run.next_uniform(tiles_of, seg, w0, w1)) {
        tiles_of.where(seg, b, grp, g);
        const int n = w1 - w0;
        const int held = warp_uniform(cached_len(rs.kv_lens, b, rs.max_len) +
                                      (TREE ? 0 : cached_len(rs.seq_lens, b, rs.T)));
        const int nslots = PAIR ? (grp * 2 + 1 < rs.tiles ? 2 : 1) : 1;
        for (int s = 0; s < nslots; ++s) {
          if (!mbar_wait_warp(&bars.q_full[s], (qph >> s) & 1u, wait_ns)) ok = false;
          qph ^= 1u << s;
        }
        if (!ok) break;
        tc_fence_after();
        // S of tile i for every slot that works on it; with !PAIR slot i & 1
        auto scores = [&](int i) -> bool {
          const int kst = take();
          if (kst < 0) return false;
          if (PAIR) {
            issue_s(0, kst);
            if (nslots == 2) issue_s(1, kst);
          } else {
            issue_s(i & 1, kst);
          }
          if (leader) tc_commit(&bars.empty[kst]);
          __syncwarp();
          return true;
        };
        ok = scores(0) && (PAIR || n < 2 || scores(1));
        for (int j = 0; j < n && ok; ++j) {
          const int vst = take();
          if (vst < 0) { ok = false; break; }
          if ((w0 + j) * 128 + 128 > held) clear_tail(vst, held - (w0 + j) * 128);
          if (PAIR) {
            int kst = -1;
            if (!issue_pv(0, vst, j > 0)) { ok = false; break; }
            if (j + 1 < n) {
              kst = take();
              if (kst < 0) { ok = false; break; }
              issue_s(0, kst);
            }
            if (nslots == 2) {
              if (!issue_pv(1, vst, j > 0)) { ok = false; break; }
              if (j + 1 < n) issue_s(1, kst);
            }
            if (leader) {
              tc_commit(&bars.empty[vst]);
              if (kst >= 0) tc_commit(&bars.empty[kst]);
            }
            __syncwarp();
          } else {
            ok = issue_pv(j & 1, vst, j > 1);
            if (!ok) break;
            if (leader) tc_commit(&bars.empty[vst]);
            __syncwarp();
            if (j + 2 < n) ok = scores(j + 2);
          }
        }
        if (leader)
          for (int s = 0; s < nslots; ++s) tc_commit(&bars.q_empty[s]);
        __syncwarp();
      }
    } else if (!TREE) {
      // -------------------------------------------------------------- zeros for the padding rows
      const int row16 = rs.H * HD * 2 / 16;
      const int w = blockIdx.x * 2 + warp - 2;
      for (int i = w; i < rs.B * rs.T; i += gridDim.x * 2) {
        if (i % rs.T < cached_len(rs.seq_lens, i / rs.T, rs.T)) continue;
        uint4* o = static_cast<uint4*>(rs.out) + (size_t)i * row16;
        for (int k = lane; k < row16; k += 32) o[k] = make_uint4(0, 0, 0, 0);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(kFlashHighRegs));
    griddep_wait_and_release();
    // ---------------------------------------------------------------- softmax (one thread per row)
    const int slot = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;            // row of the tile == TMEM lane
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const uint32_t s_tmem = tmem_base + lane_off + slot * 256;
    const uint32_t o_tmem = s_tmem + 128;
    const int t_in = row / rs.rep;                  // this row's position and head within the tile
    float2* ml = reinterpret_cast<float2*>(smem + C::OFF_ML);
    uint32_t sph = 0, oph = 0, mph = 0;
    const int score_tiles = (rs.max_len + rs.T + 127) / 128;
    bool merged = false;                            // a join is open: the other warpgroup may still read O
    run.start(tiles_of.items(), tiles_of.mult(), tiles_of, blockIdx.x, gridDim.x);
    while (run.next_uniform(tiles_of, seg, w0, w1)) {
      tiles_of.where(seg, b, grp, g);
      const int rt = PAIR ? grp * 2 + slot : grp;
      if (PAIR && rt >= rs.tiles) continue;
      const int len = warp_uniform(cached_len(rs.kv_lens, b, rs.max_len));
      const int t = rt * rs.qpt + t_in;
      const int last = TREE ? len - 1 : len + t;                     // last key this row sees
      const int last_min = TREE ? len - 1 : len + rt * rs.qpt;       // and the tile's first row
      const int n = w1 - w0;
      float m_ref = -INFINITY, l = 0.f;
      bool ok = true, first = true;
      for (int j = PAIR ? 0 : slot; j < n; j += PAIR ? 1 : 2) {
        if (!mbar_wait_warp(&bars.s_full[slot], sph, wait_ns)) { ok = false; break; }
        sph ^= 1u;
        tc_fence_after();
        const int key0 = (w0 + j) * 128;
        const bool need_mask = key0 + 127 > last_min;
        uint32_t ra[32], rb[32], rc[32], rd[32];
        flash_load_row(s_tmem, ra, rb, rc, rd);
        float m0, m1, m2, m3;
        if (need_mask) {
          m0 = flash_row_max<true>(ra, key0, last, 0);
          m1 = flash_row_max<true>(rb, key0 + 32, last, 0);
          m2 = flash_row_max<true>(rc, key0 + 64, last, 0);
          m3 = flash_row_max<true>(rd, key0 + 96, last, 0);
        } else {
          m0 = flash_row_max<false>(ra, key0, last, 0);
          m1 = flash_row_max<false>(rb, key0 + 32, last, 0);
          m2 = flash_row_max<false>(rc, key0 + 64, last, 0);
          m3 = flash_row_max<false>(rd, key0 + 96, last, 0);
        }
        if (!TREE && !PAIR && rs.scores && t_in < rs.qpt && t < rs.T) {
          float* sc = rs.scores + ((size_t)(b * rs.KV + g) * rs.rep * rs.T + row) * ((size_t)score_tiles << 7) + key0;
          rows_put_scores(ra, sc, rs.scale_log2);
          rows_put_scores(rb, sc + 32, rs.scale_log2);
          rows_put_scores(rc, sc + 64, rs.scale_log2);
          rows_put_scores(rd, sc + 96, rs.scale_log2);
        }
        const float m_tile = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3)) * rs.scale_log2;
        // the slot's previous P.V is complete: its S was issued behind it
        if (!first) oph ^= 1u;
        const bool grow = m_tile > m_ref + 8.0f;
        float alpha = 1.f;
        if (grow) {
          alpha = exp2f(m_ref - m_tile);
          l *= alpha;
          m_ref = m_tile;
        }
        if (!first && __any_sync(0xffffffffu, grow)) {
#pragma unroll 1
          for (int c = 0; c < HD / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(o_tmem + c * 16, o);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
            tmem_st16(o_tmem + c * 16, o);
          }
          tc_wait_st();
        }
        const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;
        float la, lb;
        if (need_mask)
          la = rows_exp_half<true>(ra, rb, rs.scale_log2, neg_m, s_tmem);
        else
          la = rows_exp_half<false>(ra, rb, rs.scale_log2, neg_m, s_tmem);
        if (!PAIR && merged) {
          // the first P.V of this piece overwrites O: the other warpgroup has to have read the last piece's
          if (!mbar_wait_warp(&bars.merge[1], mph ^ 1u, wait_ns)) { ok = false; break; }
          merged = false;
        }
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&bars.p_half[slot]);
        if (need_mask)
          lb = rows_exp_half<true>(rc, rd, rs.scale_log2, neg_m, s_tmem + 32);
        else
          lb = rows_exp_half<false>(rc, rd, rs.scale_log2, neg_m, s_tmem + 32);
        l += la + lb;
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(&bars.p_full[slot]);
        first = false;
      }
      if (!ok) break;
      if (!first) {
        if (!mbar_wait_warp(&bars.o_done[slot], oph, wait_ns)) break;
        oph ^= 1u;
        tc_fence_after();
      }
      // f_own, f_oth: this warpgroup's and the other one's share in the result
      float m = m_ref, f_own = 1.f, f_oth = 0.f;
      if (!PAIR) {
        if (merged) {   // this warpgroup had no tile, so it has not waited yet
          if (!mbar_wait_warp(&bars.merge[1], mph ^ 1u, wait_ns)) break;
          merged = false;
        }
        ml[slot * 128 + row] = make_float2(m_ref, l);
        tc_fence_before();
        mbar_arrive(&bars.merge[0]);
        if (!mbar_wait_warp(&bars.merge[0], mph, wait_ns)) break;
        tc_fence_after();
        const float2 oth = ml[(slot ^ 1) * 128 + row];
        m = fmaxf(m_ref, oth.x);
        f_own = m_ref == -INFINITY ? 0.f : exp2f(m_ref - m);
        f_oth = oth.x == -INFINITY ? 0.f : exp2f(oth.x - m);
        l = l * f_own + oth.y * f_oth;
        mph ^= 1u;
        merged = true;
      }
      const int live = TREE ? rs.T : cached_len(rs.seq_lens, b, rs.T);
      const bool real = t_in < rs.qpt && t < live;
      const bool whole = !TREE && w0 == 0 && w1 == seg.n;
      const int R = PAIR ? 256 : 128, rrow = PAIR ? slot * 128 + row : row;
      const size_t id = tiles_of.record(seg, blockIdx.x, run.a);
      if ((PAIR || slot == 0) && real) {
        if (whole)
          rs.nlse[((size_t)(b * rs.KV + g) * rs.tiles + rt) * 128 + row] = -(m + log2f(l));
        else
          *reinterpret_cast<float2*>(rs.part_ml + (id * R + rrow) * 2) = make_float2(m, l);
      }
      const float inv = 1.f / l;
      uint8_t* stage = smem + C::OFF_STAGE + (warp - 4) * 2048;
#pragma unroll 1
      for (int c = 0; c < HD / 32; ++c) {
        if (!PAIR && (c & 1) != slot) continue;    // the warpgroups share the columns
        uint32_t r[32];
        tmem_ld32(o_tmem + c * 32, r);
        tc_wait_ld();
        if (!PAIR) {
          uint32_t q[32];
          tmem_ld32((slot ? o_tmem - 256 : o_tmem + 256) + c * 32, q);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            // a warpgroup that saw no key has nothing in its O
            const float own = f_own == 0.f ? 0.f : __uint_as_float(r[i]) * f_own;
            r[i] = __float_as_uint(f_oth == 0.f ? own : fmaf(__uint_as_float(q[i]), f_oth, own));
          }
        }
        if (whole) {
          // as in flash_attention.cuh: through 2 KB of shared memory, 64 contiguous bytes per row
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint4 o;
            o.x = pack_bf16x2(__uint_as_float(r[8 * k + 0]) * inv, __uint_as_float(r[8 * k + 1]) * inv);
            o.y = pack_bf16x2(__uint_as_float(r[8 * k + 2]) * inv, __uint_as_float(r[8 * k + 3]) * inv);
            o.z = pack_bf16x2(__uint_as_float(r[8 * k + 4]) * inv, __uint_as_float(r[8 * k + 5]) * inv);
            o.w = pack_bf16x2(__uint_as_float(r[8 * k + 6]) * inv, __uint_as_float(r[8 * k + 7]) * inv);
            *reinterpret_cast<uint4*>(stage + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) = o;
          }
          __syncwarp();
#pragma unroll
          for (int mm = 0; mm < 4; ++mm) {
            const int rr = mm * 8 + (lane >> 2), k = lane & 3;
            const uint4 o = *reinterpret_cast<const uint4*>(stage + rr * 64 + ((k ^ ((rr >> 1) & 3)) << 4));
            const int tr = (quarter * 32 + rr) / rs.rep, jr = quarter * 32 + rr - tr * rs.rep;
            if (tr < rs.qpt && rt * rs.qpt + tr < live)
              *reinterpret_cast<uint4*>(static_cast<bf16*>(rs.out) +
                                        (((size_t)b * rs.T + rt * rs.qpt + tr) * rs.H + g * rs.rep + jr) * HD +
                                        c * 32 + k * 8) = o;
          }
          __syncwarp();
        } else if (real) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4*>(rs.part_o + ((id * (HD / 4) + c * 8 + k) * R + rrow) * 4) =
                make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
        }
      }
      tc_fence_before();
      if (!PAIR) mbar_arrive(&bars.merge[1]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// ---- joining the pieces ------------------------------------------------------
// A row's (m, l, acc): lane k holds dims 4k .. 4k+3 (k < HD / 4).
struct RowAcc {
  float m, l, a[4];
  __device__ __forceinline__ void clear() {
    m = -INFINITY;
    l = 0.f;
    a[0] = a[1] = a[2] = a[3] = 0.f;
  }
  // adds a piece; one that saw no key has nothing in its O, but one of keys that
  // are all not a number has the maximum -inf as well, and a NaN for its sum
  __device__ __forceinline__ void add(float pm, float pl, const float4& o) {
    if (pm == -INFINITY && pl == pl) return;
    const float mn = fmaxf(m, pm);
    const float f = m == -INFINITY ? 0.f : exp2f(m - mn), fp = exp2f(pm - mn);
    l = l * f + pl * fp;
    a[0] = a[0] * f + o.x * fp;
    a[1] = a[1] * f + o.y * fp;
    a[2] = a[2] * f + o.z * fp;
    a[3] = a[3] * f + o.w * fp;
    m = mn;
  }
};
__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const bf16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y));
}
__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<float4*>(p) = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(bf16* p, float a, float b, float c, float d) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}

// Joins the pieces of NR neighbouring rows of segment seg, from record row rrow on,
// into acc (whole warp; acc is empty before).  A lane per piece gathers the (m,
// l), and the first U pieces' O are asked for before those are needed.
template <int HD, int NR>
__device__ __forceinline__ void join_pieces(const RowsShape& rs, const FlatSeg& seg, int per, int rrow,
                                            RowAcc (&acc)[NR]) {
  constexpr int U = NR == 4 ? 2 : 4;
  const RowsTiles<true> tiles_of{rs};
  const int lane = threadIdx.x & 31, R = rs.slots * rs.tile_rows;
  const int c0 = seg.first_cta(per), c1 = rs.folded ? c0 : seg.last_cta(per);
  for (int cb = c0; cb <= c1; cb += 32) {
    const int c = cb + lane;
    int w0 = 0, w1 = 0;
    const bool some = c <= c1 && seg.cut(c * per, (c + 1) * per, w0, w1);
    const int id = some ? tiles_of.record(seg, c, c * per) : 0;
    uint32_t todo = __ballot_sync(0xffffffffu, some);
    float2 ml[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      ml[i] = make_float2(-INFINITY, 0.f);
      if (some) ml[i] = *reinterpret_cast<const float2*>(rs.part_ml + ((size_t)id * R + rrow + i) * 2);
    }
    float4 o[U][NR];
    int src[U];
    auto fetch = [&]() {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        src[u] = todo ? __ffs(todo) - 1 : -1;
        const int from = __shfl_sync(0xffffffffu, id, max(src[u], 0));
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          o[u][i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (src[u] >= 0 && lane < HD / 4)
            o[u][i] = load4(rs.part_o + (((size_t)from * (HD / 4) + lane) * R + rrow + i) * 4);
        }
        todo &= todo - 1;
      }
    };
    fetch();
    float fp[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const float mn = fmaxf(acc[i].m, warp_max(ml[i].x));
      const float f = acc[i].m == -INFINITY ? 0.f : exp2f(acc[i].m - mn);
      fp[i] = ml[i].x == -INFINITY ? 0.f : exp2f(ml[i].x - mn);
      acc[i].l = acc[i].l * f + warp_sum(ml[i].y * fp[i]);
      acc[i].m = mn;
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i].a[k] *= f;
    }
    for (;;) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < NR; ++i) {
          const float w = __shfl_sync(0xffffffffu, fp[i], max(src[u], 0));
          if (src[u] >= 0) {
            acc[i].a[0] = fmaf(o[u][i].x, w, acc[i].a[0]);
            acc[i].a[1] = fmaf(o[u][i].y, w, acc[i].a[1]);
            acc[i].a[2] = fmaf(o[u][i].z, w, acc[i].a[2]);
            acc[i].a[3] = fmaf(o[u][i].w, w, acc[i].a[3]);
          }
        }
      if (!todo) break;
      fetch();
    }
  }
}

// Joins the pieces of segments that many CTAs share -- a long cache of few KV
// heads -- into the record of the first, eight warps per row, so that the kernels
// below have one record to read.  blockIdx.x + 1 is the CTA whose border is the
// first within the segment, blockIdx.y a row of it.  What bounds it is the round
// trips of a row's records: 148 pieces are five rounds for eight warps of four
// pieces each, and 37 for one warp (an observed step over 60000 fp32 rows of two
// KV heads of 16: 100 us in all against 131).
constexpr int kFoldWarps = 8;
template <int HD, bool TREE>
__global__ void __launch_bounds__(32 * kFoldWarps) fold_pieces_kernel(const __grid_constant__ RowsShape rs) {
  __shared__ float ms[kFoldWarps], ls[kFoldWarps], as[kFoldWarps][HD];
  griddep_wait_and_release();
  int per, b, grp, g;
  const FlatSeg seg = flat_cut(rs.cuts, blockIdx.x + 1, per);
  if (seg.n == 0) return;
  const RowsTiles<TREE> tiles_of{rs};
  tiles_of.where(seg, b, grp, g);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, R = rs.slots * rs.tile_rows;
  const int first = seg.first_cta(per), c1 = seg.last_cta(per);
  if (first == c1) return;     // one piece
  int w0, w1;
  for (int r = blockIdx.y; r < R; r += gridDim.y) {
    const int rt = grp * rs.slots + r / rs.tile_rows, t_in = r % rs.tile_rows / rs.rep;
    if (t_in >= rs.qpt || rt * rs.qpt + t_in >= rs.T) continue;
    RowAcc acc;
    acc.clear();
    for (int cb = first + warp; cb <= c1; cb += 4 * kFoldWarps) {     // four pieces in flight
      float2 ml[4];
      float4 o[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = cb + u * kFoldWarps;
        ml[u] = make_float2(-INFINITY, 0.f);
        o[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (c > c1 || !seg.cut(c * per, (c + 1) * per, w0, w1)) continue;
        const size_t id = tiles_of.record(seg, c, c * per);
        ml[u] = *reinterpret_cast<const float2*>(rs.part_ml + (id * R + r) * 2);
        if (lane < HD / 4) o[u] = load4(rs.part_o + ((id * (HD / 4) + lane) * R + r) * 4);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) acc.add(ml[u].x, ml[u].y, o[u]);
    }
    if (lane == 0) { ms[warp] = acc.m; ls[warp] = acc.l; }
    if (lane < HD / 4) store4(&as[warp][4 * lane], acc.a[0], acc.a[1], acc.a[2], acc.a[3]);
    __syncthreads();
    if (warp == 0) {
      acc.clear();
#pragma unroll
      for (int w = 0; w < kFoldWarps; ++w)
        acc.add(ms[w], ls[w], lane < HD / 4 ? load4(&as[w][4 * lane]) : make_float4(0.f, 0.f, 0.f, 0.f));
      const size_t id = tiles_of.record(seg, first, first * per);
      if (lane == 0) *reinterpret_cast<float2*>(rs.part_ml + (id * R + r) * 2) = make_float2(acc.m, acc.l);
      if (lane < HD / 4)
        store4(rs.part_o + ((id * (HD / 4) + lane) * R + r) * 4, acc.a[0], acc.a[1], acc.a[2], acc.a[3]);
    }
    __syncthreads();
  }
}

// Tree attention, second half: a warp joins the pieces over the cache with the
// node's own ancestors, whose keys it reads one by one -- a chain is short next to
// the cache, and a product with the whole tree's values would let the infinities
// of other nodes in (0 x inf).  A warp takes NR query heads of one node: they
// share the chain and its keys, and their sums overlap.
// blockIdx.x = (sequence, KV head), blockIdx.y = kJoinWarps * NR rows.
constexpr int kJoinWarps = 8;
template <typename T, int HD, int NR>
__global__ void __launch_bounds__(32 * kJoinWarps, 2)
    tree_join_kernel(const __grid_constant__ RowsShape rs, const T* __restrict__ q, const T* __restrict__ kn,
                     const T* __restrict__ vn, const int32_t* __restrict__ parents) {
  __shared__ int32_t par[kMaxTreeNodes];
  __shared__ uint8_t chain_s[kJoinWarps][kMaxTreeNodes];
  griddep_wait_and_release();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.x / rs.KV, g = blockIdx.x % rs.KV;
  for (int i = threadIdx.x; i < rs.T; i += blockDim.x) par[i] = parents[(size_t)b * rs.T + i];
  // the plan's loads are on their way together with the parents
  const RowsTiles<true> tiles_of{rs};
  const int per = rs.G > 0 ? rs.cuts->per : 0;
  FlatSeg seg;
  seg.item = b;
  seg.n = rs.G > 0 ? tiles_of(b) : 0;
  int before = 0;
  for (int i = lane; i < b; i += 32) before += flat_cost(tiles_of(i));
  before = __reduce_add_sync(0xffffffffu, before);
  __syncthreads();
  const int r = (blockIdx.y * kJoinWarps + warp) * NR;     // row t * rep + j, NR divides rep
  if (r >= rs.T * rs.rep) return;
  const int t = r / rs.rep, h = g * rs.rep + r - t * rs.rep;
  T* o = static_cast<T*>(rs.out) + (((size_t)b * rs.T + t) * rs.H + h) * HD + 4 * lane;
  const bool on = lane < HD / 4;
  // the chain from the node up to its root
  uint8_t* chain = chain_s[warp];
  int depth = 0;
  bool live = false;
  for (int c = t;;) {
    if (lane == 0) chain[depth] = (uint8_t)c;
    ++depth;
    const int p = par[c];
    if (p >= c) record_error(LLAMA3_ERR_ARG);
    if (p < 0 || p >= c) {
      live = p == -1;
      break;
    }
    c = p;
  }
  if (!live) {
    if (on)
#pragma unroll
      for (int i = 0; i < NR; ++i) store4(o + i * HD, 0.f, 0.f, 0.f, 0.f);
    return;
  }
  __syncwarp();
  // q and the first keys of the chain are under way while the pieces are joined
  constexpr int U = NR == 4 ? 2 : 4;
  float4 qv[NR], k[U], v[U];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      k[u] = v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + u < depth && on) {
        const size_t at = (((size_t)b * rs.T + chain[i0 + u]) * rs.KV + g) * HD + 4 * lane;
        k[u] = load4(kn + at);
        v[u] = load4(vn + at);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    qv[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) qv[i] = load4(q + (((size_t)b * rs.T + t) * rs.H + h + i) * HD + 4 * lane);
  }
  fetch(0);
  RowAcc acc[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) acc[i].clear();
  if (seg.n > 0) {
    const int mult = tiles_of.mult();
    const int rt = t / rs.qpt, grp = rt / rs.slots;
    seg.sub = grp * rs.KV + g;
    seg.s0 = before * mult + seg.sub * flat_cost(seg.n);
    join_pieces<HD, NR>(rs, seg, per, (rt - grp * rs.slots) * rs.tile_rows + r - rt * rs.qpt * rs.rep, acc);
  }
  for (int i0 = 0; i0 < depth; i0 += U) {
    float sc[U][NR];
    if (i0) fetch(i0);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < NR; ++i)
        sc[u][i] = fmaf(qv[i].x, k[u].x, fmaf(qv[i].y, k[u].y, fmaf(qv[i].z, k[u].z, qv[i].w * k[u].w)));
#pragma unroll
    for (int s = 16; s > 0; s >>= 1)
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < NR; ++i) sc[u][i] += __shfl_xor_sync(0xffffffffu, sc[u][i], s);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + u < depth)
#pragma unroll
        for (int i = 0; i < NR; ++i) acc[i].add(sc[u][i] * rs.scale_log2, 1.f, v[u]);
  }
  if (on)
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const float inv = 1.f / acc[i].l;
      store4(o + i * HD, acc[i].a[0] * inv, acc[i].a[1] * inv, acc[i].a[2] * inv, acc[i].a[3] * inv);
    }
}

// Observed attention: the rows of the segments that were cut.  blockIdx.x + 1 is
// the CTA whose border cuts the segment.  The lanes of a warp are 32 neighbouring
// rows, whose records lie side by side, and a warp takes 16 columns: every load
// is contiguous, and all pieces' loads are in flight together.
template <int HD>
struct CausalJoin {
  static constexpr int WARPS = HD / 16;                       // for 32 rows
  static constexpr int ROWS = WARPS >= 4 ? 32 : 128 / WARPS;  // of a block: at least four warps
  static constexpr int THREADS = WARPS * ROWS;
};
template <typename T, int HD>
__global__ void __launch_bounds__(CausalJoin<HD>::THREADS) causal_join_kernel(const __grid_constant__ RowsShape rs) {
  griddep_wait_and_release();
  const RowsTiles<false> tiles_of{rs};
  int per, b, grp, g;
  const FlatSeg seg = flat_cut(rs.cuts, blockIdx.x + 1, per);
  if (seg.n == 0) return;
  tiles_of.where(seg, b, grp, g);
  const int warp = threadIdx.x >> 5, col = warp % CausalJoin<HD>::WARPS;    // columns 16 col ..
  const int R = rs.slots * rs.tile_rows;
  const int r = blockIdx.y * CausalJoin<HD>::ROWS + warp / CausalJoin<HD>::WARPS * 32 + (threadIdx.x & 31);
  if (r >= R) return;
  const int rt = grp * rs.slots + r / rs.tile_rows, in = r % rs.tile_rows;
  const int t_in = in / rs.rep, t = rt * rs.qpt + t_in, h = g * rs.rep + in - t_in * rs.rep;
  if (t_in >= rs.qpt || t >= cached_len(rs.seq_lens, b, rs.T)) return;
  const int c0 = seg.first_cta(per), c1 = rs.folded ? c0 : seg.last_cta(per);
  if (c0 == seg.last_cta(per)) return;       // whole: written by its CTA, no record
  float m = -INFINITY, l = 0.f, a[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) a[i] = 0.f;
  for (int c = c0; c <= c1; c += 2) {        // two pieces in flight
    float2 ml[2];
    float4 o[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      int w0, w1;
      ml[u] = make_float2(-INFINITY, 0.f);
      if (c + u > c1 || !seg.cut((c + u) * per, (c + u + 1) * per, w0, w1)) continue;
      const size_t id = tiles_of.record(seg, c + u, (c + u) * per);
      ml[u] = *reinterpret_cast<const float2*>(rs.part_ml + (id * R + r) * 2);
#pragma unroll
      for (int k = 0; k < 4; ++k) o[u][k] = load4(rs.part_o + ((id * (HD / 4) + col * 4 + k) * R + r) * 4);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      if (ml[u].x == -INFINITY && ml[u].y == ml[u].y) continue;    // no such piece, or the row saw no key in it
      const float mn = fmaxf(m, ml[u].x);
      const float f = m == -INFINITY ? 0.f : exp2f(m - mn), fp = exp2f(ml[u].x - mn);
      l = l * f + ml[u].y * fp;
      m = mn;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        a[4 * k] = a[4 * k] * f + o[u][k].x * fp;
        a[4 * k + 1] = a[4 * k + 1] * f + o[u][k].y * fp;
        a[4 * k + 2] = a[4 * k + 2] * f + o[u][k].z * fp;
        a[4 * k + 3] = a[4 * k + 3] * f + o[u][k].w * fp;
      }
    }
  }
  const float inv = 1.f / l;
  T* o = static_cast<T*>(rs.out) + (((size_t)b * rs.T + t) * rs.H + h) * HD + col * 16;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    store4(o + 4 * k, a[4 * k] * inv, a[4 * k + 1] * inv, a[4 * k + 2] * inv, a[4 * k + 3] * inv);
  if (col == 0) rs.nlse[((size_t)(b * rs.KV + g) * rs.tiles + rt) * rs.tile_rows + in] = -(m + log2f(l));
}

}  // namespace l3
