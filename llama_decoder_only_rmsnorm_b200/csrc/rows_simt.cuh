// rows_simt.cuh -- the passes of rows_attention.cuh and slot_weights.cuh on the CUDA
// cores, for what the tensor cores do not take: fp32 (whose products stay
// fp32), head_dim 16, and the plain kernel path.  Same rows, pieces and records.
//
// 256 threads as 16 x 16 on a tile of 64 rows x 64 keys held in shared memory
// as fp32: thread (ty, tx) owns rows 4 ty .. 4 ty + 3 and keys tx, tx + 16, ...
// of the scores, and its rows' share of the output columns, so a row's maximum
// and sum are shuffles within 16 lanes.  Rows of the tiles are padded by four
// floats: 16 lanes then read 16 different bank groups.  4 sequences of 1000 fp32
// keys of 16 dims take 9 us, most of it the latency of one tile per block.
#pragma once
#include "slot_weights.cuh"

namespace l3 {

constexpr int kSimtTile = 64;
template <int HD>
struct SimtCfg {
  static constexpr int LD = HD + 4;
  static constexpr int LDP = kSimtTile + 4;
  static constexpr int ATT_BYTES = (3 * kSimtTile * LD + kSimtTile * LDP) * 4;
  static constexpr int WGT_BYTES = (2 * kSimtTile * LD + 16 * kSimtTile) * 4;
  static constexpr int VW = HD % 64 == 0 ? 4 : HD % 32 == 0 ? 2 : 1;   // floats per output access
  static constexpr int NC = HD / (16 * VW);
};

// 64 packed rows of q (zeros where there is none) into shared memory.
template <typename T, int HD>
__device__ __forceinline__ void simt_load_rows(float* s, const T* q, int b, int g, int t0, int qpt, int T_, int H,
                                               int rep) {
  for (int i = threadIdx.x; i < kSimtTile * (HD / 4); i += 256) {
    const int r = i / (HD / 4), c = (i % (HD / 4)) * 4, t_in = r / rep, t = t0 + t_in;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t_in < qpt && t < T_) x = load4(q + (((size_t)b * T_ + t) * H + g * rep + r - t_in * rep) * HD + c);
    store4(s + r * SimtCfg<HD>::LD + c, x.x, x.y, x.z, x.w);
  }
}
// 64 rows of a cache from row key0 on (zeros from `held` on).
template <typename T, int HD>
__device__ __forceinline__ void simt_load_keys(float* s, const T* kc, int b, int g, int key0, int held, int cap, int KV) {
  for (int i = threadIdx.x; i < kSimtTile * (HD / 4); i += 256) {
    const int r = i / (HD / 4), c = (i % (HD / 4)) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (key0 + r < held) x = load4(kc + (((size_t)b * cap + key0 + r) * KV + g) * HD + c);
    store4(s + r * SimtCfg<HD>::LD + c, x.x, x.y, x.z, x.w);
  }
}
template <int HD>
__device__ __forceinline__ void simt_scores(const float* sq, const float* sk, float (&s)[4][4]) {
  constexpr int LD = SimtCfg<HD>::LD;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
  for (int d = 0; d < HD; d += 4) {
    float4 q[4], k[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = load4(sq + (ty * 4 + i) * LD + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) k[j] = load4(sk + (tx + 16 * j) * LD + d);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = fmaf(q[i].x, k[j].x, s[i][j]);
        s[i][j] = fmaf(q[i].y, k[j].y, s[i][j]);
        s[i][j] = fmaf(q[i].z, k[j].z, s[i][j]);
        s[i][j] = fmaf(q[i].w, k[j].w, s[i][j]);
      }
  }
}

template <typename T, int HD, bool TREE>
__global__ void __launch_bounds__(256) rows_simt_kernel(const __grid_constant__ RowsShape rs, const T* __restrict__ q,
                                                        const T* __restrict__ kc, const T* __restrict__ vc, int cap) {
  using C = SimtCfg<HD>;
  constexpr int LD = C::LD, LDP = C::LDP, VW = C::VW, NC = C::NC;
  extern __shared__ float simt_smem[];
  float *sq = simt_smem, *sk = sq + kSimtTile * LD, *sv = sk + kSimtTile * LD, *sp = sv + kSimtTile * LD;
  griddep_wait_and_release();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const RowsTiles<TREE> tiles_of{rs};
  FlatRun<RowsTiles<TREE>> run;
  FlatSeg seg;
  int w0, w1, b, rt, g;
  run.start(tiles_of.items(), tiles_of.mult(), tiles_of, blockIdx.x, gridDim.x);
  if (threadIdx.x == 0) run.leave(rs.cuts, blockIdx.x);
  while (run.next(tiles_of, seg, w0, w1)) {
    tiles_of.where(seg, b, rt, g);                  // one row tile per group
    const int len = cached_len(rs.kv_lens, b, rs.max_len);
    const int live = TREE ? rs.T : cached_len(rs.seq_lens, b, rs.T);
    const int held = TREE ? len : len + live, t0 = rt * rs.qpt;
    __syncthreads();
    simt_load_rows<T, HD>(sq, q, b, g, t0, rs.qpt, rs.T, rs.H, rs.rep);
    float m[4], l[4], acc[4][NC * VW];
    int last[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
      last[i] = TREE ? len - 1 : len + t0 + (ty * 4 + i) / rs.rep;
#pragma unroll
      for (int c = 0; c < NC * VW; ++c) acc[i][c] = 0.f;
    }
    for (int w = w0; w < w1; ++w) {
      const int key0 = w * kSimtTile;
      if (w > w0) __syncthreads();
      simt_load_keys<T, HD>(sk, kc, b, g, key0, held, cap, rs.KV);
      simt_load_keys<T, HD>(sv, vc, b, g, key0, held, cap, rs.KV);
      __syncthreads();
      float s[4][4];
      simt_scores<HD>(sq, sk, s);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int key = key0 + tx + 16 * j;
          s[i][j] = key <= last[i] && key < held ? s[i][j] * rs.scale_log2 : -INFINITY;
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mn = fmaxf(m[i], mx);
        const float f = m[i] == -INFINITY ? 0.f : exp2f(m[i] - mn);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float p = s[i][j] == -INFINITY ? 0.f : exp2f(s[i][j] - mn);
          sp[(ty * 4 + i) * LDP + tx + 16 * j] = p;
          sum += p;
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l[i] = l[i] * f + sum;
        m[i] = mn;
#pragma unroll
        for (int c = 0; c < NC * VW; ++c) acc[i][c] *= f;
      }
      __syncwarp();        // a row's probabilities are written and read by the same 16 lanes
#pragma unroll 2
      for (int k = 0; k < kSimtTile; k += 4) {
        float4 p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = load4(sp + (ty * 4 + i) * LDP + k);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          float v[NC * VW];
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const float* src = sv + (k + kk) * LD + (tx + 16 * c) * VW;
            if (VW == 4) {
              const float4 x = load4(src);
              v[c * VW] = x.x; v[c * VW + 1 % VW] = x.y; v[c * VW + 2 % VW] = x.z; v[c * VW + 3 % VW] = x.w;
            } else {
#pragma unroll
              for (int e = 0; e < VW; ++e) v[c * VW + e] = src[e];
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float pi = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
#pragma unroll
            for (int c = 0; c < NC * VW; ++c) acc[i][c] = fmaf(pi, v[c], acc[i][c]);
          }
        }
      }
    }
    const bool whole = !TREE && w0 == 0 && w1 == seg.n;
    const size_t id = tiles_of.record(seg, blockIdx.x, run.a);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = ty * 4 + i, t_in = r / rs.rep, t = t0 + t_in;
      if (t_in >= rs.qpt || t >= live) continue;
      if (tx == 0) {
        if (whole)
          rs.nlse[((size_t)(b * rs.KV + g) * rs.tiles + rt) * kSimtTile + r] = -(m[i] + log2f(l[i]));
        else
          *reinterpret_cast<float2*>(rs.part_ml + (id * kSimtTile + r) * 2) = make_float2(m[i], l[i]);
      }
      T* o = static_cast<T*>(rs.out) + (((size_t)b * rs.T + t) * rs.H + g * rs.rep + r - t_in * rs.rep) * HD;
      const float inv = 1.f / l[i];
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          const int d = (tx + 16 * c) * VW + e;
          if (whole)
            o[d] = from_f<T>(acc[i][c * VW + e] * inv);
          else
            rs.part_o[((id * (HD / 4) + d / 4) * kSimtTile + r) * 4 + d % 4] = acc[i][c * VW + e];
        }
    }
  }
  if (!TREE) {   // zeros for the padding rows
    const int row4 = rs.H * HD / 4;
    for (int i = blockIdx.x; i < rs.B * rs.T; i += gridDim.x) {
      if (i % rs.T < cached_len(rs.seq_lens, i / rs.T, rs.T)) continue;
      for (int k = threadIdx.x; k < row4; k += 256)
        store4(static_cast<T*>(rs.out) + (size_t)i * row4 * 4 + 4 * k, 0.f, 0.f, 0.f, 0.f);
    }
  }
}

template <typename T, int HD>
__global__ void __launch_bounds__(256) slot_weights_simt_kernel(const __grid_constant__ WeightShape ws,
                                                                const T* __restrict__ q, const T* __restrict__ kc,
                                                                int H) {
  constexpr int LD = SimtCfg<HD>::LD;
  extern __shared__ float simt_smem[];
  float *sq = simt_smem, *sk = sq + kSimtTile * LD, *red = sk + kSimtTile * LD;
  griddep_wait_and_release();
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const WeightTiles tiles_of{ws};
  FlatRun<WeightTiles> run;
  FlatSeg seg;
  int w0, w1;
  run.start(tiles_of.items(), ws.KV, tiles_of, blockIdx.x, gridDim.x);
  if (threadIdx.x == 0) run.leave(ws.cuts, blockIdx.x);
  while (run.next(tiles_of, seg, w0, w1)) {
    const int b = seg.item / ws.key_tiles, key0 = (seg.item % ws.key_tiles) * kSimtTile, g = seg.sub;
    const int rt0 = tiles_of.first(seg.item);
    const int len = cached_len(ws.kv_lens, b, ws.max_len), live = cached_len(ws.seq_lens, b, ws.S);
    __syncthreads();
    simt_load_keys<T, HD>(sk, kc, b, g, key0, len + live, ws.cap, ws.KV);
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int w = w0; w < w1; ++w) {
      const int t0 = (rt0 + w) * ws.qpt;
      if (w > w0) __syncthreads();
      simt_load_rows<T, HD>(sq, q, b, g, t0, ws.qpt, ws.S, H, ws.rep);
      __syncthreads();
      float s[4][4], part[4] = {0.f, 0.f, 0.f, 0.f};
      simt_scores<HD>(sq, sk, s);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = ty * 4 + i, t_in = r / ws.rep;
        if (t_in >= ws.qpt || t0 + t_in >= live) continue;
        const float n = ws.nlse[((size_t)(b * ws.KV + g) * ws.tiles + rt0 + w) * kSimtTile + r];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (key0 + tx + 16 * j <= len + t0 + t_in) part[j] += exp2f(fmaf(s[i][j], ws.scale_log2, n));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) sum[j] += part[j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) red[ty * kSimtTile + tx + 16 * j] = sum[j];
    __syncthreads();
    if (threadIdx.x < kSimtTile) {
      float all = 0.f;
      for (int y = 0; y < 16; ++y) all += red[y * kSimtTile + threadIdx.x];
      if (w0 == 0 && w1 == seg.n)
        put_weight(ws, b, g, key0 + threadIdx.x, len, live, all);
      else
        ws.part[(size_t)tiles_of.record(seg, blockIdx.x, run.a) * kSimtTile + threadIdx.x] = all;
    }
  }
}

}  // namespace l3
