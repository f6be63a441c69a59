// flat_plan.cuh -- equal shares of ragged work, planned on the device.
//
// The cache operators work on segments (a sequence, a KV head and some query
// rows or key slots) of n tiles each, where n depends on lengths that only the
// device knows.  Laid end to end, every segment of n > 0 tiles takes n +
// kFlatLead units of cost (kFlatLead stands for a segment's own start and
// end); CTA c of G takes the units [c * per, (c + 1) * per), per = ceil(total /
// G), so all CTAs carry the same load whatever the lengths are, and a segment
// that crosses a border is cut into pieces there.  Every warp derives the plan
// from the lengths alone, in the same way, so nothing is communicated.
//
// Units are counted in 32 bits; the host refuses work beyond 2^30 of them.
// Items are what has a length (a sequence, or a sequence's query block); each
// item stands for `mult` segments of the same n.  NOf is a functor int(int item).
#pragma once
#include "common.cuh"

namespace l3 {

// A segment's start and end (query load, first loads in flight, the result's
// store) in tiles: on the 8B prompt a segment costs 9200 cycles beside its tiles
// of 3350 each.
constexpr int kFlatLead = 3;

__device__ __forceinline__ int flat_cost(int n) { return n > 0 ? n + kFlatLead : 0; }

// Cost of all items; every lane gets it.  Whole warp.
template <class NOf>
__device__ __forceinline__ int flat_total(int items, int mult, const NOf& n_of) {
  int t = 0;
  for (int i = threadIdx.x & 31; i < items; i += 32) t += flat_cost(n_of(i));
  return __reduce_add_sync(0xffffffffu, t) * mult;
}

// One segment: segment `sub` of `item`, n tiles, at cost units s0 .. s0 + n + kFlatLead - 1.
struct FlatSeg {
  int item, sub, n;
  int s0;
  __device__ __forceinline__ int end() const { return s0 + n + kFlatLead; }
  // The CTAs, of runs of `per` units, that work on its first and on its last tile.
  __device__ __forceinline__ int first_cta(int per) const { return (s0 + kFlatLead) / per; }
  __device__ __forceinline__ int last_cta(int per) const { return (end() - 1) / per; }
  // The tiles [w0, w1) of this segment within the units [a, e); false if there are none.
  __device__ __forceinline__ bool cut(int a, int e, int& w0, int& w1) const {
    w0 = max(0, a - s0 - kFlatLead);
    w1 = min(e, end()) - s0 - kFlatLead;
    return w1 > w0;
  }
};

// The segment that unit `pos` (< total) lies in.  Whole warp.
template <class NOf>
__device__ __forceinline__ FlatSeg flat_seek(int items, int mult, const NOf& n_of, int pos) {
  const int lane = threadIdx.x & 31;
  int base = 0;
  FlatSeg s;
  s.item = s.sub = s.n = 0;
  s.s0 = 0;
  for (int i0 = 0; i0 < items; i0 += 32) {
    const int n = i0 + lane < items ? n_of(i0 + lane) : 0;
    const int own = flat_cost(n) * mult;
    int incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    const uint32_t hit = __ballot_sync(0xffffffffu, base + incl > pos);
    if (hit) {
      const int l = __ffs(hit) - 1;
      s.item = i0 + l;
      s.n = __shfl_sync(0xffffffffu, n, l);
      const int start = base + __shfl_sync(0xffffffffu, incl - own, l);
      s.sub = (pos - start) / flat_cost(s.n);
      s.s0 = start + s.sub * flat_cost(s.n);
      return s;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return s;
}

// What the kernels that join the pieces of cut segments need of the plan, left by
// the main kernel: entry c is the segment that the border before CTA c's run
// cuts, if that is the first border within it (n = 0 otherwise), and the run
// length `per`.
struct FlatCut {
  int item, sub, n, s0, per, pad[3];
};

// A value that all lanes hold, as one that the compiler knows to be the same for
// the whole warp: loop bounds of the plan come from shuffles, and without this a
// loop over them counts as divergent, which keeps the tcgen05 issuers' addresses
// out of the uniform registers.
__device__ __forceinline__ int warp_uniform(int x) { return __reduce_max_sync(0xffffffffu, x); }

// The pieces of one CTA, in order.
template <class NOf>
struct FlatRun {
  FlatSeg seg;
  int a, e, per;
  int items, mult;
  bool more;
  // Whole warp.
  __device__ __forceinline__ void start(int items_, int mult_, const NOf& n_of, int c, int G) {
    items = items_;
    mult = mult_;
    const int total = flat_total(items, mult, n_of);
    per = (total + G - 1) / G;
    a = per * c;
    e = min(a + per, total);
    more = a < e;
    if (more) seg = flat_seek(items, mult, n_of, a);
  }
  // After start(), by one thread of CTA c.
  __device__ __forceinline__ void leave(FlatCut* cuts, int c) const {
    const bool first = more && seg.s0 < a && seg.s0 >= a - per;
    int4* out = reinterpret_cast<int4*>(cuts + c);
    out[0] = make_int4(more ? seg.item : 0, more ? seg.sub : 0, first ? seg.n : 0, more ? seg.s0 : 0);
    out[1] = make_int4(per, 0, 0, 0);
  }
  // next() for a whole warp, with everything uniform.
  __device__ __forceinline__ bool next_uniform(const NOf& n_of, FlatSeg& s, int& w0, int& w1) {
    if (!__all_sync(0xffffffffu, next(n_of, s, w0, w1))) return false;
    s.item = warp_uniform(s.item);
    s.sub = warp_uniform(s.sub);
    s.n = warp_uniform(s.n);
    s.s0 = warp_uniform(s.s0);
    w0 = warp_uniform(w0);
    w1 = warp_uniform(w1);
    return true;
  }
  // The next piece, or false at the end of the run (any lane, no communication).
  __device__ __forceinline__ bool next(const NOf& n_of, FlatSeg& s, int& w0, int& w1) {
    while (more) {
      s = seg;
      const bool some = s.cut(a, e, w0, w1);
      seg.s0 = s.end();
      if (seg.s0 >= e) {
        more = false;
      } else if (++seg.sub == mult) {
        seg.sub = 0;
        do {
          if (++seg.item == items) {   // never reached while units below e <= total are left
            more = false;
            break;
          }
          seg.n = n_of(seg.item);
        } while (seg.n == 0);
      }
      if (some) return true;
    }
    return false;
  }
};

// A warp's run in shared memory: lane 0 steps it, all lanes read the piece, so
// that the plan takes no registers while a warp works on a piece.
template <class NOf>
struct FlatBox {
  FlatRun<NOf> run;
  FlatSeg seg;
  int w0, w1;
  int more;
  __device__ __forceinline__ void start(int items, int mult, const NOf& n_of, int c, int G) {
    FlatRun<NOf> r;
    r.start(items, mult, n_of, c, G);
    if ((threadIdx.x & 31) == 0) run = r;
    __syncwarp();
  }
  __device__ __forceinline__ bool next(const NOf& n_of) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
      FlatRun<NOf> r = run;
      FlatSeg s = r.seg;
      int a = 0, b = 0;
      more = r.next(n_of, s, a, b) ? 1 : 0;
      run = r;
      seg = s;
      w0 = a;
      w1 = b;
    }
    __syncwarp();
    return more != 0;
  }
};

__device__ __forceinline__ FlatSeg flat_cut(const FlatCut* cuts, int c, int& per) {
  const int4* in = reinterpret_cast<const int4*>(cuts + c);
  const int4 x = in[0];
  per = in[1].x;
  FlatSeg s;
  s.item = x.x;
  s.sub = x.y;
  s.n = x.z;
  s.s0 = x.w;
  return s;
}

}  // namespace l3
