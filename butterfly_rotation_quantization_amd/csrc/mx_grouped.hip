// Products of rows of microscaled 4-bit activations, grouped by expert, with
// their experts' weights: row t of group e times weight e, the groups' ends read
// on the device (format: mx.h; chunks, tiles and the epilogue: mm_dev.h).
//
// A group's rows are cut into units, numbered through all groups; the host knows
// only how many there can be (gm_units), so a grid has a place for each of those,
// and a workgroup finds its unit from the offsets, or ends.
#include "mm_dev.h"

namespace brq {
namespace {

// A unit of g.rows rows of one group.
struct GmUnit {
  int e;           // the group
  int begin, end;  // its rows
  int units;       // its units
  int first;       // the first one's number
};
// The groups, one to a lane and 64 at a time: their rows, their units and the
// inclusive sum of these.  Every lane of a wavefront makes the same calls.  No row
// is in two groups, whatever the offsets are, so there are never more units than
// the grid and the workspace have places for.
struct GmGroups {
  int at, base, low;  // of the 64: the first group, the units before it, the rows that earlier ones end at
  int b, end, n, x;

  __device__ __forceinline__ explicit GmGroups(const GmArgs& g) { load(g, 0, 0, 0); }
  __device__ __forceinline__ void next(const GmArgs& g) {
    load(g, at + 64, base + __builtin_amdgcn_readlane(x, 63), __builtin_amdgcn_readlane(end, 63));
  }
  __device__ __forceinline__ void load(const GmArgs& g, int e0, int before, int rows) {
    const int lane = threadIdx.x & 63, last = g.groups - e0 < 64 ? g.groups - e0 : 64;
    at = e0;
    base = before;
    low = rows;
    const int e = e0 + (lane < last ? lane : last - 1);
    gm_rows(g.offs[e], g.offs[e + 1], (int)g.mm.T, &b, &end);
    if (lane >= last) b = end;
    if (__builtin_amdgcn_ballot_w64(b < low || end < b)) {  // an offset below an earlier one: the greatest so far
      int top = b > end ? b : end;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const int y = __shfl_up(top, d);
        if (lane >= d && y > top) top = y;
      }
      const int y = __shfl_up(top, 1);
      if (lane > 0 && y > b) b = y;
      b = b > low ? b : low;
      end = top > low ? top : low;
      if (lane >= last) b = end;
    }
    n = (end - b + g.rows - 1) / g.rows;
    x = n;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int y = __shfl_up(x, d);
      if (lane >= d) x += y;
    }
  }
  // all groups' units
  __device__ __forceinline__ int64_t all(const GmArgs& g) {
    while (at + 64 < g.groups) next(g);
    return base + __builtin_amdgcn_readlane(x, 63);
  }
  // The group that has place p, of `places` a unit; there is one.
  __device__ __forceinline__ void find(const GmArgs& g, int64_t p, int64_t places, GmUnit& u) {
    if (p < base * places) load(g, 0, 0, 0);
    uint64_t past;
    while (!(past = __builtin_amdgcn_ballot_w64(p < (int64_t)(base + x) * places))) next(g);
    const int l = __builtin_ctzll(past);
    u.e = at + l;
    u.begin = __builtin_amdgcn_readlane(b, l);
    u.end = __builtin_amdgcn_readlane(end, l);
    u.units = __builtin_amdgcn_readlane(n, l);
    u.first = base + __builtin_amdgcn_readlane(x, l) - u.units;
  }
};
// The product's arguments as those of one group alone: rows up to its end, its
// weight.
__device__ __forceinline__ MmArgs gm_group(const GmArgs& g, const GmUnit& u) {
  MmArgs a = g.mm;
  a.T = u.end;
  a.b += (int64_t)u.e * a.m * (a.n / 2);
  a.bs += (int64_t)u.e * a.m * (a.n / kMxBlock);
  return a;
}

// Few rows a group: the stream over its weight, once for each unit.  Bound by memory
// where rows are long (32 rows, 8 groups of 11008x4096: 40 us, 4.8 TB/s), by finding the
// unit, one way from memory and the join where they are short (64 groups of 1376x2048, a row
// each 21 us, 12 each 25; 777 rows in shares that fall as the rank 32).
template <int TT, int RT, int W>
__global__ __launch_bounds__(64 * W) void gm_rows_kernel(GmArgs g, MmEpi ep) {
  __shared__ typename MmRows<TT, RT, W>::Sums sums;
  const MmArgs& a = g.mm;
  const uint32_t strips = (uint32_t)((a.m + 16 * RT - 1) / (16 * RT)), number = blockIdx.x / strips;
  GmGroups groups(g);
  if ((int)number >= groups.all(g)) return;
  GmUnit u;
  groups.find(g, number, 1, u);
  const int64_t nb = a.n / kMxBlock, weight = a.m * nb;
  const int64_t o0 = (int64_t)(blockIdx.x - number * strips) * (16 * RT);
  const int64_t t0 = u.begin + (int64_t)((int)number - u.first) * (16 * TT);
  MmRows<TT, RT, W> r;
  r.begin(a.b + u.e * weight * 16, a.bs + u.e * weight, a.m, nb, o0);
  r.sum(a, u.end, t0, sums);
  ep.bias = gm_bias(ep, u.e, a.m);
  __syncthreads();
  r.finish(a, ep, u.end, t0, o0, sums);
}

// Images of scales, of the units' rows and of the weights of groups that have some.
template <int R>
__global__ __launch_bounds__(kMxThreads) void gm_scales_kernel(GmArgs g) {
  const MmArgs& a = g.mm;
  const int64_t nb = a.n / kMxBlock, t = blockIdx.x;
  const int s0 = (int)blockIdx.y * kMmRun;
  if (t < a.gt) {
    GmGroups groups(g);
    if (t >= groups.all(g)) return;
    GmUnit u;
    groups.find(g, t, 1, u);
    mm_scale_tile<R>(a.as, u.begin + (t - u.first) * R, u.end, nb, a.stages, s0, a.ts + t * a.stages * (8 * R));
  } else {
    const int64_t i = t - a.gt, e = i / a.go, o = i - e * a.go;
    int b, end;
    gm_rows(g.offs[e], g.offs[e + 1], (int)a.T, &b, &end);
    if (end <= b) return;
    mm_scale_tile<R>(a.bs + e * a.m * nb, o * R, a.m, nb, a.stages, s0, a.os + i * a.stages * (8 * R));
  }
}

// Blocks go to the XCDs in turn, so those with one remainder by 8 take
// consecutive places, whose tiles share operands, of those that there are.
template <int WT, int WO, int TT, int TO, int NB>
__global__ __launch_bounds__(64 * WT * WO, 1) void gm_tile_kernel(GmArgs g, MmEpi) {
  using Full = MmTile<WT, WO, TT, TO, NB, true, MmEpi>;
  using Any = MmTile<WT, WO, TT, TO, NB, false, MmEpi>;
  __shared__ typename Full::Lds lds;
  GmGroups groups(g);
  const int64_t go = g.mm.go, all = groups.all(g) * go, per = (all + 7) / 8;
  const int64_t i = blockIdx.x >> 3, p = (blockIdx.x & 7) * per + i;
  if (i >= per || p >= all) return;
  GmUnit u;
  groups.find(g, p, go, u);
  MmWhere w;
  mm_place(p - u.first * go, u.units, go, g.mm.band, w);
  const MmArgs a = gm_group(g, u);
  const auto late = MmLate<MmEpi>::after<GmArgs>(u.e);
  const int64_t t0 = u.begin + w.tt * Full::BT, o0 = w.to * Full::BO;
  const uint8_t* ts = a.ts + (u.first + w.tt) * a.stages * (8 * Full::BT);
  const uint8_t* os = a.os + (u.e * go + w.to) * a.stages * (8 * Full::BO);
  if (t0 + Full::BT <= a.T && o0 + Full::BO <= a.m && a.n % kMmK == 0) Full(a, late, lds, t0, o0, 0, ts, os).run();
  else Any(a, late, reinterpret_cast<typename Any::Lds&>(lds), t0, o0, 0, ts, os).run();
}

template <int TT, int W>
void gm_rows(const GmArgs& g, const MmEpi& e, hipStream_t s) {
  gm_rows_kernel<TT, 2, W><<<dim3((unsigned)gm_stream_workgroups(g)), 64 * W, 0, s>>>(g, e);
}
template <int TT>
hipError_t gm_rows(const GmArgs& g, const MmEpi& e, hipStream_t s) {
  if (gm_stream_waves(g.mm.n) == 2) gm_rows<TT, 2>(g, e, s);
  else gm_rows<TT, 4>(g, e, s);
  return hipGetLastError();
}

template <int WT, int WO, int TT, int TO, int NB>
hipError_t gm_tiles(const GmArgs& g, const MmEpi& ep, hipStream_t s) {
  constexpr int R = 32 * TT * WT;
  static_assert(R == 32 * TO * WO, "square tiles");
  const MmArgs& a = g.mm;
  gm_scales_kernel<R><<<dim3((unsigned)(a.gt + g.groups * a.go), (unsigned)((a.stages + kMmRun - 1) / kMmRun)),
                        kMxThreads, 0, s>>>(g);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  gm_tile_kernel<WT, WO, TT, TO, NB><<<dim3((unsigned)((a.gt * a.go + 7) / 8 * 8)), 64 * WT * WO, 0, s>>>(g, ep);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_grouped(const GmArgs& g, const MmEpi& e, hipStream_t s) {
  if (g.mm.tile == 256) return gm_tiles<2, 2, 4, 4, 2>(g, e, s);
  if (g.mm.tile == 128) return gm_tiles<2, 2, 2, 2, 2>(g, e, s);
  if (g.rows == 32) return gm_rows<2>(g, e, s);
  return gm_rows<1>(g, e, s);
}

}  // namespace brq
