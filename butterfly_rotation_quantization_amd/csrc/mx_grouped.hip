// Products of rows of microscaled 4-bit activations, grouped by expert, with
// their experts' weights: row t of group e times weight e, the groups' ends read
// on the device (format: mx.h; the epilogue: mm_dev.h).
#include "mm_dev.h"

namespace brq {
namespace {

// A unit of R rows of one group.
struct GmUnit {
  int e;           // the group
  int begin, end;  // its rows
  int unit;        // of the group's units
};
// The unit of number `place` among all groups' units of R rows, in order of
// groups; false if there are fewer.  Every lane of the wavefront calls it with
// the same place: a group to a lane, 64 at a time.
__device__ __forceinline__ bool gm_find(const GmArgs& g, int R, int place, GmUnit& u) {
  const int lane = threadIdx.x & 63;
  int base = 0;
  for (int e0 = 0; e0 < g.groups; e0 += 64) {
    int b = 0, end = 0;
    if (e0 + lane < g.groups) gm_rows(g.offs[e0 + lane], g.offs[e0 + lane + 1], (int)g.mm.T, &b, &end);
    const int n = (end - b + R - 1) / R;
    int x = n;  // inclusive sum over the lanes before
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int y = __shfl_up(x, d);
      if (lane >= d) x += y;
    }
    const uint64_t past = __builtin_amdgcn_ballot_w64(place < base + x);
    if (past) {
      const int l = __builtin_ctzll(past);
      u.e = e0 + l;
      u.begin = __builtin_amdgcn_readlane(b, l);
      u.end = __builtin_amdgcn_readlane(end, l);
      u.unit = place - (base + __builtin_amdgcn_readlane(x, l) - __builtin_amdgcn_readlane(n, l));
      return true;
    }
    base += __builtin_amdgcn_readlane(x, 63);
  }
  return false;
}

// One wavefront per 16 x 16 outputs, as mm_simple_kernel.
__global__ __launch_bounds__(64) void gm_simple_kernel(GmArgs g, MmEpi ep) {
  const MmArgs& a = g.mm;
  const int lane = threadIdx.x, lr = lane & 15, lg = lane >> 4;
  const uint32_t go = (uint32_t)((a.m + 15) / 16);
  GmUnit u;
  if (!gm_find(g, 16, (int)(blockIdx.x / go), u)) return;
  const int64_t o0 = (int64_t)(blockIdx.x % go) * 16;
  const int64_t ra = u.begin + (int64_t)u.unit * 16 + lr, rb = o0 + lr;
  const int64_t nb = a.n / kMxBlock, wrow = (int64_t)u.e * a.m + rb;
  const bool va = ra < u.end, vb = rb < a.m;
  mxf4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int64_t k = 0; k < nb; k += 4) {
    const int64_t blk = k + lg;
    mxi4 x = {0, 0, 0, 0}, w = {0, 0, 0, 0};
    int sx = 127, sw = 127;
    if (va && blk < nb) {
      x = *reinterpret_cast<const mxi4*>(a.a + (ra * nb + blk) * 16);
      sx = a.as[ra * nb + blk];
    }
    if (vb && blk < nb) {
      w = *reinterpret_cast<const mxi4*>(a.b + (wrow * nb + blk) * 16);
      sw = a.bs[wrow * nb + blk];
    }
    const mxi8 X = {x[0], x[1], x[2], x[3], 0, 0, 0, 0}, W = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(X, W, acc, 4, 4, 0, sx, 0, sw);
  }
  ep.bias = gm_bias(ep, u.e, a.m);
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // D: row 4 lg + i, column lr
    const int64_t t = u.begin + (int64_t)u.unit * 16 + 4 * lg + i;
    if (t < u.end && vb) mm_store(a.y, a.yt, t * a.ldy + rb, mm_finish(ep, t, rb, acc[i]));
  }
}

}  // namespace

hipError_t launch_mx_grouped(const GmArgs& g, const MmEpi& e, hipStream_t s) {
  gm_simple_kernel<<<dim3((unsigned)(gm_units(g.mm.T, g.groups, 16) * ((g.mm.m + 15) / 16))), 64, 0, s>>>(g, e);
  return hipGetLastError();
}

}  // namespace brq
