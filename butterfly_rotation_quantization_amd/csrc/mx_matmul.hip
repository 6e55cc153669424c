// Product of two microscaled 4-bit matrices on the scaled matrix
// instructions (format: mx.h; tiles and chunks: mm_dev.h).
#include "mm_dev.h"

namespace brq {
namespace {

// For more than 64 tokens whose rows are too short (or too long) for the tiles
// below.  One wavefront per 16 x 16 outputs: lane l holds block l / 16 of a step of
// 128 values of row l % 16, of both operands, with the block's scale.  Bound by
// the outputs where they are many (2048x4096x128 12 us, 8192x8192x224 80 us, 1.7
// TB/s written two bytes a lane), by one wavefront's way through a row where that
// is long (65x64 by 2^23 values: 32 ms).
template <class E>
__global__ __launch_bounds__(64) void mm_simple_kernel(MmArgs a, E ep) {
  const int lane = threadIdx.x, lr = lane & 15, lg = lane >> 4;
  const uint32_t go = (uint32_t)((a.m + 15) / 16);
  const int64_t t0 = (int64_t)(blockIdx.x / go) * 16, o0 = (int64_t)(blockIdx.x % go) * 16;
  const int64_t ra = t0 + lr, rb = o0 + lr;
  const int64_t nb = a.n / kMxBlock;
  const bool va = ra < a.T, vb = rb < a.m;
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
      w = *reinterpret_cast<const mxi4*>(a.b + (rb * nb + blk) * 16);
      sw = a.bs[rb * nb + blk];
    }
    const mxi8 X = {x[0], x[1], x[2], x[3], 0, 0, 0, 0}, W = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(X, W, acc, 4, 4, 0, sx, 0, sw);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // D: row 4 lg + i, column lr
    const int64_t t = t0 + 4 * lg + i;
    if (t < a.T && vb) mm_store(a.y, a.yt, t * a.ldy + rb, mm_finish(ep, t, rb, acc[i]));
  }
}


template <int TT, int RT, int W, class E>
__global__ __launch_bounds__(64 * W) void mm_rows_kernel(MmArgs a, E ep) {
  __shared__ typename MmRows<TT, RT, W>::Sums sums;
  const int64_t o0 = (int64_t)blockIdx.x * (16 * RT);
  MmRows<TT, RT, W> r;
  r.begin(a.b, a.bs, a.m, a.n / kMxBlock, o0);
  r.sum(a, a.T, 0, sums);
  __syncthreads();
  r.finish(a, ep, a.T, 0, o0, sums);
}

template <int TT, int RT, class E>
void mm_rows(const MmArgs& a, const E& ep, hipStream_t s) {
  const int64_t wgs = (a.m + 16 * RT - 1) / (16 * RT);
  if (mm_stream_waves(wgs) == 8) mm_rows_kernel<TT, RT, 8><<<dim3((unsigned)wgs), 512, 0, s>>>(a, ep);
  else mm_rows_kernel<TT, RT, 4><<<dim3((unsigned)wgs), 256, 0, s>>>(a, ep);
}
template <int TT, class E>
hipError_t mm_rows(const MmArgs& a, const E& ep, hipStream_t s) {
  if (mm_stream_rows(a) == 32) mm_rows<TT, 2>(a, ep, s);
  else mm_rows<TT, 1>(a, ep, s);
  return hipGetLastError();
}

template <int BT, int BO>
__global__ __launch_bounds__(kMxThreads) void mm_scales_kernel(MmArgs a) {
  const int64_t nb = a.n / kMxBlock;
  const int stages = (int)((nb + kMmKS - 1) / kMmKS), s0 = (int)blockIdx.y * kMmRun;
  const int64_t t = blockIdx.x, o = t - a.gt;
  if (t < a.gt) mm_scale_tile<BT>(a.as, t * BT, a.T, nb, stages, s0, a.ts + t * stages * (8 * BT));
  else mm_scale_tile<BO>(a.bs, o * BO, a.m, nb, stages, s0, a.os + o * stages * (8 * BO));
}

template <int WT, int WO, int TT, int TO, int NB, class E>
__global__ __launch_bounds__(64 * WT * WO, 1) void mm_tile_kernel(MmArgs a, E) {
  using Full = MmTile<WT, WO, TT, TO, NB, true, E>;
  using Any = MmTile<WT, WO, TT, TO, NB, false, E>;
  __shared__ typename Full::Lds lds;
  MmWhere w;
  if (!mm_where(a, blockIdx.x, w)) return;
  const int64_t t0 = w.tt * Full::BT, o0 = w.to * Full::BO;
  MmLate<E> late;
  if constexpr (!std::is_same<E, MmNoEpi>::value) late = MmLate<E>::template after<MmArgs>();
  const uint8_t *ts = a.ts + w.tt * a.stages * (8 * Full::BT), *os = a.os + w.to * a.stages * (8 * Full::BO);
  if (t0 + Full::BT <= a.T && o0 + Full::BO <= a.m && a.n % kMmK == 0) Full(a, late, lds, t0, o0, w.part, ts, os).run();
  else Any(a, late, reinterpret_cast<typename Any::Lds&>(lds), t0, o0, w.part, ts, os).run();
}

// Parts of the long axis, added in order.  W: outputs per thread.
template <int W, class E>
__global__ __launch_bounds__(kMxThreads) void mm_join_kernel(MmArgs a, E ep) {
  const int64_t per = a.m / W, i = (int64_t)blockIdx.x * kMxThreads + threadIdx.x;
  if (i >= a.T * per) return;
  const int64_t t = i / per, o = (i - t * per) * W, step = a.T * a.m;
  const float* p = a.part + t * a.m + o;
  if constexpr (W == 4) {
    mxf4 v = *reinterpret_cast<const mxf4*>(p);
    for (int s = 1; s < a.splits; ++s) v += *reinterpret_cast<const mxf4*>(p + s * step);
    mm_store4(a.y, a.yt, t * a.ldy + o, mm_finish4(ep, t, o, v, 4), 4, a.wide);
  } else {
    float v = *p;
    for (int s = 1; s < a.splits; ++s) v += p[s * step];
    mm_store(a.y, a.yt, t * a.ldy + o, mm_finish(ep, t, o, v));
  }
}

template <class E>
hipError_t mm_join(const MmArgs& a, const E& ep, hipStream_t s) {
  const int64_t n = a.T * (a.m % 4 ? a.m : a.m / 4);
  const dim3 grid((unsigned)((n + kMxThreads - 1) / kMxThreads));
  if (a.m % 4) mm_join_kernel<1><<<grid, kMxThreads, 0, s>>>(a, ep);
  else mm_join_kernel<4><<<grid, kMxThreads, 0, s>>>(a, ep);
  return hipGetLastError();
}

template <int WT, int WO, int TT, int TO, int NB, class E>
hipError_t mm_tiles(const MmArgs& a, const E& ep, hipStream_t s) {
  constexpr int BT = 32 * TT * WT, BO = 32 * TO * WO;
  static_assert(BT == BO && (BT == 128 || BT == 256), "mm_plan's tiles");
  const int runs = (a.stages + kMmRun - 1) / kMmRun;
  mm_scales_kernel<BT, BO><<<dim3((unsigned)(a.gt + a.go), (unsigned)runs), kMxThreads, 0, s>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  mm_tile_kernel<WT, WO, TT, TO, NB><<<dim3((unsigned)(8 * a.per_xcd)), 64 * WT * WO, 0, s>>>(a, ep);
  e = hipGetLastError();
  return e != hipSuccess || a.splits == 1 ? e : mm_join(a, ep, s);
}

template <class E>
hipError_t mm_launch(const MmArgs& a, const E& ep, hipStream_t s) {
  if (a.tile == 256) return mm_tiles<2, 2, 4, 4, 2>(a, ep, s);
  // a compute unit that has one workgroup has LDS for a third stage
  // (65x8192x28672: 48 -> 44 us, 128: 50 -> 48.5)
  if (a.tile == 128 && a.gt * a.go * a.splits <= 256) return mm_tiles<2, 2, 2, 2, 3>(a, ep, s);
  if (a.tile == 128) return mm_tiles<2, 2, 2, 2, 2>(a, ep, s);
  if (a.T <= 16) return mm_rows<1>(a, ep, s);
  if (a.T <= 32) return mm_rows<2>(a, ep, s);
  if (a.T <= 64) return mm_rows<4>(a, ep, s);
  mm_simple_kernel<<<dim3((unsigned)(((a.m + 15) / 16) * ((a.T + 15) / 16))), 64, 0, s>>>(a, ep);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_matmul(const MmArgs& a, hipStream_t s) { return mm_launch(a, MmNoEpi{}, s); }
hipError_t launch_mx_linear(const MmArgs& a, const MmEpi& e, hipStream_t s) { return mm_launch(a, e, s); }

}  // namespace brq
