// Quantize rows to the microscaled 4-bit format and back (format: mx.h).
//
// Per block of 32: A = max |v|, scale 2^(floor(log2 A) - 2), codes of
// v / scale.  One pass, each value read once, the transform ahead of it in
// registers and lane exchanges.  Memory-bound: 8192x28672 bfloat16 in 98 us
// without a transform and 100 with one of 128, back in 116 and, with it undone
// at eight values a lane, 146; 2048x4096 in 5.0 and 6.0, back in 5.7 and 7.0 (one
// launch after the other).  Under the profiler, 124 us either way; with eight
// values a lane, and so twice the exchanges, 193; with the size of the transform
// not known to the compiler and the signs asked for after the values, 129, and
// 9.2 us for 2048x4096, which then took 7.6.
#include "mx_dev.h"

namespace brq {
namespace {

// D: the transform, 0 for none.  N values per lane: 16 with a transform, else 8
// (whole lines to a load).
template <int XT, int D>
__global__ __launch_bounds__(kMxThreads) void mx_quant_kernel(MxArgs a) {
  constexpr int N = D ? 16 : 8;
  const int lane = threadIdx.x & 63;
  const uint64_t li = (uint64_t)blockIdx.x * kMxThreads + threadIdx.x;
  if (li >= a.lanes) return;  // whole blocks and whole transforms leave together
  int64_t row = 0, col = (int64_t)li * N;  // rows without a gap are one
  if (a.gap) mx_lane(a.lpr, N, li, &row, &col);
  float v[N], sign[N];
  if constexpr (D) mx_signs(a.signs, (int)(col & (D - 1)), sign);
#pragma unroll
  for (int q = 0; q < N / 8; ++q) mx_load8<XT>(a.x, row * a.ldx + col + 8 * q, *reinterpret_cast<float (*)[8]>(&v[8 * q]));
  if constexpr (D) mx_rotate<D>(v, sign, a.rnorm, lane);
  uint32_t byte, w[N / 8];
  mx_round(v, w, &byte);
  if constexpr (N == 16) reinterpret_cast<uint2*>(a.codes)[li] = make_uint2(w[0], w[1]);
  else reinterpret_cast<uint32_t*>(a.codes)[li] = w[0];
  if ((lane & (32 / N - 1)) == 0) a.scales[li / (32 / N)] = (uint8_t)byte;
}

template <int YT, int D>
__global__ __launch_bounds__(kMxThreads) void mx_dequant_kernel(MxArgs a) {
  const int lane = threadIdx.x & 63;
  const uint64_t li = (uint64_t)blockIdx.x * kMxThreads + threadIdx.x;
  if (li >= a.lanes) return;
  int64_t row = 0, col = (int64_t)li * kMxPerLane;
  if (a.gap) mx_lane(a.lpr, kMxPerLane, li, &row, &col);
  float v[8], sign[8];
  if constexpr (D) mx_signs(a.signs, (int)(col & (D - 1)), sign);
  mx_values8(reinterpret_cast<const uint32_t*>(a.codes)[li], a.scales[li >> 2], v);
  if constexpr (D) mx_unrotate<D>(v, sign, a.rnorm, lane);
  mx_store8<YT>(a.y, row * a.ldy + col, v);
}

template <int T, int D>
void mx_launch(const MxArgs& a, bool quantize, hipStream_t s) {
  const dim3 grid((unsigned)((a.lanes + kMxThreads - 1) / kMxThreads));
  if (quantize) mx_quant_kernel<T, D><<<grid, kMxThreads, 0, s>>>(a);
  else mx_dequant_kernel<T, D><<<grid, kMxThreads, 0, s>>>(a);
}
template <int T>
void mx_launch(const MxArgs& a, bool quantize, hipStream_t s) {
  if (a.d == 0) mx_launch<T, 0>(a, quantize, s);
  else if (a.d == 32) mx_launch<T, 32>(a, quantize, s);
  else if (a.d == 64) mx_launch<T, 64>(a, quantize, s);
  else if (a.d == 128) mx_launch<T, 128>(a, quantize, s);
  else mx_launch<T, 256>(a, quantize, s);
}
hipError_t mx_launch(const MxArgs& a, int type, bool quantize, hipStream_t s) {
  if (type == BRQ_F32) mx_launch<BRQ_F32>(a, quantize, s);
  else if (type == BRQ_BF16) mx_launch<BRQ_BF16>(a, quantize, s);
  else mx_launch<BRQ_F16>(a, quantize, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quant(const MxArgs& a, hipStream_t s) { return mx_launch(a, a.xt, true, s); }
hipError_t launch_mx_dequant(const MxArgs& a, hipStream_t s) { return mx_launch(a, a.yt, false, s); }

}  // namespace brq
