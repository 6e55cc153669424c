// Quantize rows to the microscaled 4-bit format and back (format: mx.h).
//
// Per block of 32: A = max |v|, scale 2^(floor(log2 A) - 2), codes of
// v / scale.  One pass, each value read once, the transform ahead of it in
// registers and lane exchanges.  Memory-bound: 8192x28672 bfloat16 in 124 us
// without a transform (4.8 TB/s; back: 116 us), 129 us with one of 128 (with
// eight values a lane, and so twice the exchanges, 193).
#include "mx_dev.h"

namespace brq {
namespace {

// N values per lane: 16 with a transform, else 8 (whole lines to a load).
template <int XT, int N>
__global__ __launch_bounds__(kMxThreads) void mx_quant_kernel(MxArgs a) {
  const int lane = threadIdx.x & 63;
  const uint64_t li = (uint64_t)blockIdx.x * kMxThreads + threadIdx.x;
  if (li >= a.lanes) return;  // whole blocks and whole transforms leave together
  int64_t row = 0, col = (int64_t)li * N;  // rows without a gap are one
  if (a.gap) mx_lane(a.lpr, N, li, &row, &col);
  float v[N];
#pragma unroll
  for (int q = 0; q < N / 8; ++q) mx_load8<XT>(a.x, row * a.ldx + col + 8 * q, *reinterpret_cast<float (*)[8]>(&v[8 * q]));
  if constexpr (N == 16) mx_rotate(v, a.signs, a.d, a.rnorm, (int)(col & (a.d - 1)), lane);
  uint32_t byte, w[N / 8];
  mx_round(v, w, &byte);
  if constexpr (N == 16) reinterpret_cast<uint2*>(a.codes)[li] = make_uint2(w[0], w[1]);
  else reinterpret_cast<uint32_t*>(a.codes)[li] = w[0];
  if ((lane & (32 / N - 1)) == 0) a.scales[li / (32 / N)] = (uint8_t)byte;
}

template <int YT>
__global__ __launch_bounds__(kMxThreads) void mx_dequant_kernel(MxArgs a) {
  const int lane = threadIdx.x & 63;
  const uint64_t li = (uint64_t)blockIdx.x * kMxThreads + threadIdx.x;
  if (li >= a.lanes) return;
  int64_t row = 0, col = (int64_t)li * kMxPerLane;
  if (a.gap || a.d) mx_lane(a.lpr, kMxPerLane, li, &row, &col);
  float v[8];
  mx_values8(reinterpret_cast<const uint32_t*>(a.codes)[li], a.scales[li >> 2], v);
  if (a.d) mx_unrotate(v, a.signs, a.d, a.rnorm, (int)(col & (a.d - 1)), lane);
  mx_store8<YT>(a.y, row * a.ldy + col, v);
}

}  // namespace

namespace {
template <int XT>
void mx_quant(const MxArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.lanes + kMxThreads - 1) / kMxThreads));
  if (a.per == 16) mx_quant_kernel<XT, 16><<<grid, kMxThreads, 0, s>>>(a);
  else mx_quant_kernel<XT, 8><<<grid, kMxThreads, 0, s>>>(a);
}
}  // namespace

hipError_t launch_mx_quant(const MxArgs& a, hipStream_t s) {
  if (a.xt == BRQ_F32) mx_quant<BRQ_F32>(a, s);
  else if (a.xt == BRQ_BF16) mx_quant<BRQ_BF16>(a, s);
  else mx_quant<BRQ_F16>(a, s);
  return hipGetLastError();
}

hipError_t launch_mx_dequant(const MxArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.lanes + kMxThreads - 1) / kMxThreads));
  if (a.yt == BRQ_F32) mx_dequant_kernel<BRQ_F32><<<grid, kMxThreads, 0, s>>>(a);
  else if (a.yt == BRQ_BF16) mx_dequant_kernel<BRQ_BF16><<<grid, kMxThreads, 0, s>>>(a);
  else mx_dequant_kernel<BRQ_F16><<<grid, kMxThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace brq
