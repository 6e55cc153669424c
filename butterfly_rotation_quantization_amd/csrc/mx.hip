// Quantize rows to the microscaled 4-bit format and back (format: mx.h).
//
// Per block of 32: A = max |v|, scale 2^(floor(log2 A) - 2), codes of
// v / scale.  Memory-bound: one pass, each value read once; the transform
// ahead of it stays in registers and lane exchanges.
#include "mx_dev.h"

namespace brq {
namespace {

template <int XT>
__global__ __launch_bounds__(kMxThreads) void mx_quant_kernel(MxArgs a) {
  const int lane = threadIdx.x & 63;
  const uint64_t li = (uint64_t)blockIdx.x * kMxThreads + threadIdx.x;
  if (li >= a.lanes) return;  // whole blocks and whole transforms leave together
  int64_t row, col;
  mx_lane(a.lpr, li, &row, &col);
  float v[8];
  mx_load8<XT>(a.x, row * a.ldx + col, v);
  if (a.d) mx_rotate(v, a.signs, a.d, a.rnorm, (int)(col & (a.d - 1)), lane);
  uint32_t byte;
  const uint32_t w = mx_round8(v, &byte);
  reinterpret_cast<uint32_t*>(a.codes)[li] = w;
  if ((lane & 3) == 0) a.scales[li >> 2] = (uint8_t)byte;
}

template <int YT>
__global__ __launch_bounds__(kMxThreads) void mx_dequant_kernel(MxArgs a) {
  const int lane = threadIdx.x & 63;
  const uint64_t li = (uint64_t)blockIdx.x * kMxThreads + threadIdx.x;
  if (li >= a.lanes) return;
  int64_t row, col;
  mx_lane(a.lpr, li, &row, &col);
  float v[8];
  mx_values8(reinterpret_cast<const uint32_t*>(a.codes)[li], a.scales[li >> 2], v);
  if (a.d) mx_unrotate(v, a.signs, a.d, a.rnorm, (int)(col & (a.d - 1)), lane);
  mx_store8<YT>(a.y, row * a.ldy + col, v);
}

}  // namespace

hipError_t launch_mx_quant(const MxArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.lanes + kMxThreads - 1) / kMxThreads));
  if (a.xt == BRQ_F32) mx_quant_kernel<BRQ_F32><<<grid, kMxThreads, 0, s>>>(a);
  else if (a.xt == BRQ_BF16) mx_quant_kernel<BRQ_BF16><<<grid, kMxThreads, 0, s>>>(a);
  else mx_quant_kernel<BRQ_F16><<<grid, kMxThreads, 0, s>>>(a);
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
