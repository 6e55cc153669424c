// Product of two microscaled 4-bit matrices on the scaled matrix
// instructions (format: mx.h).
#include "mx_dev.h"

namespace brq {
namespace {

__device__ __forceinline__ void mm_store(void* y, int yt, int64_t off, float v) {
  if (yt == BRQ_F32) static_cast<float*>(y)[off] = v;
  else if (yt == BRQ_BF16) static_cast<uint16_t*>(y)[off] = (uint16_t)mx_bf16(v);
  else static_cast<uint16_t*>(y)[off] = (uint16_t)mx_f16(v);
}

// One wavefront per 16 x 16 outputs: lane l holds block l / 16 of a step of
// 128 values of row l % 16, of both operands, with the block's scale.
__global__ __launch_bounds__(64) void mm_simple_kernel(MmArgs a) {
  const int lane = threadIdx.x, lr = lane & 15, lg = lane >> 4;
  const int64_t t0 = (int64_t)blockIdx.y * 16, o0 = (int64_t)blockIdx.x * 16;
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
    if (t < a.T && vb) mm_store(a.y, a.yt, t * a.ldy + rb, acc[i]);
  }
}

}  // namespace

hipError_t launch_mx_matmul(const MmArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.m + 15) / 16), (unsigned)((a.T + 15) / 16));
  mm_simple_kernel<<<grid, 64, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace brq
