// Append to and read from the paged 4-bit key-value cache (layout: KvPage in
// mx.h).  A row is one head of one token, its D values on D / 8 lanes; keys
// are rows [0, R), values rows [R, 2R), R = tokens * heads.
#include "mx_dev.h"

namespace brq {
namespace {

template <int T>
__global__ __launch_bounds__(kMxThreads) void kv_append_kernel(KvArgs a) {
  const int D = a.pg.D, lane = threadIdx.x & 63;
  const uint32_t lpr = (uint32_t)D / kMxPerLane;
  const uint64_t li = (uint64_t)blockIdx.x * kMxThreads + threadIdx.x;
  const int64_t row = (int64_t)(li / lpr);
  const int c = (int)(li % lpr) * kMxPerLane;
  const int64_t rows = a.tokens * a.heads;
  if (row >= rows) return;
  const bool val = blockIdx.y != 0;
  const int64_t tok = row / a.heads;
  const int h = (int)(row - tok * a.heads);
  const int64_t slot = a.slots[tok];
  if (slot < 0 || (slot >> a.lgP) >= a.pages) return;  // uniform over the row's lanes
  float v[8];
  if (val) mx_load8<T>(a.v, tok * a.ldv + (int64_t)h * D + c, v);
  else mx_load8<T>(a.k, tok * a.ldk + (int64_t)h * D + c, v);
  if (a.d) mx_rotate(v, a.signs, a.d, a.rnorm, c, lane);
  uint32_t byte;
  const uint32_t w = mx_round8(v, &byte);
  uint8_t* pb = a.cache + ((slot >> a.lgP) * a.heads + h) * a.pg.bytes();
  const int t = (int)(slot & (a.pg.P - 1));
  if (!val) {
    *reinterpret_cast<uint32_t*>(pb + a.pg.kcode(t) + c / 2) = w;
    if ((c & 31) == 0) pb[a.pg.kscale(t) + c / 32] = (uint8_t)byte;
    return;
  }
  if (D == 64) {  // the lane holds two runs of four values
    *reinterpret_cast<uint16_t*>(pb + a.pg.vcode(t, c / 4)) = (uint16_t)w;
    *reinterpret_cast<uint16_t*>(pb + a.pg.vcode(t, c / 4 + 1)) = (uint16_t)(w >> 16);
  } else {        // one run of eight, or half a run of sixteen
    const int run = D / 16;
    *reinterpret_cast<uint32_t*>(pb + a.pg.vcode(t, c / run) + (c % run) / 2) = w;
  }
  if ((c & 31) == 0) pb[a.pg.vscale(t, c / 32)] = (uint8_t)byte;
}

template <int T>
__global__ __launch_bounds__(kMxThreads) void kv_read_kernel(KvArgs a) {
  const int D = a.pg.D, lane = threadIdx.x & 63;
  const uint32_t lpr = (uint32_t)D / kMxPerLane;
  const uint64_t li = (uint64_t)blockIdx.x * kMxThreads + threadIdx.x;
  const int64_t row = (int64_t)(li / lpr);
  const int c = (int)(li % lpr) * kMxPerLane;
  const int64_t rows = a.tokens * a.heads;
  if (row >= rows) return;
  const bool val = blockIdx.y != 0;
  const int64_t tok = row / a.heads;
  const int h = (int)(row - tok * a.heads);
  const int64_t slot = a.slots[tok];
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (slot >= 0 && (slot >> a.lgP) < a.pages) {  // uniform over the row's lanes
    const uint8_t* pb = a.cache + ((slot >> a.lgP) * a.heads + h) * a.pg.bytes();
    const int t = (int)(slot & (a.pg.P - 1));
    uint32_t w;
    if (!val) {
      w = *reinterpret_cast<const uint32_t*>(pb + a.pg.kcode(t) + c / 2);
    } else if (D == 64) {
      w = *reinterpret_cast<const uint16_t*>(pb + a.pg.vcode(t, c / 4)) |
          (uint32_t) * reinterpret_cast<const uint16_t*>(pb + a.pg.vcode(t, c / 4 + 1)) << 16;
    } else {
      const int run = D / 16;
      w = *reinterpret_cast<const uint32_t*>(pb + a.pg.vcode(t, c / run) + (c % run) / 2);
    }
    mx_values8(w, val ? pb[a.pg.vscale(t, c / 32)] : pb[a.pg.kscale(t) + c / 32], v);
    if (a.d) mx_unrotate(v, a.signs, a.d, a.rnorm, c, lane);
  }
  if (val) mx_store8<T>(const_cast<void*>(a.v), tok * a.ldv + (int64_t)h * D + c, v);
  else mx_store8<T>(const_cast<void*>(a.k), tok * a.ldk + (int64_t)h * D + c, v);
}

dim3 kv_grid(const KvArgs& a) {
  const int64_t lanes = a.tokens * a.heads * (a.pg.D / kMxPerLane);
  return dim3((unsigned)((lanes + kMxThreads - 1) / kMxThreads), 2);
}

}  // namespace

hipError_t launch_kv_append(const KvArgs& a, hipStream_t s) {
  if (a.t == BRQ_F32) kv_append_kernel<BRQ_F32><<<kv_grid(a), kMxThreads, 0, s>>>(a);
  else if (a.t == BRQ_BF16) kv_append_kernel<BRQ_BF16><<<kv_grid(a), kMxThreads, 0, s>>>(a);
  else kv_append_kernel<BRQ_F16><<<kv_grid(a), kMxThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvArgs& a, hipStream_t s) {
  if (a.t == BRQ_F32) kv_read_kernel<BRQ_F32><<<kv_grid(a), kMxThreads, 0, s>>>(a);
  else if (a.t == BRQ_BF16) kv_read_kernel<BRQ_BF16><<<kv_grid(a), kMxThreads, 0, s>>>(a);
  else kv_read_kernel<BRQ_F16><<<kv_grid(a), kMxThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace brq
