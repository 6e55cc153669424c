// Append to and read from the paged 4-bit key-value cache (layout: KvPage in
// mx.h).  A row is one head of one token, its D values on D / 16 lanes (append)
// or D / 8 (read); keys are the first half of the grid, values the second.
// Memory-bound for prompts, latency for single tokens: 8190 tokens of 8 heads
// of 128 are appended in 7.5 us without a transform and 11.6 with one, read in
// 10.8 and, with it undone, 14.6 (one launch after the other; under the
// profiler, like the figure of kv_rows, 13.5 with one and 11.4); 33 tokens in 3
// us each.
#include "mx_dev.h"

namespace brq {
namespace {

template <int T, int D>
__global__ __launch_bounds__(kMxThreads) void kv_append_kernel(KvArgs a) {
  constexpr int LPR = D / kKvPerLane, RUN = D / 16;  // lanes per row; dimensions of a run of the values' layout
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * (kMxThreads / LPR) + threadIdx.x / LPR;
  const int c = (int)(threadIdx.x % LPR) * kKvPerLane;
  int64_t tok;
  int h;
  kv_row((uint32_t)row, a.heads, &tok, &h);
  if (tok >= a.tokens) return;
  const bool val = blockIdx.y != 0;
  const int64_t slot = a.slots[tok];
  float v[16], sign[16];
  if (a.d) mx_signs(a.signs, c, sign);
  const void* x = val ? a.v : a.k;
  const int64_t at = tok * (val ? a.ldv : a.ldk) + (int64_t)h * D + c;
#pragma unroll
  for (int q = 0; q < 2; ++q) mx_load8<T>(x, at + 8 * q, *reinterpret_cast<float (*)[8]>(&v[8 * q]));
  if (slot < 0 || (slot >> a.lgP) >= a.pages) return;  // uniform over the row's lanes
  if (a.d) mx_rotate<D>(v, sign, a.rnorm, lane);
  uint32_t byte, w[2];
  mx_round(v, w, &byte);
  const KvPage pg{D, a.pg.P};
  uint8_t* pb = a.cache + ((slot >> a.lgP) * a.heads + h) * pg.bytes();
  const int t = (int)(slot & (a.pg.P - 1));
  if (!val) {
    *reinterpret_cast<uint2*>(pb + pg.kcode(t) + c / 2) = make_uint2(w[0], w[1]);
    if ((c & 31) == 0) pb[pg.kscale(t) + c / 32] = (uint8_t)byte;
    return;
  }
  uint8_t* d = pb + pg.vcode(t, c / RUN);  // runs are D / 8 bytes apart
  if constexpr (D == 64) {         // the lane holds four runs of four values
#pragma unroll
    for (int q = 0; q < 4; ++q) *reinterpret_cast<uint16_t*>(d + q * (D / 8)) = (uint16_t)(w[q / 2] >> (16 * (q & 1)));
  } else if constexpr (D == 128) {  // two of eight
    *reinterpret_cast<uint32_t*>(d) = w[0];
    *reinterpret_cast<uint32_t*>(d + D / 8) = w[1];
  } else {                          // one of sixteen
    *reinterpret_cast<uint2*>(d) = make_uint2(w[0], w[1]);
  }
  if ((c & 31) == 0) pb[pg.vscale(t, c / 32)] = (uint8_t)byte;
}

template <int T, int D>
__global__ __launch_bounds__(kMxThreads) void kv_read_kernel(KvArgs a) {
  const int lane = threadIdx.x & 63;
  constexpr uint32_t lpr = D / kMxPerLane;
  const uint64_t li = (uint64_t)blockIdx.x * kMxThreads + threadIdx.x;
  const int64_t row = (int64_t)(li / lpr);
  const int c = (int)(li % lpr) * kMxPerLane;
  int64_t tok;
  int h;
  kv_row((uint32_t)row, a.heads, &tok, &h);
  if (tok >= a.tokens) return;
  const bool val = blockIdx.y != 0;
  const int64_t slot = a.slots[tok];
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sign[8];
  if (a.d) mx_signs(a.signs, c, sign);
  if (slot >= 0 && (slot >> a.lgP) < a.pages) {  // uniform over the row's lanes
    const KvPage pg{D, a.pg.P};
    const uint8_t* pb = a.cache + ((slot >> a.lgP) * a.heads + h) * pg.bytes();
    const int t = (int)(slot & (a.pg.P - 1));
    uint32_t w;
    if (!val) {
      w = *reinterpret_cast<const uint32_t*>(pb + pg.kcode(t) + c / 2);
    } else if constexpr (D == 64) {
      w = *reinterpret_cast<const uint16_t*>(pb + pg.vcode(t, c / 4)) |
          (uint32_t) * reinterpret_cast<const uint16_t*>(pb + pg.vcode(t, c / 4 + 1)) << 16;
    } else {
      constexpr int run = D / 16;
      w = *reinterpret_cast<const uint32_t*>(pb + pg.vcode(t, c / run) + (c % run) / 2);
    }
    mx_values8(w, val ? pb[pg.vscale(t, c / 32)] : pb[pg.kscale(t) + c / 32], v);
    if (a.d) mx_unrotate<D>(v, sign, a.rnorm, lane);
  }
  if (val) mx_store8<T>(const_cast<void*>(a.v), tok * a.ldv + (int64_t)h * D + c, v);
  else mx_store8<T>(const_cast<void*>(a.k), tok * a.ldk + (int64_t)h * D + c, v);
}

template <int T, int D>
void kv_launch(const KvArgs& a, bool append, hipStream_t s) {
  const int64_t lanes = kv_rows(a.tokens, a.heads) * (D / (append ? kKvPerLane : kMxPerLane));
  const dim3 grid((unsigned)((lanes + kMxThreads - 1) / kMxThreads), 2);
  if (append) kv_append_kernel<T, D><<<grid, kMxThreads, 0, s>>>(a);
  else kv_read_kernel<T, D><<<grid, kMxThreads, 0, s>>>(a);
}
template <int T>
void kv_launch(const KvArgs& a, bool append, hipStream_t s) {
  if (a.pg.D == 64) kv_launch<T, 64>(a, append, s);
  else if (a.pg.D == 128) kv_launch<T, 128>(a, append, s);
  else kv_launch<T, 256>(a, append, s);
}
hipError_t kv_launch(const KvArgs& a, bool append, hipStream_t s) {
  if (a.t == BRQ_F32) kv_launch<BRQ_F32>(a, append, s);
  else if (a.t == BRQ_BF16) kv_launch<BRQ_BF16>(a, append, s);
  else kv_launch<BRQ_F16>(a, append, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const KvArgs& a, hipStream_t s) { return kv_launch(a, true, s); }
hipError_t launch_kv_read(const KvArgs& a, hipStream_t s) { return kv_launch(a, false, s); }

}  // namespace brq
