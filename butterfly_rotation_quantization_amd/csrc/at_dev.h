// Device code shared by the attention kernels over the paged 4-bit cache
// (kv_attn.hip, kv_tree.hip): queries in pieces, the deal of tiles to
// workgroups, finished rows.
#pragma once

#include <type_traits>

#include "mx_dev.h"

namespace brq {
namespace {

__device__ __forceinline__ mxb2 at_pair(uint32_t w, float s, int byte) {
  switch (byte & 3) {
    case 0: return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0);
    case 1: return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1);
    case 2: return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2);
    default: return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3);
  }
}
__device__ __forceinline__ uint32_t at_bits(mxb2 x) { return __builtin_bit_cast(uint32_t, x); }

__device__ __forceinline__ float at_ror8(float x) { return __uint_as_float(mx_dpp<0x128>(__float_as_uint(x))); }
// maximum / sum over the four lanes of a column
__device__ __forceinline__ float at_colmax(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  const auto q = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ __forceinline__ float at_colsum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  const auto q = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

__device__ __forceinline__ void at_load8(int t, const void* p, int64_t off, float (&v)[8]) {
  if (t == BRQ_F32) mx_load8<BRQ_F32>(p, off, v);
  else if (t == BRQ_BF16) mx_load8<BRQ_BF16>(p, off, v);
  else mx_load8<BRQ_F16>(p, off, v);
}
__device__ __forceinline__ void at_store8(int t, void* p, int64_t off, const float (&v)[8]) {
  if (t == BRQ_F32) mx_store8<BRQ_F32>(p, off, v);
  else if (t == BRQ_BF16) mx_store8<BRQ_BF16>(p, off, v);
  else mx_store8<BRQ_F16>(p, off, v);
}

// Eight values of a head's finished output: normalise, undo the transform,
// store (m in units of log2).
template <int D>
__device__ __forceinline__ void at_finish(const AtArgs& a, int64_t b, int head, int c, int lane, float (&o)[8],
                                          float m, float l) {
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;  // a NaN sum stays one
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = l != 0.0f ? o[e] * inv : 0.0f;
  if (a.d) {
    float sign[8];
    mx_signs(a.signs, c, sign);
    mx_unrotate<D>(o, sign, a.rnorm, lane);
  }
  at_store8(a.qt, a.out, b * a.ldo + (int64_t)head * D + c, o);
  if (a.lse && c == 0)
    a.lse[b * a.q_heads + head] = l != 0.0f ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// A query enters the scores as eight 4-bit floating-point pieces, each the
// rounding of what the ones before it left.  The first has half the scale of
// the largest exponent of its block of 32, so that it lies below 4, where the
// format's steps are 1/2 and less, or 1: half of that is left, 4 of the next
// piece, whose scale is an eighth.  Together the pieces are within 2^-23 of the
// block's largest magnitude.  Products of 4-bit values lose nothing that a
// float32 sum would keep; those of 8-bit ones, which would need four pieces for
// 16 bits, drop what lies 14 bits below the largest of a block (a key's code of
// 6 beside one of 1/2: scores 2^-14 of the sum of magnitudes off).
// The eight values of a lane (its block is four lanes): the pieces' codes and
// scale bytes.
__device__ __forceinline__ void at_pieces(float (&v)[8], uint32_t (&piece)[8], uint32_t (&byte)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
  top = max(top, mx_xor<1>(top));
  top = max(top, mx_xor<2>(top));
  const int ex = (int)(top >> 23);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int x = ex - 1 - 3 * k;
    byte[k] = ex == 255 ? 255u : x > 0 ? (uint32_t)x : 0u;  // an infinity or a NaN: a NaN scale
    const float sc = mx_scale(byte[k]);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], sc, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], sc, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], sc, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], sc, 3);
    piece[k] = w;
    if (k < 7) {
      float back[8];
      mx_values8(w, byte[k], back);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] -= back[e];  // exact
    }
  }
}

// c += K Q, both 4-bit; the queries' scale is byte w of qs.
__device__ __forceinline__ mxf4 at_score(mxi8 K, mxi8 Q, mxf4 c, int ks, int qs, int w) {
  switch (w & 3) {
    case 0: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(K, Q, c, 4, 4, 0, ks, 0, qs);
    case 1: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(K, Q, c, 4, 4, 0, ks, 1, qs);
    case 2: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(K, Q, c, 4, 4, 0, ks, 2, qs);
    default: return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(K, Q, c, 4, 4, 0, ks, 3, qs);
  }
}

// Sum over the workgroup's threads (every thread gets it); scratch: one value
// per wavefront.
__device__ __forceinline__ int64_t at_block_sum(int64_t x, int64_t* scratch) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) x += __shfl_xor(x, d);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) scratch[threadIdx.x >> 6] = x;
  __syncthreads();
  int64_t s = 0;
#pragma unroll
  for (int w = 0; w < kAtWaves; ++w) s += scratch[w];
  return s;
}

// A workgroup's share of the places of all units: [pos, end), of which pos is
// in sequence b, whose first place is base.
struct AtShare {
  int64_t total, pos, end, base;
  int64_t b;
  int w, wgs;  // the workgroup's number among those that have places
};
struct AtShareLds {
  int64_t sums[kAtWaves];
  int found[1];
  int64_t found_base[1];
};
// `cost` gives a sequence's places for one of its `units`; `number` the
// workgroup's number among `wgs` that have places, or one beyond them.  False: none
// for this one.
template <class Cost, class Number>
__device__ __forceinline__ bool at_share(int64_t batch, int wgs, int units, AtShareLds& lds, Cost cost, Number number,
                                         AtShare& s) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  s.base = 0;
  // all tiles; with more sequences than threads, by a pass of its own
  if (batch > kAtThreads) {
    int64_t mine = 0;
    for (int64_t i = tid; i < batch; i += kAtThreads) mine += cost(i);
    s.total = at_block_sum(mine, lds.sums) * units;
  }
  for (int64_t i0 = 0;; i0 += kAtThreads) {
    const int64_t i = i0 + tid;
    const int64_t n = i < batch ? (int64_t)cost(i) * units : 0;
    int64_t x = n;  // inclusive sum over the threads before
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int64_t y = __shfl_up(x, d);
      if (lane >= d) x += y;
    }
    __syncthreads();
    if (lane == 63) lds.sums[wave] = x;
    __syncthreads();
    int64_t all = 0;
#pragma unroll
    for (int w = 0; w < kAtWaves; ++w) {
      if (w < wave) x += lds.sums[w];
      all += lds.sums[w];
    }
    if (i0 == 0) {
      if (batch <= kAtThreads) s.total = all;
      s.wgs = at_dealt(s.total, wgs);
      s.w = number(s.wgs);
      if (s.w >= s.wgs) return false;
      s.pos = at_start(s.w, s.total, s.wgs);
      s.end = at_start((int64_t)s.w + 1, s.total, s.wgs);
    }
    if (s.pos >= s.base + x - n && s.pos < s.base + x) {  // the sequence that has place pos
      lds.found[0] = (int)i;
      lds.found_base[0] = s.base + x - n;
    }
    __syncthreads();
    if (s.pos < s.base + all) break;  // it is one of these: pos < total
    s.base += all;
  }
  s.b = lds.found[0];
  s.base = lds.found_base[0];
  return true;
}

}  // namespace
}  // namespace brq
