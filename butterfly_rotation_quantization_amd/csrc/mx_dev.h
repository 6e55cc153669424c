// Device helpers of the microscaled 4-bit kernels: loads and stores of eight
// values, lane exchanges, the fixed-order Hadamard transform, and rounding to
// and from the 4-bit format.
#pragma once

#include "mx.h"

namespace brq {

typedef float mxf2 __attribute__((ext_vector_type(2)));
typedef float mxf4 __attribute__((ext_vector_type(4)));
typedef float mxf16 __attribute__((ext_vector_type(16)));
typedef int mxi4 __attribute__((ext_vector_type(4)));
typedef int mxi8 __attribute__((ext_vector_type(8)));
typedef __bf16 mxb2 __attribute__((ext_vector_type(2)));
typedef __bf16 mxb8 __attribute__((ext_vector_type(8)));

// Eight consecutive values (16-byte aligned) of type t as float32.
template <int T>
__device__ __forceinline__ void mx_load8(const void* base, int64_t off, float (&v)[8]) {
  if constexpr (T == BRQ_F32) {
    const mxf4* p = reinterpret_cast<const mxf4*>(static_cast<const float*>(base) + off);
    const mxf4 a = p[0], b = p[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[e] = a[e];
      v[4 + e] = b[e];
    }
  } else {
    const uint4 r = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + off);
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (T == BRQ_BF16) {
        v[2 * e] = __uint_as_float(w[e] << 16);
        v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      } else {
        v[2 * e] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[e] & 0xffffu));
        v[2 * e + 1] = (float)__builtin_bit_cast(_Float16, (uint16_t)(w[e] >> 16));
      }
    }
  }
}

__device__ __forceinline__ uint32_t mx_bf16(float f) {  // nearest, ties to even
  return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)f);
}
__device__ __forceinline__ uint32_t mx_f16(float f) {
  return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)f);
}

template <int T>
__device__ __forceinline__ void mx_store8(void* base, int64_t off, const float (&v)[8]) {
  if constexpr (T == BRQ_F32) {
    mxf4* p = reinterpret_cast<mxf4*>(static_cast<float*>(base) + off);
    p[0] = mxf4{v[0], v[1], v[2], v[3]};
    p[1] = mxf4{v[4], v[5], v[6], v[7]};
  } else {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e] = T == BRQ_BF16 ? (mx_bf16(v[2 * e]) | (mx_bf16(v[2 * e + 1]) << 16))
                           : (mx_f16(v[2 * e]) | (mx_f16(v[2 * e + 1]) << 16));
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + off) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The value of lane (lane ^ X), X = 1, 2, 4, 8 (moves within a row of 16).
template <int CTRL>
__device__ __forceinline__ uint32_t mx_dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)x, CTRL, 0xf, 0xf, false);
}
template <int X>
__device__ __forceinline__ uint32_t mx_xor(uint32_t x) {
  static_assert(X == 1 || X == 2 || X == 4 || X == 8, "moves within 16 lanes");
  if constexpr (X == 1) return mx_dpp<0xb1>(x);       // swap neighbours
  else if constexpr (X == 2) return mx_dpp<0x4e>(x);  // swap pairs
  else if constexpr (X == 4) return (uint32_t)__builtin_amdgcn_ds_swizzle((int)x, 4 << 10 | 0x1f);  // no one move does
  else return mx_dpp<0x128>(x);                       // rotate 16 lanes by 8
}
template <int X>
__device__ __forceinline__ float mx_xorf(float x) {
  return __uint_as_float(mx_xor<X>(__float_as_uint(x)));
}

// One butterfly stage between lanes: the lower lane gets lo + hi, the upper
// one lo - hi, each one addition (the product with +-1 is exact).
template <int X, int N>
__device__ __forceinline__ void mx_stage(float (&v)[N], int lane) {
  if constexpr (X == 16) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const uint32_t u = __float_as_uint(v[e]);
      const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
      const float lo = __uint_as_float(r[0]), hi = __uint_as_float(r[1]);
      v[e] = (lane & 16) ? lo - hi : lo + hi;
    }
  } else {
    const float s = (lane & X) ? -1.0f : 1.0f;
#pragma unroll
    for (int e = 0; e < N; ++e) v[e] = fmaf(v[e], s, mx_xorf<X>(v[e]));
  }
}

// H_d v for the d / N lanes of a transform (d = 32..256, N = 8 or 16 values a
// lane), unnormalised: the additions in the order of strides 1, 2, 4, ..., d / 2.
template <int d, int N>
__device__ __forceinline__ void mx_hadamard(float (&v)[N], int lane) {
#pragma unroll
  for (int s = 1; s < N; s *= 2)
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (!(e & s)) {
        const float a = v[e], b = v[e + s];
        v[e] = a + b;
        v[e + s] = a - b;
      }
  mx_stage<1>(v, lane);
  if constexpr (d > 2 * N) mx_stage<2>(v, lane);
  if constexpr (d > 4 * N) mx_stage<4>(v, lane);
  if constexpr (d > 8 * N) mx_stage<8>(v, lane);
  if constexpr (d > 16 * N) mx_stage<16>(v, lane);
}

// The plan's signs at positions c .. of its d values (none: all 1).  Asked for
// before the values they go with, so that both loads travel together.
template <int N>
__device__ __forceinline__ void mx_signs(const float* signs, int c, float (&s)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) s[e] = 1.0f;
  if (signs)
#pragma unroll
    for (int q = 0; q < N / 8; ++q) mx_load8<BRQ_F32>(signs, c + 8 * q, *reinterpret_cast<float (*)[8]>(&s[8 * q]));
}

// The plan's transform of the lane's values: signs, additions, one product.
template <int d, int N>
__device__ __forceinline__ void mx_rotate(float (&v)[N], const float (&signs)[N], float rnorm, int lane) {
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] *= signs[e];
  mx_hadamard<d>(v, lane);
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] *= rnorm;
}
// Its inverse (the transform is symmetric): additions, product, signs.
template <int d>
__device__ __forceinline__ void mx_unrotate(float (&v)[8], const float (&signs)[8], float rnorm, int lane) {
  mx_hadamard<d>(v, lane);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= rnorm;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= signs[e];
}

// 2^(byte - 127); byte 0 is the subnormal 2^-127.  Byte 255, which stands for
// NaN, gives infinity's bits: of a scale the conversions read the exponent
// only, and take that one for NaN.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return __uint_as_float(byte ? byte << 23 : 0x400000u);
}

// Round the lane's N values (8 or 16): the codes, eight to a word (the first in
// the lowest half-byte), and the block's scale byte.  The block is the lane's
// aligned group of 32 / N lanes; magnitudes are compared as integers, which
// order NaN above infinity above every number.
template <int N>
__device__ __forceinline__ void mx_round(const float (&v)[N], uint32_t (&w)[N / 8], uint32_t* byte) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
  top = max(top, mx_xor<1>(top));
  if constexpr (N == 8) top = max(top, mx_xor<2>(top));
  const bool bad = top >= 0x7f800000u;
  const int b = (int)(top >> 23) - 2;  // floor(log2 A) - 2 + 127
  *byte = bad ? 255u : b > 0 ? (uint32_t)b : 0u;
  const float s = mx_scale(*byte);
#pragma unroll
  for (int q = 0; q < N / 8; ++q) {  // the conversion divides by the scale, rounds half to even and saturates
    uint32_t x = 0;
    x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(x, v[8 * q], v[8 * q + 1], s, 0);
    x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(x, v[8 * q + 2], v[8 * q + 3], s, 1);
    x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(x, v[8 * q + 4], v[8 * q + 5], s, 2);
    x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(x, v[8 * q + 6], v[8 * q + 7], s, 3);
    w[q] = bad ? 0u : x;
  }
}

// Eight codes times a block's scale.
__device__ __forceinline__ void mx_values8(uint32_t w, uint32_t byte, float (&v)[8]) {
  const float s = mx_scale(byte);
  const mxf2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0);
  const mxf2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
  const mxf2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2);
  const mxf2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
  v[0] = a[0]; v[1] = a[1]; v[2] = b[0]; v[3] = b[1];
  v[4] = c[0]; v[5] = c[1]; v[6] = d[0]; v[7] = d[1];
  if (byte == 255u) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(0x7fc00000u);
  }
}

}  // namespace brq
