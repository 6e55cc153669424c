// Device code of the products of microscaled 4-bit matrices, shared by the
// plain product, the one with an epilogue (mx_matmul.hip) and the one grouped
// by expert (mx_grouped.hip): the chunks of the stream over a weight, the tiles
// through LDS, the epilogue.  Format: mx.h.
#pragma once

#include <type_traits>

#include "mx_dev.h"

namespace brq {
namespace {

__device__ __forceinline__ void mm_store(void* y, int yt, int64_t off, float v) {
  if (yt == BRQ_F32) static_cast<float*>(y)[off] = v;
  else if (yt == BRQ_BF16) static_cast<uint16_t*>(y)[off] = (uint16_t)mx_bf16(v);
  else static_cast<uint16_t*>(y)[off] = (uint16_t)mx_f16(v);
}

__device__ __forceinline__ void mm_store4(void* y, int yt, int64_t off, mxf4 v, int valid, bool wide) {
  if (wide && valid >= 4) {
    if (yt == BRQ_F32) {
      *reinterpret_cast<mxf4*>(static_cast<float*>(y) + off) = v;
    } else {
      uint2 w;
      w.x = yt == BRQ_BF16 ? (mx_bf16(v[0]) | mx_bf16(v[1]) << 16) : (mx_f16(v[0]) | mx_f16(v[1]) << 16);
      w.y = yt == BRQ_BF16 ? (mx_bf16(v[2]) | mx_bf16(v[3]) << 16) : (mx_f16(v[2]) | mx_f16(v[3]) << 16);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + off) = w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < valid) mm_store(y, yt, off + i, v[i]);
}

// ---- the epilogue

__device__ __forceinline__ float mm_read(const void* p, int t, int64_t i) {
  if (t == BRQ_F32) return static_cast<const float*>(p)[i];
  const uint16_t w = static_cast<const uint16_t*>(p)[i];
  return t == BRQ_BF16 ? __uint_as_float((uint32_t)w << 16) : (float)__builtin_bit_cast(_Float16, w);
}
// Four values, of which the first `valid` are there.
__device__ __forceinline__ mxf4 mm_read4(const void* p, int t, int64_t i, int valid, bool wide) {
  mxf4 v = {0.f, 0.f, 0.f, 0.f};
  if (wide && valid >= 4) {
    if (t == BRQ_F32) return *reinterpret_cast<const mxf4*>(static_cast<const float*>(p) + i);
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
    if (t == BRQ_BF16)
      return mxf4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                  __uint_as_float(w.y & 0xffff0000u)};
    return mxf4{(float)__builtin_bit_cast(_Float16, (uint16_t)(w.x & 0xffffu)),
                (float)__builtin_bit_cast(_Float16, (uint16_t)(w.x >> 16)),
                (float)__builtin_bit_cast(_Float16, (uint16_t)(w.y & 0xffffu)),
                (float)__builtin_bit_cast(_Float16, (uint16_t)(w.y >> 16))};
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (e < valid) v[e] = mm_read(p, t, i + e);
  return v;
}

// x times the logistic function of g, by its tail, which keeps the digits of
// large negative g; the exponential enters as two factors of half the exponent,
// since a single one would be zero below 2^-126, where the product is not yet.
__device__ __forceinline__ float mm_logistic(float x, float g) {
  const float h = __builtin_amdgcn_exp2f(-0.72134752044448170f * fabsf(g)), r = __builtin_amdgcn_rcpf(fmaf(h, h, 1.f));
  return g < 0.f ? x * r * h * h : x * r;
}
// x times the normal distribution function of x, by its tail too, mm_gelu_tail.  (The library's erfcf took more than twice the
// time: 2048x28672x8192 with bias and gelu 478 us, with this 349.)
__device__ __forceinline__ float mm_gelu(float x) {
  const float t = __builtin_amdgcn_rcpf(fmaf(fabsf(x), 0.35355339059327373f, 1.f));
  const float p = mm_gelu_tail(t);
  const float h = __builtin_amdgcn_exp2f(-0.36067376022224085f * (x * x)), q = 0.5f * p * t;
  return x < 0.f ? q * x * h * h : x * (1.f - q * h * h);
}
template <int N>
__device__ __forceinline__ void mm_act(int act, float (&v)[N]) {
  switch (act) {
    case BRQ_ACT_RELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];  // a NaN stays one
      return;
    case BRQ_ACT_GELU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = mm_gelu(v[i]);
      return;
    case BRQ_ACT_GELU_TANH:  // (1 + tanh(g)) / 2 is the logistic function of 2 g
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = mm_logistic(v[i], 1.5957691216057308f * (v[i] + 0.044715f * v[i] * v[i] * v[i]));
      return;
    case BRQ_ACT_SILU:
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = mm_logistic(v[i], v[i]);
      return;
    default: return;
  }
}
// The output of row t, column o from its sum.
__device__ __forceinline__ float mm_finish(const MmNoEpi&, int64_t, int64_t, float v) { return v; }
__device__ __forceinline__ float mm_finish(const MmEpi& e, int64_t t, int64_t o, float v) {
  const float mul = e.mul ? mm_read(e.mul, e.mt, t * e.ldm + o) : 1.f;  // asked for before what they wait for
  const float res = e.res ? mm_read(e.res, e.rt, t * e.ldr + o) : 0.f;
  float x[1] = {e.bias ? v + mm_read(e.bias, e.bt, o) : v};
  mm_act(e.act, x);
  if (e.mul) x[0] *= mul;
  return e.res ? x[0] + res : x[0];
}
// Four consecutive values of each of N rows `step` apart, those below T (past it the
// last one again); one decision on the type for all of them.
template <int N, class F>
__device__ __forceinline__ void mm_each(int64_t t, int step, int64_t T, F f) {
#pragma unroll
  for (int i = 0; i < N; ++i) f(i, t + i * step < T ? t + i * step : T - 1);
}
template <int N>
__device__ __forceinline__ void mm_read_rows(const void* p, int type, int64_t ld, int64_t t, int step, int64_t T, int64_t o,
                                             int valid, bool wide, mxf4 (&v)[N]) {
  if (!wide || valid < 4) {
    mm_each<N>(t, step, T, [&](int i, int64_t row) { v[i] = mm_read4(p, type, row * ld + o, valid, false); });
  } else if (type == BRQ_F32) {
    mm_each<N>(t, step, T, [&](int i, int64_t row) {
      v[i] = *reinterpret_cast<const mxf4*>(static_cast<const float*>(p) + row * ld + o);
    });
  } else {
    uint2 w[N];
    mm_each<N>(t, step, T, [&](int i, int64_t row) {
      w[i] = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + row * ld + o);
    });
    if (type == BRQ_BF16) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        v[i] = mxf4{__uint_as_float(w[i].x << 16), __uint_as_float(w[i].x & 0xffff0000u), __uint_as_float(w[i].y << 16),
                    __uint_as_float(w[i].y & 0xffff0000u)};
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        v[i] = mxf4{(float)__builtin_bit_cast(_Float16, (uint16_t)(w[i].x & 0xffffu)),
                    (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i].x >> 16)),
                    (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i].y & 0xffffu)),
                    (float)__builtin_bit_cast(_Float16, (uint16_t)(w[i].y >> 16))};
    }
  }
}
template <int N>
__device__ __forceinline__ void mm_store_rows(void* y, int yt, int64_t ldy, int64_t t, int step, int64_t T, int64_t o,
                                              int valid, bool wide, const mxf4 (&v)[N]) {
  if (!wide || valid < 4) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (t + i * step < T) mm_store4(y, yt, (t + i * step) * ldy + o, v[i], valid, false);
  } else if (yt == BRQ_F32) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (t + i * step < T) *reinterpret_cast<mxf4*>(static_cast<float*>(y) + (t + i * step) * ldy + o) = v[i];
  } else {
    uint2 w[N];
    if (yt == BRQ_BF16) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        w[i] = make_uint2(mx_bf16(v[i][0]) | mx_bf16(v[i][1]) << 16, mx_bf16(v[i][2]) | mx_bf16(v[i][3]) << 16);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        w[i] = make_uint2(mx_f16(v[i][0]) | mx_f16(v[i][1]) << 16, mx_f16(v[i][2]) | mx_f16(v[i][3]) << 16);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (t + i * step < T) *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + (t + i * step) * ldy + o) = w[i];
  }
}
// Such rows' epilogue: what they take from memory is asked for before anything
// waits for it, and every part is done for all of them under one condition.
template <int N, class EP>
struct MmFinish;
template <int N>
struct MmFinish<N, MmNoEpi> {
  __device__ __forceinline__ void ask(const MmNoEpi&, int64_t, int, int64_t, int64_t, int) {}
  __device__ __forceinline__ void apply(const MmNoEpi&, mxf4, mxf4 (&)[N]) const {}
};
template <int N>
struct MmFinish<N, MmEpi> {
  mxf4 mul[N], res[N];

  // rows below T, the first `valid` of four columns
  __device__ __forceinline__ void ask(const MmEpi& e, int64_t t, int step, int64_t T, int64_t o, int valid) {
    if (e.mul) mm_read_rows<N>(e.mul, e.mt, e.ldm, t, step, T, o, valid, e.wide, mul);
    if (e.res) mm_read_rows<N>(e.res, e.rt, e.ldr, t, step, T, o, valid, e.wide, res);
  }
  __device__ __forceinline__ void apply(const MmEpi& e, mxf4 bias, mxf4 (&v)[N]) const {
    float x[4 * N];
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) x[i] = v[i / 4][i & 3] + bias[i & 3];  // without one, -0
    mm_act(e.act, x);
    if (e.mul)
#pragma unroll
      for (int i = 0; i < 4 * N; ++i) x[i] *= mul[i / 4][i & 3];
    if (e.res)
#pragma unroll
      for (int i = 0; i < 4 * N; ++i) x[i] += res[i / 4][i & 3];
#pragma unroll
    for (int i = 0; i < 4 * N; ++i) v[i / 4][i & 3] = x[i];
  }
};
constexpr float kMmNoBias = -0.f;  // adds nothing, not even to a zero's sign
__device__ __forceinline__ mxf4 mm_finish4(const MmNoEpi&, int64_t, int64_t, mxf4 v, int) { return v; }
__device__ __forceinline__ mxf4 mm_finish4(const MmEpi& e, int64_t t, int64_t o, mxf4 v, int valid) {
  MmFinish<1, MmEpi> f;
  f.ask(e, t, 0, t + 1, o, valid);
  mxf4 x[1] = {v};
  f.apply(e, e.bias ? mm_read4(e.bias, e.bt, o, valid, e.wide) : mxf4{kMmNoBias, kMmNoBias, kMmNoBias, kMmNoBias}, x);
  return x[0];
}

// ---- few tokens: a stream over the weight

// 512 values of 16 rows: lane l holds blocks 4 s + l / 16 of row l % 16.
struct MmChunk {
  mxi4 c[4];
  uint4 s;  // the 16 scales of the row
};
// row: the lane's row of codes at its block l / 16; srow: of scales.  k: the
// chunk's first block, nb: blocks of a row.  Past the end of a row: zeros.
__device__ __forceinline__ void mm_chunk(MmChunk& f, const uint8_t* row, const uint8_t* srow, int64_t k, int64_t nb,
                                         int lg) {
  if (k + kMmChunk / kMxBlock <= nb) {
#pragma unroll
    for (int s = 0; s < 4; ++s) f.c[s] = *reinterpret_cast<const mxi4*>(row + (k + 4 * s) * 16);
    __builtin_memcpy(&f.s, srow + k, 16);
  } else {
    uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      f.c[s] = mxi4{0, 0, 0, 0};
      const int64_t b = k + 4 * s + lg;
      if (b < nb) {
        f.c[s] = *reinterpret_cast<const mxi4*>(row + (k + 4 * s) * 16);
        w[s] = (uint32_t)srow[b] << (8 * lg);
      }
    }
    f.s = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
// The scale of step s for this lane, in the lowest byte.
__device__ __forceinline__ int mm_scale_of(const uint4& v, int s, int sh) {
  const uint32_t w = s == 0 ? v.x : s == 1 ? v.y : s == 2 ? v.z : v.w;
  return (int)(w >> sh);
}

// 16 RT outputs, up to 16 TT tokens: outputs from o0 on, tokens t0 .. t0 + 16 TT - 1
// as far as there are a.T.  The workgroup's W wavefronts take chunks of the weight's
// rows in turn, 2 KB of each row in flight at a time, and join their sums in LDS:
// the weight is read once, in one launch.  Bound by memory: one token at
// 8192x28672 23 us, 5.4 TB/s of the weight.
template <int TT, int RT, int W>
struct MmRows {
  static constexpr int B = kMmChunk / kMxBlock;
  typedef float Sums[W][RT][TT][16][17];
  int lane, wave, lr, lg;
  const uint8_t *wrow[RT], *wsrow[RT];
  MmChunk w[RT];

  __device__ __forceinline__ MmRows() : lane(threadIdx.x & 63), wave(threadIdx.x >> 6), lr(lane & 15), lg(lane >> 4) {}

  // the first chunk of the weight's rows
  __device__ __forceinline__ void begin(const uint8_t* b, const uint8_t* bs, int64_t m, int64_t nb, int64_t o0) {
#pragma unroll
    for (int i = 0; i < RT; ++i) {  // rows past the end: the last one, not stored
      const int64_t o = o0 + 16 * i + lr < m ? o0 + 16 * i + lr : m - 1;
      wrow[i] = b + (o * nb + lg) * 16;
      wsrow[i] = bs + o * nb;
    }
    const int64_t k = (int64_t)wave * B;
    if (k < nb)
#pragma unroll
      for (int i = 0; i < RT; ++i) mm_chunk(w[i], wrow[i], wsrow[i], k, nb, lg);
  }
  // the sums of rows begun before, into LDS
  __device__ __forceinline__ void sum(const MmArgs& a, int64_t T, int64_t t0, Sums& sums) {
    const int sh = 8 * lg;
    const int64_t nb = a.n / kMxBlock;
    const uint8_t *xrow[TT], *xsrow[TT];
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      const int64_t t = t0 + 16 * j + lr < T ? t0 + 16 * j + lr : T - 1;
      xrow[j] = a.a + (t * nb + lg) * 16;
      xsrow[j] = a.as + t * nb;
    }
    mxf4 acc[RT][TT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < TT; ++j) acc[i][j] = mxf4{0.f, 0.f, 0.f, 0.f};
    int64_t k = (int64_t)wave * B;
    while (k < nb) {
      const int64_t next = k + W * B;
      MmChunk wn[RT], x[TT];
#pragma unroll
      for (int j = 0; j < TT; ++j) mm_chunk(x[j], xrow[j], xsrow[j], k, nb, lg);
      if (next < nb)
#pragma unroll
        for (int i = 0; i < RT; ++i) mm_chunk(wn[i], wrow[i], wsrow[i], next, nb, lg);
#pragma unroll
      for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int j = 0; j < TT; ++j) {
          const mxi8 A8 = {x[j].c[s][0], x[j].c[s][1], x[j].c[s][2], x[j].c[s][3], 0, 0, 0, 0};
          const int sx = mm_scale_of(x[j].s, s, sh);
#pragma unroll
          for (int i = 0; i < RT; ++i) {
            const mxi8 B8 = {w[i].c[s][0], w[i].c[s][1], w[i].c[s][2], w[i].c[s][3], 0, 0, 0, 0};
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(B8, A8, acc[i][j], 4, 4, 0,
                                                                         mm_scale_of(w[i].s, s, sh), 0, sx);
          }
        }
#pragma unroll
      for (int i = 0; i < RT; ++i) w[i] = wn[i];
      k = next;
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < TT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) sums[wave][i][j][lr][4 * lg + e] = acc[i][j][e];  // token lr, output 4 lg + e
  }
  // the wavefronts' sums joined and stored
  template <class E>
  __device__ __forceinline__ void finish(const MmArgs& a, const E& ep, int64_t T, int64_t t0, int64_t o0, const Sums& sums) {
    for (int e = threadIdx.x; e < 256 * TT * RT; e += 64 * W) {
      const int c = e & 15, i = (e >> 4) % RT, t = (e >> 4) / RT, j = t >> 4;  // a token's outputs on consecutive lanes
      float v = sums[0][i][j][t & 15][c];
#pragma unroll
      for (int u = 1; u < W; ++u) v += sums[u][i][j][t & 15][c];
      const int64_t o = o0 + 16 * i + c;
      if (t0 + t < T && o < a.m) mm_store(a.y, a.yt, (t0 + t) * a.ldy + o, mm_finish(ep, t0 + t, o, v));
    }
  }
};

// ---- tiles through LDS

// c += a b with byte SA of sa and SB of sb as the scales; c stays in the
// accumulation registers.  Written out because with all 256 of them in use the
// register allocator moved sums to and fro between the two files (90 moves in
// a stage of 128 products of 16 x 16 x 128).  The hardware orders these among themselves and
// after the loads of their operands; two wait states cover a move into an
// operand just before (the matrix unit is busy longer than that with the
// product before); mm_settle and mm_settled come before other reads of c.
template <int SA, int SB>
__device__ __forceinline__ void mm_mfma(mxi4 a, mxi4 b, mxf16& c, int sa, int sb) {
  asm volatile(
      "s_nop 1\n\tv_mfma_scale_f32_32x32x64_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[%5,%6,0] op_sel_hi:[%7,%8,0] cbsz:4 blgp:4"
      : "+a"(c)
      : "v"(a), "v"(b), "v"(sa), "v"(sb), "n"(SA & 1), "n"(SB & 1), "n"(SA >> 1), "n"(SB >> 1));
}
// More wait states than any product needs until its result can be read; then,
// for each sum, a statement that passes it on, behind which its reads stay (they
// are register moves, which a clobber of memory does not hold back).
__device__ __forceinline__ void mm_settle() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }
__device__ __forceinline__ void mm_settled(mxf16& c) { asm volatile("" : "+a"(c)); }
// byte ia of sa and byte ib of sb (constants once the loops are unrolled)
__device__ __forceinline__ void mm_step(mxi4 a, mxi4 b, mxf16& c, int sa, int ia, int sb, int ib) {
  switch ((ia & 3) * 4 + (ib & 3)) {
    case 0: return mm_mfma<0, 0>(a, b, c, sa, sb);
    case 1: return mm_mfma<0, 1>(a, b, c, sa, sb);
    case 2: return mm_mfma<0, 2>(a, b, c, sa, sb);
    case 3: return mm_mfma<0, 3>(a, b, c, sa, sb);
    case 4: return mm_mfma<1, 0>(a, b, c, sa, sb);
    case 5: return mm_mfma<1, 1>(a, b, c, sa, sb);
    case 6: return mm_mfma<1, 2>(a, b, c, sa, sb);
    case 7: return mm_mfma<1, 3>(a, b, c, sa, sb);
    case 8: return mm_mfma<2, 0>(a, b, c, sa, sb);
    case 9: return mm_mfma<2, 1>(a, b, c, sa, sb);
    case 10: return mm_mfma<2, 2>(a, b, c, sa, sb);
    case 11: return mm_mfma<2, 3>(a, b, c, sa, sb);
    case 12: return mm_mfma<3, 0>(a, b, c, sa, sb);
    case 13: return mm_mfma<3, 1>(a, b, c, sa, sb);
    case 14: return mm_mfma<3, 2>(a, b, c, sa, sb);
    default: return mm_mfma<3, 3>(a, b, c, sa, sb);
  }
}

constexpr int kMmKB = kMmK / 2;     // code bytes of a row in a stage
constexpr int kMmKS = kMmK / kMxBlock;

__device__ const uint4 kMmZero = {0u, 0u, 0u, 0u};

// 16 bytes per lane from p straight to LDS, lane l's to byte at + 16 l (at
// uniform over the wavefront).  Written out because the compiler, which takes any LDS
// read to depend on such a load, would wait for it before the next one; the
// kernel waits for vmcnt(0) and a barrier before it reads what was brought.
__device__ __forceinline__ void mm_to_lds(const void* p, uint32_t at) {
  uint32_t m0;  // written, not read
  asm volatile("s_mov_b32 %0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, off"
               : "=&{m0}"(m0)
               : "s"(at), "v"(p)
               : "memory");
}
// The same from base + (off + step), to byte at + to; off is left there.
template <int TO>
__device__ __forceinline__ void mm_to_lds(const void* base, uint32_t& off, uint32_t step, uint32_t at) {
  uint32_t m0;
  asm volatile("s_add_u32 %1, %4, %5\n\tv_add_u32 %0, %3, %0\n\tglobal_load_lds_dwordx4 %0, %2"
               : "+&v"(off), "=&{m0}"(m0)
               : "s"(base), "s"(step), "s"(at), "n"(TO)
               : "memory", "scc");
}

// Scales of one operand in the order the tiles take them: for each tile of R
// rows and each stage, as mm_scale_at says, so that a stage's are one run of
// 8 R bytes, fetched straight to LDS, in which a lane finds those of its tiles
// in one word.  Read from the rows they are 8 bytes out of a line
// for each row and stage (measured at 4096x8192x28672, rows read by the tile
// kernel: 15% of its time; this pass: 2%).  Rows and blocks past the end
// get zeros (2^-127, times codes of zero).  One workgroup: a tile, kMmRun
// stages.
constexpr int kMmRun = 4;
// Of rows row0 .. of a tile; `out`: the tile's image.
template <int R>
__device__ __forceinline__ void mm_scale_tile(const uint8_t* src, int64_t row0, int64_t rows, int64_t nb, int stages,
                                              int s0, uint8_t* out) {
  constexpr int W = kMmRun * kMmKS, LD = W + 4;
  __shared__ uint8_t lds[R][LD];
  const int tid = threadIdx.x;
  const int64_t k0 = (int64_t)s0 * kMmKS;
  if (nb % 4 == 0) {  // whole words (the base is aligned)
    for (int e = tid; e < R * (W / 4); e += kMxThreads) {
      const int r = e / (W / 4), c = 4 * (e % (W / 4));
      const int64_t row = row0 + r;
      *reinterpret_cast<uint32_t*>(&lds[r][c]) =
          row < rows && k0 + c < nb ? *reinterpret_cast<const uint32_t*>(src + row * nb + k0 + c) : 0u;
    }
  } else {
    for (int e = tid; e < R * W; e += kMxThreads) {
      const int r = e / W, c = e % W;
      const int64_t row = row0 + r;
      lds[r][c] = row < rows && k0 + c < nb ? src[row * nb + k0 + c] : 0;
    }
  }
  __syncthreads();
  for (int e = tid; e < kMmRun * kMmKS * 32; e += kMxThreads) {
    const int r = e & 31, c = e >> 5, s = s0 + c / kMmKS;  // block c of the run
    if (s >= stages) break;
    uint8_t* d = out + (int64_t)s * (8 * R) + mm_scale_at(R, c % kMmKS, r);
#pragma unroll
    for (int q = 0; q < R / 128; ++q) {
      uint32_t w = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) w |= (uint32_t)lds[r + 32 * (4 * q + j)][c] << (8 * j);
      reinterpret_cast<uint32_t*>(d)[q] = w;
    }
  }
}
// A kernel's epilogue, its second argument after ARGS, read from where the
// arguments are when it is wanted: taken at the kernel's beginning, as arguments
// are, it would hold registers that the addresses of the main loop need.
template <class EP>
struct MmLate;
template <>
struct MmLate<MmNoEpi> {
};
template <>
struct MmLate<MmEpi> {
  typedef const __attribute__((address_space(4))) char* Ptr;
  Ptr p;
  int64_t group;  // of a bias for each

  template <class ARGS>
  static __device__ __forceinline__ MmLate after(int64_t group = 0) {
    return {(Ptr)__builtin_amdgcn_kernarg_segment_ptr() + (sizeof(ARGS) + 7) / 8 * 8, group};
  }
  __device__ __forceinline__ MmEpi get(int64_t m) const {
    Ptr q = p;
    asm volatile("" : "+s"(q));
    MmEpi e;
    __builtin_memcpy(&e, (const void*)q, sizeof e);
    e.bias = gm_bias(e, group, m);
    return e;
  }
};

// Operands of a step of 128 values: two of 64, and the scales of the tiles.
template <int TT, int TO>
struct MmFrag {
  mxi4 x[2][TT], w[2][TO];
  int xs[2], ws[2];
};

// One workgroup's tile, WT x WO wavefronts of TT x TO tiles of 32 tokens x 32
// outputs; NB stages in LDS.  FULL: no row of the tile is past the end and rows are whole
// stages, so that a piece takes three instructions to fetch.
template <int WT, int WO, int TT, int TO, int NB, bool FULL, class EP>
struct MmTile {
  static constexpr int NTH = 64 * WT * WO;
  static constexpr int BT = 32 * TT * WT, BO = 32 * TO * WO, ROWS = BT + BO;
  static constexpr int NL = ROWS * (kMmKB / 16) / NTH;  // 16-byte pieces per thread and stage
  static constexpr int RS = NTH / 8;                    // rows between a thread's pieces
  static constexpr int NTT = BT / 32, NTO = BO / 32;
  static constexpr int NM = 2 * TT * TO;                // products of a step
  static constexpr int NG = 2 * (TT + TO);              // operand reads of a step
  static_assert(ROWS % NTH == 0 && BT % RS == 0 && BT % 64 == 0 && BO % 64 == 0, "whole rows per thread and wavefront");
  using Frag = MmFrag<TT, TO>;

  struct Lds {
    uint4 codes[NB][ROWS * 8];     // piece c of row r at mm_piece
    uint8_t scales[NB][ROWS * 8];  // mm_scale_at, tokens first
  };

  const MmArgs& a;
  const MmLate<EP> late;
  Lds& lds;
  const int tid, lane, wave, lr, lg, wt, wo;
  const int64_t t0, o0, nb, ld;
  const uint8_t *ts, *os;   // the tile's images of scales
  const int first, stages;  // the part's first stage, its number of stages
  // where the sums go: the output, or the part's float32 partial sums
  const bool whole;
  void* y;
  int yt;
  int64_t ldy;
  bool wide;
  // The thread's LDS slots: row pr + j RS, piece pc of the row.  Rows past the
  // end repeat the last one (their products are not stored).
  const int pr, pc, lt, lo;
  const uint8_t *ab, *bb;
  const uint32_t base, at;  // LDS addresses: of the workgroup, of the wavefront's first piece
  uint32_t off0;
  mxf16 acc[TO][TT];
  mxf4 bias;  // of the lane's four outputs

  __device__ __forceinline__ MmTile(const MmArgs& a_, const MmLate<EP>& e, Lds& l, int64_t t0_, int64_t o0_, int part,
                                    const uint8_t* ts_, const uint8_t* os_)
      : a(a_), late(e), lds(l), tid(threadIdx.x), lane(tid & 63), wave(tid >> 6), lr(lane & 31), lg(lane >> 5), wt(wave % WT),
        wo(wave / WT), t0(t0_), o0(o0_), nb(a_.n / kMxBlock), ld(a_.n / 2),
        ts(ts_), os(os_),
        first(part * a_.per), stages(a_.stages - first < a_.per ? a_.stages - first : a_.per), whole(a_.splits == 1), pr(tid >> 3), pc((tid & 7) ^ (pr >> 1 & 7)),
        lt((int)(a_.T - t0_ < BT ? a_.T - t0_ : BT) - 1), lo((int)(a_.m - o0_ < BO ? a_.m - o0_ : BO) - 1),
        base((uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) void*)&l)),
        at(__builtin_amdgcn_readfirstlane(base + 16 * (tid & ~63))) {
    y = whole ? a.y : a.part + (int64_t)part * a.T * a.m;
    yt = whole ? a.yt : (int)BRQ_F32;
    ldy = whole ? a.ldy : a.m;
    wide = whole ? a.wide != 0 : a.m % 4 == 0;
    ab = a.a + t0 * ld;
    bb = a.b + o0 * ld;
    off0 = (uint32_t)(pr * (int)ld + 16 * pc) - (uint32_t)(RS * (int)ld);
  }

  // Where the pieces of stage s come from.  Past the end of a row (the ragged
  // last stage, stages that do not exist) zeros are fetched instead; with FULL
  // only whole stages exist, and the last one is fetched again after it.
  struct Source {
    const uint8_t *x, *w;
    unsigned ld;
    int row;
    uint32_t off;
  };
  __device__ __forceinline__ Source source(int s) const {
    Source f;
    if constexpr (FULL) {
      const int64_t kb = (int64_t)(first + (s < stages ? s : stages - 1)) * kMmKB;
      f.x = ab + kb;
      f.w = bb + kb;
      f.ld = (unsigned)(RS * (int)ld);
      f.row = 0;
    } else {
      const int64_t kb = (int64_t)(first + s) * kMmKB + 16 * pc;
      const bool in = kb < ld;
      f.x = in ? ab + kb : reinterpret_cast<const uint8_t*>(&kMmZero);
      f.w = in ? bb + kb : reinterpret_cast<const uint8_t*>(&kMmZero);
      f.ld = in ? (unsigned)ld : 0u;
      f.row = pr;
      asm volatile("" : "+v"(f.row));  // offsets are computed at each use, or NL of them would be kept
    }
    f.off = off0;
    return f;
  }
  template <int BUF, int J>
  __device__ __forceinline__ void fetch(Source& f) const {
    constexpr int to = (int)sizeof(lds.codes[0]) * BUF + J * NTH * 16;
    if constexpr (FULL) {
      if constexpr (J == BT / RS) f.off = off0;
      mm_to_lds<to>(J * RS < BT ? f.x : f.w, f.off, f.ld, at);
    } else {  // row < 256 and ld < 2^23: a 24-bit product
      const int r = J * RS < BT ? f.row + J * RS : f.row + J * RS - BT, last = J * RS < BT ? lt : lo;
      mm_to_lds((J * RS < BT ? f.x : f.w) + __umul24((unsigned)(r < last ? r : last), f.ld), at + to);
    }
  }
  // Scales of stage s, from their image (mm_scales_kernel): the wavefronts
  // bring 1 KB each, in turn from the start when there are fewer pieces.
  template <int BUF>
  __device__ __forceinline__ void fetch_scales(int s) const {
    constexpr int from = (int)sizeof(lds.codes) + BUF * (int)sizeof(lds.scales[0]);
    const int piece = __builtin_amdgcn_readfirstlane(wave % (8 * ROWS / 1024)) * 1024;
    const int64_t st = first + (s < stages ? s : stages - 1);
    const uint8_t* g = piece < 8 * BT ? ts + st * (8 * BT) + piece : os + st * (8 * BO) + (piece - 8 * BT);
    mm_to_lds(g + 16 * lane, base + from + piece);
  }
  template <int E>  // operand E of step k2: the first 64 values, tokens first, then the second
  __device__ __forceinline__ void read(Frag& f, int buf, int k2) const {
    constexpr int u = E / (TT + TO), e = E % (TT + TO);
    const int c = 4 * k2 + 2 * u + lg;
    if constexpr (e < TT) f.x[u][e] = *reinterpret_cast<const mxi4*>(&lds.codes[buf][mm_piece(32 * (TT * wt + e) + lr, c)]);
    else f.w[u][e - TT] = *reinterpret_cast<const mxi4*>(&lds.codes[buf][mm_piece(BT + 32 * (TO * wo + e - TT) + lr, c)]);
  }
  __device__ __forceinline__ void read_scales(Frag& f, int buf, int k2) const {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int at = (4 * k2 + 2 * u + lg) * 32 + lr;
      const uint8_t* xq = &lds.scales[buf][at * NTT + TT * wt];
      const uint8_t* wq = &lds.scales[buf][8 * BT + at * NTO + TO * wo];
      f.xs[u] = TT == 4 ? *reinterpret_cast<const int*>(xq) : *reinterpret_cast<const uint16_t*>(xq);
      f.ws[u] = TO == 4 ? *reinterpret_cast<const int*>(wq) : *reinterpret_cast<const uint16_t*>(wq);
    }
  }

  // A stage's first step: the products of f, and spread between them, so that
  // the matrix unit is not left waiting for this wavefront's next issue, the
  // reads of g, the operands of the second step.
  template <int BUF, int X>
  __device__ __forceinline__ void first_step(const Frag& f, Frag& g) {
    if constexpr (X < NM) {
      constexpr int e0 = X * NG / NM, e1 = (X + 1) * NG / NM;
      multiply<X>(f);
      if constexpr (e1 > e0) read<e0>(g, BUF, 1);
      if constexpr (e1 > e0 + 1) read<e0 + 1>(g, BUF, 1);
      static_assert(e1 <= e0 + 2, "reads per product");
      __builtin_amdgcn_sched_barrier(0);
      first_step<BUF, X + 1>(f, g);
    }
  }
  // Its second step: the products of g; between them, the pieces of stage
  // s + NB into buffer BUF; half way, once the next stage has arrived (all
  // but this step's fetches so far), the reads of f, the operands of its first
  // step.  Waiting this late leaves a fetch 3/4 of a stage at least (half
  // way through the stage, with the reads spread over the step: 488 us where
  // this took 473 at 4096x8192x28672).
  template <int BUF, int X>
  __device__ __forceinline__ void second_step(const Frag& g, Frag& f, Source& src) {
    if constexpr (X < NM) {
      constexpr int H = NM / 2, Y = X < H ? 0 : X - H;
      constexpr int e0 = Y * NG / H, e1 = X < H ? 0 : (Y + 1) * NG / H;
      constexpr int j0 = X * NL / NM, j1 = (X + 1) * NL / NM;
      constexpr int next = (BUF + 1) % NB;
      if constexpr (X == H) {
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NB - 2) * (1 + NL) + 1 + NL / 2) : "memory");
        __syncthreads();
        read_scales(f, next, 0);
      }
      multiply<X>(g);
      if constexpr (e1 > e0) read<e0>(f, next, 0);
      if constexpr (e1 > e0 + 1) read<e0 + 1>(f, next, 0);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (j1 > j0) fetch<BUF, j0>(src);
      if constexpr (j1 > j0 + 1) fetch<BUF, j0 + 1>(src);
      static_assert(j1 <= j0 + 2 && e1 <= e0 + 2 && NL % 2 == 0, "pieces and reads per product");
      __builtin_amdgcn_sched_barrier(0);
      second_step<BUF, X + 1>(g, f, src);
    }
  }
  template <int X>
  __device__ __forceinline__ void multiply(const Frag& f) {
    constexpr int u = X / (TT * TO), i = X % (TT * TO) / TT, j = X % TT;
    mm_step(f.w[u][i], f.x[u][j], acc[i][j], f.ws[u], i, f.xs[u], j);
  }
  template <int BUF, int J>
  __device__ __forceinline__ void fetch_all(Source& f) const {
    if constexpr (J < NL) {
      fetch<BUF, J>(f);
      fetch_all<BUF, J + 1>(f);
    }
  }
  // The first NB stages, into their buffers.
  template <int BUF>
  __device__ __forceinline__ void begin(Source& src) const {
    if constexpr (BUF < NB) {
      src = source(BUF);
      fetch_scales<BUF>(BUF);
      fetch_all<BUF, 0>(src);
      begin<BUF + 1>(src);
    }
  }
  template <int E>
  __device__ __forceinline__ void read_all(Frag& f, int buf, int k2) const {
    if constexpr (E < NG) {
      read<E>(f, buf, k2);
      read_all<E + 1>(f, buf, k2);
    }
  }

  // Stage s, in buffer BUF, which is free for stage s + NB once every wavefront
  // has its second step's operands.
  template <int BUF>
  __device__ __forceinline__ void stage(int s, Frag& f0, Frag& f1, Source& src) {
    read_scales(f1, BUF, 1);
    __builtin_amdgcn_sched_barrier(0);
    first_step<BUF, 0>(f0, f1);
    __syncthreads();
    src = source(s + NB);
    fetch_scales<BUF>(s + NB);
    __builtin_amdgcn_sched_barrier(0);
    second_step<BUF, 0>(f1, f0, src);
  }

  __device__ __forceinline__ void run() {
#pragma unroll
    for (int i = 0; i < TO; ++i)
#pragma unroll
      for (int j = 0; j < TT; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;
    Source src;
    begin<0>(src);
    // all but the first stage may be on their way still
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NB - 1) * (1 + NL)) : "memory");
    __syncthreads();
    Frag f0, f1;
    read_scales(f0, 0, 0);
    read_all<0>(f0, 0, 0);
    int s = 0;
    for (; s + NB <= stages; s += NB) {
      stage<0>(s, f0, f1, src);
      stage<1>(s + 1, f0, f1, src);
      if constexpr (NB > 2) stage<2>(s + 2, f0, f1, src);
    }
    if (s < stages) stage<0>(s, f0, f1, src);
    if constexpr (NB > 2) {
      if (s + 1 < stages) stage<1>(s + 1, f0, f1, src);
    }
    mm_settle();
#pragma unroll
    for (int i = 0; i < TO; ++i)
#pragma unroll
      for (int j = 0; j < TT; ++j) mm_settled(acc[i][j]);
    // LDS is about to hold the sums: the last pieces, fetched for no stage,
    // have to be in it before, and every wavefront's reads done
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    EP ep;
    if constexpr (!std::is_same<EP, MmNoEpi>::value) {
      ep = late.get(a.m);
      const int64_t o = o0 + 32 * TO * wo + 4 * (lane % (8 * TO)), left = a.m - o;
      bias = mxf4{kMmNoBias, kMmNoBias, kMmNoBias, kMmNoBias};
      if (ep.bias && left > 0) bias = mm_read4(ep.bias, ep.bt, o, left < 4 ? (int)left : 4, ep.wide);
    }
    store<0>(ep);
  }

  // The sums of 32 tokens at a time through the wavefront's part of LDS, so
  // that a row's outputs leave in runs of 128 TO bytes and more, by code small
  // enough to stay in the instruction cache (one store a register, unrolled,
  // cost 25 us of fetching instructions).
  template <int J>
  __device__ __forceinline__ void store(const EP& ep) {
    if constexpr (J < TT) {
      constexpr int LD = 32 * TO + 4, LPR = 8 * TO;  // floats a row, lanes a row
      static_assert(32 * LD * 4 * WT * WO <= (int)sizeof(Lds), "sums of 32 tokens of every wavefront");
      float* my = reinterpret_cast<float*>(&lds) + wave * (32 * LD);
#pragma unroll
      for (int i = 0; i < TO; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e)  // D: outputs 8 e + 4 lg .. + 3 of tile i, token lr of tile J
          *reinterpret_cast<mxf4*>(&my[lr * LD + 32 * i + 8 * e + 4 * lg]) =
              mxf4{acc[i][J][4 * e], acc[i][J][4 * e + 1], acc[i][J][4 * e + 2], acc[i][J][4 * e + 3]};
      __builtin_amdgcn_wave_barrier();
      const int64_t o = o0 + 32 * TO * wo + 4 * (lane % LPR), left = a.m - o;
      const int64_t tj = t0 + 32 * (TT * wt + J);
      const int valid = left < 4 ? (int)left : 4;
      // four rows at a time, whose operands travel together
      constexpr int N = 4, S = 64 / LPR;
#pragma unroll 1
      for (int r = lane / LPR; r < 32; r += N * S) {
        if (tj + r >= a.T || left <= 0) break;
        MmFinish<N, EP> f;
        if (whole) f.ask(ep, tj + r, S, a.T, o, valid);
        mxf4 v[N];
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = *reinterpret_cast<const mxf4*>(&my[(r + i * S) * LD + 4 * (lane % LPR)]);
        if (whole) f.apply(ep, bias, v);
        mm_store_rows<N>(y, yt, ldy, tj + r, S, a.T, o, valid, wide, v);
      }
      __builtin_amdgcn_wave_barrier();
      store<J + 1>(ep);
    }
  }
};

}  // namespace
}  // namespace brq
