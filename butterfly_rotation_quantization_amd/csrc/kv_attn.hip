// Attention of one new token per sequence over the paged 4-bit cache
// (layout: KvPage in mx.h).
//
// Per key-value head the scores and the output are products on the bfloat16
// matrix instructions, S^T = K Q^T and O^T = V^T P^T, with the query heads of
// the group as columns.  Codes times their scale are exact in bfloat16; each
// query and each probability enters as a pair of bfloat16 (its rounding and
// the rest), the pair in columns c and c + 8, so products keep 16 bits and
// more of them; sums, maxima and normalisers are float32.
//
// Lane l = 16 g + c of a wavefront: of 16 keys x D it holds key c, dimensions
// [g D/4, (g + 1) D/4) as the A operand of the scores; the scores come out as
// column c, keys 4 g + i, which is where the B operand of O^T wants the
// probabilities when the values' A operand takes keys 4 g + i as well: nothing
// moves between lanes in between.  The values of four keys lie together in the
// cache for that reason.
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
__device__ __forceinline__ void at_finish(const AtArgs& a, int64_t b, int head, int c, int lane, float (&o)[8],
                                          float m, float l) {
  const float inv = l != 0.0f ? 1.0f / l : 0.0f;  // a NaN sum stays one
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = l != 0.0f ? o[e] * inv : 0.0f;
  if (a.d) mx_unrotate(o, a.signs, a.d, a.rnorm, c, lane);
  at_store8(a.qt, a.out, b * a.ldo + (int64_t)head * a.pg.D + c, o);
  if (a.lse && c == 0)
    a.lse[b * a.q_heads + head] = l != 0.0f ? (m + __log2f(l)) * 0.69314718055994531f : -INFINITY;
}

// Tokens of sequence b that the table has room for.
__device__ __forceinline__ int at_length(const AtArgs& a, int64_t b) {
  const int n = a.lens[b];
  return n < 0 ? 0 : (n < a.cap ? n : a.cap);
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

// One workgroup: its share of the tiles of all units (or, without a deal, the
// unit of its number); its wavefronts take 32 keys at a time in turn.
template <int D, int NT>
__global__ __launch_bounds__(kAtThreads, at_workgroups(D, NT) / 256) void at_kernel(AtArgs a) {
  constexpr int KW = D / 32;          // words of codes a lane holds per key (of the scores) or four keys (values)
  constexpr int NS = D / 32;          // matrix steps of a score
  constexpr int R = D / 16;           // dimensions of a run = output tiles
  constexpr int H = kAtCols * NT;     // query heads
  constexpr int LD = D + 4;
  constexpr int LPH = D / kMxPerLane; // lanes of a head's row
  __shared__ float os[kAtWaves][H][LD];
  __shared__ float ms[kAtWaves][H], ls[kAtWaves][H];
  __shared__ int64_t sums[kAtWaves];
  __shared__ int found[1];
  __shared__ int64_t found_base[1];
  float (*qs)[LD] = os[0];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = lane & 15, g = lane >> 4;
  const int units = a.heads * a.ht;   // of a sequence
  int64_t total = 0, pos = 0, end = 0, base = 0;  // tiles: all, this workgroup's, before sequence b
  int64_t b = 0;
  int wgs = 0;
  if (a.wgs) {
    int64_t mine = 0;
    for (int64_t i = tid; i < a.batch; i += kAtThreads) mine += at_tiles(at_length(a, i), a.window);
    total = at_block_sum(mine, sums) * units;
    wgs = at_dealt(total, a.wgs);
    if ((int)blockIdx.x >= wgs) return;
    pos = at_start(blockIdx.x, total, wgs);
    end = at_start((int64_t)blockIdx.x + 1, total, wgs);
    // the sequence that has tile pos
    for (int64_t i0 = 0;; i0 += kAtThreads) {
      const int64_t i = i0 + tid;
      const int64_t n = i < a.batch ? (int64_t)at_tiles(at_length(a, i), a.window) * units : 0;
      int64_t x = n;  // inclusive sum over the threads before
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const int64_t y = __shfl_up(x, d);
        if (lane >= d) x += y;
      }
      __syncthreads();
      if (lane == 63) sums[wave] = x;
      __syncthreads();
      int64_t all = 0;
#pragma unroll
      for (int w = 0; w < kAtWaves; ++w) {
        if (w < wave) x += sums[w];
        all += sums[w];
      }
      if (pos >= base + x - n && pos < base + x) {
        found[0] = (int)i;
        found_base[0] = base + x - n;
      }
      __syncthreads();
      if (pos < base + all) break;  // it is one of these: pos < total
      base += all;
    }
    b = found[0];
    base = found_base[0];
  } else {
    b = blockIdx.x / (uint32_t)units;
    const int tiles = at_tiles(at_length(a, b), a.window);
    pos = (int64_t)(blockIdx.x - (uint32_t)b * (uint32_t)units) * tiles;
    end = pos + tiles;
    if (pos == end) {  // no key: the unit's rows get what an empty sum gives
      const int u = (int)(blockIdx.x - (uint32_t)b * (uint32_t)units);
      for (int r = tid / LPH; r < H; r += kAtThreads / LPH) {
        const int in = u % a.ht * H + r;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (in < a.group) at_finish(a, b, u / a.ht * a.group + in, (tid % LPH) * kMxPerLane, lane, v, 0.f, 0.f);
      }
      return;
    }
  }
  while (pos < end) {
  // the part's keys: tiles [tb, te) of unit u of sequence b
  const int n = at_length(a, b);
  const int first = a.window > 0 && n > a.window ? n - a.window : 0;
  const int s0 = at_skip(n, a.window), tiles = at_tiles(n, a.window);
  if (pos >= base + (int64_t)tiles * units) {  // on to the next sequence (one without keys has no tiles)
    base += (int64_t)tiles * units;
    ++b;
    continue;
  }
  const int u = (int)((pos - base) / tiles);
  const int64_t g0 = base + (int64_t)u * tiles;
  const int tb = (int)(pos - g0), te = (int)(end - g0 < tiles ? end - g0 : tiles);
  pos = g0 + te;
  const int h = u / a.ht, h0 = (u - h * a.ht) * H;  // key-value head; first query head within its group

  // queries: rotated, in float32, then as pairs
  for (int r = tid / LPH; r < H; r += kAtThreads / LPH) {
    const int e0 = (tid % LPH) * kMxPerLane;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (h0 + r < a.group) {
      at_load8(a.qt, a.q, b * a.ldq + (int64_t)(h * a.group + h0 + r) * D + e0, v);
      if (a.d) mx_rotate(v, a.signs, a.d, a.rnorm, e0, lane);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) qs[r][e0 + e] = v[e];
  }
  __syncthreads();
  const float sl = a.scale * 1.44269504088896341f;  // scores in units of log2
  mxb8 qf[NT][NS];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x = qs[8 * t + (c & 7)][g * (D / 4) + 8 * s + j] * sl;
        const __bf16 hi = (__bf16)x;
        qf[t][s][j] = c < 8 ? hi : (__bf16)(x - (float)hi);
      }
  __syncthreads();

  mxf4 o[NT][R];
  float m[NT], l[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t] = -INFINITY;
    l[t] = 0.f;
#pragma unroll
    for (int j = 0; j < R; ++j) o[t][j] = mxf4{0.f, 0.f, 0.f, 0.f};
  }
  const int64_t pbytes = a.pg.bytes();
  for (int tile = tb; tile < te; ++tile) {
    const int k0 = s0 + tile * kAtTile + wave * kAtKeys;
    if (k0 >= n) break;  // only in the last tile
    uint32_t kw[2][KW], vw[2][KW], ks[2][(KW + 3) / 4], vs[2];
    bool ok[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int kk = k0 + 16 * t;  // 16 keys of one page
      int64_t page = -1;
      if (kk < n) page = a.table[b * a.ldt + (kk >> a.lgP)];
      ok[t] = page >= 0 && page < a.pages;
#pragma unroll
      for (int i = 0; i < KW; ++i) kw[t][i] = vw[t][i] = 0u;
      ks[t][0] = 127u;
      if constexpr (D == 256) ks[t][1] = 127u;
      vs[t] = 0x7f7f7f7fu;
      if (ok[t]) {
        const uint8_t* pb = a.cache + (page * a.heads + h) * pbytes;
        const int p = kk & (a.pg.P - 1);
        const uint8_t* kp = pb + a.pg.kcode(p + c) + g * (D / 8);
        const uint8_t* vp = pb + a.pg.vcode(p + 4 * g, c);
        if constexpr (D == 64) {
          const uint2 x = *reinterpret_cast<const uint2*>(kp), y = *reinterpret_cast<const uint2*>(vp);
          kw[t][0] = x.x; kw[t][1] = x.y;
          vw[t][0] = y.x; vw[t][1] = y.y;
          ks[t][0] = pb[a.pg.kscale(p + c) + (g >> 1)];
        } else {
#pragma unroll
          for (int q = 0; q < KW / 4; ++q) {
            const uint4 x = reinterpret_cast<const uint4*>(kp)[q], y = reinterpret_cast<const uint4*>(vp)[q];
            kw[t][4 * q] = x.x; kw[t][4 * q + 1] = x.y; kw[t][4 * q + 2] = x.z; kw[t][4 * q + 3] = x.w;
            vw[t][4 * q] = y.x; vw[t][4 * q + 1] = y.y; vw[t][4 * q + 2] = y.z; vw[t][4 * q + 3] = y.w;
          }
          if constexpr (D == 128) {
            ks[t][0] = pb[a.pg.kscale(p + c) + g];
          } else {
            const uint32_t x = *reinterpret_cast<const uint16_t*>(pb + a.pg.kscale(p + c) + 2 * g);
            ks[t][0] = x & 255u;
            ks[t][1] = x >> 8;
          }
        }
        vs[t] = *reinterpret_cast<const uint32_t*>(pb + a.pg.vscale(p + 4 * g, c * D / 512));
      }
    }
    // scores: column c, keys kk + 4 g + i
    float s[NT][2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      mxf4 acc[NT];
#pragma unroll
      for (int u = 0; u < NT; ++u) acc[u] = mxf4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < NS; ++q) {
        const float sc = mx_scale(ks[t][D == 256 ? q / 4 : 0]);
        uint4 w;
        w.x = at_bits(at_pair(kw[t][q], sc, 0));
        w.y = at_bits(at_pair(kw[t][q], sc, 1));
        w.z = at_bits(at_pair(kw[t][q], sc, 2));
        w.w = at_bits(at_pair(kw[t][q], sc, 3));
#pragma unroll
        for (int u = 0; u < NT; ++u)
          acc[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(mxb8, w), qf[u][q], acc[u], 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < NT; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[u][t][i] = acc[u][i] + at_ror8(acc[u][i]);
    }
    // a tile with masked keys: scores to -infinity, values to zero
    if (k0 < first || k0 + kAtKeys > n || !ok[0] || !ok[1]) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = k0 + 16 * t + 4 * g + i;
          if (key < first || key >= n || !ok[t]) {
#pragma unroll
            for (int u = 0; u < NT; ++u) s[u][t][i] = -INFINITY;
            vs[t] = (vs[t] & ~(255u << (8 * i))) | 127u << (8 * i);
            if constexpr (D == 64) {
              vw[t][i / 2] &= ~(0xffffu << (16 * (i & 1)));
            } else {
#pragma unroll
              for (int q = 0; q < KW / 4; ++q) vw[t][i * (KW / 4) + q] = 0u;
            }
          }
        }
    }
    mxb8 pf[NT];
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      float mx = s[u][0][0];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) mx = fmaxf(mx, s[u][t][i]);
      mx = fmaxf(at_colmax(mx), m[u]);
      const float base = mx == -INFINITY ? 0.f : mx;
      const float f = __builtin_amdgcn_exp2f(m[u] - base);
      m[u] = mx;
      float sum = 0.f;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float p = __builtin_amdgcn_exp2f(s[u][t][i] - base);
          sum += p;
          const __bf16 hi = (__bf16)p;
          pf[u][4 * t + i] = c < 8 ? hi : (__bf16)(p - (float)hi);
        }
      l[u] = l[u] * f + sum;
#pragma unroll
      for (int j = 0; j < R; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[u][j][i] *= f;
    }
    // values: keys in pairs, one run of dimensions per lane
    float vsc[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) vsc[t][i] = mx_scale((vs[t] >> (8 * i)) & 255u);
#pragma unroll
    for (int q = 0; q < R / 2; ++q) {  // dimensions 2 q and 2 q + 1 of the run
      uint32_t lo[4], hi[4];
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const int ba = i * (R / 2) + q, bb = (i + 1) * (R / 2) + q;  // bytes of the lane's words
          const uint32_t x = at_bits(at_pair(vw[t][ba / 4], vsc[t][i], ba));
          const uint32_t y = at_bits(at_pair(vw[t][bb / 4], vsc[t][i + 1], bb));
          lo[2 * t + i / 2] = __builtin_amdgcn_perm(y, x, 0x05040100u);
          hi[2 * t + i / 2] = __builtin_amdgcn_perm(y, x, 0x07060302u);
        }
      const mxb8 va = __builtin_bit_cast(mxb8, make_uint4(lo[0], lo[1], lo[2], lo[3]));
      const mxb8 vb = __builtin_bit_cast(mxb8, make_uint4(hi[0], hi[1], hi[2], hi[3]));
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        o[u][2 * q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, pf[u], o[u][2 * q], 0, 0, 0);
        o[u][2 * q + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vb, pf[u], o[u][2 * q + 1], 0, 0, 0);
      }
    }
  }

  // join the wavefronts: all parts to the common maximum, summed in order
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    l[t] = at_colsum(l[t]);
    if (lane < 8) {
      ms[wave][8 * t + lane] = m[t];
      ls[wave][8 * t + lane] = l[t];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const float x = o[t][j][i] + at_ror8(o[t][j][i]);
        if (c < 8) os[wave][8 * t + c][(4 * g + i) * R + j] = x;
      }
  }
  __syncthreads();
  for (int r = tid / LPH; r < H; r += kAtThreads / LPH) {
    if (h0 + r >= a.group) continue;  // uniform over the row's lanes
    const int e0 = (tid % LPH) * kMxPerLane;
    float M = ms[0][r];
#pragma unroll
    for (int w = 1; w < kAtWaves; ++w) M = fmaxf(M, ms[w][r]);
    const float base = M == -INFINITY ? 0.f : M;
    float L = 0.f, v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kAtWaves; ++w) {
      const float f = __builtin_amdgcn_exp2f(ms[w][r] - base);
      L += ls[w][r] * f;
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] += os[w][r][e0 + e] * f;
    }
    if (tb == 0 && te == tiles) {
      at_finish(a, b, h * a.group + h0 + r, e0, lane, v, M, L);
    } else {
      float* p = a.part + (at_slot(blockIdx.x, g0, total, wgs) * H + r) * (D + 4);
      mx_store8<BRQ_F32>(p, e0, v);
      if (e0 == 0) *reinterpret_cast<float2*>(p + D) = make_float2(M, L);
    }
  }
  __syncthreads();  // the next part's queries go where these sums were
  }
}

// Joins the parts of units that span workgroups, in order, and writes the rows
// of sequences without keys.  ROWS query heads of one unit to a workgroup;
// each has G groups of D / 8 lanes, which take its parts in turn and are
// joined in LDS.
template <int D>
__global__ __launch_bounds__(kAtThreads) void at_join_kernel(AtArgs a, int rows) {
  constexpr int LPH = D / kMxPerLane;
  constexpr int LD = D + 4;
  __shared__ float os[kAtThreads / LPH][LD];
  __shared__ int64_t sums[kAtWaves];
  const int tid = threadIdx.x, lane = tid & 63;
  const int H = kAtCols * a.nt, units = a.heads * a.ht, per = H / rows;
  const int64_t ub = blockIdx.x / (uint32_t)per;
  const int r0 = (int)(blockIdx.x - (uint32_t)ub * (uint32_t)per) * rows;
  const int64_t b = ub / units;
  const int u = (int)(ub - b * units);
  const int tiles = at_tiles(at_length(a, b), a.window);
  const int h = u / a.ht, h0 = (u - h * a.ht) * H;
  const int r = r0 + tid / LPH % rows, grp = tid / (LPH * rows), groups = kAtThreads / (LPH * rows);
  const int e0 = (tid % LPH) * kMxPerLane;
  const bool mine = h0 + r < a.group;
  int64_t before = 0, all = 0;
  for (int64_t i = tid; i < a.batch; i += kAtThreads) {
    const int t = at_tiles(at_length(a, i), a.window);
    all += t;
    if (i < b) before += t;
  }
  const int64_t total = at_block_sum(all, sums) * units;
  const int64_t g0 = at_block_sum(before, sums) * units + (int64_t)u * tiles;
  float M = -INFINITY, L = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (tiles > 0) {
    const int wgs = at_dealt(total, a.wgs);
    const int w0 = at_owner(g0, total, wgs), w1 = at_owner(g0 + tiles - 1, total, wgs);
    if (w0 == w1) return;  // finished by its workgroup
    for (int w = w0 + grp; w <= w1; w += groups) {
      const float* p = a.part + (at_slot(w, g0, total, wgs) * H + r) * (int64_t)LD;
      const float2 ml = *reinterpret_cast<const float2*>(p + D);
      float v[8];
      mx_load8<BRQ_F32>(p, e0, v);
      const float m = fmaxf(M, ml.x), base = m == -INFINITY ? 0.f : m;
      const float f = __builtin_amdgcn_exp2f(M - base), q = __builtin_amdgcn_exp2f(ml.x - base);
      M = m;
      L = L * f + ml.y * q;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = o[e] * f + v[e] * q;
    }
  }
  mx_store8<BRQ_F32>(&os[tid / LPH][0], e0, o);
  if (e0 == 0) *reinterpret_cast<float2*>(&os[tid / LPH][D]) = make_float2(M, L);
  __syncthreads();
  if (grp != 0 || !mine) return;
  for (int s = 1; s < groups; ++s) {
    const float* p = os[tid / LPH + s * rows];
    const float2 ml = *reinterpret_cast<const float2*>(p + D);
    const float m = fmaxf(M, ml.x), base = m == -INFINITY ? 0.f : m;
    const float f = __builtin_amdgcn_exp2f(M - base), q = __builtin_amdgcn_exp2f(ml.x - base);
    M = m;
    L = L * f + ml.y * q;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = o[e] * f + p[e0 + e] * q;
  }
  at_finish(a, b, h * a.group + h0 + r, e0, lane, o, M, L);
}

template <int D>
hipError_t at_launch(const AtArgs& a, hipStream_t s) {
  const int64_t units = a.batch * a.heads * a.ht;
  const dim3 grid((unsigned)(a.wgs ? a.wgs : units));
  if (a.nt == 1) at_kernel<D, 1><<<grid, kAtThreads, 0, s>>>(a);
  else at_kernel<D, 2><<<grid, kAtThreads, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.wgs) return e;
  // few units: each has many parts, and a workgroup for every row; many: most
  // were finished in one place, and a workgroup looks after several rows
  const int H = kAtCols * a.nt, most = kAtThreads / (D / kMxPerLane);
  const int rows = units * H <= 2048 ? 1 : (H < most ? H : most);
  at_join_kernel<D><<<dim3((unsigned)(units * (H / rows))), kAtThreads, 0, s>>>(a, rows);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_paged_attention(const AtArgs& a, hipStream_t s) {
  if (a.pg.D == 64) return at_launch<64>(a, s);
  if (a.pg.D == 128) return at_launch<128>(a, s);
  return at_launch<256>(a, s);
}

}  // namespace brq
