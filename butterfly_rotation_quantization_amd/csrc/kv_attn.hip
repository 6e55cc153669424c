// Attention of one new token per sequence over the paged 4-bit cache
// (layout: KvPage in mx.h).
//
// Per key-value head the scores are products S^T = K Q^T on the scaled matrix
// instructions: the keys' codes and scale bytes as they lie in the cache, the
// queries of the group as columns, each in four 8-bit floating-point pieces
// (at_pieces) of which columns c and c + 8 of two products hold one each.  The
// output is O^T = V^T P^T on the bfloat16 ones: a value's code times its scale
// is exact in bfloat16, and a probability is a pair of bfloat16 (its upper 16
// bits and the rest), in columns c and c + 8 again.  Sums, maxima and
// normalisers are float32.  With float32 queries the scores are bfloat16
// products too, and queries and probabilities three pieces.
//
// Lane l = 16 g + c of a wavefront holds block g of key c as the A operand of
// the scores; these come out as column c, keys 4 g + i, which is where the B
// operand of O^T wants the probabilities when the values' A operand takes keys
// 4 g + i as well: nothing moves between lanes in between.  The values of four
// keys lie together in the cache for that reason.
//
// A tile is 128 keys of one unit (workgroup: four wavefronts, 32 keys each);
// which workgroup takes which tiles: kAtLead in mx.h.  64 query heads over 8
// of 128: 4 sequences of 131072 tokens take 114 us, 5.0 TB/s of the cache,
// bound by memory; 96 of 17 to 16384 tokens 67 us, 3.9 TB/s, the rest being
// what beginning and joining 768 units takes.  The loads of the next 32 keys
// are under way while these are worked on; that needs the queries in LDS
// rather than in registers (in registers, with four workgroups a compute unit:
// spilled, 132 and 88 us; without loads ahead 122 and 72).  With the keys
// converted and the queries in pairs of bfloat16 the two took 139 and 84 us.
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

// A query enters the scores as four 8-bit floating-point pieces, each the
// rounding of what the ones before it left (4 bits each: together within
// 2^-17 of its block's largest magnitude), with a scale for each block of 32.
// The eight values of a lane (its block is four lanes): the pieces' words and
// scale bytes.
__device__ __forceinline__ void at_pieces(float (&v)[8], uint2 (&piece)[4], int (&byte)[4]) {
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(v[e]) & 0x7fffffffu);
  top = max(top, mx_xor<1>(top));
  top = max(top, mx_xor<2>(top));
  const int ex = (int)(top >> 23);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    // times 2^(7 - 4 k) of the largest exponent: the first piece lies below
    // 256, what is left of it below 128; an infinity or a NaN: a NaN scale
    const int x = ex - 7 - 4 * k;
    byte[k] = ex == 255 ? 255 : x > 0 ? x : 0;
    const float inv = __uint_as_float((uint32_t)(254 - (x > 0 ? x : 0)) << 23);
    const float back = __uint_as_float(x > 0 ? (uint32_t)x << 23 : 0x400000u);
    int w[2] = {0, 0};
    // Beside 2^7 the matrix unit drops bits below 2^-6 (measured: 2^-7 counted
    // as zero, 1.5 2^-6 as 2^-6), so a value that would have such bits is left
    // to the next piece.
    float t[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      t[e] = v[e] * inv;
      t[e] = fabsf(t[e]) < 0.125f ? 0.0f : t[e];
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      w[e] = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * e], t[4 * e + 1], w[e], false);
      w[e] = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * e + 2], t[4 * e + 3], w[e], true);
      v[4 * e] -= __builtin_amdgcn_cvt_f32_fp8(w[e], 0) * back;
      v[4 * e + 1] -= __builtin_amdgcn_cvt_f32_fp8(w[e], 1) * back;
      v[4 * e + 2] -= __builtin_amdgcn_cvt_f32_fp8(w[e], 2) * back;
      v[4 * e + 3] -= __builtin_amdgcn_cvt_f32_fp8(w[e], 3) * back;
    }
    piece[k] = make_uint2((uint32_t)w[0], (uint32_t)w[1]);
  }
}

// For float32 a query, like a probability, is three bfloat16 pieces (24 bits):
// the upper 16 bits, those of what they leave, and the rest.
__device__ __forceinline__ void at_pieces(const float (&v)[8], uint4 (&piece)[3]) {
  uint32_t x[3][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float r = v[e];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      x[k][e] = __float_as_uint(r);
      r -= __uint_as_float(x[k][e] & 0xffff0000u);
    }
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = __builtin_amdgcn_perm(x[k][2 * e + 1], x[k][2 * e], 0x07060302u);
    piece[k] = make_uint4(w[0], w[1], w[2], w[3]);
  }
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
// F32: queries and outputs are float32, and the scores and the output keep 24
// bits.  The scaled instructions, which drop low bits of the smaller products
// (scores within some 2^-18), do not: the keys are converted like the values.
template <int D, int NT, bool F32>
__global__ __launch_bounds__(kAtThreads, at_workgroups(D, NT) / 256) void at_kernel(AtArgs a) {
  constexpr int KW = D / 32;          // words of codes a lane holds per key (of the scores) or four keys (values)
  constexpr int NQ = D == 256 ? 2 : 1;  // matrix steps of 128 values of a score
  constexpr int NP = D == 64 ? 1 : 2;   // products of a step: two of a query's four pieces each (D = 64: all four)
  constexpr int NJ = D == 64 ? 2 : 4;   // F32: products of 32 values in a step
  constexpr int R = D / 16;           // dimensions of a run = output tiles
  constexpr int H = kAtCols * NT;     // query heads
  constexpr int LD = D + 4;
  constexpr int LPH = D / kMxPerLane; // lanes of a head's row
  __shared__ __align__(16) float os[kAtWaves][H][LD];
  __shared__ float ms[kAtWaves][H], ls[kAtWaves][H];
  __shared__ int64_t sums[kAtWaves];
  __shared__ int found[1];
  __shared__ int64_t found_base[1];
  // the queries' pieces, with scales or (F32) of bfloat16; the gap in a row
  // keeps a column's lanes on banks of their own
  __shared__ uint8_t qb[H][4][D / 32];
  constexpr int QD = D + 16, FD = D + 8;
  uint8_t (*qs)[4][QD] = reinterpret_cast<uint8_t (*)[4][QD]>(&os[0]);
  uint16_t (*qh)[3][FD] = reinterpret_cast<uint16_t (*)[3][FD]>(&os[0]);
  static_assert(sizeof(uint8_t[H][4][QD]) <= sizeof(os) && sizeof(uint16_t[H][3][FD]) <= sizeof(os),
                "the pieces lie where the sums will");

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const uint32_t low = c < 8 ? 0u : 0xffff0000u;
  const uint32_t one2 = 0x3f803f80u;
  const mxb8 ones = __builtin_bit_cast(mxb8, make_uint4(one2, one2, one2, one2));
  const int units = a.heads * a.ht;   // of a sequence
  int64_t total = 0, pos = 0, end = 0, base = 0;  // places: all, this workgroup's, before sequence b
  int64_t b = 0;
  int wgs = 0;
  if (a.wgs) {
    // all tiles; with more sequences than threads, by a pass of its own
    if (a.batch > kAtThreads) {
      int64_t mine = 0;
      for (int64_t i = tid; i < a.batch; i += kAtThreads) mine += at_cost(at_tiles(at_length(a, i), a.window));
      total = at_block_sum(mine, sums) * units;
    }
    for (int64_t i0 = 0;; i0 += kAtThreads) {
      const int64_t i = i0 + tid;
      const int64_t n = i < a.batch ? (int64_t)at_cost(at_tiles(at_length(a, i), a.window)) * units : 0;
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
      if (i0 == 0) {
        if (a.batch <= kAtThreads) total = all;
        wgs = at_dealt(total, a.wgs);
        if ((int)blockIdx.x >= wgs) return;
        pos = at_start(blockIdx.x, total, wgs);
        end = at_start((int64_t)blockIdx.x + 1, total, wgs);
      }
      if (pos >= base + x - n && pos < base + x) {  // the sequence that has place pos
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
    const int cost = at_cost(at_tiles(at_length(a, b), a.window));
    pos = (int64_t)(blockIdx.x - (uint32_t)b * (uint32_t)units) * cost;
    end = pos + cost;
    if (pos == end) {  // no key: the unit's rows get what an empty sum gives
      const int u = (int)(blockIdx.x - (uint32_t)b * (uint32_t)units);
      for (int r = tid / LPH; r < H; r += kAtThreads / LPH) {
        const int in = u % a.ht * H + r;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (in < a.group) at_finish<D>(a, b, u / a.ht * a.group + in, (tid % LPH) * kMxPerLane, lane, v, 0.f, 0.f);
      }
      return;
    }
  }
  while (pos < end) {
  // the part's keys: tiles [tb, te) of unit u of sequence b
  const int n = at_length(a, b);
  const int first = a.window > 0 && n > a.window ? n - a.window : 0;
  const int s0 = at_skip(n, a.window), tiles = at_tiles(n, a.window);
  const int cost = at_cost(tiles);
  if (pos >= base + (int64_t)cost * units) {  // on to the next sequence (one without keys has no place)
    base += (int64_t)cost * units;
    ++b;
    continue;
  }
  const int u = (int)((pos - base) / cost);
  const int64_t g0 = base + (int64_t)u * cost + kAtLead;  // place of the unit's first tile
  const int tb = pos > g0 ? (int)(pos - g0) : 0;
  const int te = end - g0 < tiles ? (int)(end - g0) : tiles;
  pos = g0 + tiles < end ? g0 + tiles : end;
  if (te <= tb) continue;  // only of the unit's lead
  const int h = u / a.ht, h0 = (u - h * a.ht) * H;  // key-value head; first query head within its group
  if (wgs && tb == 0 && tid == 0)  // who has the unit's parts, and the first one's slot, for the join
    a.who[b * units + u] = make_int2((int)at_slot(blockIdx.x, g0, total, wgs),
                                     te == tiles ? 0 : at_owner(g0 + tiles - 1, total, wgs) - (int)blockIdx.x);

  const int64_t pbytes = a.pg.bytes();
  const int32_t* row = a.table + b * a.ldt;
  int k0 = s0 + tb * kAtTile + wave * kAtKeys;
  const int kend = s0 + te * kAtTile < n ? s0 + te * kAtTile : n;
  // Operands of 32 keys, 16 of them from one page.  The next keys are fetched
  // once the scores have used these, the next values once the output has, so
  // each travels during the other's arithmetic without registers of its own.
  // Where there is no key, or no page, page 0 is read and masked below: loads
  // under no condition, or the wait for one would be a wait for all.
  int page[2], pg[2];
  bool ok[2];
  mxi4 kw[2][NQ];
  uint32_t vw[2][KW], vs[2];
  int ks[2][NQ];
  auto look_up = [&](int k) {
#pragma unroll
    for (int t = 0; t < 2; ++t) page[t] = row[(k + 16 * t < n ? k + 16 * t : n - 1) >> a.lgP];
  };
  auto fetch_keys = [&](int k) {  // looked up before; looks up the next
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      pg[t] = __builtin_amdgcn_readfirstlane(page[t]);
      ok[t] = pg[t] >= 0 && pg[t] < a.pages && k + 16 * t < n;
      pg[t] = ok[t] ? pg[t] : 0;
      const uint8_t* pb = a.cache + ((int64_t)pg[t] * a.heads + h) * pbytes;
      const int p = (k + 16 * t) & (a.pg.P - 1);
#pragma unroll
      for (int e = 0; e < NQ; ++e) {
        const int blk = D == 64 ? (g & 1) : 4 * e + g;  // D = 64: both halves of the lanes hold the 64 values
        kw[t][e] = *reinterpret_cast<const mxi4*>(pb + a.pg.kcode(p) + (uint32_t)(c * (D / 2) + 16 * blk));
        ks[t][e] = pb[a.pg.kscale(p) + (uint32_t)(c * (D / 32) + blk)];
      }
    }
    look_up(k + kAtTile);
  };
  auto fetch_values = [&](int k) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const uint8_t* pb = a.cache + ((int64_t)pg[t] * a.heads + h) * pbytes;
      const int p = (k + 16 * t) & (a.pg.P - 1);
      const uint8_t* vp = pb + a.pg.vcode(p, 0) + (uint32_t)(g * (2 * D) + c * (D / 8));
      if constexpr (D == 64) {
        const uint2 y = *reinterpret_cast<const uint2*>(vp);
        vw[t][0] = y.x; vw[t][1] = y.y;
      } else {
#pragma unroll
        for (int q = 0; q < KW / 4; ++q) {
          const uint4 y = reinterpret_cast<const uint4*>(vp)[q];
          vw[t][4 * q] = y.x; vw[t][4 * q + 1] = y.y; vw[t][4 * q + 2] = y.z; vw[t][4 * q + 3] = y.w;
        }
      }
      vs[t] = *reinterpret_cast<const uint32_t*>(pb + a.pg.vscale(p, 0) + (uint32_t)(g * (D / 8) + (c * D / 512) * 4));
    }
  };
  if (k0 < kend) {
    look_up(k0);
    fetch_keys(k0);
    fetch_values(k0);
  }
  // queries: rotated, times the scale, in pieces
  const float sl = a.scale * 1.44269504088896341f;  // scores in units of log2
  for (int r = tid / LPH; r < H; r += kAtThreads / LPH) {
    const int e0 = (tid % LPH) * kMxPerLane;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (h0 + r < a.group) {
      at_load8(a.qt, a.q, b * a.ldq + (int64_t)(h * a.group + h0 + r) * D + e0, v);
      if (a.d) {
        if (a.signs)  // after the query: registers are short here
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= a.signs[e0 + e];
        mx_hadamard<D>(v, lane);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= a.rnorm;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= sl;
    if constexpr (F32) {
      uint4 piece[3];
      at_pieces(v, piece);
#pragma unroll
      for (int k = 0; k < 3; ++k) *reinterpret_cast<uint4*>(&qh[r][k][e0]) = piece[k];
    } else {
      uint2 piece[4];
      int byte[4];
      at_pieces(v, piece, byte);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        *reinterpret_cast<uint2*>(&qs[r][k][e0]) = piece[k];
        if ((e0 & 31) == 0) qb[r][k][e0 / 32] = (uint8_t)byte[k];
      }
    }
  }
  __syncthreads();
  // The B operand: column c < 8 holds pieces 1 and 3 of query head c, column
  // c + 8 its pieces 2 and 4; product w takes the first or the second.  A
  // lane's words hold dimensions 16 g .. + 15 and 64 + 16 g .. + 15 of a step,
  // and its scale is that of block g.  With D = 64 one product takes all: the
  // second half of the words repeats dimensions 16 g .. with pieces 3 and 4,
  // as the keys' lanes repeat theirs.
  int qsc[NT][NQ][NP];
  if constexpr (!F32) {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int e = 0; e < NQ; ++e)
#pragma unroll
        for (int w = 0; w < NP; ++w) {
          const int r = 8 * t + (c & 7), k = (c >> 3) + 2 * w;
          qsc[t][e][w] = D == 64 ? qb[r][k + 2 * (g >> 1)][g & 1] : qb[r][k][4 * e + g];
        }
  }
  auto query = [&](int t, int e, int w) {
    const int r = 8 * t + (c & 7), k = (c >> 3) + 2 * w;
    const mxi4 x = *reinterpret_cast<const mxi4*>(&qs[r][k][128 * e + 16 * g]);
    const mxi4 y = D == 64 ? *reinterpret_cast<const mxi4*>(&qs[r][k + 2][16 * g])
                           : *reinterpret_cast<const mxi4*>(&qs[r][k][128 * e + 64 + 16 * g]);
    return mxi8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
  };
  // F32: word j of a lane's keys is 8 j .. + 7 of its block (with D = 64, where
  // two lanes have the same block, word j + 2 for the second); piece k of the
  // query's values there
  auto query_f32 = [&](int t, int e, int j, int k) {
    const int at = D == 64 ? 32 * (g & 1) + 8 * (j + 2 * (g >> 1)) : 128 * e + 32 * g + 8 * j;
    return *reinterpret_cast<const uint4*>(&qh[8 * t + (c & 7)][k][at]);
  };

  mxf4 o[NT][R], l[NT];
  float m[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t] = -INFINITY;
    l[t] = mxf4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < R; ++j) o[t][j] = mxf4{0.f, 0.f, 0.f, 0.f};
  }
  // One step of 32 keys.  The last one fetches nothing (and is code of its own:
  // under a condition in the loop, the fetches would be waited for at once).
  auto step = [&](auto last) {
    constexpr bool more = !decltype(last)::value;
    asm volatile("" ::: "memory");  // the queries stay in LDS
    // scores: column c, keys 16 t + 4 g + i
    float s[NT][2][4];
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      mxf4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
      if constexpr (F32) {  // columns c < 8: the first and third pieces, c + 8: the second
#pragma unroll
        for (int e = 0; e < NQ; ++e)
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            const mxb8 q1 = __builtin_bit_cast(mxb8, query_f32(u, e, j, c >> 3));
            uint4 third = query_f32(u, e, j, 2);
            if (low) third = make_uint4(0u, 0u, 0u, 0u);
            const mxb8 q2 = __builtin_bit_cast(mxb8, third);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const uint32_t x = D == 64 && g >= 2 ? kw[t][e][(j + 2) & 3] : kw[t][e][j];
              const float sc = __uint_as_float((uint32_t)ks[t][e] << 23);
              const mxb8 K = __builtin_bit_cast(mxb8, make_uint4(at_bits(at_pair(x, sc, 0)), at_bits(at_pair(x, sc, 1)),
                                                                 at_bits(at_pair(x, sc, 2)), at_bits(at_pair(x, sc, 3))));
              acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(K, q1, acc[t], 0, 0, 0);
              acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(K, q2, acc[t], 0, 0, 0);
            }
          }
      } else {
#pragma unroll
        for (int e = 0; e < NQ; ++e)
#pragma unroll
          for (int w = 0; w < NP; ++w) {
            const mxi8 Q = query(u, e, w);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              const mxi8 K = {kw[t][e][0], kw[t][e][1], kw[t][e][2], kw[t][e][3], 0, 0, 0, 0};
              acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(K, Q, acc[t], 4, 0, 0, ks[t][e], 0, qsc[u][e][w]);
            }
          }
      }
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[u][t][i] = acc[t][i] + at_ror8(acc[t][i]);
    }
    // masked keys: scores to -infinity, values to zero
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
    if constexpr (more) fetch_keys(k0 + kAtTile);
    mxb8 pf[NT], pl[NT];
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      float mx = fmaxf(fmaxf(s[u][0][0], s[u][0][1]), fmaxf(s[u][0][2], s[u][0][3]));
      mx = fmaxf(mx, fmaxf(fmaxf(s[u][1][0], s[u][1][1]), fmaxf(s[u][1][2], s[u][1][3])));
      mx = fmaxf(at_colmax(mx), m[u]);
      const float base = mx == -INFINITY ? 0.f : mx;
      if (__builtin_amdgcn_ballot_w64(mx != m[u])) {  // seldom after the first tiles
        const float f = __builtin_amdgcn_exp2f(m[u] - base);
        m[u] = mx;
#pragma unroll
        for (int i = 0; i < 4; ++i) l[u][i] *= f;
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[u][j][i] *= f;
      }
      // columns 0..7 take a probability's upper 16 bits, columns 8..15 the
      // rest, rounded toward zero to 8 bits (2^-16 of the probability); for
      // float32 a second product's columns 0..7 take what is left then.  The
      // sum below is of what the products use.
      uint32_t w[4], y[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float x[2], z[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float p = __builtin_amdgcn_exp2f(s[u][q / 2][2 * (q & 1) + e] - base);
          x[e] = p - __uint_as_float(__float_as_uint(p) & low);
          if constexpr (F32) {
            const float r = p - __uint_as_float(__float_as_uint(p) & 0xffff0000u);
            z[e] = r - __uint_as_float(__float_as_uint(r) & 0xffff0000u);
          }
        }
        w[q] = __builtin_amdgcn_perm(__float_as_uint(x[1]), __float_as_uint(x[0]), 0x07060302u);
        if constexpr (F32)
          y[q] = low ? 0u : __builtin_amdgcn_perm(__float_as_uint(z[1]), __float_as_uint(z[0]), 0x07060302u);
      }
      pf[u] = __builtin_bit_cast(mxb8, make_uint4(w[0], w[1], w[2], w[3]));
      l[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, pf[u], l[u], 0, 0, 0);
      if constexpr (F32) {
        pl[u] = __builtin_bit_cast(mxb8, make_uint4(y[0], y[1], y[2], y[3]));
        l[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, pl[u], l[u], 0, 0, 0);
      }
    }
    // values: keys in pairs, one run of dimensions per lane (of a scale the
    // conversion reads the exponent, so byte 0 is 2^-127 and 255 NaN)
    float vsc[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) vsc[t][i] = __uint_as_float(i == 3 ? vs[t] >> 24 << 23 : (vs[t] >> (8 * i) & 255u) << 23);
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
        if constexpr (F32) {
          o[u][2 * q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, pl[u], o[u][2 * q], 0, 0, 0);
          o[u][2 * q + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vb, pl[u], o[u][2 * q + 1], 0, 0, 0);
        }
      }
    }
    if constexpr (more) fetch_values(k0 + kAtTile);
  };
  for (; k0 + kAtTile < kend; k0 += kAtTile) step(std::false_type{});
  if (k0 < kend) step(std::true_type{});

  // join the wavefronts: all parts to the common maximum, summed in order
  __syncthreads();  // the sums go where the queries were
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const float sum = l[t][0] + at_ror8(l[t][0]);  // every row of the product is the column's sum
    if (lane < 8) {
      ms[wave][8 * t + lane] = m[t];
      ls[wave][8 * t + lane] = sum;
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
      at_finish<D>(a, b, h * a.group + h0 + r, e0, lane, v, M, L);
    } else {
      float* p = a.part + (at_slot(blockIdx.x, g0, total, wgs) * H + r) * (D + 4);
      mx_store8<BRQ_F32>(p, e0, v);
      if (e0 == 0) *reinterpret_cast<float2*>(p + D) = make_float2(M, L);
    }
  }
  __syncthreads();  // the next part's queries go where these sums were
  }
}

// Joins the parts of units that span workgroups and writes the rows of
// sequences without keys.  ROWS query heads of one unit to a workgroup;
// each has G groups of D / 8 lanes, which take its parts in turn and are
// joined in LDS.
template <int D>
__global__ __launch_bounds__(kAtThreads) void at_join_kernel(AtArgs a, int rows) {
  constexpr int LPH = D / kMxPerLane;
  constexpr int LD = D + 4;
  __shared__ float os[kAtThreads / LPH][LD];
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
  float M = -INFINITY, L = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (tiles > 0) {
    const int2 who = a.who[ub];
    if (who.y == 0) return;  // finished by its workgroup
    // part s (of who.y + 1) is the first of workgroup who.x / 2 + s
    const float* p0 = a.part + r * (int64_t)LD;
#pragma unroll 2
    for (int s = grp; s <= who.y; s += groups) {
      const float* p = p0 + (s == 0 ? who.x : (who.x / 2 + s) * 2) * (int64_t)(H * LD);
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
  // the maximum first, so that the parts' factors do not wait for one another
  const float own = M;
#pragma unroll 4
  for (int s = 1; s < groups; ++s) M = fmaxf(M, os[tid / LPH + s * rows][D]);
  const float base = M == -INFINITY ? 0.f : M, f = __builtin_amdgcn_exp2f(own - base);
  L *= f;
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] *= f;
#pragma unroll 4
  for (int s = 1; s < groups; ++s) {
    const float* p = os[tid / LPH + s * rows];
    const float q = __builtin_amdgcn_exp2f(p[D] - base);
    L += p[D + 1] * q;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] += p[e0 + e] * q;
  }
  at_finish<D>(a, b, h * a.group + h0 + r, e0, lane, o, M, L);
}

template <int D>
hipError_t at_launch(const AtArgs& a, hipStream_t s) {
  const int64_t units = a.batch * a.heads * a.ht;
  const dim3 grid((unsigned)(a.wgs ? a.wgs : units));
  const bool f32 = a.qt == BRQ_F32;
  if (a.nt == 1 && f32) at_kernel<D, 1, true><<<grid, kAtThreads, 0, s>>>(a);
  else if (a.nt == 1) at_kernel<D, 1, false><<<grid, kAtThreads, 0, s>>>(a);
  else if (f32) at_kernel<D, 2, true><<<grid, kAtThreads, 0, s>>>(a);
  else at_kernel<D, 2, false><<<grid, kAtThreads, 0, s>>>(a);
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
