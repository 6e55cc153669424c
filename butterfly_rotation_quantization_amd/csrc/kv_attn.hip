// Attention of one new token per sequence over the paged 4-bit cache
// (layout: KvPage in mx.h).
//
// Per key-value head the scores are products S^T = K Q^T on the scaled matrix
// instructions: the keys' codes and scale bytes as they lie in the cache, the
// queries of the group as columns, each in eight 4-bit floating-point pieces
// (at_pieces) of which columns c and c + 8 of four products hold one each.  The
// output is O^T = V^T P^T on the bfloat16 ones: a value's code times its scale
// is exact in bfloat16, and a probability is three pieces of 8 bits, in columns c
// and c + 8 of one product and c of another.  Nothing is held in fewer than 24
// bits, so a result is as near to the formula as one in plain float32.
//
// Lane l = 16 g + c of a wavefront holds block g of key c as the A operand of
// the scores; these come out as column c, keys 4 g + i, which is where the B
// operand of O^T wants the probabilities when the values' A operand takes keys
// 4 g + i as well: nothing moves between lanes in between.  The values of four
// keys lie together in the cache for that reason.
//
// A tile is 128 keys of one unit (workgroup: four wavefronts, 32 keys each);
// which workgroup takes which tiles: kAtLead in mx.h.  64 query heads over 8
// of 128: 4 sequences of 131072 tokens take 117 us, 4.9 TB/s of the cache,
// bound by memory; 96 of 17 to 16384 tokens 68 us, 3.8 TB/s, the rest being
// what beginning and joining 768 units takes; the same with float32 queries.
// The loads of the next 32 keys are under way while these are worked on; that
// needs the queries in LDS rather than in registers.  (Measured while a query
// had 16 bits and a probability too, and the two took 114 and 67 us: queries in
// registers, with four workgroups a compute unit, spilled, 132 and 88 us; no
// loads ahead 122 and 72; keys converted and queries in pairs of bfloat16, then
// without loads ahead, 139 and 84.)  A group of 16 heads takes 161 us for the four,
// one of 128 over a single key-value head 146: 16 heads at a time, the products,
// exponentials and the values' conversions of each pass bound it.
#include "at_dev.h"

namespace brq {
namespace {

// Tokens of sequence b that the table has room for.
__device__ __forceinline__ int at_length(const AtArgs& a, int64_t b) {
  const int n = a.lens[b];
  return n < 0 ? 0 : (n < a.cap ? n : a.cap);
}

// One workgroup: its share of the tiles of all units (or, without a deal, the
// unit of its number); its wavefronts take 32 keys at a time in turn.
template <int D, int NT>
__global__ __launch_bounds__(kAtThreads, at_workgroups(D, NT) / 256) void at_kernel(AtArgs a) {
  constexpr int KW = D / 32;          // words of codes a lane holds per key (of the scores) or four keys (values)
  constexpr int NQ = D == 256 ? 2 : 1;  // matrix steps of 128 values of a score
  constexpr int NP = D == 64 ? 2 : 4;   // products of a step: two of a query's eight pieces each (D = 64: four)
  constexpr int R = D / 16;           // dimensions of a run = output tiles
  constexpr int H = kAtCols * NT;     // query heads
  constexpr int LD = D + 4;
  constexpr int LPH = D / kMxPerLane; // lanes of a head's row
  __shared__ __align__(16) float os[kAtWaves][H][LD];
  __shared__ float ms[kAtWaves][H], ls[kAtWaves][H];
  __shared__ AtShareLds share;
  // The queries' pieces in the order of the operands, 16 columns of 16 bytes for
  // each column tile, product and block: a read's lanes find column c at place c
  // of the banks' 256 bytes, whatever their block (four sequences of 131072:
  // conflicts in 13% of the LDS's cycles; 46% with pieces in rows and a gap
  // between them; the time is the same).  And their scales.
  constexpr int NB = D == 64 ? 4 : D / 32;
  __shared__ __align__(4) uint8_t qb[H][2][D / 32][4];  // of head, column half, block: the products' scales
  uint8_t* qs = reinterpret_cast<uint8_t*>(&os[0]);
  static_assert(NT * NP * NB * 256 <= (int)sizeof(os), "the pieces lie where the sums will");

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const bool first8 = c < 8;
  const uint32_t third = first8 ? 0x07060302u : 0x0c0c0c0cu;  // columns 8..15 of the second product are zero
  const int units = a.heads * a.ht;   // of a sequence
  int64_t total = 0, pos = 0, end = 0, base = 0;  // places: all, this workgroup's, before sequence b
  int64_t b = 0;
  int wgs = 0;
  if (a.wgs) {
    AtShare s;
    if (!at_share(a.batch, a.wgs, units, share,
                  [&](int64_t i) { return at_cost(at_tiles(at_length(a, i), a.window)); },
                  [](int) { return (int)blockIdx.x; }, s))
      return;
    total = s.total;
    pos = s.pos;
    end = s.end;
    base = s.base;
    b = s.b;
    wgs = s.wgs;
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
    uint32_t piece[8], byte[8];
    at_pieces(v, piece, byte);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int w = D == 64 ? k >> 2 : k >> 1, half = k >> 1 & 1;
      const int chunk = (r / 8 * NP + w) * NB + e0 / 32 + (D == 64 ? 2 * half : 0);
      *reinterpret_cast<uint32_t*>(qs + chunk * 256 + ((k & 1) * 8 + r % 8) * 16 + e0 % 32 / 2) = piece[k];
      if ((e0 & 31) == 0) qb[r][k & 1][e0 / 32][D == 64 ? half * 2 + w : w] = (uint8_t)byte[k];
    }
  }
  __syncthreads();
  // The B operand: in product w column c < 8 holds piece 2 w of query head c,
  // column c + 8 its piece 2 w + 1; a lane's words are block g of a step.  With
  // D = 64 blocks 2 and 3 repeat the two, as the keys' lanes repeat theirs, with
  // the pieces after next: piece 4 w + 2 (g / 2) and the one after it.
  int qsc[NT][NQ];  // the products' scales, a byte each
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < NQ; ++e) {
      const int r = 8 * t + (c & 7);
      qsc[t][e] = D == 64 ? *reinterpret_cast<const uint16_t*>(&qb[r][c >> 3][g & 1][2 * (g >> 1)])
                          : *reinterpret_cast<const int*>(&qb[r][c >> 3][4 * e + g][0]);
    }
  const uint8_t* ql = qs + lane * 16;  // g * 256 + c * 16
  auto query = [&](int t, int e, int w) {
    const mxi4 x = *reinterpret_cast<const mxi4*>(ql + ((t * NP + w) * NB + 4 * e) * 256);
    return mxi8{x[0], x[1], x[2], x[3], 0, 0, 0, 0};
  };

  mxf4 o[NT][R];
  float m[NT], l[NT];  // l: of the lane's keys
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t] = -INFINITY;
    l[t] = 0.f;
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
#pragma unroll
      for (int e = 0; e < NQ; ++e)
#pragma unroll
        for (int w = 0; w < NP; ++w) {
          const mxi8 Q = query(u, e, w);
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            const mxi8 K = {kw[t][e][0], kw[t][e][1], kw[t][e][2], kw[t][e][3], 0, 0, 0, 0};
            acc[t] = at_score(K, Q, acc[t], ks[t][e], qsc[u][e], w);
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
        l[u] *= f;
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[u][j][i] *= f;
      }
      // A probability's first 8 bits go to columns 0..7 of a product, the next
      // 8 to columns 8..15, the last 8 to columns 0..7 of a second one (with
      // pairs, of 17 bits, the outputs of 96 sequences in bfloat16 were 7e-5 of
      // their norm away from the formula's rounding, where float32 sums are 3e-5;
      // the second product takes 4% of their time, of four long ones' 2%).  The normaliser is the sum of the probabilities as they are.
      uint32_t w[4], y[4];
      float sum = 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float x[2], z[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float p = __builtin_amdgcn_exp2f(s[u][q / 2][2 * (q & 1) + e] - base);
          sum += p;
          const float r = p - __uint_as_float(__float_as_uint(p) & 0xffff0000u);
          x[e] = first8 ? p : r;
          z[e] = r - __uint_as_float(__float_as_uint(r) & 0xffff0000u);
        }
        w[q] = __builtin_amdgcn_perm(__float_as_uint(x[1]), __float_as_uint(x[0]), 0x07060302u);
        y[q] = __builtin_amdgcn_perm(__float_as_uint(z[1]), __float_as_uint(z[0]), third);
      }
      l[u] += sum;
      pf[u] = __builtin_bit_cast(mxb8, make_uint4(w[0], w[1], w[2], w[3]));
      pl[u] = __builtin_bit_cast(mxb8, make_uint4(y[0], y[1], y[2], y[3]));
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
        o[u][2 * q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, pl[u], o[u][2 * q], 0, 0, 0);
        o[u][2 * q + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vb, pl[u], o[u][2 * q + 1], 0, 0, 0);
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
    const float sum = at_colsum(l[t]);
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
  if (a.nt == 1) at_kernel<D, 1><<<grid, kAtThreads, 0, s>>>(a);
  else at_kernel<D, 2><<<grid, kAtThreads, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.wgs) return e;
  const int rows = at_join_rows(units, a.nt, D);
  at_join_kernel<D><<<dim3((unsigned)(units * (kAtCols * a.nt / rows))), kAtThreads, 0, s>>>(a, rows);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_paged_attention(const AtArgs& a, hipStream_t s) {
  if (a.pg.D == 64) return at_launch<64>(a, s);
  if (a.pg.D == 128) return at_launch<128>(a, s);
  return at_launch<256>(a, s);
}

}  // namespace brq
