// Attention of a tree of drafted tokens per sequence over the paged 4-bit cache
// (layout: KvPage in mx.h; what it shares with the attention of one token:
// at_dev.h).
//
// The rows of a unit are 16 nt of the (draft, query head) pairs over one
// key-value head of one sequence, in columns of the matrix products: the scores
// S^T = K Q^T from the codes as they lie in the cache and the queries in eight
// 4-bit pieces, a column a row, one product after the other into the same sums;
// the output O^T = V^T P^T with the values in bfloat16 (exact) and a probability
// in three pieces of 8 bits, whatever the rows' type, so that it has its 24 bits, as in the
// attention of one token (of 7 drafts over 1000 tokens, two pieces left 31 to 62 of 28672 bfloat16
// outputs other than the formula's rounding, three 2 to 8, elementary float32 operations 10 to 14;
// the third takes 16% of the largest call's time).
//
// Which keys a row sees differs only among the drafts, and at a window's far
// end: a step of 32 keys that lies clear of both is computed without a mask.
//
// Four wavefronts of a workgroup take 32 keys each in turn over the same rows, of one
// or two column tiles (tr_nt), and join at the part's end.  64 drafts over 8 key-value
// heads of 128 and 64 query heads, four sequences of 32768 tokens: 608 us, bound by what two
// wavefronts a SIMD issue: 80 products and some 240 vector instructions a step.  8 drafts, 32
// sequences of 17 to 16384: 84 us, half of it 512 units' beginnings and ends.
#include "at_dev.h"

namespace brq {
namespace {

// Keys of sequence b: context and drafts, as many as the table has room for.
__device__ __forceinline__ int tr_keys(const TrArgs& a, int64_t b) {
  const int64_t n = a.at.lens[b];
  return n < 0 ? 0 : n + a.tokens < a.at.cap ? (int)n + a.tokens : a.at.cap;
}
__device__ __forceinline__ int tr_tiles_of(const TrArgs& a, int64_t b) {
  return tr_tiles(tr_keys(a, b), tr_skip(a.at.lens[b], a.at.window));
}

// A row's mask, of the drafts that there are.
__device__ __forceinline__ uint64_t tr_mask(const TrArgs& a, int64_t row) {
  return (uint64_t)a.mask[row] & ~0ull >> (kTrTokens - a.tokens);
}

// What a row sees: context from position `from` on, and drafts by their bits.
// Of a window, drafts come last: bits below the last `window` set ones go.
struct TrSeen {
  int from;
  uint32_t lo, hi;
};
__device__ __forceinline__ TrSeen tr_seen(uint64_t m, int ctx, int window) {
  TrSeen s;
  const int ones = __popcll(m);
  s.from = 0;
  if (window > 0) {
    const int64_t from = (int64_t)ctx + ones - window;
    s.from = from <= 0 ? 0 : from < INT32_MAX ? (int)from : INT32_MAX;
    for (int drop = ones - window; drop > 0; --drop) m &= m - 1;  // the lowest set bit
  }
  s.lo = (uint32_t)m;
  s.hi = (uint32_t)(m >> 32);
  return s;
}

__device__ __forceinline__ bool tr_sees(const TrSeen& z, int key, int ctx) {
  const int j = key - ctx;
  return j < 0 ? key >= z.from : ((j < 32 ? z.lo >> (j & 31) : z.hi >> (j & 31)) & 1u) != 0;
}

// Not 0 if one of w's bytes is 253 or more: subtracted from 252 in every byte, the lowest such one
// borrows and has its own highest bit (and no byte below it does).
__device__ __forceinline__ uint32_t tr_large(uint32_t w) { return (0xfcfcfcfcu - w) & w & 0x80808080u; }

// A unit's row: its row of the batch's and its query head; false past the last.
__device__ __forceinline__ bool tr_row(const TrArgs& a, int64_t b, int h, int r, int64_t* row, int* head) {
  const int group = a.at.group, i = r / group;
  *row = b * a.tokens + i;
  *head = h * group + (r - i * group);
  return i < a.tokens;
}
// A row of the output, with nothing seen where its mask is 0.
template <int D>
__device__ __forceinline__ void tr_finish(const TrArgs& a, int64_t row, int head, int c, int lane, float (&o)[8],
                                          float m, float l) {
  const bool there = tr_mask(a, row) != 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = there ? o[e] : 0.f;
  at_finish<D>(a.at, row, head, c, lane, o, m, there ? l : 0.f);
}

template <int D, int NT>
__global__ __launch_bounds__(kAtThreads, tr_workgroups(D, NT) / 256) void tr_kernel(TrArgs t) {
  const AtArgs& a = t.at;
  constexpr int KW = D / 32;            // words of codes a lane holds per key (of the scores) or four keys (values)
  constexpr int NQ = D == 256 ? 2 : 1;  // matrix steps of 128 values of a score
  constexpr int NP = D == 64 ? 4 : 8;   // products of a step: a piece each (D = 64: two)
  constexpr int R = D / 16;             // dimensions of a run = output tiles
  constexpr int H = 16 * NT;            // rows
  constexpr int LD = D + 4;
  constexpr int LPH = D / kMxPerLane;   // lanes of a row
  constexpr int PP = 3;                 // pieces of a probability
  constexpr int NB = D == 64 ? 4 : D / 32;
  // the queries' pieces in the order of the operands (16 columns of 16 bytes for
  // each column tile, product and block); later the wavefronts' sums of a column tile
  constexpr int kPieces = NT * NP * NB * 256, kSums = kAtWaves * 16 * LD * 4;
  __shared__ __align__(16) uint8_t lds[kPieces > kSums ? kPieces : kSums];
  __shared__ __align__(8) uint8_t qb[H][D / 32][8];  // the pieces' scales
  __shared__ TrSeen seen[H];
  __shared__ float ms[kAtWaves][16], ls[kAtWaves][16];
  __shared__ AtShareLds share;
  __shared__ int far[1];  // the first position that every row's window has reached
  uint8_t* qs = lds;
  float (*os)[16][LD] = reinterpret_cast<float (*)[16][LD]>(lds);

  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c = lane & 15, g = lane >> 4;
  const int units = a.heads * a.ht;  // of a sequence
  int64_t total = 0, pos = 0, end = 0, base = 0, b = 0;
  int wgs = 0, number = 0;
  if (a.wgs) {
    AtShare s;
    // neighbours in the deal, which read the same keys, on one XCD
    if (!at_share(a.batch, a.wgs, units, share, [&](int64_t i) { return tr_cost(tr_tiles_of(t, i)); },
                  [](int n) { return tr_number(blockIdx.x, n); }, s))
      return;
    total = s.total;
    pos = s.pos;
    end = s.end;
    base = s.base;
    b = s.b;
    wgs = s.wgs;
    number = s.w;
  } else {
    b = blockIdx.x / (uint32_t)units;
    const int cost = tr_cost(tr_tiles_of(t, b)), u = (int)(blockIdx.x - (uint32_t)b * (uint32_t)units);
    pos = (int64_t)u * cost;
    end = pos + cost;
    if (pos == end) {  // no key: the unit's rows get what an empty sum gives
      for (int r = tid / LPH; r < H; r += kAtThreads / LPH) {
        int64_t row;
        int head;
        float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (tr_row(t, b, u / a.ht, u % a.ht * H + r, &row, &head))
          tr_finish<D>(t, row, head, (tid % LPH) * kMxPerLane, lane, v, 0.f, 0.f);
      }
      return;
    }
  }
  while (pos < end) {
  // the part's keys: tiles [tb, te) of unit u of sequence b
  const int ctx = a.lens[b], n = tr_keys(t, b);
  const int s0 = tr_skip(ctx, a.window), tiles = tr_tiles(n, s0);
  const int cost = tr_cost(tiles);
  if (pos >= base + (int64_t)cost * units) {  // on to the next sequence (one without keys has no place)
    base += (int64_t)cost * units;
    ++b;
    continue;
  }
  const int u = (int)((pos - base) / cost);
  const int64_t g0 = base + (int64_t)u * cost + kTrLead;  // place of the unit's first tile
  const int tb = pos > g0 ? (int)(pos - g0) : 0;
  const int te = end - g0 < tiles ? (int)(end - g0) : tiles;
  pos = g0 + tiles < end ? g0 + tiles : end;
  if (te <= tb) continue;  // only of the unit's lead
  const int h = u / a.ht, r0 = (u - h * a.ht) * H;  // key-value head; the unit's first row
  if (wgs && tb == 0 && tid == 0)  // who has the unit's parts, and the first one's slot, for the join
    a.who[b * units + u] = make_int2((int)at_slot(number, g0, total, wgs),
                                     te == tiles ? 0 : at_owner(g0 + tiles - 1, total, wgs) - number);

  // Places in a page, with the dimension known; of the 16 tokens from p on, keys and
  // values of either kind lie p times as many bytes into their part of it.
  const KvPage pp{D, a.pg.P};
  const int64_t pbytes = pp.bytes(), stride = a.heads * pbytes;
  const uint8_t* head = a.cache + h * pbytes;
  typedef const __attribute__((address_space(4))) int32_t* Table;  // not written while this runs: scalar loads
  const Table table = (Table)(a.table + b * a.ldt);
  const uint32_t pages = (uint32_t)(a.pages < kAtMaxKeys ? a.pages : kAtMaxKeys);
  int k0 = s0 + tb * kAtTile + wave * kAtKeys;
  const int kend = s0 + te * kAtTile < n ? s0 + te * kAtTile : n;
  // Operands of 32 keys, 16 of them from one page, fetched a step ahead as in
  // the attention of one token.  Where there is no key, or no page, page 0 is read and
  // masked below.
  int page[2];
  bool ok[2];
  const uint8_t *code[2], *scale[2];  // of the 16 keys: in the keys' codes; from the page's beginning on in scales
  mxi4 kw[2][NQ];
  uint32_t vw[2][KW], vs[2];
  int ks[2][NQ];
  const int blk0 = D == 64 ? (g & 1) : g;  // D = 64: both halves of the lanes hold the 64 values
  uint32_t kc_at = c * (D / 2) + 16 * blk0, ks_at = (uint32_t)pp.kscale(0) + c * (D / 32) + blk0;
  uint32_t vc_at = (uint32_t)pp.vcode(0, 0) + g * (2 * D) + c * (D / 8);
  uint32_t vs_at = (uint32_t)pp.vscale(0, 0) + g * (D / 8) + (c * D / 512) * 4;
  auto look_up = [&](int k) {
#pragma unroll
    for (int t = 0; t < 2; ++t) page[t] = table[(k + 16 * t < n ? k + 16 * t : n - 1) >> a.lgP];
  };
  auto fetch_keys = [&](int k) {  // looked up before; looks up the next
    asm volatile("" : "+v"(kc_at), "+v"(ks_at));  // offsets of 32 bits stay such
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int pg = __builtin_amdgcn_readfirstlane(page[t]);
      ok[t] = (uint32_t)pg < pages && k + 16 * t < n;
      const uint8_t* pb = head + (uint64_t)(uint32_t)(ok[t] ? pg : 0) * stride;
      const uint32_t p = (uint32_t)(k + 16 * t) & (uint32_t)(a.pg.P - 1);
      code[t] = pb + p * (D / 2);
      scale[t] = pb + p * (D / 32);
#pragma unroll
      for (int e = 0; e < NQ; ++e) {
        kw[t][e] = *reinterpret_cast<const mxi4*>(code[t] + 64 * e + kc_at);
        ks[t][e] = *(scale[t] + 4 * e + ks_at);
      }
    }
    look_up(k + kAtTile);
  };
  auto fetch_values = [&]() {  // of the keys fetched last
    asm volatile("" : "+v"(vc_at), "+v"(vs_at));
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if constexpr (D == 64) {
        const uint2 y = *reinterpret_cast<const uint2*>(code[t] + vc_at);
        vw[t][0] = y.x; vw[t][1] = y.y;
      } else {
#pragma unroll
        for (int q = 0; q < KW / 4; ++q) {
          const uint4 y = *reinterpret_cast<const uint4*>(code[t] + 16 * q + vc_at);
          vw[t][4 * q] = y.x; vw[t][4 * q + 1] = y.y; vw[t][4 * q + 2] = y.z; vw[t][4 * q + 3] = y.w;
        }
      }
      vs[t] = *reinterpret_cast<const uint32_t*>(scale[t] + vs_at);
    }
  };
  if (k0 < kend) {
    look_up(k0);
    fetch_keys(k0);
    fetch_values();
  }
  // what the rows see; one that sees nothing is given all here and cleared at the end
  if (tid == 0) far[0] = 0;
  __syncthreads();
  if (tid < H) {
    int64_t row;
    int head;
    TrSeen s = {0, 0u, 0u};
    if (tr_row(t, b, h, r0 + tid, &row, &head)) {
      const uint64_t m = tr_mask(t, row);
      s = tr_seen(m, ctx, a.window);
      if (m == 0) s.from = 0;
    }
    seen[tid] = s;
    if (s.from > 0) atomicMax(&far[0], s.from);
  }
  // queries: rotated, times the scale, in pieces
  const float sl = a.scale * 1.44269504088896341f;  // scores in units of log2
  constexpr int kPass = kAtThreads / LPH, kRows = H < kPass ? 1 : H / kPass;  // rows of a pass, passes
  const int e0 = (tid % LPH) * kMxPerLane;
  float qv[kRows][8];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {  // all on their way before the first is waited for
    int64_t row;
    int head;
#pragma unroll
    for (int e = 0; e < 8; ++e) qv[i][e] = 0.f;
    if (tid / LPH < H && tr_row(t, b, h, r0 + tid / LPH + i * kPass, &row, &head))
      at_load8(a.qt, a.q, row * a.ldq + (int64_t)head * D + e0, qv[i]);
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int r = tid / LPH + i * kPass;
    if (r >= H) break;  // uniform over the row's lanes
    float (&v)[8] = qv[i];
    if (a.d) {
      if (a.signs)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= a.signs[e0 + e];
      mx_hadamard<D>(v, lane);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= a.rnorm;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= sl;
    uint32_t piece[8], byte[8];
    at_pieces(v, piece, byte);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int w = D == 64 ? k >> 1 : k;
      const int chunk = (r / 16 * NP + w) * NB + e0 / 32 + (D == 64 ? 2 * (k & 1) : 0);
      *reinterpret_cast<uint32_t*>(qs + chunk * 256 + r % 16 * 16 + e0 % 32 / 2) = piece[k];
      // D = 64: the even pieces' scales, then the odd ones'
      if ((e0 & 31) == 0) qb[r][e0 / 32][D == 64 ? (k & 1) * 4 + w : k] = (uint8_t)byte[k];
    }
  }
  __syncthreads();
  // scales of a column's pieces, four to a word
  int qsc[NT][NQ][NP / 4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < NQ; ++e)
#pragma unroll
      for (int q = 0; q < NP / 4; ++q)
        qsc[t][e][q] = D == 64 ? *reinterpret_cast<const int*>(&qb[16 * t + c][g & 1][4 * (g >> 1)])
                               : *reinterpret_cast<const int*>(&qb[16 * t + c][4 * e + g][4 * q]);
  const uint8_t* ql = qs + lane * 16;  // g * 256 + c * 16
  auto query = [&](int t, int e, int w) {
    return *reinterpret_cast<const mxi4*>(ql + ((t * NP + w) * NB + 4 * e) * 256);
  };
  const int reach = far[0];  // from here to the context's end nothing is masked

  mxf4 o[NT][R];
  // m: the maximum, 0 while no key was seen; then least is -infinity, afterwards 0; l: of the lane's keys
  float m[NT], least[NT], l[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    m[t] = 0.f;
    least[t] = -INFINITY;
    l[t] = 0.f;
#pragma unroll
    for (int j = 0; j < R; ++j) o[t][j] = mxf4{0.f, 0.f, 0.f, 0.f};
  }
  auto no_value = [&](int t, int i) {  // key i of the lane's four: zero
    vs[t] = (vs[t] & ~(255u << (8 * i))) | 127u << (8 * i);
    if constexpr (D == 64) {
      vw[t][i / 2] &= ~(0xffffu << (16 * (i & 1)));
    } else {
#pragma unroll
      for (int q = 0; q < KW / 4; ++q) vw[t][i * (KW / 4) + q] = 0u;
    }
  };
  // One step of 32 keys.  The last one fetches nothing (and is code of its own:
  // under a condition in the loop, the fetches would be waited for at once).
  auto step = [&](auto last) {
    constexpr bool more = !decltype(last)::value;
    asm volatile("" ::: "memory");  // the queries stay in LDS
    // scores: column c, keys 16 t + 4 g + i
    float s[NT][2][4];
    // A piece takes as long to come from LDS as six of these products take, so
    // four are on their way ahead (left to itself, the compiler waits for each: four
    // sequences of 32768 tokens and 64 drafts took 646 us, so 584).
    mxf4 acc[NT][2];
#pragma unroll
    for (int u = 0; u < NT; ++u) acc[u][0] = acc[u][1] = mxf4{0.f, 0.f, 0.f, 0.f};
    constexpr int kAhead = 4, kReads = NQ * NP * NT;
    mxi4 Q[kReads];  // piece i: column tile i % NT, product i / NT of them
#pragma unroll
    for (int i = 0; i < kAhead; ++i) Q[i] = query(i % NT, i / NT / NP, i / NT % NP);
#pragma unroll
    for (int i = 0; i < kReads; ++i) {
      const int j = i + kAhead, u = i % NT, e = i / NT / NP, w = i / NT % NP;
      __builtin_amdgcn_sched_barrier(0);
      if (j < kReads) Q[j] = query(j % NT, j / NT / NP, j / NT % NP);
      __builtin_amdgcn_sched_barrier(0);
      const mxi8 B = {Q[i][0], Q[i][1], Q[i][2], Q[i][3], 0, 0, 0, 0};
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const mxi8 K = {kw[t][e][0], kw[t][e][1], kw[t][e][2], kw[t][e][3], 0, 0, 0, 0};
        acc[u][t] = at_score(K, B, acc[u][t], ks[t][e], qsc[u][e][w / 4], w);
      }
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < NT; ++u)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[u][t][i] = acc[u][t][i];
    // masked keys: scores to -infinity, values that no row sees to zero
    if (k0 < reach || k0 + kAtKeys > ctx || !ok[0] || !ok[1]) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = k0 + 16 * t + 4 * g + i;
          const bool none = key >= n || !ok[t];
#pragma unroll
          for (int u = 0; u < NT; ++u) {
            if (none || !tr_sees(seen[16 * u + c], key, ctx)) s[u][t][i] = -INFINITY;
          }
          if (none) no_value(t, i);
        }
    }
    if constexpr (more) fetch_keys(k0 + kAtTile);
    // Scores relative to the rows' maxima so far.  Seldom after the first tiles is one
    // larger; only then are the four lanes of a column compared and the sums rescaled.
    bool moved = false;
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      float top = -INFINITY;
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[u][t][i] -= m[u];
          top = fmaxf(top, s[u][t][i]);
        }
      moved |= top > least[u];
    }
    if (__builtin_amdgcn_ballot_w64(moved)) {
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        float top = least[u];
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) top = fmaxf(top, s[u][t][i]);
        top = at_colmax(top);
        if (top > -INFINITY) {
          const float f = __builtin_amdgcn_exp2f(tr_rescale(top));
          m[u] += top;
          least[u] = 0.f;
          l[u] *= f;
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[u][t][i] -= top;
#pragma unroll
          for (int j = 0; j < R; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[u][j][i] *= f;
        }
      }
    }
    // A probability's first 8 bits, the next ones, the last ones.
    mxb8 pf[NT][PP];
#pragma unroll
    for (int u = 0; u < NT; ++u) {
      uint32_t w[PP][4];
      float sum = 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float x[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          x[e] = __builtin_amdgcn_exp2f(s[u][q / 2][2 * (q & 1) + e]);
          sum += x[e];
        }
#pragma unroll
        for (int z = 0; z < PP; ++z) {
          w[z][q] = __builtin_amdgcn_perm(__float_as_uint(x[1]), __float_as_uint(x[0]), 0x07060302u);
#pragma unroll
          for (int e = 0; e < 2; ++e) x[e] -= __uint_as_float(__float_as_uint(x[e]) & 0xffff0000u);
        }
      }
      l[u] += sum;
#pragma unroll
      for (int z = 0; z < PP; ++z) pf[u][z] = __builtin_bit_cast(mxb8, make_uint4(w[z][0], w[z][1], w[z][2], w[z][3]));
    }
    // A value is multiplied by the zeros of rows that do not see it, and by those that a
    // probability's lower pieces can be, so one that is not finite (its scale's byte
    // is 253 or more) is taken out here and added below to the rows that see it.
    uint32_t odd = 0u;  // such keys of the lane's block: bit 4 t + i
    const bool any = __builtin_amdgcn_ballot_w64((tr_large(vs[0]) | tr_large(vs[1])) != 0u) != 0;  // of the step's
    if (any) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if ((vs[t] >> (8 * i) & 255u) >= 253u) {
            odd |= 1u << (4 * t + i);
            no_value(t, i);
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
      for (int z = 0; z < PP; ++z)
#pragma unroll
        for (int u = 0; u < NT; ++u) {
          o[u][2 * q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(va, pf[u][z], o[u][2 * q], 0, 0, 0);
          o[u][2 * q + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vb, pf[u][z], o[u][2 * q + 1], 0, 0, 0);
        }
    }
    if (any) {
      // The values that were taken out, a key at a time, from the cache again: a
      // product of that key alone, added where the row sees it.
#pragma unroll 1
      for (int kk = 0; kk < 32; ++kk) {
        const int tt = kk >> 4, gg = kk >> 2 & 3, i = kk & 3, key = k0 + kk;
        if (!__builtin_amdgcn_ballot_w64(g == gg && (odd >> (4 * tt + i) & 1u) != 0)) continue;
        const uint8_t* pb = head + (uint64_t)(uint32_t)table[key >> a.lgP] * stride;
        const int p = key & (a.pg.P - 1);
        const uint32_t byte = pb[pp.vscale(p, c * D / 512)];
        const bool keep = g == gg && byte >= 253u;
        uint32_t run[KW / 4 + 1] = {};  // the lane's run of the key, eight codes a word
        if (keep) {
          const uint8_t* vp = pb + pp.vcode(p, c);
          if constexpr (D == 64) run[0] = *reinterpret_cast<const uint16_t*>(vp);
#pragma unroll
          for (int q = 0; q < KW / 4; ++q) run[q] = reinterpret_cast<const uint32_t*>(vp)[q];
        }
        const float scale = __uint_as_float(byte << 23);
        const uint32_t half = keep ? (i & 1 ? 0xffff0000u : 0x0000ffffu) : 0u;  // of the pair of keys
        const int pair = 2 * tt + i / 2;
        bool sees[NT];
#pragma unroll
        for (int u = 0; u < NT; ++u) sees[u] = tr_sees(seen[16 * u + c], key, ctx);
#pragma unroll
        for (int q = 0; q < R / 2; ++q) {
          const uint32_t x = at_bits(at_pair(run[q / 4], scale, q));
          const uint32_t xl = __builtin_amdgcn_perm(x, x, 0x01000100u) & half, xh = __builtin_amdgcn_perm(x, x, 0x03020302u) & half;
          // an infinity times a piece that is 0 would be NaN: only the first piece, which is not, meets it
          auto place = [&](uint32_t y, bool first) {
            const uint32_t inf = 0x7f807f80u & half;
            y = !first && (y & inf) == inf ? 0u : y;
            return __builtin_bit_cast(mxb8, make_uint4(pair == 0 ? y : 0u, pair == 1 ? y : 0u, pair == 2 ? y : 0u, pair == 3 ? y : 0u));
          };
#pragma unroll
          for (int u = 0; u < NT; ++u) {
            mxf4 x0 = {0.f, 0.f, 0.f, 0.f}, x1 = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int z = 0; z < PP; ++z) {
              x0 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(place(xl, z == 0), pf[u][z], x0, 0, 0, 0);
              x1 = __builtin_amdgcn_mfma_f32_16x16x32_bf16(place(xh, z == 0), pf[u][z], x1, 0, 0, 0);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              o[u][2 * q][e] += sees[u] ? x0[e] : 0.f;
              o[u][2 * q + 1][e] += sees[u] ? x1[e] : 0.f;
            }
          }
        }
      }
    }
    if constexpr (more) fetch_values();
  };
  for (; k0 + kAtTile < kend; k0 += kAtTile) step(std::false_type{});
  if (k0 < kend) step(std::true_type{});

  // join the wavefronts, a column tile at a time: all parts to the common
  // maximum, summed in order
#pragma unroll
  for (int u16 = 0; u16 < NT; ++u16) {
    __syncthreads();  // the sums go where the queries were, or the tile before
    const float sum = at_colsum(l[u16]);
    if (lane < 16) {
      ms[wave][lane] = least[u16] == 0.f ? m[u16] : -INFINITY;
      ls[wave][lane] = sum;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < R; ++j) os[wave][c][(4 * g + i) * R + j] = o[u16][j][i];
    __syncthreads();
    for (int r = tid / LPH; r < 16; r += kAtThreads / LPH) {
      int64_t row;
      int head;
      if (!tr_row(t, b, h, r0 + 16 * u16 + r, &row, &head)) continue;  // uniform over the row's lanes
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
        tr_finish<D>(t, row, head, e0, lane, v, M, L);
      } else {
        float* p = a.part + (at_slot(number, g0, total, wgs) * H + 16 * u16 + r) * (D + 4);
        mx_store8<BRQ_F32>(p, e0, v);
        if (e0 == 0) *reinterpret_cast<float2*>(p + D) = make_float2(M, L);
      }
    }
  }
  __syncthreads();  // the next part's queries go where these sums were
  }
}

// Joins the parts of units that span workgroups and writes the rows of
// sequences without keys, as at_join_kernel; `rows` rows of one unit to a workgroup.
template <int D>
__global__ __launch_bounds__(kAtThreads) void tr_join_kernel(TrArgs t, int rows) {
  const AtArgs& a = t.at;
  constexpr int LPH = D / kMxPerLane;
  constexpr int LD = D + 4;
  __shared__ float os[kAtThreads / LPH][LD];
  const int tid = threadIdx.x, lane = tid & 63;
  const int H = 16 * a.nt, units = a.heads * a.ht, per = H / rows;
  const int64_t ub = blockIdx.x / (uint32_t)per;
  const int64_t b = ub / units;
  const int u = (int)(ub - b * units);
  const int tiles = tr_tiles_of(t, b);
  const int r = (int)(blockIdx.x - (uint32_t)ub * (uint32_t)per) * rows + tid / LPH % rows;
  const int grp = tid / (LPH * rows), groups = kAtThreads / (LPH * rows);
  const int e0 = (tid % LPH) * kMxPerLane;
  int64_t row;
  int head;
  const bool mine = tr_row(t, b, u / a.ht, u % a.ht * H + r, &row, &head);
  float M = -INFINITY, L = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (tiles > 0) {
    const int2 who = a.who[ub];
    if (who.y == 0) return;  // finished by its workgroup
    // part s (of who.y + 1) is the first of workgroup who.x / 2 + s
    const float* p0 = a.part + r * (int64_t)LD;
#pragma unroll 2
    for (int s = grp; s <= who.y && mine; s += groups) {
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
  tr_finish<D>(t, row, head, e0, lane, o, M, L);
}

template <int D>
hipError_t tr_launch(const TrArgs& t, hipStream_t s) {
  const AtArgs& a = t.at;
  const int64_t units = a.batch * a.heads * a.ht;
  const dim3 grid((unsigned)(a.wgs ? a.wgs : units));
  if (D == 256 || a.nt == 1) tr_kernel<D, 1><<<grid, kAtThreads, 0, s>>>(t);
  else if constexpr (D != 256) tr_kernel<D, 2><<<grid, kAtThreads, 0, s>>>(t);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || !a.wgs) return e;
  const int rows = tr_join_rows(units, a.nt, D);
  tr_join_kernel<D><<<dim3((unsigned)(units * (16 * a.nt / rows))), kAtThreads, 0, s>>>(t, rows);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_tree_attention(const TrArgs& t, hipStream_t s) {
  if (t.at.pg.D == 64) return tr_launch<64>(t, s);
  if (t.at.pg.D == 128) return tr_launch<128>(t, s);
  return tr_launch<256>(t, s);
}

}  // namespace brq
