// Microscaled 4-bit rows (MX4): launch arguments and the index arithmetic
// shared by the kernels (mx.hip, mx_matmul.hip, kv.hip, kv_attn.hip) and the
// host dry-run checker.
//
// Element lanes: a lane holds 8 consecutive values of a row (16 where it also
// transforms them for the quantizer: half the exchanges between lanes), so a
// block of 32 spans 4 (2) lanes and a transform of d values d / 8 (d / 16);
// both are aligned, since rows are whole blocks (whole transforms).
#pragma once

#include "brq_internal.h"

namespace brq {

constexpr int kMxBlock = 32;      // values that share a scale
constexpr int kMxPerLane = 8;
constexpr int kMxThreads = 256;   // four wavefronts per workgroup
constexpr int64_t kMxMost = (int64_t)1 << 34;  // values of a call: within 2^32 threads a launch

// ---- quantize / dequantize (mx.hip)

struct MxArgs {
  const void* x;         // quantize input [rows][ldx]
  int xt;
  int64_t ldx;
  void* y;               // dequantize output [rows][ldy]
  int yt;
  int64_t ldy;
  int64_t rows;
  int per;               // values per lane: 8 or 16
  uint32_t lpr;          // lanes per row: n / per
  uint64_t lanes;        // rows * lpr
  int gap;               // rows do not follow one another in x or y
  uint8_t* codes;        // [rows][n/2]
  uint8_t* scales;       // [rows][n/32]
  const float* signs;    // the transform's signs, or null
  int d;                 // transform length (0: none)
  float rnorm;           // fl(1 / sqrt(d))
};

// Row and first column of lane li (li < a.lanes).
__host__ __device__ inline void mx_lane(uint32_t lpr, int per, uint64_t li, int64_t* row, int64_t* col) {
  const uint64_t r = (li >> 32) ? li / lpr : (uint64_t)((uint32_t)li / lpr);
  *row = (int64_t)r;
  *col = (int64_t)(li - r * lpr) * per;
}

hipError_t launch_mx_quant(const MxArgs& a, hipStream_t s);
hipError_t launch_mx_dequant(const MxArgs& a, hipStream_t s);

// ---- product (mx_matmul.hip)

struct MmArgs {
  const uint8_t* a;      // [T][n/2]
  const uint8_t* as;     // [T][n/32]
  const uint8_t* b;      // [m][n/2]
  const uint8_t* bs;     // [m][n/32]
  int64_t T, m, n;
  void* y;
  int yt;
  int64_t ldy;
  int wide;              // four consecutive outputs may be stored at once
  // tiles (tile > 0)
  int tile;              // rows and columns of a workgroup's tile: 256, 128; 0: no tiles
  int stages;            // of kMmK values
  int64_t gt, go;        // tiles along tokens and outputs
  int band;              // rows of tiles taken together
  int64_t per_xcd;       // tiles per XCD
  int splits, per;       // parts of the long axis, stages per part
  uint8_t *ts, *os;      // scale images of the operands, in the workspace
  float* part;           // [splits][T][m] partial sums, in the workspace
};

constexpr int kMmK = 256;      // values of a row per stage
constexpr int kMmChunk = 512;  // values of a row that a wavefront of the stream takes at a time

// What follows a product's sums: y = act(sum + bias) * mul + res, each part
// where its pointer is not null; in float32, rounded once to y's type.
struct MmEpi {
  int act;               // brq_act
  const void* bias;      // [m], or [groups][m]
  int bt;
  const void* mul;       // [T][ldm]
  int mt;
  int64_t ldm;
  const void* res;       // [T][ldr]
  int rt;
  int64_t ldr;
  int wide;              // four consecutive values of each may be read at once
};
struct MmNoEpi {};       // the plain product

// erfc(z) exp(z^2) is t times this, t = 1 / (1 + z / 2): a polynomial of degree 8, fitted to
// erfc, whose value is within 1.4 2^-24 of it up to z = 12 (float32's exp(-z^2) is 0 beyond).
__host__ __device__ inline float mm_fma(float a, float b, float c) { return __builtin_fmaf(a, b, c); }
__host__ __device__ inline double mm_fma(double a, double b, double c) { return __builtin_fma(a, b, c); }
template <class F>
__host__ __device__ inline F mm_gelu_tail(F t) {
  F p = -0.059385716915130615f;
  p = mm_fma(p, t, F(0.28612077236175537f));
  p = mm_fma(p, t, F(-0.49040067195892334f));
  p = mm_fma(p, t, F(0.28172776103019714f));
  p = mm_fma(p, t, F(-0.029145410284399986f));
  p = mm_fma(p, t, F(0.20375148952007294f));
  p = mm_fma(p, t, F(0.24283531308174133f));
  p = mm_fma(p, t, F(0.2824120819568634f));
  return mm_fma(p, t, F(0.2820843458175659f));
}

// Launches within 2^32 threads (at most 64 per 16 x 16 outputs, 32 per row).
inline bool mm_supported(int64_t T, int64_t m, int64_t n) {
  const int64_t most = (int64_t)1 << 28;
  return T <= most && m <= most && n <= most && (m == 0 || T <= kMxMost / 2 / m);
}

// Kernel and workspace of a product (a.T, a.m, a.n set), with an epilogue or
// without: returns the workspace bytes.
inline size_t mm_plan(MmArgs& a, uint8_t* ws, bool epilogue) {
  a.tile = 0;
  a.splits = 1;
  if (a.n < kMmK || a.n > (1 << 23)) return 0;
  // The stream over the weight up to 64 tokens; above 32 only while the tiles'
  // three launches weigh more (64 tokens: 8192x28672 stream 53 us, tiles 47;
  // 16384x8192 35 and 31; 4096x4096 10 and 16).
  if (a.T <= 32 || (a.T <= 64 && a.m * a.n < ((int64_t)1 << 27))) return 0;
  auto tiles = [&](int64_t t) { return ((a.T + t - 1) / t) * ((a.m + t - 1) / t); };
  // One 256 x 256 tile per compute unit at a time, two of 128 x 128; such a
  // pair takes about 2/3 of a large tile's time for half its work.
  // An epilogue's operands and activations are worked on while the other tile of a pair
  // is multiplied, but by a large tile alone, for as long as 11 stages take it
  // (2048x28672x8192 with bias and gelu: large 318 us, small 299; with factor and
  // residual too 396 and 348; 4096x8192x8192 169 and 173, 186 and 180).
  a.stages = (int)((a.n + kMmK - 1) / kMmK);
  const int64_t large = (tiles(256) + 255) / 256 * 3, small = (tiles(128) + 511) / 512 * 2;
  a.tile = (epilogue ? large * (a.stages + 11) <= small * (a.stages + 3) : large <= small) ? 256 : 128;
  a.gt = (a.T + a.tile - 1) / a.tile;
  a.go = (a.m + a.tile - 1) / a.tile;
  // Too few tiles for the chip: the long axis in parts, of eight stages or more
  // up to a workgroup for each compute unit, of 28 or more up to two (their
  // sums written and read cost what shorter parts save: 384x4096 by 8192, 2
  // parts 24 us, 4 parts 27; by 65536, 2 parts 120 us, 5 parts 97;
  // 128x8192x28672, 2, 4 and 8 parts 62, 50 and 53 us).
  a.per = a.stages;
  if (a.tile == 128 && tiles(128) <= 256) {
    auto least = [](int64_t x, int64_t y) { return x < y ? x : y; };
    const int64_t one = least(256 / tiles(128), a.stages / 8), two = least(512 / tiles(128), a.stages / 28);
    const int64_t parts = one > two ? one : two;
    if (parts > 1) a.per = (int)((a.stages + parts - 1) / parts);
  }
  a.splits = (a.stages + a.per - 1) / a.per;
  a.per_xcd = (a.gt * a.go * a.splits + 7) / 8;
  a.band = 4;
  const int64_t image = (int64_t)a.stages * (kMmK / kMxBlock) * a.tile;
  a.ts = ws;
  a.os = ws + a.gt * image;
  a.part = reinterpret_cast<float*>(a.os + a.go * image);
  return (size_t)((a.gt + a.go) * image) + (a.splits > 1 ? (size_t)a.splits * a.T * a.m * sizeof(float) : 0);
}

// Index arithmetic of the tile kernels.

// A workgroup's tile and part.  Blocks go to the XCDs in turn, so those with
// one remainder by 8 take consecutive places, whose tiles share operands; a
// place is a part, in it a band of rows of tiles, in it the rows fastest.
// False: no tile for this workgroup.
struct MmWhere {
  int64_t tt, to;  // the tile, along tokens and outputs
  int part;
};
__host__ __device__ inline void mm_place(int64_t p, int64_t gt, int64_t go, int rows, MmWhere& w) {
  const int64_t band = p / (rows * go), q = p - band * rows * go;
  const int64_t h = gt - band * rows < rows ? gt - band * rows : rows;  // rows of tiles in this band
  w.tt = band * rows + q % h;
  w.to = q / h;
}
__host__ __device__ inline bool mm_where(const MmArgs& a, uint32_t block, MmWhere& w) {
  int64_t p = (int64_t)(block & 7) * a.per_xcd + (block >> 3);
  if (p >= a.gt * a.go * a.splits) return false;
  w.part = (int)(p / (a.gt * a.go));
  mm_place(p - w.part * (a.gt * a.go), a.gt, a.go, a.band, w);
  return true;
}
// Place in LDS of 16-byte piece c of row r, in pieces: the pieces c of sixteen
// consecutive rows lie in sixteen different places of 256 bytes, the width of
// the banks (by r & 7, eight of 128 bytes, half of the reads' cycles were
// conflicts; 384x4096x65536 100 -> 99 us).  XOR: piece of place, too.
__host__ __device__ constexpr int mm_piece(int r, int c) { return r * 8 + (c ^ (r >> 1 & 7)); }
// Place of the scale of block c of row r in a stage of a tile of R rows.
__host__ __device__ constexpr int mm_scale_at(int R, int c, int r) { return (c * 32 + r % 32) * (R / 32) + r / 32; }

// Rows of the weight per workgroup of the stream.  32 where that still gives
// every compute unit one: the activations are read half as often (8192x28672:
// 16 tokens 37 -> 30 us, 64 tokens 83 -> 53 us).
inline int mm_stream_rows(const MmArgs& a) { return a.m >= 32 * 256 ? 32 : 16; }
// Wavefronts of a workgroup of the stream.  With one workgroup for each compute
// unit or less, eight: more of a long row is in flight (one token at 4096x28672
// 14.0 us, with four 16.9; at 4096x4096 4.1 both).  Beyond that four, or one
// workgroup of eight keeps the next off its unit: 257 and more workgroups of 32
// rows take 3 to 18% less with four at lengths of 512 to 28672 (16x9216x4000 9.8
// us, with eight 11.3; 16x9216x5120 10.1 and 10.8), of 16 rows up to 25% less
// above 16 tokens, otherwise the same within 4%.
inline int mm_stream_waves(int64_t wgs) { return wgs > 256 ? 4 : 8; }

hipError_t launch_mx_matmul(const MmArgs& a, hipStream_t s);
hipError_t launch_mx_linear(const MmArgs& a, const MmEpi& e, hipStream_t s);

// ---- products grouped by expert (mx_grouped.hip)

struct GmArgs {
  MmArgs mm;             // T rows, m outputs; b, bs: of group 0, the others' behind
  const int32_t* offs;   // [groups + 1]
  int groups;
  int rows;              // of a unit: 16 or 32 of the stream, a tile's 128 or 256
};

// Rows [b, end) of a group from its two offsets, within the T rows there are; of
// offsets that do not decrease.
__host__ __device__ inline void gm_rows(int from, int to, int T, int* b, int* end) {
  *b = from < 0 ? 0 : from < T ? from : T;
  *end = to < 0 ? 0 : to < T ? to : T;
}
// The most units of R rows that the groups can have: each begins at most one
// that is not whole.
inline int64_t gm_units(int64_t T, int64_t groups, int64_t R) { return T / R + (groups < T ? groups : T); }
__host__ __device__ inline const void* gm_bias(const MmEpi& e, int64_t group, int64_t m) {
  if (!e.bias) return nullptr;
  return static_cast<const char*>(e.bias) + group * m * (e.bt == BRQ_F32 ? 4 : 2);
}
// Kernel of a grouped product (g.mm.T, m, n and g.groups set, none of the first two and the
// last 0): a group's units are taken by the stream over its weight, or by tiles through LDS.
inline void gm_choose(GmArgs& g) {
  MmArgs& a = g.mm;
  a.tile = 0;
  a.splits = 1;
  g.rows = 16;
  if (a.n > (1 << 23) || a.n < kMmK) return;
  // Rows a group in the mean, up to which the stream takes less time than tiles
  // (8 groups of 11008x4096, 16, 32 and 40 rows: 46, 61 and 103 us, tiles of 128 66, 66 and 69).
  const int64_t mean = a.T / g.groups;
  if (mean <= 32) {
    g.rows = mean <= 16 ? 16 : 32;
    return;
  }
  // as many units as are to be expected: half of a group's last one is empty, none all of it
  const int64_t some = g.groups < a.T ? g.groups : a.T;
  auto tiles = [&](int64_t t) {
    const int64_t units = a.T / t + some / 2;
    return (units > some ? units : some) * ((a.m + t - 1) / t);
  };
  // As for one product (mm_plan), what follows the stages for an epilogue and without one
  // alike, and rounds in fractions, since the groups' sizes are not known.
  auto most = [](int64_t x, int64_t y) { return x > y ? x : y; };
  a.stages = (int)((a.n + kMmK - 1) / kMmK);
  const int64_t large = most(tiles(256), 256) * 2 * (3 * a.stages + 16), small = most(tiles(128), 512) * (2 * a.stages + 4);
  a.tile = large <= small ? 256 : 128;
  g.rows = a.tile;
  a.per = a.stages;
  a.gt = gm_units(a.T, g.groups, a.tile);
  a.go = (a.m + a.tile - 1) / a.tile;
  a.band = 4;
}
// The same and the workspace's bytes: the tiles' images of scales, of every unit and of every
// group's weight.
inline size_t gm_plan(GmArgs& g, uint8_t* ws) {
  gm_choose(g);
  MmArgs& a = g.mm;
  if (!a.tile) return 0;
  const int64_t image = (int64_t)a.stages * (kMmK / kMxBlock) * a.tile;
  a.ts = ws;
  a.os = ws + a.gt * image;
  return (size_t)((a.gt + g.groups * a.go) * image);
}
// The stream's workgroups, 32 outputs of a unit each, and their wavefronts: rows of up to four
// chunks take two, longer ones four.
inline int64_t gm_stream_workgroups(const GmArgs& g) { return (g.mm.m + 31) / 32 * gm_units(g.mm.T, g.groups, g.rows); }
inline int gm_stream_waves(int64_t n) { return n <= 4 * kMmChunk ? 2 : 4; }
// Launches within 2^32 threads, of the kernel that is chosen: rows shorter than a stage, or longer
// than 2^23, are the stream's however many a group has, in units of 16.
inline bool gm_supported(int64_t T, int64_t groups, int64_t m, int64_t n) {
  if (!mm_supported(T, m, n) || groups > 1 << 20) return false;
  if (T == 0 || groups == 0 || m == 0) return true;
  GmArgs g = {};
  g.mm.T = T;
  g.mm.m = m;
  g.mm.n = n;
  g.groups = (int)groups;
  gm_choose(g);
  const int64_t most = (int64_t)1 << 32;
  if (!g.mm.tile) return gm_stream_workgroups(g) * 64 * gm_stream_waves(n) < most;
  return (g.mm.gt * g.mm.go + 7) * 256 < most && (g.mm.gt + groups * g.mm.go) * kMxThreads < most;
}

hipError_t launch_mx_grouped(const GmArgs& g, const MmEpi& e, hipStream_t s);

// ---- paged cache (kv.hip) and attention (kv_attn.hip)

constexpr int kKvQuad = 4;        // tokens whose value codes are interleaved
constexpr int kKvRuns = 16;       // runs of D / 16 dimensions

// Layout of one head's page for head dimension D and P tokens (bytes).
struct KvPage {
  int D, P;
  __host__ __device__ int64_t bytes() const { return (int64_t)P * (D + D / 16); }
  // keys' codes of token t (D / 2 bytes)
  __host__ __device__ int64_t kcode(int t) const { return (int64_t)t * (D / 2); }
  // values' codes of run r of token t (D / 32 bytes)
  __host__ __device__ int64_t vcode(int t, int r) const {
    return (int64_t)P * (D / 2) + (int64_t)(t / kKvQuad) * (2 * D) + r * (D / 8) + (t % kKvQuad) * (D / 32);
  }
  // keys' scales of token t (D / 32 bytes)
  __host__ __device__ int64_t kscale(int t) const { return (int64_t)P * D + (int64_t)t * (D / 32); }
  // values' scale of block e of token t
  __host__ __device__ int64_t vscale(int t, int e) const {
    return (int64_t)P * D + (int64_t)P * (D / 32) + (int64_t)(t / kKvQuad) * (D / 8) + e * kKvQuad + t % kKvQuad;
  }
};

struct KvArgs {
  const void* k;         // append: inputs; read: outputs
  const void* v;
  int64_t ldk, ldv;
  int t;                 // their type
  const int64_t* slots;
  int64_t tokens;
  int heads;
  KvPage pg;
  int lgP;               // log2 of the page's tokens
  int64_t pages;
  uint8_t* cache;
  const float* signs;
  int d;                 // transform length: 0 or the head dimension
  float rnorm;
};

constexpr int kKvPerLane = 16;    // values per lane of an append
// Rows of a call: four tokens of one head follow one another, as their value
// codes do in the cache (when their slots do), then the next head.  8190 tokens of 8
// heads of 128 are read in 11.4 us so, in 12.1 token by token.
inline int64_t kv_rows(int64_t tokens, int heads) { return (tokens + kKvQuad - 1) / kKvQuad * kKvQuad * heads; }
__host__ __device__ inline void kv_row(uint32_t row, int heads, int64_t* tok, int* h) {  // rows < 2^31
  const uint32_t quad = row / (uint32_t)(kKvQuad * heads), r = row - quad * (uint32_t)(kKvQuad * heads);
  *tok = (int64_t)quad * kKvQuad + r % kKvQuad;
  *h = (int)(r / kKvQuad);
}
hipError_t launch_kv_append(const KvArgs& a, hipStream_t s);
hipError_t launch_kv_read(const KvArgs& a, hipStream_t s);

// ---- tokens and pages moved, shared, taken, given back (kv_pages.hip)

struct KpMove {
  const int64_t *src, *dst;  // slots
  int64_t tokens;
  int heads;
  KvPage pg;
  int lgP;
  int64_t pages;
  uint8_t* cache;
  uint8_t* ws;           // rows: runs of kKpRun tokens of a head, the heads, then the next run
};
// Bytes of a row of the workspace: the codes and scales of a token's head.
__host__ __device__ constexpr int64_t kp_row_bytes(int D) { return D + D / 16; }
constexpr int64_t kKpTokens = (int64_t)1 << 27;  // heads of tokens of a move: within 2^31 threads of 16 a token and head
constexpr int kKpThreads = 1024;  // of a workgroup that does by itself what has an order: a move, a reservation
constexpr int kKpFew = 512;       // tokens that such a workgroup holds in registers, of one head
constexpr int kKpRun = 4;         // tokens of a head that 16 lanes move at a time
inline int64_t kp_runs(int64_t tokens) { return (tokens + kKpRun - 1) / kKpRun; }
// Whether a move is one launch, of a workgroup for each head: within 2^32 threads.
inline bool kp_few(int64_t tokens, int64_t heads) { return tokens <= kKpFew && heads < ((int64_t)1 << 32) / kKpThreads; }
// Bytes of a move's workspace.
inline size_t kp_move_bytes(int64_t tokens, int64_t heads, int D) {
  return kp_few(tokens, heads) ? 0 : (size_t)(kp_runs(tokens) * kKpRun * heads * kp_row_bytes(D) + 15) / 16 * 16;
}

struct KpFork {
  const int32_t *table, *lens, *parents;
  int64_t batch, width, children, pages;
  int32_t *refs, *out_table, *out_lens;
};
struct KpFree {
  int32_t* table;
  int64_t batch, width, pages, n;
  int32_t* refs;
  const int32_t* rows;   // [n], or null: all rows
};

struct KpReserve {
  uint8_t* cache;
  int32_t* table;
  const int32_t* lens;
  int64_t batch, width;
  int32_t* refs;
  int64_t pages, tokens;
  int heads;
  KvPage pg;
  int lgP;
  int64_t* slots;        // [batch][tokens]
  int64_t per;           // table entries that a row's new tokens can lie in
  // in the workspace
  int4* copy;            // [batch]: page to copy from and to, its tokens
  int32_t* item;         // [batch * per]: the page of an entry, or -1; kp_want's while it has none
  int32_t* fresh;        // free pages
};
// Entries that `tokens` tokens can lie in, from any place of a page on.
__host__ __device__ inline int64_t kp_per(int64_t tokens, int64_t page) { return (tokens + page - 2) / page + 1; }
inline size_t kp_bytes(int64_t batch, int64_t tokens, int64_t page, int64_t pages) {
  const int64_t items = batch * kp_per(tokens, page);
  return (size_t)(16 * batch + 4 * items + 4 * (items < pages ? items : pages) + 15) / 16 * 16;
}

struct KpItem {
  int64_t row, entry;    // of the table
  int used;              // tokens that the entry's page holds already
};
// Item i of a reservation; false: no entry, since the row's new tokens end
// before it, its table does, or its length is negative.
__host__ __device__ inline bool kp_item(const KpReserve& a, int64_t i, KpItem& it) {
  it.row = i / a.per;
  const int64_t k = i - it.row * a.per, n = a.lens[it.row];
  if (n < 0) return false;
  const int64_t first = n >> a.lgP;
  it.entry = first + k;
  it.used = k == 0 ? (int)(n & (a.pg.P - 1)) : 0;
  return it.entry < a.width && it.entry <= (n + a.tokens - 1) >> a.lgP;
}
// An entry that needs a page, before it has one: the how manieth such one it is, and whether
// it leaves a page that others hold.  Below -1, in 32 bits: ranks from kKpRanks on (a pool
// beyond a terabyte) count as that, and get none.
constexpr int kKpRanks = (1 << 30) - 2;
__host__ __device__ inline int32_t kp_want(int rank, bool shared) {
  return -2 - (2 * (rank < kKpRanks ? rank : kKpRanks) + (shared ? 1 : 0));
}
__host__ __device__ inline int kp_rank(int32_t want) { return (-2 - want) >> 1; }
__host__ __device__ inline bool kp_shared(int32_t want) { return ((-2 - want) & 1) != 0; }
// Place in a page, in 16-byte pieces, of piece i of the first tokens' codes (keys',
// then values') and scales (keys', then values'), of `codes` and `scales` pieces each.
__host__ __device__ inline int kp_piece(const KvPage& pg, int codes, int scales, int i) {
  if (i < 2 * codes) return i < codes ? i : pg.P * (pg.D / 32) + i - codes;
  i -= 2 * codes;
  const int base = pg.P * (pg.D / 16);
  return i < scales ? base + i : base + pg.P * pg.D / 512 + i - scales;
}

hipError_t launch_kv_move(const KpMove& a, hipStream_t s);
hipError_t launch_kv_fork(const KpFork& a, hipStream_t s);
hipError_t launch_kv_free(const KpFree& a, hipStream_t s);
hipError_t launch_kv_reserve(const KpReserve& a, hipStream_t s);

constexpr int kAtWaves = 4;       // wavefronts of an attention workgroup
constexpr int kAtThreads = 64 * kAtWaves;
constexpr int kAtKeys = 32;       // keys a wavefront takes at a time
constexpr int kAtTile = kAtWaves * kAtKeys;
constexpr int kAtCols = 8;        // query heads per 16 matrix columns (two pieces of each)

constexpr int kAtMaxKeys = 1 << 30;

constexpr int kAtMaxBatch = 4096;  // sequences whose tiles are dealt out evenly

// A unit is the group of query heads of one workgroup over one sequence's
// keys, in tiles of kAtTile keys.  Up to kAtMaxBatch sequences the tiles of
// all units, in order, are dealt out evenly to a fixed number of workgroups
// that the chip holds at once, whatever the lengths.  Ahead of its tiles a unit
// has kAtLead empty places, since beginning one (its queries, its join) takes
// as long as some tiles: without them a workgroup got fourteen short sequences
// where another got fourteen tiles of a long one, and 96 sequences of 17 to
// 16384 tokens took 117 us (with 1, 2, 3 and 4 places 83, 75, 69 and 68; 64
// sequences of 1000 tokens, none to 4 places, 26, 28, 28, 30 and 30).  Workgroup w has places
// [at_start(w), at_start(w + 1)).  A unit whose tiles lie within one workgroup
// is finished there; the parts of the others go to the workspace, two slots a
// workgroup (a part from before its first place, one that it begins), and are
// joined.
constexpr int kAtLead = 4;
__host__ __device__ inline int at_cost(int tiles) { return tiles > 0 ? tiles + kAtLead : 0; }
// Workgroups that get places: no more than there are, so each has one.
__host__ __device__ inline int at_dealt(int64_t total, int wgs) { return total < wgs ? (int)total : wgs; }
__host__ __device__ inline int64_t at_start(int64_t w, int64_t total, int wgs) { return w * total / wgs; }
// The workgroup that has place g.
__host__ __device__ inline int at_owner(int64_t g, int64_t total, int wgs) {
  return (int)(((g + 1) * wgs - 1) / total);
}
// Slot of the part that workgroup w has of a unit whose first tile is place g0.
__host__ __device__ inline int64_t at_slot(int64_t w, int64_t g0, int64_t total, int wgs) {
  return 2 * w + (at_start(w, total, wgs) < g0 ? 1 : 0);
}
// Keys before the first tile of n keys with a window, and their tiles.
__host__ __device__ inline int at_skip(int n, int window) {
  return window > 0 && n > window ? (n - window) & ~(kAtKeys - 1) : 0;
}
__host__ __device__ inline int at_tiles(int n, int window) {
  return (n - at_skip(n, window) + kAtTile - 1) / kAtTile;
}
// Workgroups that the chip holds at once, by the registers of their kernel.
constexpr int at_workgroups(int head_dim, int nt) {
  if (head_dim == 256) return nt == 1 ? 512 : 256;
  return nt == 1 ? 1024 : head_dim == 64 ? 768 : 512;
}

struct AtArgs {
  const void* q;
  int64_t ldq;
  void* out;
  int64_t ldo;
  int qt;
  const uint8_t* cache;
  int64_t pages;
  KvPage pg;
  int lgP;
  const int32_t* table;
  int64_t ldt;
  const int32_t* lens;
  int cap;               // tokens a sequence may have: ldt * P, at most kAtMaxKeys
  int64_t batch;
  int q_heads, heads;
  int group;             // query heads per key-value head
  int nt;                // column tiles per workgroup (1 or 2)
  int ht;                // workgroups of query heads per key-value head
  float scale;
  int window;
  float* lse;
  const float* signs;
  int d;
  float rnorm;
  int wgs;               // workgroups the tiles are dealt out to (0: one for each unit)
  float* part;           // [2 wgs][nt * kAtCols][D + 4]: o, then m and l
  int2* who;             // [batch][heads][ht]: a unit's first slot, workgroups after its first
};

// Rows of a workgroup of the join.  Few units: each has many parts, and a
// workgroup for every row; many: most were finished in one place, and a
// workgroup looks after several rows.
inline int at_join_rows(int64_t units, int nt, int head_dim) {
  const int rows = kAtCols * nt, most = kAtThreads / (head_dim / kMxPerLane);
  return units * rows <= 2048 ? 1 : (rows < most ? rows : most);
}

// Workspace bytes with and without the units' records.
inline size_t at_part_bytes(int head_dim, int nt) {
  return (size_t)2 * at_workgroups(head_dim, nt) * nt * kAtCols * (head_dim + 4) * sizeof(float);
}
inline size_t at_bytes(int head_dim, int nt, int64_t units) {
  return at_part_bytes(head_dim, nt) + (size_t)units * sizeof(int2);
}

hipError_t launch_paged_attention(const AtArgs& a, hipStream_t s);

// ---- attention of a tree of drafted tokens (kv_tree.hip)

constexpr int kTrTokens = 64;     // drafted tokens of a sequence: a mask's bits

// A unit is 16 nt rows (pairs of a draft and a query head over one key-value
// head) over one sequence's keys; the deal of their tiles as above.
struct TrArgs {
  AtArgs at;             // q, out: a row for each draft; group, q_heads: of one
  const int64_t* mask;   // [batch][tokens]
  int tokens;
};
inline int64_t tr_rows(int tokens, int q_heads, int heads) { return (int64_t)tokens * (q_heads / heads); }
// Column tiles of 16 rows of a workgroup: one where a second would be empty.  Two share
// the conversion of the values, which saves less than a fourth, empty one would cost, so three
// rather go one by one (64 rows over 20000 tokens, eight sequences: two at a time 125 us, one
// 129; 32 rows over 130000, four: 207 and 227; 40 rows, sixteen of 300 to 3000: 39 and 32).
// A head of 256 has registers for one.
inline int tr_nt(int64_t rows, int head_dim) {
  const int64_t tiles = (rows + 15) / 16;
  return tiles == 1 || tiles == 3 || head_dim == 256 ? 1 : 2;
}
// Workgroups that the chip holds at once, by the registers of their kernel.
constexpr int tr_workgroups(int head_dim, int nt) { return nt == 1 && head_dim != 256 ? 768 : 512; }
// Empty places ahead of a unit's tiles (kAtLead): beginning one takes longer here, with
// more queries to bring in and more sums to hand on (32 sequences of 17 to 16384 tokens, 8
// drafts, in the mean of six such, 4, 5, 6 and 7 places: 93, 90, 90 and 92 us, with 10 6% more;
// sixteen of 300 to 3000, 5 drafts: 31, 32, 32 and 33).
constexpr int kTrLead = 7;
__host__ __device__ inline int tr_cost(int tiles) { return tiles > 0 ? tiles + kTrLead : 0; }
// Keys before the first tile of a context of ctx tokens with a window (a row sees
// one draft at least), and the tiles of n keys after them.
__host__ __device__ inline int tr_skip(int ctx, int window) {
  const int64_t first = (int64_t)ctx + 1 - window;
  return window > 0 && first > 0 ? (int)(first & ~(int64_t)(kAtKeys - 1)) : 0;
}
__host__ __device__ inline int tr_tiles(int n, int skip) { return n > skip ? (n - skip + kAtTile - 1) / kAtTile : 0; }
// A row's running maximum goes up by `top`, the largest of a step's scores relative to it: the
// exponent of the factor on the row's sums.  At the first keys that the row sees, top is relative
// to 0 and can be far below it; the sums are 0 then, and stay so with any finite factor
// (2^200 is not one: times 0 it is NaN), so the factor is never above 1.
__host__ __device__ inline float tr_rescale(float top) { return top > 0.f ? -top : 0.f; }
// The number in the deal of workgroup `block` of n that have places: blocks go
// to the XCDs in turn, so those of one remainder by 8 take neighbouring numbers.
// n or more: none.
__host__ __device__ inline int tr_number(uint32_t block, int n) {
  const int per = (n + 7) / 8, i = (int)(block >> 3);
  return i < per ? (int)(block & 7) * per + i : n;
}
inline int tr_join_rows(int64_t units, int nt, int head_dim) {
  const int rows = 16 * nt, most = kAtThreads / (head_dim / kMxPerLane);
  return units * rows <= 2048 ? 1 : (rows < most ? rows : most);
}
// Whether the tiles are dealt out evenly: not where the join's launch would have 2^32 threads
// (from 2^23 units of a head of 256 on, two workgroups each), and enough units fill the chip.
inline bool tr_dealt(int64_t batch, int64_t units, int nt, int head_dim) {
  return batch <= kAtMaxBatch && units * (16 * nt / tr_join_rows(units, nt, head_dim)) < (int64_t)1 << 24;
}
inline size_t tr_part_bytes(int head_dim, int nt) {
  return (size_t)2 * tr_workgroups(head_dim, nt) * nt * 16 * (head_dim + 4) * sizeof(float);
}

hipError_t launch_tree_attention(const TrArgs& t, hipStream_t s);

}  // namespace brq
