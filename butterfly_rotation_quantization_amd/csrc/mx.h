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

constexpr int kMmK = 256;  // values of a row per stage

// Launches within 2^32 threads (at most 64 per 16 x 16 outputs, 32 per row).
inline bool mm_supported(int64_t T, int64_t m, int64_t n) {
  const int64_t most = (int64_t)1 << 28;
  return T <= most && m <= most && n <= most && (m == 0 || T <= kMxMost / 2 / m);
}

// Kernel and workspace of a product (a.T, a.m, a.n set): returns the
// workspace bytes.
inline size_t mm_plan(MmArgs& a, uint8_t* ws) {
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
  const int64_t large = (tiles(256) + 255) / 256 * 3, small = (tiles(128) + 511) / 512 * 2;
  a.tile = large <= small ? 256 : 128;
  a.stages = (int)((a.n + kMmK - 1) / kMmK);
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
__host__ __device__ inline bool mm_where(const MmArgs& a, uint32_t block, MmWhere& w) {
  int64_t p = (int64_t)(block & 7) * a.per_xcd + (block >> 3);
  if (p >= a.gt * a.go * a.splits) return false;
  w.part = (int)(p / (a.gt * a.go));
  p -= w.part * (a.gt * a.go);
  const int64_t band = p / ((int64_t)a.band * a.go);
  const int64_t q = p - band * a.band * a.go;
  const int64_t h = a.gt - band * a.band < a.band ? a.gt - band * a.band : a.band;  // rows of tiles in this band
  w.tt = band * a.band + q % h;
  w.to = q / h;
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

}  // namespace brq
