// Dry-run walks of the microscaled 4-bit operators: every lane's reads and
// writes of rows, codes, scales, cache pages and partial results, from the
// index functions the kernels use.
#include <vector>

#include "mx.h"

namespace brq {

bool dry_violation(const char* fmt, long long a, long long b);
void dry_launch();

static hipError_t bad(const char* fmt, long long a, long long b) {
  dry_violation(fmt, a, b);
  return hipErrorInvalidValue;
}
// A launch has fewer than 2^32 threads along a dimension.
static bool launchable(int64_t workgroups, int64_t threads) { return workgroups * threads < (int64_t)1 << 32; }

static hipError_t walk_mx(const MxArgs& a, int64_t ld) {
  dry_launch();
  const int64_t n = (int64_t)a.lpr * a.per;
  if ((a.per != 8 && a.per != 16) || n % kMxBlock || a.lanes != (uint64_t)a.rows * a.lpr || ld < n || (a.d && n % a.d))
    return bad("mx geometry (row of %lld, d %lld)", n, a.d);
  if (!launchable((int64_t)(a.lanes + kMxThreads - 1) / kMxThreads, kMxThreads)) return bad("mx grid of %lld lanes", (long long)a.lanes, 0);
  if (a.lanes > (1 << 22)) return hipSuccess;  // walked in full at test sizes
  std::vector<uint8_t> cover((size_t)(a.rows * n), 0);
  for (uint64_t li = 0; li < a.lanes; ++li) {
    int64_t row, col;
    mx_lane(a.lpr, a.per, li, &row, &col);
    if (row < 0 || row >= a.rows || col < 0 || col + a.per > n) return bad("mx lane at (%lld, %lld)", row, col);
    if ((row * n + col) / a.per != (int64_t)li) return bad("mx codes word %lld of lane %lld", row * n + col, li);
    if (li % (kMxBlock / a.per) == 0 && col % kMxBlock) return bad("mx block at column %lld", col, 0);
    for (int e = 0; e < a.per; ++e) cover[(size_t)(row * n + col + e)]++;
  }
  for (size_t i = 0; i < cover.size(); ++i)
    if (cover[i] != 1) return bad("mx value %lld handled %lld times", (long long)i, cover[i]);
  return hipSuccess;
}

hipError_t launch_mx_quant(const MxArgs& a, hipStream_t) { return walk_mx(a, a.ldx); }
hipError_t launch_mx_dequant(const MxArgs& a, hipStream_t) { return walk_mx(a, a.ldy); }

// Tiles, parts, scale images and LDS places of the tile kernels of a matmul.
static hipError_t walk_tiles(const MmArgs& a) {
  MmArgs b = a;
  const size_t bytes = mm_plan(b, a.ts);
  const int R = a.tile;
  const int64_t image = (int64_t)a.stages * 8 * R, images = (a.gt + a.go) * image;
  if (b.os != a.os || b.part != a.part || b.splits != a.splits || (R != 128 && R != 256) || a.os != a.ts + a.gt * image ||
      reinterpret_cast<uint8_t*>(a.part) != a.ts + images ||
      (int64_t)bytes != images + (a.splits > 1 ? a.splits * a.T * a.m * 4 : 0))
    return bad("mx matmul workspace (%lld bytes, tile %lld)", (long long)bytes, R);
  if (a.gt * R < a.T || a.go * R < a.m || (int64_t)a.stages * kMmK < a.n || !launchable(8 * a.per_xcd, 256) ||
      !launchable(a.gt + a.go, kMxThreads))
    return bad("mx matmul tiles (%lld x %lld)", a.gt, a.go);
  for (int p = 0; p < a.splits; ++p)
    if (a.stages - p * a.per < 1 || (p + 1 == a.splits && a.stages > (p + 1) * a.per))
      return bad("mx matmul part %lld of %lld", p, a.splits);
  // addresses in the kernel are offsets in 32 bits from a tile's first row
  if (R * (a.n / 2) >= (int64_t)1 << 31) return bad("mx matmul row of %lld", a.n, 0);
  const int64_t places = a.gt * a.go * a.splits;
  if (places <= 1 << 16) {
    std::vector<uint8_t> cover((size_t)places, 0);
    for (int64_t x = 0; x < 8 * a.per_xcd; ++x) {
      MmWhere w;
      if (!mm_where(a, (uint32_t)x, w)) continue;
      if (w.tt < 0 || w.tt >= a.gt || w.to < 0 || w.to >= a.go || w.part < 0 || w.part >= a.splits)
        return bad("mx matmul tile (%lld, %lld)", w.tt, w.to);
      cover[(size_t)((w.part * a.gt + w.tt) * a.go + w.to)]++;
    }
    for (size_t i = 0; i < cover.size(); ++i)
      if (cover[i] != 1) return bad("mx matmul tile %lld taken %lld times", (long long)i, cover[i]);
  }
  // a stage of an image: every byte one block's scale of one row, words of
  // tiles of 32 rows whole
  std::vector<uint8_t> cover((size_t)(8 * R), 0);
  for (int c = 0; c < 8; ++c)
    for (int r = 0; r < R; ++r) {
      const int at = mm_scale_at(R, c, r);
      if (at < 0 || at >= 8 * R || cover[(size_t)at]++ || at != mm_scale_at(R, c, r % 32) + r / 32)
        return bad("mx matmul scale of block %lld, row %lld", c, r);
    }
  // codes in LDS: thread tid brings piece (tid & 7) ^ (row / 2 & 7) of row tid / 8
  // + 32 j to its own 16 bytes; sixteen rows' pieces c are in different places
  // of 256 bytes
  const int threads = 256;
  for (int j = 0; j < 2 * R * 8 / threads; ++j)
    for (int tid = 0; tid < threads; ++tid) {
      const int row = tid / 8 + j * (threads / 8), c = (tid & 7) ^ (tid / 16 & 7);
      if (mm_piece(row, c) != j * threads + tid) return bad("mx matmul piece of row %lld, thread %lld", row, tid);
    }
  for (int c = 0; c < 8; ++c)
    for (int r = 0; r < 2 * R; r += 16) {
      unsigned seen = 0;
      for (int i = 0; i < 16; ++i) seen |= 1u << (mm_piece(r + i, c) & 15);
      if (seen != 0xffff) return bad("mx matmul piece %lld of rows from %lld", c, r);
    }
  return hipSuccess;
}

hipError_t launch_mx_matmul(const MmArgs& a, hipStream_t) {
  dry_launch();
  if (a.T < 1 || a.m < 1 || a.n % kMxBlock || a.ldy < a.m) return bad("mx matmul geometry (%lld x %lld)", a.T, a.m);
  if (a.tile) return walk_tiles(a);
  if (a.T <= 64) {
    const int rows = mm_stream_rows(a);
    const int64_t wgs = (a.m + rows - 1) / rows;
    if ((rows != 16 && rows != 32) || !launchable(wgs, 64 * mm_stream_waves(wgs)))
      return bad("mx matmul stream of %lld rows", a.m, 0);
  } else if (!launchable(((a.T + 15) / 16) * ((a.m + 15) / 16), 64)) {
    return bad("mx matmul grid (%lld x %lld)", a.T, a.m);
  }
  return hipSuccess;
}

// Every byte of a page is written by exactly one lane of one token, and every
// access is aligned to its width.
static hipError_t walk_page(const KvPage& pg) {
  const int D = pg.D, P = pg.P;
  std::vector<uint8_t> cover((size_t)pg.bytes(), 0);
  auto put = [&](int64_t at, int w) {
    if (at < 0 || at + w > pg.bytes() || at % w) return false;
    for (int i = 0; i < w; ++i) cover[(size_t)(at + i)]++;
    return true;
  };
  for (int t = 0; t < P; ++t)
    for (int c = 0; c < D; c += kKvPerLane) {
      const int run = D / 16, w = D / 32;  // a run's dimensions and bytes; runs are D / 8 bytes apart
      bool ok = put(pg.kcode(t) + c / 2, 8);
      for (int q = 0; q < kKvPerLane / run; ++q)
        ok = ok && pg.vcode(t, c / run + q) == pg.vcode(t, c / run) + q * (D / 8) && put(pg.vcode(t, c / run + q), w);
      if (c % kMxBlock == 0) ok = ok && put(pg.kscale(t) + c / 32, 1) && put(pg.vscale(t, c / 32), 1);
      if (!ok) return bad("cache page access of token %lld, value %lld", t, c);
    }
  for (size_t i = 0; i < cover.size(); ++i)
    if (cover[i] != 1) return bad("cache page byte %lld written %lld times", (long long)i, cover[i]);
  return hipSuccess;
}

static hipError_t walk_kv(const KvArgs& a) {
  dry_launch();
  if ((1 << a.lgP) != a.pg.P || a.ldk < (int64_t)a.heads * a.pg.D || a.ldv < (int64_t)a.heads * a.pg.D ||
      (a.d && a.d != a.pg.D))
    return bad("cache geometry (page %lld, D %lld)", a.pg.P, a.pg.D);
  const int64_t rows = kv_rows(a.tokens, a.heads);
  if (rows >= (int64_t)1 << 31 || !launchable(rows * (a.pg.D / kMxPerLane) / kMxThreads + 1, kMxThreads))
    return bad("cache rows of %lld tokens", a.tokens, 0);
  if (rows <= 1 << 22) {  // every head of every token once
    std::vector<uint8_t> cover((size_t)(a.tokens * a.heads), 0);
    for (int64_t r = 0; r < rows; ++r) {
      int64_t tok;
      int h;
      kv_row((uint32_t)r, a.heads, &tok, &h);
      if (tok < 0 || h < 0 || h >= a.heads) return bad("cache row %lld of head %lld", r, h);
      if (tok < a.tokens) cover[(size_t)(tok * a.heads + h)]++;
    }
    for (size_t i = 0; i < cover.size(); ++i)
      if (cover[i] != 1) return bad("cache row %lld handled %lld times", (long long)i, cover[i]);
  }
  return walk_page(a.pg);
}

hipError_t launch_kv_append(const KvArgs& a, hipStream_t) { return walk_kv(a); }
hipError_t launch_kv_read(const KvArgs& a, hipStream_t) { return walk_kv(a); }

hipError_t launch_paged_attention(const AtArgs& a, hipStream_t) {
  dry_launch();
  const KvPage& pg = a.pg;
  const int D = pg.D;
  if ((1 << a.lgP) != pg.P || a.group * a.heads != a.q_heads || a.ht * a.nt * kAtCols < a.group ||
      (int64_t)a.cap > a.ldt << a.lgP || a.cap > kAtMaxKeys || a.wgs < 0 || (a.wgs > 0 && !a.part))
    return bad("attention geometry (group %lld, workgroups %lld)", a.group, a.wgs);
  const int64_t units = a.batch * a.heads * a.ht;
  if (!launchable(a.wgs ? a.wgs : units, kAtThreads) ||
      (a.wgs && !launchable(units * (kAtCols * a.nt / at_join_rows(units, a.nt, D)), kAtThreads)))
    return bad("attention launch for %lld units", units, 0);
  // the deal of tiles to workgroups for some lengths: every part has a slot of
  // its own, and the join finds the workgroups that have one
  for (int seed = 0; a.wgs && a.batch <= 64 && seed < 6; ++seed) {
    std::vector<int> tiles;
    int64_t total = 0, units = (int64_t)a.heads * a.ht;
    for (int64_t b = 0; b < a.batch; ++b) {
      const int64_t n = seed == 0 ? 0 : seed == 1 ? a.cap : (b * 7919 + seed * 104729) % (a.cap + 1) >> (seed * b % 5);
      tiles.push_back(at_tiles((int)n, seed == 3 ? 100 : 0));
      total += at_cost(tiles.back()) * units;
    }
    if (!total) continue;
    const int wgs = at_dealt(total, a.wgs);
    std::vector<int> owner, uses(2 * (size_t)wgs, 0);
    for (int w = 0; w < wgs; ++w)
      for (int64_t g = at_start(w, total, wgs); g < at_start(w + 1, total, wgs); ++g) owner.push_back(w);
    if ((int64_t)owner.size() != total || at_start(wgs, total, wgs) != total)
      return bad("attention deal of %lld tiles covers %lld", total, owner.size());
    int64_t g0 = 0;
    for (int64_t b = 0; b < a.batch; ++b)
      for (int64_t u = 0; u < units && tiles[(size_t)b]; ++u, g0 += tiles[(size_t)b]) {
        g0 += kAtLead;  // the lead's places come before the first tile
        const int64_t g1 = g0 + tiles[(size_t)b] - 1;
        if (at_owner(g0, total, wgs) != owner[(size_t)g0] || at_owner(g1, total, wgs) != owner[(size_t)g1])
          return bad("attention owner of tile %lld of %lld", g0, total);
        int last = -1;
        for (int64_t g = g0; owner[(size_t)g0] != owner[(size_t)g1] && g <= g1; ++g)
          if (owner[(size_t)g] != last) {
            last = owner[(size_t)g];
            if (uses[(size_t)at_slot(last, g0, total, wgs)]++)
              return bad("attention slot of workgroup %lld used twice (tile %lld)", last, g);
          }
      }
  }
  // the wide loads of 16 keys at every place of a page
  for (int p = 0; p < pg.P; p += 16)
    for (int lane = 0; lane < 64; ++lane) {
      const int c = lane & 15, g = lane >> 4, w = D / 8;
      const int64_t kc = pg.kcode(p + c) + g * w, vc = pg.vcode(p + 4 * g, c);
      const int64_t ks = pg.kscale(p + c) + (int64_t)g * D / 128, vs = pg.vscale(p + 4 * g, c * D / 512);
      const int wide = w < 16 ? w : 16, kb = D == 256 ? 2 : 1;
      if (kc % wide || vc % wide || kc + w > pg.vcode(0, 0) || vc + w > pg.kscale(0))
        return bad("attention codes of lane %lld at token %lld", lane, p);
      if (ks % kb || ks + kb > pg.vscale(0, 0) || vs % 4 || vs + 4 > pg.bytes())
        return bad("attention scales of lane %lld at token %lld", lane, p);
      // the four keys of a lane's values follow one another, as do their scales
      for (int i = 0; i < 4; ++i)
        if (pg.vcode(p + 4 * g + i, c) != vc + i * (D / 32) || pg.vscale(p + 4 * g + i, c * D / 512) != vs + i)
          return bad("attention values of lane %lld, key %lld", lane, i);
    }
  return walk_page(pg);
}

}  // namespace brq
