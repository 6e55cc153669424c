// Dry-run walks of the microscaled 4-bit operators: every lane's reads and
// writes of rows, codes, scales, cache pages and partial results, from the
// index functions the kernels use.
#include <cmath>
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
static hipError_t walk_tiles(const MmArgs& a, bool epilogue) {
  MmArgs b = a;
  const size_t bytes = mm_plan(b, a.ts, epilogue);
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

static hipError_t walk_matmul(const MmArgs& a, bool epilogue) {
  dry_launch();
  if (a.T < 1 || a.m < 1 || a.n % kMxBlock || a.ldy < a.m) return bad("mx matmul geometry (%lld x %lld)", a.T, a.m);
  if (a.tile) return walk_tiles(a, epilogue);
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

hipError_t launch_mx_matmul(const MmArgs& a, hipStream_t) { return walk_matmul(a, false); }
hipError_t launch_mx_linear(const MmArgs& a, const MmEpi& e, hipStream_t) {
  if ((e.mul && e.ldm < a.m) || (e.res && e.ldr < a.m) || (e.wide && ((e.mul && a.T > 1 && e.ldm % 4) || (e.res && a.T > 1 && e.ldr % 4))))
    return bad("mx linear epilogue (%lld, %lld)", e.ldm, e.ldr);
  return walk_matmul(a, true);
}

hipError_t launch_mx_grouped(const GmArgs& g, const MmEpi& e, hipStream_t) {
  dry_launch();
  const MmArgs& a = g.mm;
  if (a.T < 1 || a.m < 1 || a.n % kMxBlock || a.ldy < a.m || g.groups < 1 || (e.mul && e.ldm < a.m) ||
      (e.res && e.ldr < a.m))
    return bad("mx grouped geometry (%lld x %lld)", a.T, a.m);
  const int64_t units = gm_units(a.T, g.groups, g.rows);
  if (!a.tile) {
    if ((g.rows != 16 && g.rows != 32) || !launchable(gm_stream_workgroups(g), 64 * gm_stream_waves(a.n)))
      return bad("mx grouped stream (%lld units of %lld rows)", units, g.rows);
  } else {
    GmArgs h = g;
    const size_t bytes = gm_plan(h, a.ts);
    const int64_t image = (int64_t)a.stages * 8 * a.tile;
    if (g.rows != a.tile || (a.tile != 128 && a.tile != 256) || a.gt != units || a.go * a.tile < a.m || a.os != a.ts + units * image ||
        (int64_t)bytes != (units + g.groups * a.go) * image || (int64_t)a.stages * kMmK < a.n || a.per != a.stages ||
        !launchable(units * a.go + 7, 256) || !launchable(units + g.groups * a.go, kMxThreads) || a.tile * (a.n / 2) >= (int64_t)1 << 31)
      return bad("mx grouped tiles (%lld units, %lld bytes)", units, (long long)bytes);
    // every tile of a group of some units once
    for (int64_t gt : {1, 2, 4, 5, 11}) {
      std::vector<uint8_t> cover((size_t)(gt * a.go), 0);
      for (int64_t p = 0; p < gt * a.go && a.go < 1 << 16; ++p) {
        MmWhere w;
        mm_place(p, gt, a.go, a.band, w);
        if (w.tt < 0 || w.tt >= gt || w.to < 0 || w.to >= a.go || cover[(size_t)(w.tt * a.go + w.to)]++)
          return bad("mx grouped tile (%lld, %lld)", w.tt, w.to);
      }
    }
  }
  // groups of every kind have no more units than the grid has places, and no
  // row beyond the last
  for (int seed = 0; seed < 6 && a.T <= 1 << 20; ++seed)
    for (int R : {16, 32, 128, 256}) {
      int64_t units = 0, at = 0;
      for (int64_t e = 0; e < g.groups; ++e) {
        const int64_t left = a.T - at, share = a.T / g.groups;
        const int64_t n = seed == 0 ? share : seed == 1 ? (e ? 0 : a.T) : seed == 2 ? (left ? 1 : 0)
                          : seed == 3 ? (e * 7919 + 13) % (2 * share + 2) : seed == 4 ? R + 1 : (e + 1 == g.groups ? left : 1);
        int b, end;
        gm_rows((int)at - (seed == 3 && e == 0 ? 5 : 0), (int)(at + n), (int)a.T, &b, &end);
        if (b < 0 || b > a.T || end < 0 || end > a.T || (seed != 3 && end < b)) return bad("mx grouped rows [%lld, %lld)", b, end);
        units += end > b ? (end - b + R - 1) / R : 0;
        at = end;
      }
      if (units > gm_units(a.T, g.groups, R)) return bad("mx grouped units %lld of %lld rows", units, R);
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

// The deal of a batch's tiles to workgroups: every part has a slot of its own, and
// the join finds the workgroups that have one.
static hipError_t walk_deal(const std::vector<int>& tiles, int64_t units, int of, int lead) {
  int64_t total = 0;
  for (int t : tiles) total += (t > 0 ? t + lead : 0) * units;
  if (!total) return hipSuccess;
  const int wgs = at_dealt(total, of);
  std::vector<int> owner, uses(2 * (size_t)wgs, 0);
  for (int w = 0; w < wgs; ++w)
    for (int64_t g = at_start(w, total, wgs); g < at_start(w + 1, total, wgs); ++g) owner.push_back(w);
  if ((int64_t)owner.size() != total || at_start(wgs, total, wgs) != total)
    return bad("attention deal of %lld tiles covers %lld", total, owner.size());
  int64_t g0 = 0;
  for (size_t b = 0; b < tiles.size(); ++b)
    for (int64_t u = 0; u < units && tiles[b]; ++u, g0 += tiles[b]) {
      g0 += lead;  // the lead's places come before the first tile
      const int64_t g1 = g0 + tiles[b] - 1;
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
  return hipSuccess;
}

static hipError_t walk_loads(const KvPage& pg) {
  const int D = pg.D;
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
  for (int seed = 0; a.wgs && a.batch <= 64 && seed < 6; ++seed) {  // some lengths
    std::vector<int> tiles;
    for (int64_t b = 0; b < a.batch; ++b) {
      const int64_t n = seed == 0 ? 0 : seed == 1 ? a.cap : (b * 7919 + seed * 104729) % (a.cap + 1) >> (seed * b % 5);
      tiles.push_back(at_tiles((int)n, seed == 3 ? 100 : 0));
    }
    const hipError_t e = walk_deal(tiles, (int64_t)a.heads * a.ht, a.wgs, kAtLead);
    if (e != hipSuccess) return e;
  }
  return walk_loads(pg);
}

hipError_t launch_tree_attention(const TrArgs& t, hipStream_t) {
  dry_launch();
  const AtArgs& a = t.at;
  const int D = a.pg.D, H = 16 * a.nt;
  const int64_t rows = (int64_t)t.tokens * a.group, units = a.batch * a.heads * a.ht;
  if ((1 << a.lgP) != a.pg.P || a.group * a.heads != a.q_heads || (int64_t)a.ht * H < rows || (int64_t)(a.ht - 1) * H >= rows ||
      (a.nt != 1 && (a.nt != 2 || D == 256)) || (int64_t)a.cap > a.ldt << a.lgP || a.cap > kAtMaxKeys ||
      t.tokens < 1 || t.tokens > kTrTokens || a.wgs < 0 || a.wgs % 8 || (a.wgs > 0 && !a.part))
    return bad("tree attention geometry (group %lld, tokens %lld)", a.group, t.tokens);
  const int join = tr_join_rows(units, a.nt, D);
  if (H % join || kAtThreads % (D / kMxPerLane * join) || !launchable(a.wgs ? a.wgs : units, kAtThreads) ||
      (a.wgs && !launchable(units * (H / join), kAtThreads)))
    return bad("tree attention launch for %lld units", units, 0);
  // every number of the deal is one workgroup's
  for (int n : {0, 1, 7, 8, 9, 100, a.wgs}) {
    std::vector<int> uses((size_t)n, 0);
    for (int x = 0; x < a.wgs && n <= a.wgs; ++x)
      if (tr_number((uint32_t)x, n) < n) uses[(size_t)tr_number((uint32_t)x, n)]++;
    for (int i = 0; a.wgs && n <= a.wgs && i < n; ++i)
      if (uses[(size_t)i] != 1) return bad("tree attention number %lld of %lld", i, n);
  }
  for (int seed = 0; a.wgs && a.batch <= 64 && seed < 6; ++seed) {  // some lengths, windows too
    std::vector<int> tiles;
    for (int64_t b = 0; b < a.batch; ++b) {
      const int64_t ctx = seed == 0 ? 0 : seed == 1 ? a.cap : (b * 7919 + seed * 104729) % (a.cap + 1) >> (seed * b % 5);
      const int n = (int)(ctx + t.tokens < a.cap ? ctx + t.tokens : a.cap), window = seed == 3 ? 100 : seed == 4 ? 1 : 0;
      const int skip = tr_skip((int)ctx, window);
      if (skip < 0 || skip % kAtKeys || (window && skip > (ctx + 1 > window ? ctx + 1 - window : 0)))
        return bad("tree attention skips %lld of %lld keys", skip, ctx);
      tiles.push_back(tr_tiles(n, skip));
    }
    const hipError_t e = walk_deal(tiles, (int64_t)a.heads * a.ht, a.wgs, kTrLead);
    if (e != hipSuccess) return e;
  }
  return walk_loads(a.pg);
}

// A row of a move's workspace, byte by byte; the pieces that a reservation
// copies of a page, against the places of the tokens it copies.
hipError_t launch_kv_move(const KpMove& a, hipStream_t) {
  dry_launch();
  const int D = a.pg.D;
  const int64_t rows = kp_runs(a.tokens) * a.heads;
  const bool few = kp_few(a.tokens, a.heads);
  if ((1 << a.lgP) != a.pg.P || a.tokens < 1 || (few && a.tokens > kKpFew) || kKpFew % (kKpThreads / 16) ||
      !(few ? launchable(a.heads, kKpThreads) : launchable(rows / (kMxThreads / 16) + 1, kMxThreads)))
    return bad("cache move of %lld tokens", a.tokens, 0);
  if (!few) {  // rows past the last run stay in the workspace only if they move nothing
    const int64_t last = (rows - 1) * kKpRun * kp_row_bytes(D) + kKpRun * kp_row_bytes(D);
    if (!a.ws || last > (int64_t)kp_move_bytes(a.tokens, a.heads, D) || rows >= (int64_t)1 << 32)
      return bad("cache move workspace of %lld bytes", last, 0);
  }
  std::vector<uint8_t> cover((size_t)kp_row_bytes(D), 0);
  for (int r = 0; r < 16; ++r)
    for (int i = 0; i < D / 32; ++i) {
      cover[(size_t)(r * (D / 32) + i)]++;
      cover[(size_t)(D / 2 + r * (D / 32) + i)]++;
      if (r == 0) cover[(size_t)(D + i)]++, cover[(size_t)(D + D / 32 + i)]++;
    }
  for (size_t i = 0; i < cover.size(); ++i)
    if (cover[i] != 1) return bad("cache move byte %lld written %lld times", (long long)i, cover[i]);
  return walk_page(a.pg);
}
hipError_t launch_kv_fork(const KpFork& a, hipStream_t) {
  dry_launch();
  const int64_t n = a.children * (a.width > 0 ? a.width : 1);
  return launchable((n + kMxThreads - 1) / kMxThreads, kMxThreads) ? hipSuccess : bad("cache fork of %lld", n, 0);
}
hipError_t launch_kv_free(const KpFree& a, hipStream_t) {
  dry_launch();
  return launchable((a.n * a.width + kMxThreads - 1) / kMxThreads, kMxThreads) ? hipSuccess
                                                                             : bad("cache free of %lld", a.n, 0);
}
hipError_t launch_kv_reserve(const KpReserve& a, hipStream_t) {
  dry_launch();
  const KvPage& pg = a.pg;
  const int P = pg.P, D = pg.D;
  if ((1 << a.lgP) != P || a.per != kp_per(a.tokens, P) || !launchable(a.batch, kMxThreads) || a.heads > 65535)
    return bad("cache reservation geometry (%lld tokens)", a.tokens, 0);
  for (int used = 16; used <= P; used += 16) {
    std::vector<uint8_t> cover((size_t)pg.bytes(), 0);
    const int codes = used * (D / 32), scales = used * D / 512;
    for (int i = 0; i < 2 * (codes + scales); ++i) {
      const int64_t at = (int64_t)kp_piece(pg, codes, scales, i) * 16;
      if (at < 0 || at + 16 > pg.bytes()) return bad("cache reservation piece %lld of %lld tokens", i, used);
      for (int e = 0; e < 16; ++e) cover[(size_t)(at + e)]++;
    }
    for (int t = 0; t < P; ++t) {  // the first tokens' bytes once, no other's
      bool ok = true;
      for (int r = 0; r < 16; ++r)
        for (int e = 0; e < D / 32; ++e)
          ok = ok && cover[(size_t)(pg.kcode(t) + r * (D / 32) + e)] == (t < used) &&
               cover[(size_t)(pg.vcode(t, r) + e)] == (t < used);
      for (int e = 0; e < D / 32; ++e)
        ok = ok && cover[(size_t)(pg.kscale(t) + e)] == (t < used) && cover[(size_t)pg.vscale(t, e)] == (t < used);
      if (!ok) return bad("cache reservation copy of token %lld of %lld", t, used);
    }
  }
  for (int rank : {0, 1, 1000, kKpRanks - 1, kKpRanks, INT32_MAX})  // what an entry wants is no page
    for (bool shared : {false, true}) {
      const int32_t w = kp_want(rank, shared);
      if (w >= -1 || kp_shared(w) != shared || kp_rank(w) != (rank < kKpRanks ? rank : kKpRanks))
        return bad("cache reservation rank %lld as %lld", rank, w);
    }
  // the entries that new tokens lie in, for lengths around page and table ends
  std::vector<int32_t> lens;
  for (int64_t n : {(int64_t)-1, (int64_t)0, (int64_t)1, (int64_t)P - 1, (int64_t)P, a.width * P - 1, a.width * P, a.width * P + 5})
    if (n < (int64_t)1 << 31) lens.push_back((int32_t)n);
  KpReserve b = a;
  b.lens = lens.data();
  b.batch = (int64_t)lens.size();
  for (int64_t i = 0; i < b.batch * b.per && b.per < 1 << 16; ++i) {
    KpItem it;
    if (!kp_item(b, i, it)) continue;
    const int64_t n = lens[(size_t)it.row];
    if (it.entry < 0 || it.entry >= a.width || it.entry < n / P || it.entry > (n + a.tokens - 1) / P ||
        it.used != (it.entry == n / P ? n % P : 0))
      return bad("cache reservation entry %lld of a row of %lld tokens", it.entry, n);
  }
  return walk_page(pg);
}

}  // namespace brq

// A row's maximum and sum over n scores (in units of log2, -infinity where masked), as a
// wavefront of the tree attention holds them: `step` scores at a time, relative to
// the maximum so far.
extern "C" void brq_dryrun_tree_row(const float* scores, int n, int step, float* max, float* sum) {
  float m = 0.f, least = -INFINITY, l = 0.f;
  for (int k = 0; k < n; k += step) {
    const int end = n < k + step ? n : k + step;
    float top = least;
    for (int i = k; i < end; ++i) top = std::fmax(top, scores[i] - m);
    const bool moved = top > least;
    float up = 0.f;
    if (moved) {
      l *= std::exp2(brq::tr_rescale(top));
      up = top;
    }
    for (int i = k; i < end; ++i) l += std::exp2(scores[i] - m - up);
    if (moved) {
      m += top;
      least = 0.f;
    }
  }
  *max = least == 0.f ? m : -INFINITY;
  *sum = l;
}

// gelu's polynomial for erfc(z) exp(z^2), with its own error alone.
extern "C" double brq_dryrun_gelu_tail(double z) {
  const double t = 1 / (1 + z / 2);
  return t * brq::mm_gelu_tail(t);
}
