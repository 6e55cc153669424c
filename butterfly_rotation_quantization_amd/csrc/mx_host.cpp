// C ABI of the microscaled 4-bit operators: argument checks and dispatch of
// quantize, dequantize, product, paged cache and attention (mx.h).
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "mx.h"

namespace brq {
namespace {

brq_status refuse(brq_status s, const char* fmt, ...) {
  char buf[256];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  return report_error(s, buf);
}

bool dtype_ok(int32_t t) { return t == BRQ_F32 || t == BRQ_BF16 || t == BRQ_F16; }
int64_t dtype_size(int32_t t) { return t == BRQ_F32 ? 4 : 2; }
bool misaligned(const void* p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)a != 0; }
// rows of `ld` elements of type t starting at p, every row 16-byte aligned
bool rows_misaligned(const void* p, int64_t ld, int32_t t) {
  return misaligned(p, 16) || (ld * dtype_size(t)) % 16 != 0;
}

brq_status launched(hipError_t e, const char* what) {
  return e == hipSuccess ? BRQ_OK : refuse(BRQ_ERR_HIP, "%s launch: %s", what, hipGetErrorString(e));
}

brq_status workspace_ok(const void* ws, size_t bytes, size_t need) {
  if (need && (!ws || bytes < need))
    return refuse(BRQ_ERR_WORKSPACE, "workspace of %zu bytes, %zu needed", ws ? bytes : (size_t)0, need);
  if (need && misaligned(ws, 16)) return refuse(BRQ_ERR_ALIGNMENT, "the workspace must be 16-byte aligned");
  return BRQ_OK;
}

// The transform of a plan these kernels apply in registers: Hadamard, d in
// 32..256 (want > 0: exactly that d).
brq_status transform_of(const brq_plan* plan, int want, const float** signs, int* d, float* rnorm) {
  *signs = nullptr;
  *d = 0;
  *rnorm = 1.0f;
  const Plan* p = nullptr;
  const brq_status st = plan_data(plan, &p);
  if (st != BRQ_OK || !p) return st;
  if (p->mode != BRQ_HADAMARD) return refuse(BRQ_ERR_UNSUPPORTED, "the plan must be a Hadamard plan");
  if (want ? p->d != want : (p->d < 32 || p->d > 256))
    return refuse(BRQ_ERR_UNSUPPORTED, want ? "the plan's d = %d must be the head dimension %d"
                                            : "the plan's d = %d must be 32, 64, 128 or 256", p->d, want);
  *signs = p->signs;
  *d = p->d;
  *rnorm = (float)(1.0 / std::sqrt((double)p->d));
  return BRQ_OK;
}

int log2_of(int64_t x) {
  int l = 0;
  while (((int64_t)1 << l) < x) ++l;
  return l;
}

// Shared checks of brq_mx_quantize and brq_mx_dequantize; *done set when
// there is nothing to do.
brq_status mx_setup(MxArgs& a, const brq_plan* right, int64_t rows, int64_t n, const void* x, int32_t t, int64_t ld,
                    const uint8_t* codes, const uint8_t* scales, bool quantize, bool* done) {
  clear_error();
  *done = false;
  std::memset(&a, 0, sizeof a);
  if (!dtype_ok(t)) return refuse(BRQ_ERR_INVALID_ARGUMENT, "bad dtype %d", t);
  if (rows < 0 || n < 0 || ld < n) return refuse(BRQ_ERR_INVALID_ARGUMENT, "bad shape or leading dimension");
  if (n % kMxBlock)
    return refuse(BRQ_ERR_INVALID_ARGUMENT, "n = %lld must be a multiple of %d", (long long)n, kMxBlock);
  const brq_status st = transform_of(right, 0, &a.signs, &a.d, &a.rnorm);
  if (st != BRQ_OK) return st;
  if (a.d && n % a.d)
    return refuse(BRQ_ERR_INVALID_ARGUMENT, "d = %d must divide n = %lld", a.d, (long long)n);
  if (rows == 0 || n == 0) {
    *done = true;
    return BRQ_OK;
  }
  if (n > kMxMost || rows > kMxMost / n) return refuse(BRQ_ERR_UNSUPPORTED, "more than 2^34 values");
  if (!x || !codes || !scales) return refuse(BRQ_ERR_INVALID_ARGUMENT, "NULL data pointer");
  if (rows_misaligned(x, ld, t)) return refuse(BRQ_ERR_ALIGNMENT, "rows must be 16-byte aligned");
  if (misaligned(codes, 16) || misaligned(scales, 4))
    return refuse(BRQ_ERR_ALIGNMENT, "codes must be 16-byte and scales 4-byte aligned");
  a.rows = rows;
  a.per = quantize && a.d ? 16 : kMxPerLane;
  a.lpr = (uint32_t)(n / a.per);
  a.lanes = (uint64_t)rows * a.lpr;
  a.gap = ld != n;
  a.codes = const_cast<uint8_t*>(codes);
  a.scales = const_cast<uint8_t*>(scales);
  return BRQ_OK;
}

// The epilogue of a product of T x m outputs (`groups` rows of bias).
brq_status epilogue_of(const brq_mx_epilogue* ep, int64_t T, int64_t m, int64_t groups, MmEpi* e) {
  std::memset(e, 0, sizeof *e);
  if (!ep) return BRQ_OK;
  if (ep->act < BRQ_ACT_NONE || ep->act > BRQ_ACT_SILU)
    return refuse(BRQ_ERR_INVALID_ARGUMENT, "bad activation %d", ep->act);
  if ((ep->bias && !dtype_ok(ep->bias_type)) || (ep->mul && !dtype_ok(ep->mul_type)) ||
      (ep->residual && !dtype_ok(ep->residual_type)))
    return refuse(BRQ_ERR_INVALID_ARGUMENT, "bad dtype in the epilogue");
  if ((ep->mul && ep->ldmul < m) || (ep->residual && ep->ldresidual < m))
    return refuse(BRQ_ERR_INVALID_ARGUMENT, "leading dimension of mul or residual below m");
  if ((ep->bias && misaligned(ep->bias, dtype_size(ep->bias_type))) ||
      (ep->mul && misaligned(ep->mul, dtype_size(ep->mul_type))) ||
      (ep->residual && misaligned(ep->residual, dtype_size(ep->residual_type))))
    return refuse(BRQ_ERR_ALIGNMENT, "bias, mul and residual must be aligned to their types");
  auto wide = [](const void* p, int32_t t, int64_t ld, int64_t rows) {
    return !p || (!misaligned(p, 4 * dtype_size(t)) && (ld % 4 == 0 || rows == 1));
  };
  e->act = ep->act;
  e->bias = ep->bias;
  e->bt = ep->bias_type;
  e->mul = ep->mul;
  e->mt = ep->mul_type;
  e->ldm = ep->ldmul;
  e->res = ep->residual;
  e->rt = ep->residual_type;
  e->ldr = ep->ldresidual;
  e->wide = wide(ep->bias, ep->bias_type, m, groups) && wide(ep->mul, ep->mul_type, ep->ldmul, T) &&
            wide(ep->residual, ep->residual_type, ep->ldresidual, T);
  return BRQ_OK;
}

// Shared checks of the products; *done set when there is nothing to do.
brq_status mm_setup(MmArgs& a, MmEpi& e, const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
                    const uint8_t* b_scales, int64_t T, int64_t m, int64_t n, int64_t groups, const brq_mx_epilogue* ep,
                    void* y, int32_t yt, int64_t ldy, bool* done) {
  *done = false;
  std::memset(&a, 0, sizeof a);
  if (!dtype_ok(yt)) return refuse(BRQ_ERR_INVALID_ARGUMENT, "bad output dtype %d", yt);
  if (T < 0 || m < 0 || n < 0 || ldy < m)
    return refuse(BRQ_ERR_INVALID_ARGUMENT, "bad shape or leading dimension");
  if (n % kMxBlock)
    return refuse(BRQ_ERR_INVALID_ARGUMENT, "n = %lld must be a multiple of %d", (long long)n, kMxBlock);
  if (!mm_supported(T, m, n)) return refuse(BRQ_ERR_UNSUPPORTED, "T, m or n above 2^28, or more than 2^33 outputs");
  const brq_status st = epilogue_of(ep, T, m, groups, &e);
  if (st != BRQ_OK) return st;
  if (T == 0 || m == 0 || groups == 0) {
    *done = true;
    return BRQ_OK;
  }
  if (!y || (n > 0 && (!a_codes || !a_scales || !b_codes || !b_scales)))
    return refuse(BRQ_ERR_INVALID_ARGUMENT, "NULL data pointer");
  if (misaligned(a_codes, 16) || misaligned(b_codes, 16) || misaligned(a_scales, 4) || misaligned(b_scales, 4))
    return refuse(BRQ_ERR_ALIGNMENT, "codes must be 16-byte and scales 4-byte aligned");
  if (misaligned(y, dtype_size(yt))) return refuse(BRQ_ERR_ALIGNMENT, "the output must be aligned to its type");
  a.a = a_codes;
  a.as = a_scales;
  a.b = b_codes;
  a.bs = b_scales;
  a.T = T;
  a.m = m;
  a.n = n;
  a.y = y;
  a.yt = yt;
  a.ldy = ldy;
  a.wide = ldy % 4 == 0 && !misaligned(y, 4 * dtype_size(yt));
  return BRQ_OK;
}

}  // namespace
}  // namespace brq

using namespace brq;

extern "C" {

brq_status brq_mx_quantize(const brq_plan* right, const void* x, int32_t xt, int64_t ldx, int64_t rows, int64_t n,
                           uint8_t* codes, uint8_t* scales, void* stream) {
  MxArgs a;
  bool done;
  const brq_status st = mx_setup(a, right, rows, n, x, xt, ldx, codes, scales, true, &done);
  if (st != BRQ_OK || done) return st;
  a.x = x;
  a.xt = xt;
  a.ldx = ldx;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int tok = prof_begin("mx quantize", s);
  const hipError_t e = launch_mx_quant(a, s);
  prof_end(tok, s);
  return launched(e, "mx quantize");
}

brq_status brq_mx_dequantize(const brq_plan* right, const uint8_t* codes, const uint8_t* scales, int64_t rows,
                             int64_t n, void* out, int32_t ot, int64_t ldo, void* stream) {
  MxArgs a;
  bool done;
  const brq_status st = mx_setup(a, right, rows, n, out, ot, ldo, codes, scales, false, &done);
  if (st != BRQ_OK || done) return st;
  a.y = out;
  a.yt = ot;
  a.ldy = ldo;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int tok = prof_begin("mx dequantize", s);
  const hipError_t e = launch_mx_dequant(a, s);
  prof_end(tok, s);
  return launched(e, "mx dequantize");
}

size_t brq_mx_matmul_workspace_bytes(int64_t T, int64_t m, int64_t n) {
  if (T <= 0 || m <= 0 || n <= 0 || n % kMxBlock || !mm_supported(T, m, n)) return 0;
  MmArgs a;
  std::memset(&a, 0, sizeof a);
  a.T = T;
  a.m = m;
  a.n = n;
  const size_t plain = mm_plan(a, nullptr, false), with = mm_plan(a, nullptr, true);
  return plain > with ? plain : with;
}

brq_status brq_mx_matmul(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
                         const uint8_t* b_scales, int64_t T, int64_t m, int64_t n, void* y, int32_t yt, int64_t ldy,
                         void* ws, size_t ws_bytes, void* stream) {
  return brq_mx_linear(a_codes, a_scales, b_codes, b_scales, T, m, n, nullptr, y, yt, ldy, ws, ws_bytes, stream);
}

brq_status brq_mx_linear(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
                         const uint8_t* b_scales, int64_t T, int64_t m, int64_t n, const brq_mx_epilogue* ep, void* y,
                         int32_t yt, int64_t ldy, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  MmArgs a;
  MmEpi e;
  bool done;
  brq_status st = mm_setup(a, e, a_codes, a_scales, b_codes, b_scales, T, m, n, 1, ep, y, yt, ldy, &done);
  if (st != BRQ_OK || done) return st;
  const size_t need = brq_mx_matmul_workspace_bytes(T, m, n);
  if ((st = workspace_ok(ws, ws_bytes, need)) != BRQ_OK) return st;
  mm_plan(a, static_cast<uint8_t*>(ws), ep != nullptr);
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int tok = prof_begin("mx matmul", s);
  const hipError_t err = ep ? launch_mx_linear(a, e, s) : launch_mx_matmul(a, s);
  prof_end(tok, s);
  return launched(err, "mx matmul");
}

size_t brq_mx_grouped_matmul_workspace_bytes(int64_t T, int64_t groups, int64_t m, int64_t n) {
  if (T <= 0 || groups <= 0 || m <= 0 || n <= 0 || n % kMxBlock || !gm_supported(T, groups, m, n)) return 0;
  GmArgs g;
  std::memset(&g, 0, sizeof g);
  g.mm.T = T;
  g.mm.m = m;
  g.mm.n = n;
  g.groups = (int)groups;
  return gm_plan(g, nullptr);
}

brq_status brq_mx_grouped_matmul(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* b_codes,
                                 const uint8_t* b_scales, const int32_t* offsets, int64_t T, int64_t groups, int64_t m,
                                 int64_t n, const brq_mx_epilogue* ep, void* y, int32_t yt, int64_t ldy, void* ws,
                                 size_t ws_bytes, void* stream) {
  clear_error();
  GmArgs g;
  std::memset(&g, 0, sizeof g);
  MmEpi e;
  bool done;
  if (groups < 0) return refuse(BRQ_ERR_INVALID_ARGUMENT, "bad number of groups");
  if (T > 0 && m > 0 && n >= 0 && !gm_supported(T, groups, m, n))
    return refuse(BRQ_ERR_UNSUPPORTED, "T, m or n above 2^28, more than 2^33 outputs, 2^20 groups or 2^32 threads");
  brq_status st = mm_setup(g.mm, e, a_codes, a_scales, b_codes, b_scales, T, m, n, groups, ep, y, yt, ldy, &done);
  if (st != BRQ_OK || done) return st;
  if (!offsets) return refuse(BRQ_ERR_INVALID_ARGUMENT, "NULL offsets");
  if (misaligned(offsets, 4)) return refuse(BRQ_ERR_ALIGNMENT, "offsets must be 4-byte aligned");
  const size_t need = brq_mx_grouped_matmul_workspace_bytes(T, groups, m, n);
  if ((st = workspace_ok(ws, ws_bytes, need)) != BRQ_OK) return st;
  g.offs = offsets;
  g.groups = (int)groups;
  gm_plan(g, static_cast<uint8_t*>(ws));
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int tok = prof_begin("mx grouped matmul", s);
  const hipError_t err = launch_mx_grouped(g, e, s);
  prof_end(tok, s);
  return launched(err, "mx grouped matmul");
}

}  // extern "C"

namespace brq {
namespace {

brq_status page_ok(int32_t head_dim, int32_t page) {
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return refuse(BRQ_ERR_UNSUPPORTED, "head_dim %d must be 64, 128 or 256", head_dim);
  if (page < 16 || page > 1024 || (page & (page - 1)))
    return refuse(BRQ_ERR_UNSUPPORTED, "page %d must be a power of two in 16..1024", page);
  return BRQ_OK;
}

brq_status kv_setup(KvArgs& a, const brq_plan* plan, const void* k, int64_t ldk, const void* v, int64_t ldv, int32_t t,
                    const int64_t* slots, int64_t tokens, int32_t heads, int32_t head_dim, int32_t page, int64_t pages,
                    const uint8_t* cache, bool* done) {
  clear_error();
  *done = false;
  std::memset(&a, 0, sizeof a);
  if (!dtype_ok(t)) return refuse(BRQ_ERR_INVALID_ARGUMENT, "bad dtype %d", t);
  if (tokens < 0 || heads < 1 || pages < 0) return refuse(BRQ_ERR_INVALID_ARGUMENT, "bad shape");
  brq_status st = page_ok(head_dim, page);
  if (st != BRQ_OK) return st;
  const int64_t row = (int64_t)heads * head_dim;
  if (ldk < row || ldv < row) return refuse(BRQ_ERR_INVALID_ARGUMENT, "leading dimension below heads * head_dim");
  if ((st = transform_of(plan, head_dim, &a.signs, &a.d, &a.rnorm)) != BRQ_OK) return st;
  if (tokens == 0) {
    *done = true;
    return BRQ_OK;
  }
  if (tokens + (kKvQuad - 1) > kMxMost / row) return refuse(BRQ_ERR_UNSUPPORTED, "more than 2^34 values");
  if (!k || !v || !slots || (!cache && pages > 0)) return refuse(BRQ_ERR_INVALID_ARGUMENT, "NULL data pointer");
  if (rows_misaligned(k, ldk, t) || rows_misaligned(v, ldv, t))
    return refuse(BRQ_ERR_ALIGNMENT, "rows must be 16-byte aligned");
  if (misaligned(cache, 16) || misaligned(slots, 8))
    return refuse(BRQ_ERR_ALIGNMENT, "the cache must be 16-byte and slots 8-byte aligned");
  a.k = k;
  a.v = v;
  a.ldk = ldk;
  a.ldv = ldv;
  a.t = t;
  a.slots = slots;
  a.tokens = tokens;
  a.heads = heads;
  a.pg = KvPage{head_dim, page};
  a.lgP = log2_of(page);
  a.pages = pages;
  a.cache = const_cast<uint8_t*>(cache);
  return BRQ_OK;
}

constexpr int64_t kKpMost = ((int64_t)1 << 31) - 1;
// A table whose entries a launch of a thread for each can have.
bool entries_ok(int64_t rows, int64_t width) { return rows <= kKpMost && (width == 0 || rows <= kKpMost / width); }
// A reservation whose entries have ranks in 32 bits and whose sequences a launch can have.
bool reserve_ok(int64_t batch, int64_t tokens, int64_t page) {
  return batch < (int64_t)1 << 24 && tokens <= kKpMost && batch <= kKpMost / kp_per(tokens, page);
}

// Query heads per workgroup and their number of workgroups (AtArgs::nt, ht).
void at_shape(int32_t q_heads, int32_t heads, int* nt, int* ht) {
  const int group = q_heads / heads;
  *nt = group > kAtCols ? 2 : 1;
  *ht = (group + kAtCols * *nt - 1) / (kAtCols * *nt);
}

// Shared checks of the attentions, `tokens` rows a sequence; *done set when
// there is nothing to do.
brq_status at_setup(AtArgs& a, const brq_plan* plan, const void* q, int64_t ldq, int32_t qt, const uint8_t* cache,
                    int64_t pages, const int32_t* table, int64_t ldt, const int32_t* lens, int64_t batch,
                    int32_t tokens, int32_t q_heads, int32_t heads, int32_t head_dim, int32_t page, float scale,
                    int32_t window, void* out, int64_t ldo, float* lse, bool* done) {
  *done = false;
  std::memset(&a, 0, sizeof a);
  if (!dtype_ok(qt)) return refuse(BRQ_ERR_INVALID_ARGUMENT, "bad dtype %d", qt);
  if (batch < 0 || heads < 1 || q_heads < 1 || pages < 0 || ldt < 0 || window < 0)
    return refuse(BRQ_ERR_INVALID_ARGUMENT, "bad shape or window");
  if (q_heads % heads)
    return refuse(BRQ_ERR_INVALID_ARGUMENT, "%d query heads are not a multiple of %d key-value heads", q_heads, heads);
  if (!std::isfinite(scale)) return refuse(BRQ_ERR_INVALID_ARGUMENT, "scale must be finite");
  brq_status st = page_ok(head_dim, page);
  if (st != BRQ_OK) return st;
  const int64_t row = (int64_t)q_heads * head_dim;
  if (ldq < row || ldo < row)
    return refuse(BRQ_ERR_INVALID_ARGUMENT, "leading dimension below q_heads * head_dim");
  if ((st = transform_of(plan, head_dim, &a.signs, &a.d, &a.rnorm)) != BRQ_OK) return st;
  if (batch == 0 || tokens == 0) {
    *done = true;
    return BRQ_OK;
  }
  if (batch > (((int64_t)1 << 24) - 1) / q_heads / tokens)  // up to one workgroup of 256 threads for each
    return refuse(BRQ_ERR_UNSUPPORTED, "2^24 rows times query heads or more");
  if (!q || !out || !lens || (ldt > 0 && !table) || (pages > 0 && !cache))
    return refuse(BRQ_ERR_INVALID_ARGUMENT, "NULL data pointer");
  if (rows_misaligned(q, ldq, qt) || rows_misaligned(out, ldo, qt))
    return refuse(BRQ_ERR_ALIGNMENT, "query and output rows must be 16-byte aligned");
  if (misaligned(cache, 16) || misaligned(table, 4) || misaligned(lens, 4) || misaligned(lse, 4))
    return refuse(BRQ_ERR_ALIGNMENT, "the cache must be 16-byte, table, lens and lse 4-byte aligned");
  a.q = q;
  a.ldq = ldq;
  a.out = out;
  a.ldo = ldo;
  a.qt = qt;
  a.cache = cache;
  a.pages = pages;
  a.pg = KvPage{head_dim, page};
  a.lgP = log2_of(page);
  a.table = table;
  a.ldt = ldt;
  a.lens = lens;
  // without a page there is no visible token (and none to read where there is no other)
  a.cap = pages == 0 ? 0 : (int)(ldt < (kAtMaxKeys >> a.lgP) ? ldt << a.lgP : kAtMaxKeys);
  a.batch = batch;
  a.q_heads = q_heads;
  a.heads = heads;
  a.group = q_heads / heads;
  a.scale = scale;
  a.window = window;
  a.lse = lse;
  return BRQ_OK;
}

}  // namespace
}  // namespace brq

extern "C" {

size_t brq_kv_page_bytes(int32_t head_dim, int32_t page) {
  if (page_ok(head_dim, page) != BRQ_OK) return 0;
  return (size_t)KvPage{head_dim, page}.bytes();
}

brq_status brq_kv_append(const brq_plan* plan, const void* k, int64_t ldk, const void* v, int64_t ldv, int32_t xt,
                         const int64_t* slots, int64_t tokens, int32_t heads, int32_t head_dim, int32_t page,
                         int64_t pages, uint8_t* cache, void* stream) {
  KvArgs a;
  bool done;
  const brq_status st =
      kv_setup(a, plan, k, ldk, v, ldv, xt, slots, tokens, heads, head_dim, page, pages, cache, &done);
  if (st != BRQ_OK || done) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int tok = prof_begin("kv append", s);
  const hipError_t e = launch_kv_append(a, s);
  prof_end(tok, s);
  return launched(e, "kv append");
}

brq_status brq_kv_read(const brq_plan* plan, const uint8_t* cache, const int64_t* slots, int64_t tokens, int32_t heads,
                       int32_t head_dim, int32_t page, int64_t pages, void* k, int64_t ldk, void* v, int64_t ldv,
                       int32_t ot, void* stream) {
  KvArgs a;
  bool done;
  const brq_status st =
      kv_setup(a, plan, k, ldk, v, ldv, ot, slots, tokens, heads, head_dim, page, pages, cache, &done);
  if (st != BRQ_OK || done) return st;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int tok = prof_begin("kv read", s);
  const hipError_t e = launch_kv_read(a, s);
  prof_end(tok, s);
  return launched(e, "kv read");
}

size_t brq_kv_move_workspace_bytes(int64_t tokens, int32_t heads, int32_t head_dim) {
  if (tokens <= 0 || heads < 1 || (head_dim != 64 && head_dim != 128 && head_dim != 256) ||
      tokens > kKpTokens / heads)
    return 0;
  return kp_move_bytes(tokens, heads, head_dim);
}

brq_status brq_kv_move(uint8_t* cache, const int64_t* src, const int64_t* dst, int64_t tokens, int32_t heads,
                       int32_t head_dim, int32_t page, int64_t pages, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  if (tokens < 0 || heads < 1 || pages < 0) return refuse(BRQ_ERR_INVALID_ARGUMENT, "bad shape");
  brq_status st = page_ok(head_dim, page);
  if (st != BRQ_OK) return st;
  if (tokens == 0 || pages == 0) return BRQ_OK;
  if (tokens > kKpTokens / heads) return refuse(BRQ_ERR_UNSUPPORTED, "more than 2^27 tokens times heads");
  if (!cache || !src || !dst) return refuse(BRQ_ERR_INVALID_ARGUMENT, "NULL data pointer");
  if (misaligned(cache, 16) || misaligned(src, 8) || misaligned(dst, 8))
    return refuse(BRQ_ERR_ALIGNMENT, "the cache must be 16-byte and slots 8-byte aligned");
  if ((st = workspace_ok(ws, ws_bytes, brq_kv_move_workspace_bytes(tokens, heads, head_dim))) != BRQ_OK) return st;
  const KpMove a = {src, dst, tokens, heads, KvPage{head_dim, page}, log2_of(page), pages, cache,
                    static_cast<uint8_t*>(ws)};
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int tok = prof_begin("kv move", s);
  const hipError_t e = launch_kv_move(a, s);
  prof_end(tok, s);
  return launched(e, "kv move");
}

brq_status brq_kv_fork(const int32_t* table, const int32_t* lens, int64_t batch, int64_t width, const int32_t* parents,
                       int64_t children, int32_t* refs, int64_t pages, int32_t* out_table, int32_t* out_lens,
                       void* stream) {
  clear_error();
  if (batch < 0 || width < 0 || children < 0 || pages < 0) return refuse(BRQ_ERR_INVALID_ARGUMENT, "bad shape");
  if (children == 0) return BRQ_OK;
  if (!entries_ok(batch, width) || !entries_ok(children, width) || pages > kKpMost)
    return refuse(BRQ_ERR_UNSUPPORTED, "2^31 entries or pages or more");
  if (!parents || !out_lens || (batch > 0 && !lens) || (width > 0 && (!out_table || (batch > 0 && !table))) ||
      (pages > 0 && !refs))
    return refuse(BRQ_ERR_INVALID_ARGUMENT, "NULL data pointer");
  if (misaligned(table, 4) || misaligned(lens, 4) || misaligned(parents, 4) || misaligned(refs, 4) ||
      misaligned(out_table, 4) || misaligned(out_lens, 4))
    return refuse(BRQ_ERR_ALIGNMENT, "tables, lengths, parents and refs must be 4-byte aligned");
  const KpFork a = {table, lens, parents, batch, width, children, pages, refs, out_table, out_lens};
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int tok = prof_begin("kv fork", s);
  const hipError_t e = launch_kv_fork(a, s);
  prof_end(tok, s);
  return launched(e, "kv fork");
}

size_t brq_kv_reserve_workspace_bytes(int64_t batch, int64_t tokens, int32_t page, int64_t pages) {
  if (batch <= 0 || tokens <= 0 || pages < 0 || page_ok(64, page) != BRQ_OK || !reserve_ok(batch, tokens, page)) return 0;
  return kp_bytes(batch, tokens, page, pages);
}

brq_status brq_kv_reserve(uint8_t* cache, int32_t* table, const int32_t* lens, int64_t batch, int64_t width,
                          int32_t* refs, int64_t pages, int64_t tokens, int32_t heads, int32_t head_dim, int32_t page,
                          int64_t* slots, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  if (batch < 0 || width < 0 || pages < 0 || tokens < 0 || heads < 1)
    return refuse(BRQ_ERR_INVALID_ARGUMENT, "bad shape");
  brq_status st = page_ok(head_dim, page);
  if (st != BRQ_OK) return st;
  if (batch == 0 || tokens == 0) return BRQ_OK;
  if (!entries_ok(batch, width) || !reserve_ok(batch, tokens, page) || pages > kKpMost || heads > 65535)
    return refuse(BRQ_ERR_UNSUPPORTED, "2^31 entries or pages or more, 2^24 sequences or more, or above 65535 heads");
  if (!lens || !slots || (width > 0 && !table) || (pages > 0 && (!cache || !refs)))
    return refuse(BRQ_ERR_INVALID_ARGUMENT, "NULL data pointer");
  if (misaligned(cache, 16) || misaligned(slots, 8) || misaligned(table, 4) || misaligned(lens, 4) || misaligned(refs, 4))
    return refuse(BRQ_ERR_ALIGNMENT, "the cache must be 16-byte, slots 8-byte, table, lens and refs 4-byte aligned");
  if ((st = workspace_ok(ws, ws_bytes, kp_bytes(batch, tokens, page, pages))) != BRQ_OK) return st;
  KpReserve a;
  std::memset(&a, 0, sizeof a);
  a.cache = cache;
  a.table = table;
  a.lens = lens;
  a.batch = batch;
  a.width = width;
  a.refs = refs;
  a.pages = pages;
  a.tokens = tokens;
  a.heads = heads;
  a.pg = KvPage{head_dim, page};
  a.lgP = log2_of(page);
  a.slots = slots;
  a.per = kp_per(tokens, page);
  a.copy = static_cast<int4*>(ws);
  a.item = reinterpret_cast<int32_t*>(a.copy + batch);
  a.fresh = a.item + batch * a.per;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int tok = prof_begin("kv reserve", s);
  const hipError_t e = launch_kv_reserve(a, s);
  prof_end(tok, s);
  return launched(e, "kv reserve");
}

brq_status brq_kv_free(int32_t* table, int64_t batch, int64_t width, int32_t* refs, int64_t pages, const int32_t* rows,
                       int64_t n, void* stream) {
  clear_error();
  if (batch < 0 || width < 0 || pages < 0 || n < 0 || (!rows && n > batch))
    return refuse(BRQ_ERR_INVALID_ARGUMENT, "bad shape");
  if (batch == 0 || width == 0 || n == 0) return BRQ_OK;
  if (!entries_ok(batch, width) || !entries_ok(n, width) || pages > kKpMost)
    return refuse(BRQ_ERR_UNSUPPORTED, "2^31 entries or pages or more");
  if (!table || (pages > 0 && !refs)) return refuse(BRQ_ERR_INVALID_ARGUMENT, "NULL data pointer");
  if (misaligned(table, 4) || misaligned(refs, 4) || misaligned(rows, 4))
    return refuse(BRQ_ERR_ALIGNMENT, "table, refs and rows must be 4-byte aligned");
  const KpFree a = {table, batch, width, pages, n, refs, rows};
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int tok = prof_begin("kv free", s);
  const hipError_t e = launch_kv_free(a, s);
  prof_end(tok, s);
  return launched(e, "kv free");
}

size_t brq_paged_attention_workspace_bytes(int64_t batch, int32_t q_heads, int32_t heads, int32_t head_dim) {
  if (batch <= 0 || heads < 1 || q_heads < heads || q_heads % heads || head_dim < 1) return 0;
  int nt, ht;
  at_shape(q_heads, heads, &nt, &ht);
  if (batch > kAtMaxBatch) return 0;
  return at_bytes(head_dim, nt, batch * heads * ht);
}

brq_status brq_paged_attention(const brq_plan* plan, const void* q, int64_t ldq, int32_t qt, const uint8_t* cache,
                               int64_t pages, const int32_t* table, int64_t ldt, const int32_t* lens, int64_t batch,
                               int32_t q_heads, int32_t heads, int32_t head_dim, int32_t page, float scale,
                               int32_t window, void* out, int64_t ldo, float* lse, void* ws, size_t ws_bytes,
                               void* stream) {
  clear_error();
  AtArgs a;
  bool done;
  brq_status st = at_setup(a, plan, q, ldq, qt, cache, pages, table, ldt, lens, batch, 1, q_heads, heads, head_dim, page,
                           scale, window, out, ldo, lse, &done);
  if (st != BRQ_OK || done) return st;
  if ((st = workspace_ok(ws, ws_bytes, brq_paged_attention_workspace_bytes(batch, q_heads, heads, head_dim))) != BRQ_OK)
    return st;
  at_shape(q_heads, heads, &a.nt, &a.ht);
  a.wgs = batch <= kAtMaxBatch ? at_workgroups(head_dim, a.nt) : 0;
  a.part = static_cast<float*>(ws);
  a.who = a.wgs ? reinterpret_cast<int2*>(static_cast<char*>(ws) + at_part_bytes(head_dim, a.nt)) : nullptr;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int tok = prof_begin("paged attention", s);
  const hipError_t e = launch_paged_attention(a, s);
  prof_end(tok, s);
  return launched(e, "paged attention");
}

size_t brq_tree_attention_workspace_bytes(int64_t batch, int32_t tokens, int32_t q_heads, int32_t heads,
                                          int32_t head_dim) {
  if (batch <= 0 || tokens < 1 || tokens > kTrTokens || heads < 1 || q_heads < heads ||
      q_heads % heads || (head_dim != 64 && head_dim != 128 && head_dim != 256))
    return 0;
  const int64_t rows = tr_rows(tokens, q_heads, heads);
  const int nt = tr_nt(rows, head_dim);
  if (batch > kAtMaxBatch) return 0;
  const int64_t units = batch * heads * ((rows + 16 * nt - 1) / (16 * nt));
  return tr_dealt(batch, units, nt, head_dim) ? tr_part_bytes(head_dim, nt) + (size_t)units * sizeof(int2) : 0;
}

brq_status brq_tree_attention(const brq_plan* plan, const void* q, int64_t ldq, int32_t qt, const uint8_t* cache,
                              int64_t pages, const int32_t* table, int64_t ldt, const int32_t* lens,
                              const int64_t* mask, int64_t batch, int32_t tokens, int32_t q_heads, int32_t heads,
                              int32_t head_dim, int32_t page, float scale, int32_t window, void* out, int64_t ldo,
                              float* lse, void* ws, size_t ws_bytes, void* stream) {
  clear_error();
  TrArgs t;
  bool done;
  if (tokens < 0) return refuse(BRQ_ERR_INVALID_ARGUMENT, "bad shape");
  if (tokens > kTrTokens)
    return refuse(BRQ_ERR_UNSUPPORTED, "%d drafted tokens, a mask has %d bits", tokens, kTrTokens);
  brq_status st = at_setup(t.at, plan, q, ldq, qt, cache, pages, table, ldt, lens, batch, tokens, q_heads, heads,
                           head_dim, page, scale, window, out, ldo, lse, &done);
  if (st != BRQ_OK || done) return st;
  if (!mask) return refuse(BRQ_ERR_INVALID_ARGUMENT, "NULL data pointer");
  if (misaligned(mask, 8)) return refuse(BRQ_ERR_ALIGNMENT, "the mask must be 8-byte aligned");
  if ((st = workspace_ok(ws, ws_bytes,
                         brq_tree_attention_workspace_bytes(batch, tokens, q_heads, heads, head_dim))) != BRQ_OK)
    return st;
  t.mask = mask;
  t.tokens = tokens;
  const int64_t rows = tr_rows(tokens, q_heads, heads);
  t.at.nt = tr_nt(rows, head_dim);
  t.at.ht = (int)((rows + 16 * t.at.nt - 1) / (16 * t.at.nt));
  t.at.wgs = tr_dealt(batch, batch * heads * t.at.ht, t.at.nt, head_dim) ? tr_workgroups(head_dim, t.at.nt) : 0;
  t.at.part = static_cast<float*>(ws);
  t.at.who =
      t.at.wgs ? reinterpret_cast<int2*>(static_cast<char*>(ws) + tr_part_bytes(head_dim, t.at.nt)) : nullptr;
  hipStream_t s = static_cast<hipStream_t>(stream);
  const int tok = prof_begin("tree attention", s);
  const hipError_t e = launch_tree_attention(t, s);
  prof_end(tok, s);
  return launched(e, "tree attention");
}

}  // extern "C"
