// Tokens and pages of the paged 4-bit cache moved, shared, taken and given back
// (layout: KvPage in mx.h).  Nothing is requantized: codes and scales are copied
// as they are.
//
// A token of one head is moved by 16 lanes: lane r takes the D / 32 bytes of run
// r of its values' codes and as many of its keys' codes, the first D / 32 lanes
// one scale of each.  Counts change by whole numbers, so their order does not
// show.
#include <type_traits>

#include "mx_dev.h"

namespace brq {
namespace {

// A lane's bytes of a token's codes, keys and values, and of its scales.
template <int D>
struct KpWord {
  using W = std::conditional_t<D == 64, uint16_t, std::conditional_t<D == 128, uint32_t, uint2>>;
  W k, v;
  uint8_t ks, vs;

  __device__ __forceinline__ void load(const uint8_t* head, const KvPage& pg, int t, int r) {
    k = *reinterpret_cast<const W*>(head + pg.kcode(t) + r * (D / 32));
    v = *reinterpret_cast<const W*>(head + pg.vcode(t, r));
    if (r < D / 32) {
      ks = head[pg.kscale(t) + r];
      vs = head[pg.vscale(t, r)];
    }
  }
  // the same in a row of the workspace: codes of keys and values, scales of either
  __device__ __forceinline__ void load(const uint8_t* row, int r) {
    k = *reinterpret_cast<const W*>(row + r * (D / 32));
    v = *reinterpret_cast<const W*>(row + D / 2 + r * (D / 32));
    if (r < D / 32) {
      ks = row[D + r];
      vs = row[D + D / 32 + r];
    }
  }
  __device__ __forceinline__ void store(uint8_t* row, int r) const {
    *reinterpret_cast<W*>(row + r * (D / 32)) = k;
    *reinterpret_cast<W*>(row + D / 2 + r * (D / 32)) = v;
    if (r < D / 32) {
      row[D + r] = ks;
      row[D + D / 32 + r] = vs;
    }
  }
  __device__ __forceinline__ void store(uint8_t* head, const KvPage& pg, int t, int r) const {
    *reinterpret_cast<W*>(head + pg.kcode(t) + r * (D / 32)) = k;
    *reinterpret_cast<W*>(head + pg.vcode(t, r)) = v;
    if (r < D / 32) {
      head[pg.kscale(t) + r] = ks;
      head[pg.vscale(t, r)] = vs;
    }
  }
};

// The slots of a pair, or one outside the cache: not moved.
__device__ __forceinline__ bool kp_pair(const KpMove& a, int64_t tok, int64_t* src, int64_t* dst) {
  if (tok >= a.tokens) return false;
  *src = a.src[tok];
  *dst = a.dst[tok];
  return *src >= 0 && (*src >> a.lgP) < a.pages && *dst >= 0 && (*dst >> a.lgP) < a.pages;
}
template <int D>
__device__ __forceinline__ uint8_t* kp_head(const KpMove& a, int64_t slot, int h, int* t) {
  *t = (int)(slot & (a.pg.P - 1));
  return a.cache + ((slot >> a.lgP) * a.heads + h) * KvPage{D, a.pg.P}.bytes();
}

// Up to kKpFew tokens: a workgroup for each head reads them all into registers, then
// writes them.
template <int D>
__global__ __launch_bounds__(kKpThreads) void kp_few_kernel(KpMove a) {
  constexpr int N = kKpFew / (kKpThreads / 16);
  const int h = blockIdx.x, r = threadIdx.x & 15;
  const KvPage pg{D, a.pg.P};
  KpWord<D> w[N];
  int64_t src, dst[N];
  bool ok[N];
  int t;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    ok[i] = kp_pair(a, i * (kKpThreads / 16) + threadIdx.x / 16, &src, &dst[i]);
    if (ok[i]) {
      const uint8_t* head = kp_head<D>(a, src, h, &t);
      w[i].load(head, pg, t, r);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // every wavefront has what it read
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (ok[i]) {
      uint8_t* head = kp_head<D>(a, dst[i], h, &t);
      w[i].store(head, pg, t, r);
    }
}

// More: tokens to the workspace and from it, one launch each, so that everything is
// read before anything is written; 16 lanes take kKpRun tokens of a head, whose loads
// travel together (15000 tokens of 8 heads of 128, one at a time 14.7 and 12.6 us, so
// 12.8 and 10.4: bound by the number of pieces, a run of values being 4 bytes).
template <int D, bool OUT>
__global__ __launch_bounds__(kMxThreads) void kp_move_kernel(KpMove a) {
  const uint32_t row = blockIdx.x * (kMxThreads / 16) + threadIdx.x / 16, run = row / (uint32_t)a.heads;
  const int h = (int)(row - run * (uint32_t)a.heads), r = threadIdx.x & 15;
  const KvPage pg{D, a.pg.P};
  KpWord<D> w[kKpRun];
  int64_t src[kKpRun], dst[kKpRun];
  bool ok[kKpRun];
  int t;
#pragma unroll
  for (int i = 0; i < kKpRun; ++i) ok[i] = kp_pair(a, (int64_t)run * kKpRun + i, &src[i], &dst[i]);
  uint8_t* keep = a.ws + (int64_t)row * kKpRun * kp_row_bytes(D);
#pragma unroll
  for (int i = 0; i < kKpRun; ++i)
    if (ok[i]) {
      if constexpr (OUT) {
        w[i].load(keep + i * kp_row_bytes(D), r);
      } else {
        const uint8_t* head = kp_head<D>(a, src[i], h, &t);
        w[i].load(head, pg, t, r);
      }
    }
#pragma unroll
  for (int i = 0; i < kKpRun; ++i)
    if (ok[i]) {
      if constexpr (OUT) {
        uint8_t* head = kp_head<D>(a, dst[i], h, &t);
        w[i].store(head, pg, t, r);
      } else {
        w[i].store(keep + i * kp_row_bytes(D), r);
      }
    }
}

// A row of the table for each child: its parent's pages, which it holds too.
__global__ __launch_bounds__(kMxThreads) void kp_fork_kernel(KpFork a) {
  const int64_t i = (int64_t)blockIdx.x * kMxThreads + threadIdx.x;
  if (i >= a.children * (a.width > 0 ? a.width : 1)) return;
  const int64_t f = a.width > 0 ? i / a.width : i, c = a.width > 0 ? i - f * a.width : 0;
  const int parent = a.parents[f];
  const bool there = parent >= 0 && parent < a.batch;
  if (c == 0) a.out_lens[f] = there ? a.lens[parent] : 0;
  if (a.width == 0) return;
  int p = there ? a.table[parent * a.width + c] : -1;
  if (p < 0 || p >= a.pages) p = -1;
  a.out_table[i] = p;
  if (p >= 0) atomicAdd(&a.refs[p], 1);
}

// The pages of rows given back, their entries cleared (by an exchange: a row
// that is named twice is given back once).
__global__ __launch_bounds__(kMxThreads) void kp_free_kernel(KpFree a) {
  const int64_t i = (int64_t)blockIdx.x * kMxThreads + threadIdx.x;
  if (i >= a.n * a.width) return;
  const int64_t f = i / a.width, c = i - f * a.width, row = a.rows ? a.rows[f] : f;
  if (row < 0 || row >= a.batch) return;
  const int p = atomicExch(&a.table[row * a.width + c], -1);
  if (p >= 0 && p < a.pages) atomicSub(&a.refs[p], 1);
}

// ---- reservation

// Inclusive sum over the workgroup's threads; *all the whole sum.
__device__ __forceinline__ int kp_scan(int n, int* scratch, int* all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = n;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  __syncthreads();
  if (lane == 63) scratch[wave] = x;
  __syncthreads();
  int s = 0;
#pragma unroll
  for (int w = 0; w < kKpThreads / 64; ++w) {
    if (w < wave) x += scratch[w];
    s += scratch[w];
  }
  *all = s;
  return x;
}

// One workgroup decides: which entries need a page, in order (their ranks); as
// many free pages, the lowest first; then who gets which.  Counts are read
// before any is changed, that of an entry's page too: one that nobody holds (refs below 1) is
// free, may be another's a moment later, and is neither counted nor copied here.  (128 sequences over 5000 pages 5 us, of which most is waiting for
// one read after the other; a search through all of a pool takes 1 us for some 4000 pages.)
__global__ __launch_bounds__(kKpThreads) void kp_reserve_kernel(KpReserve a) {
  __shared__ int scratch[kKpThreads / 64];
  const int tid = threadIdx.x;
  const int64_t items = a.batch * a.per;
  int total = 0;
  for (int64_t i0 = 0; i0 < items; i0 += kKpThreads) {
    const int64_t i = i0 + tid;
    KpItem it;
    const bool here = i < items && kp_item(a, i, it);
    int p = -1;
    if (here) p = a.table[it.row * a.width + it.entry];
    const int holders = here && p >= 0 && p < a.pages ? a.refs[p] : 0;
    const bool need = here && holders != 1;
    int all;
    const int rank = total + kp_scan(need, scratch, &all) - 1;
    if (i < items) a.item[i] = need ? kp_want(rank, holders > 1) : here ? p : -1;
    total += all;
  }
  // free pages
  int found = 0;
  for (int64_t p0 = 0; p0 < a.pages && found < total; p0 += kKpThreads) {
    const int64_t p = p0 + tid;
    const bool free = p < a.pages && a.refs[p] <= 0;
    int all;
    const int at = found + kp_scan(free, scratch, &all) - 1;
    if (free && at < total) a.fresh[at] = (int)p;
    found += all;
  }
  __syncthreads();  // with the list's stores and the counts' loads done
  for (int64_t i0 = 0; i0 < items; i0 += kKpThreads) {
    const int64_t i = i0 + tid;
    if (i >= items) break;
    const int r = a.item[i];
    KpItem it;
    if (!kp_item(a, i, it)) {
      if (i % a.per == 0) a.copy[i / a.per] = make_int4(-1, -1, 0, 0);
      continue;
    }
    int4 copy = make_int4(-1, -1, 0, 0);
    if (r <= -2) {
      const int rank = kp_rank(r);
      int page = -1;
      if (rank < found && rank < kKpRanks) {
        int* entry = &a.table[it.row * a.width + it.entry];
        const int old = *entry;
        page = a.fresh[rank];
        *entry = page;
        a.refs[page] = 1;
        if (kp_shared(r)) {
          atomicSub(&a.refs[old], 1);
          if (it.used > 0) copy = make_int4(old, page, it.used, 0);
        }
      }
      a.item[i] = page;
    }
    if (i % a.per == 0) a.copy[i / a.per] = copy;
  }
}

// The slots of the new tokens, and the first tokens of shared pages (128 sequences with
// 32 tokens of 8 heads of 128 each in the mean 4 us):
// whole sixteens of them, of each of a page's four parts the first bytes, 16 at a time.
__global__ __launch_bounds__(kMxThreads) void kp_copy_kernel(KpReserve a) {
  const int64_t b = blockIdx.x;
  const int part = blockIdx.y, tid = threadIdx.x;
  for (int64_t j = (int64_t)part * kMxThreads + tid; j < a.tokens; j += (int64_t)gridDim.y * kMxThreads) {
    const int64_t n = a.lens[b], pos = n + j;
    int64_t slot = -1;
    if (n >= 0 && (pos >> a.lgP) < a.width) {
      const int page = a.item[b * a.per + ((pos >> a.lgP) - (n >> a.lgP))];
      if (page >= 0) slot = ((int64_t)page << a.lgP) + (pos & (a.pg.P - 1));
    }
    a.slots[b * a.tokens + j] = slot;
  }
  const int4 c = a.copy[b];
  if (c.z <= 0) return;
  const int D = a.pg.D, used = (c.z + 15) / 16 * 16;
  // 16-byte pieces of the keys' codes, the values' codes, and of either's scales
  const int codes = used * (D / 32), scales = used * D / 512, pieces = 2 * (codes + scales);
  for (int h = part; h < a.heads; h += gridDim.y) {
    const uint4* from = reinterpret_cast<const uint4*>(a.cache + ((int64_t)c.x * a.heads + h) * a.pg.bytes());
    uint4* to = reinterpret_cast<uint4*>(a.cache + ((int64_t)c.y * a.heads + h) * a.pg.bytes());
    for (int i = tid; i < pieces; i += kMxThreads) {
      const int at = kp_piece(a.pg, codes, scales, i);
      to[at] = from[at];
    }
  }
}

template <int D>
void kp_move(const KpMove& a, hipStream_t s) {
  if (kp_few(a.tokens, a.heads)) {
    kp_few_kernel<D><<<dim3((unsigned)a.heads), kKpThreads, 0, s>>>(a);
    return;
  }
  const int64_t rows = kp_runs(a.tokens) * a.heads;
  const dim3 grid((unsigned)((rows + kMxThreads / 16 - 1) / (kMxThreads / 16)));
  kp_move_kernel<D, false><<<grid, kMxThreads, 0, s>>>(a);
  kp_move_kernel<D, true><<<grid, kMxThreads, 0, s>>>(a);
}

}  // namespace

hipError_t launch_kv_move(const KpMove& a, hipStream_t s) {
  if (a.pg.D == 64) kp_move<64>(a, s);
  else if (a.pg.D == 128) kp_move<128>(a, s);
  else kp_move<256>(a, s);
  return hipGetLastError();
}

hipError_t launch_kv_fork(const KpFork& a, hipStream_t s) {
  const int64_t n = a.children * (a.width > 0 ? a.width : 1);
  kp_fork_kernel<<<dim3((unsigned)((n + kMxThreads - 1) / kMxThreads)), kMxThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_kv_free(const KpFree& a, hipStream_t s) {
  kp_free_kernel<<<dim3((unsigned)((a.n * a.width + kMxThreads - 1) / kMxThreads)), kMxThreads, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_kv_reserve(const KpReserve& a, hipStream_t s) {
  kp_reserve_kernel<<<dim3(1), kKpThreads, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  kp_copy_kernel<<<dim3((unsigned)a.batch, (unsigned)a.heads), kMxThreads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace brq
