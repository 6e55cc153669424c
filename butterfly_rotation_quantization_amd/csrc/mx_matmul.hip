// Product of two microscaled 4-bit matrices on the scaled matrix
// instructions (format: mx.h).
#include "mx_dev.h"

namespace brq {
namespace {

__device__ __forceinline__ void mm_store(void* y, int yt, int64_t off, float v) {
  if (yt == BRQ_F32) static_cast<float*>(y)[off] = v;
  else if (yt == BRQ_BF16) static_cast<uint16_t*>(y)[off] = (uint16_t)mx_bf16(v);
  else static_cast<uint16_t*>(y)[off] = (uint16_t)mx_f16(v);
}

// One wavefront per 16 x 16 outputs: lane l holds block l / 16 of a step of
// 128 values of row l % 16, of both operands, with the block's scale.
__global__ __launch_bounds__(64) void mm_simple_kernel(MmArgs a) {
  const int lane = threadIdx.x, lr = lane & 15, lg = lane >> 4;
  const int64_t t0 = (int64_t)blockIdx.y * 16, o0 = (int64_t)blockIdx.x * 16;
  const int64_t ra = t0 + lr, rb = o0 + lr;
  const int64_t nb = a.n / kMxBlock;
  const bool va = ra < a.T, vb = rb < a.m;
  mxf4 acc = {0.f, 0.f, 0.f, 0.f};
  for (int64_t k = 0; k < nb; k += 4) {
    const int64_t blk = k + lg;
    mxi4 x = {0, 0, 0, 0}, w = {0, 0, 0, 0};
    int sx = 127, sw = 127;
    if (va && blk < nb) {
      x = *reinterpret_cast<const mxi4*>(a.a + (ra * nb + blk) * 16);
      sx = a.as[ra * nb + blk];
    }
    if (vb && blk < nb) {
      w = *reinterpret_cast<const mxi4*>(a.b + (rb * nb + blk) * 16);
      sw = a.bs[rb * nb + blk];
    }
    const mxi8 X = {x[0], x[1], x[2], x[3], 0, 0, 0, 0}, W = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
    acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(X, W, acc, 4, 4, 0, sx, 0, sw);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {  // D: row 4 lg + i, column lr
    const int64_t t = t0 + 4 * lg + i;
    if (t < a.T && vb) mm_store(a.y, a.yt, t * a.ldy + rb, acc[i]);
  }
}


// ---- tiles through LDS

// c += a b with byte SA of sa and SB of sb as the scales; c stays in the
// accumulation registers.  Written out because with all 256 of them in use the
// register allocator moved sums to and fro between the two files (90 moves in
// a stage of 128 products).  The hardware orders these among themselves and
// after the loads of their operands; mm_settle comes before other reads of c.
template <int SA, int SB>
__device__ __forceinline__ void mm_mfma(mxi4 a, mxi4 b, mxf4& c, int sa, int sb) {
  asm volatile(
      "v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[%5,%6,0] op_sel_hi:[%7,%8,0] cbsz:4 blgp:4"
      : "+a"(c)
      : "v"(a), "v"(b), "v"(sa), "v"(sb), "n"(SA & 1), "n"(SB & 1), "n"(SA >> 1), "n"(SB >> 1));
}
// More wait states than any product needs until its result can be read.
__device__ __forceinline__ void mm_settle() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }
// byte ia of sa and byte ib of sb (constants once the loops are unrolled)
__device__ __forceinline__ void mm_step(mxi4 a, mxi4 b, mxf4& c, int sa, int ia, int sb, int ib) {
  switch ((ia & 3) * 4 + (ib & 3)) {
    case 0: return mm_mfma<0, 0>(a, b, c, sa, sb);
    case 1: return mm_mfma<0, 1>(a, b, c, sa, sb);
    case 2: return mm_mfma<0, 2>(a, b, c, sa, sb);
    case 3: return mm_mfma<0, 3>(a, b, c, sa, sb);
    case 4: return mm_mfma<1, 0>(a, b, c, sa, sb);
    case 5: return mm_mfma<1, 1>(a, b, c, sa, sb);
    case 6: return mm_mfma<1, 2>(a, b, c, sa, sb);
    case 7: return mm_mfma<1, 3>(a, b, c, sa, sb);
    case 8: return mm_mfma<2, 0>(a, b, c, sa, sb);
    case 9: return mm_mfma<2, 1>(a, b, c, sa, sb);
    case 10: return mm_mfma<2, 2>(a, b, c, sa, sb);
    case 11: return mm_mfma<2, 3>(a, b, c, sa, sb);
    case 12: return mm_mfma<3, 0>(a, b, c, sa, sb);
    case 13: return mm_mfma<3, 1>(a, b, c, sa, sb);
    case 14: return mm_mfma<3, 2>(a, b, c, sa, sb);
    default: return mm_mfma<3, 3>(a, b, c, sa, sb);
  }
}

__device__ __forceinline__ void mm_store4(void* y, int yt, int64_t off, mxf4 v, int valid, bool wide) {
  if (wide && valid >= 4) {
    if (yt == BRQ_F32) {
      *reinterpret_cast<mxf4*>(static_cast<float*>(y) + off) = v;
    } else {
      uint2 w;
      w.x = yt == BRQ_BF16 ? (mx_bf16(v[0]) | mx_bf16(v[1]) << 16) : (mx_f16(v[0]) | mx_f16(v[1]) << 16);
      w.y = yt == BRQ_BF16 ? (mx_bf16(v[2]) | mx_bf16(v[3]) << 16) : (mx_f16(v[2]) | mx_f16(v[3]) << 16);
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(y) + off) = w;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i < valid) mm_store(y, yt, off + i, v[i]);
}

constexpr int kMmK = 256;           // values of a row per stage
constexpr int kMmKB = kMmK / 2;     // their code bytes
constexpr int kMmKS = kMmK / kMxBlock;

__device__ const uint4 kMmZero = {0u, 0u, 0u, 0u};

// Byte g of the words of lanes c, c + 16, c + 32, c + 48 (g = lane / 16,
// c = lane % 16): a transpose of 4 x 4 bytes over the four rows of lanes.
__device__ __forceinline__ uint32_t mm_transpose(uint32_t w, uint32_t sel) {
  const auto h = __builtin_amdgcn_permlane32_swap(w, w, false, false);       // rows 0 1 0 1, 2 3 2 3
  const auto p = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);  // row 0, row 1
  const auto q = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);  // row 2, row 3
  const uint32_t lo = __builtin_amdgcn_perm(p[1], p[0], sel), hi = __builtin_amdgcn_perm(q[1], q[0], sel);
  return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

// 16 bytes per lane from p straight to LDS, lane l's to dst + l (dst uniform
// over the wavefront).  Written out because the compiler, which takes any LDS
// read to depend on such a load, would wait for it before the next one; the
// kernel waits for vmcnt(0) and a barrier before it reads what was brought.
__device__ __forceinline__ void mm_to_lds(const void* p, uint4* dst) {
  const uint32_t at = __builtin_amdgcn_readfirstlane(
      (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) void*)dst));
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(p) : "memory");
}

// Operands of one matrix step of 128 values.
template <int TT, int TO>
struct MmFrag {
  mxi4 x[TT], w[TO];
  int xs[(TT + 3) / 4], ws[(TO + 3) / 4];
};

// WT x WO wavefronts, each TT x TO tiles of 16 tokens x 16 outputs.
template <int WT, int WO, int TT, int TO>
__global__ __launch_bounds__(64 * WT * WO, 1) void mm_tile_kernel(MmArgs a) {
  constexpr int NTH = 64 * WT * WO;
  constexpr int BT = 16 * TT * WT, BO = 16 * TO * WO, ROWS = BT + BO;
  constexpr int NL = ROWS * (kMmKB / 16) / NTH;  // 16-byte pieces per thread and stage
  constexpr int RS = NTH / 8;                    // rows between a thread's pieces
  constexpr int NR = ROWS / NTH;                 // rows whose scales a thread brings
  constexpr int NTT = BT / 16, NTO = BO / 16;
  static_assert(ROWS % NTH == 0 && BT % RS == 0 && BT % 64 == 0 && BO % 64 == 0, "whole rows per thread and wavefront");
  __shared__ uint4 codes[2][ROWS * 8];           // piece c of row r at r * 8 + (c ^ (r & 7))
  __shared__ uint8_t scales[2][ROWS * 8];        // [block][row % 16][tile], tokens first

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lr = lane & 15, lg = lane >> 4;
  const int wt = wave % WT, wo = wave / WT;
  // tile of this workgroup
  const int64_t p = (int64_t)(blockIdx.x & 7) * a.per_xcd + (blockIdx.x >> 3);
  if (p >= (int64_t)a.gt * a.go) return;
  const int64_t band = p / ((int64_t)a.band * a.go);
  const int64_t q = p - band * a.band * a.go;
  const int64_t h = a.gt - band * a.band < a.band ? a.gt - band * a.band : a.band;  // rows of tiles in this band
  const int64_t t0 = (band * a.band + q % h) * BT, o0 = q / h * BO;

  const int64_t nb = a.n / kMxBlock, ld = a.n / 2;
  const int stages = (int)((nb + kMmKS - 1) / kMmKS);
  // The thread's LDS slots: row pr + j RS, piece pc of the row.  Rows past the
  // end repeat the last one (their products are not stored).
  const int pr = tid >> 3, pc = (tid & 7) ^ (pr & 7);
  const int lt = (int)(a.T - t0 < BT ? a.T - t0 : BT) - 1, lo = (int)(a.m - o0 < BO ? a.m - o0 : BO) - 1;
  const uint8_t* ab = a.a + t0 * ld + 16 * pc;
  const uint8_t* bb = a.b + o0 * ld + 16 * pc;
  const uint8_t* sp[NR];
#pragma unroll
  for (int j = 0; j < NR; ++j) {
    const int r = tid + j * NTH;
    sp[j] = r < BT ? a.as + (t0 + (r < lt ? r : lt)) * nb : a.bs + (o0 + (r - BT < lo ? r - BT : lo)) * nb;
  }
  const uint32_t tsel = (uint32_t)lg | (uint32_t)(4 + lg) << 8 | 0x0c0c0000u;

  // Pieces of stage s: straight to LDS; past the end of a row (the ragged last
  // stage, stages that do not exist) zeros are fetched instead.
  struct Source {
    const uint8_t *x, *w;
    unsigned ld;
    int row;
  };
  auto source = [&](int s) {
    const int64_t kb = (int64_t)s * kMmKB;
    const bool in = kb + 16 * pc < ld;
    Source f;
    f.x = in ? ab + kb : reinterpret_cast<const uint8_t*>(&kMmZero);
    f.w = in ? bb + kb : reinterpret_cast<const uint8_t*>(&kMmZero);
    f.ld = in ? (unsigned)ld : 0u;
    f.row = pr;
    asm volatile("" : "+v"(f.row));  // offsets are computed at each use, or NL of them would be kept
    return f;
  };
  auto fetch = [&](const Source& f, int buf, int j) {  // row < 256 and ld < 2^23: a 24-bit product
    const int r = j * RS < BT ? f.row + j * RS : f.row + j * RS - BT, last = j * RS < BT ? lt : lo;
    const uint8_t* g = (j * RS < BT ? f.x : f.w) + __umul24((unsigned)(r < last ? r : last), f.ld);
    mm_to_lds(g, &codes[buf][(tid & ~63) + j * NTH]);
  };
  auto fetch_scales = [&](int s, uint64_t (&v)[NR]) {
    // the row's last eight bytes where the stage is ragged, moved into place:
    // zeros (2^-127, times codes of zero) follow
    const int64_t k0 = (int64_t)s * kMmKS, k = k0 < nb - kMmKS ? k0 : nb - kMmKS;
    const int sh = k0 - k < kMmKS ? 8 * (int)(k0 - k) : 8 * (kMmKS - 1);
#pragma unroll
    for (int j = 0; j < NR; ++j) {
      __builtin_memcpy(&v[j], sp[j] + k, 8);
    }
    return sh;
  };
  auto put_scales = [&](int buf, const uint64_t (&v)[NR], int sh) {
#pragma unroll
    for (int j = 0; j < NR; ++j) {  // 64 rows of one operand: four tiles; lane (lr, lg) stores blocks lg and lg + 4
      const int r0 = (tid & ~63) + j * NTH;
      const int nt = r0 < BT ? NTT : NTO;
      uint8_t* d = &scales[buf][r0 < BT ? 0 : 8 * BT] + (lg * 16 + lr) * nt + (r0 < BT ? r0 : r0 - BT) / 16;
      *reinterpret_cast<uint32_t*>(d) = mm_transpose((uint32_t)(v[j] >> sh), tsel);
      *reinterpret_cast<uint32_t*>(d + 64 * nt) = mm_transpose((uint32_t)(v[j] >> sh >> 32), tsel);
    }
  };
  using Frag = MmFrag<TT, TO>;
  const int xr = 16 * TT * wt + lr, wr = BT + 16 * TO * wo + lr;  // LDS rows of the lane's first tiles
  // operand tile e of step k2 (tokens first), and the scales
  auto read = [&](Frag& f, int buf, int k2, int e) {
    const int c = (4 * k2 + lg) ^ (lr & 7);
    if (e < TT) f.x[e] = *reinterpret_cast<const mxi4*>(&codes[buf][(xr + 16 * e) * 8 + c]);
    else f.w[e - TT] = *reinterpret_cast<const mxi4*>(&codes[buf][(wr + 16 * (e - TT)) * 8 + c]);
  };
  auto read_scales = [&](Frag& f, int buf, int k2) {
    const uint8_t* xq = &scales[buf][((4 * k2 + lg) * 16 + lr) * NTT + TT * wt];
    const uint8_t* wq = &scales[buf][8 * BT + ((4 * k2 + lg) * 16 + lr) * NTO + TO * wo];
#pragma unroll
    for (int j = 0; j < (TT + 3) / 4; ++j)
      f.xs[j] = TT >= 4 ? reinterpret_cast<const int*>(xq)[j] : *reinterpret_cast<const uint16_t*>(xq);
#pragma unroll
    for (int i = 0; i < (TO + 3) / 4; ++i)
      f.ws[i] = TO >= 4 ? reinterpret_cast<const int*>(wq)[i] : *reinterpret_cast<const uint16_t*>(wq);
  };

  mxf4 acc[TO][TT];
#pragma unroll
  for (int i = 0; i < TO; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[i][j] = mxf4{0.f, 0.f, 0.f, 0.f};
  constexpr int NG = TT + TO, PER = (TT * TO + NG - 1) / NG;  // groups of one operand read and PER products
  auto products = [&](const Frag& f, int e) {
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int x = e * PER + u, i = x / TT, j = x % TT;
      if (x < TT * TO) mm_step(f.w[i], f.x[j], acc[i][j], f.ws[i / 4], i, f.xs[j / 4], j);
    }
  };

  // Stage s's first step multiplies while its second step's operands come from
  // LDS; then, once every wavefront has them and stage s + 1 has arrived, the
  // second step multiplies while stage s + 2 is fetched over stage s and the
  // first step's operands of stage s + 1 are read.
  uint64_t sv[NR];
  int sh;
  {
    const Source f = source(0);
#pragma unroll
    for (int j = 0; j < NL; ++j) fetch(f, 0, j);
    sh = fetch_scales(0, sv);
    put_scales(0, sv, sh);
    sh = fetch_scales(1, sv);
    put_scales(1, sv, sh);
    const Source g = source(1);
#pragma unroll
    for (int j = 0; j < NL; ++j) fetch(g, 1, j);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  Frag f0, f1;
  read_scales(f0, 0, 0);
#pragma unroll
  for (int e = 0; e < NG; ++e) read(f0, 0, 0, e);
  for (int s = 0; s < stages; ++s) {
    const int buf = s & 1;
    sh = fetch_scales(s + 2, sv);
    __builtin_amdgcn_sched_barrier(0);
    read_scales(f1, buf, 1);
#pragma unroll
    for (int e = 0; e < NG; ++e) {
      read(f1, buf, 1, e);
      products(f0, e);
      __builtin_amdgcn_sched_barrier(0);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NR; ++j) asm volatile("" : "+v"(sv[j]));  // they are here: the compiler's own wait belongs here
    const Source f = source(s + 2);
    __builtin_amdgcn_sched_barrier(0);
    read_scales(f0, buf ^ 1, 0);
#pragma unroll
    for (int e = 0; e < NG; ++e) {
#pragma unroll
      for (int j = e * NL / NG; j < (e + 1) * NL / NG; ++j) fetch(f, buf, j);
      read(f0, buf ^ 1, 0, e);
      products(f1, e);
      if (e == NG / 2) put_scales(buf, sv, sh);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  mm_settle();
  // D: outputs 4 lg .. + 3 of tile i, token lr of tile j
#pragma unroll
  for (int j = 0; j < TT; ++j) {
    const int64_t t = t0 + 16 * (TT * wt + j) + lr;
    if (t >= a.T) continue;
#pragma unroll
    for (int i = 0; i < TO; ++i) {
      const int64_t o = o0 + 16 * (TO * wo + i) + 4 * lg;
      const int64_t left = a.m - o;
      if (left > 0) mm_store4(a.y, a.yt, t * a.ldy + o, acc[i][j], left < 4 ? (int)left : 4, a.wide);
    }
  }
}

template <int WT, int WO, int TT, int TO>
hipError_t mm_tiles(MmArgs a, hipStream_t s) {
  constexpr int BT = 16 * TT * WT, BO = 16 * TO * WO;
  a.gt = (int)((a.T + BT - 1) / BT);
  a.go = (int)((a.m + BO - 1) / BO);
  const int64_t total = (int64_t)a.gt * a.go;
  a.per_xcd = (total + 7) / 8;
  a.band = 4;
  mm_tile_kernel<WT, WO, TT, TO><<<dim3((unsigned)(8 * a.per_xcd)), 64 * WT * WO, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_matmul(const MmArgs& a, hipStream_t s) {
  if (a.n >= kMmK && a.T > 16 && a.n <= (1 << 23)) {
    if (a.T > 512 && a.m > 512) return mm_tiles<2, 2, 8, 8>(a, s);
    return mm_tiles<2, 2, 4, 4>(a, s);
  }
  const dim3 grid((unsigned)((a.m + 15) / 16), (unsigned)((a.T + 15) / 16));
  mm_simple_kernel<<<grid, 64, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace brq
