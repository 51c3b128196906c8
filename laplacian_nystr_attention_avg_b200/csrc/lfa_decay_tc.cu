// Decay attention on bf16 tensors: the chunked run of lfa_decay.cu on tcgen05 tensor cores.
//
// A CTA takes one segment of one unit's tokens (one run: DecayJob) and walks its chunks of 128 tokens. Per chunk,
// with x, y, z tiles brought in by TMA and the carried state R [da][db] held in fp32 registers:
//   S  = x y^T                              (M 128 tokens, N 128 tokens, K da)
//   P  = c_intra l^(i-j) S, j <= i, in bf16   (P warps; the only rounding of the weights)
//   Oz = P z,  Ox = x bf16(R)               (M 128, N db; K 128 and K da)
//   O  = Oz + c_inter l^i Ox                (epilogue warps, fp32, rounded once)
//   D  = (y c_state l^(n-j))^T z            (M da, N db, K 128 tokens), R' = l^n R + D   (state warps)
// The decayed rows of y enter as bf16 parts (value and remainders, one product each): two parts (2^-17) where R
// only meets x, whose products are rounded to bf16 anyway, three (2^-25) where the run's state is returned. D
// starts from zero in every chunk and is added to R by CUDA cores: tensor-core accumulation truncates and would
// drift over thousands of chunks. All widths are padded to DP = 64 or 128 by TMA's zero fill.
//
// Warps: 4 for P, 4 for y's decayed rows, 8 for R and the epilogue, one thread each to issue TMA loads, the products
// of the state and those of the output. Every hand-over is an mbarrier; every wait is bounded (on expiry the device's status
// word is set, the CTA stops waiting for anything and drains what it has in flight).
//
// Few units over long sequences: segments run at once. k_decay_tc<.., true> sums up each segment's own
// state, k_decay_prefix carries them over the segments, and the main kernel starts every segment from its state.
#include <string.h>

#include "lfa_internal.h"
#include "lfa_sm100.cuh"
#include "lfa_tma_host.h"
#include "lfa_token.h"

namespace lfa {
namespace {

using namespace sm100;

__device__ int g_decay_status;   // sticky until decay_take_status reads it

constexpr int kC = kDecayChunk;
constexpr int kPanelB = kC * 128;   // bytes of a 128-token x 64-channel panel

struct TcJob {
  CUtensorMap x, y, z;
  __nv_bfloat16* O;
  long long os[3];
  const float* init;      // state before the run ([da][db], or [db][da] with trans), or null
  const float* seg_init;  // segs > 1: R at the start of each segment, [units][segs]
  float* fin;
  float* local;           // state kernel: sums of each segment, [units][segs]
  int da, db, rev, trans, init_decays, fin_sub;
  int wide;               // O's rows are whole, aligned 32-byte sectors
  int parts;              // bf16 parts of y's decayed rows: 3 where a state is returned, else 2
  float c_inter, c_intra, c_state;
};
struct TcArgs {
  TcJob job[3];
  const float* log_decay;
  const int* lengths;
  int heads, N, segs, seg_chunks;
};

template <int DP, bool STATE>
struct Cfg {
  static constexpr int kTile = DP / 64 * kPanelB;          // bytes of a token tile, one ring slot
  static constexpr int kPer = STATE ? 2 : 3;               // tiles of a chunk: y, [x], z
  static constexpr int kSlots = DP == 64 ? (STATE ? 8 : 9) : (STATE ? 5 : 4);
  // y's decayed rows are formed in steps of kStep tokens: four 16-byte vectors per thread
  static constexpr int kStep = 4096 / DP;
  static constexpr int kSteps = kC / kStep;
  static constexpr int kPart = kStep * DP * 2;             // bytes of one part of a step
  static constexpr int kOffPart = kSlots * kTile;          // 2 buffers of 3 parts
  static constexpr int kOffR = kOffPart + 6 * kPart;
  static constexpr int kOffBar = kOffR + (STATE ? 0 : DP * DP * 2);
  static constexpr int kOffPw = kOffBar + 320;
  static constexpr int kOffWt = kOffPw + 4 * (kC + 4 + 32 + kC + 32);
  static constexpr int kSmem = kOffWt + 16 * (kC + 1) + 1024;   // + alignment of the base to 1024
  static_assert(kSmem <= 232448, "shared memory over the sm_100 per-block limit");
  // warps: 4 for P (not STATE), 4 for y's decayed rows, 8 for the state and the epilogue, loads, products (two)
  static constexpr int kY0 = STATE ? 0 : 4;
  static constexpr int kR0 = kY0 + 4;
  static constexpr int kLoad = kR0 + 8;
  static constexpr int kMma = kLoad + 1;      // products of the state
  static constexpr int kMmaO = kMma + 1;      // products of the output (not STATE)
  static constexpr int kThreads = 32 * (STATE ? kMma + 1 : kMmaO + 1);
  // 608 threads have 96 registers each; with 64 of them R, the state warps take 24 more from the P warps (16 each)
  // and the y warps (32 each): 128 (80 + 64) + 256 120 + 96 96 = 608 96
  static constexpr bool kSplitRegs = DP == 128 && !STATE;
  // tensor memory columns; P (bf16 pairs) takes the first half of S's columns, row by row as S is read
  static constexpr int kTs = 0, kToz = STATE ? 0 : kC, kTox = kToz + (STATE ? 0 : DP), kTd = kTox + (STATE ? 0 : DP);
  static constexpr int kTmem = STATE ? DP : 512;
};
enum Bar {
  kFull = 0, kEmpty = 9, kSFull = 18, kPReady, kYdReady, kPartFree = kYdReady + 2, kDFull = kPartFree + 2, kDRead,
  kRbReady, kXDone, kOFull, kOFree, kZClean, kFin, kNumBars = kFin + 2
};
static_assert(kNumBars * 8 <= 304, "barriers overlap the TMEM slot");

struct Waiter {
  uint64_t* bars;
  volatile int* gave_up;
  __device__ __forceinline__ void operator()(int bar, uint32_t phase) const {
    if (mbar_try_wait(bars + bar, phase & 1)) return;
    const long long t0 = clock64();
    while (!mbar_try_wait_ns(bars + bar, phase & 1, 2000)) {
      if (*gave_up) return;
      if (clock64() - t0 > kSpinBudget) {
        *gave_up = 1;
        atomicOr(&g_decay_status, 1);
        return;
      }
    }
  }
  // for what is in flight at the end: not cut short by gave_up
  __device__ __forceinline__ void drain(int bar, uint32_t phase) const {
    const long long t0 = clock64();
    while (!mbar_try_wait(bars + bar, phase & 1))
      if (clock64() - t0 > kSpinBudget) {
        atomicOr(&g_decay_status, 1);
        return;
      }
  }
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
// y w for a pair y of bf16 and w = w.x + w.y + w.z in bf16 parts, as a + b + c in bf16: a = y w.x rounded, its
// remainder y w.x - a is a bf16 itself (8 by 8 bits make 16), and so on down; about 2^-25 of y w is left out
__device__ __forceinline__ __nv_bfloat162 as_b2(uint32_t v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); }
__device__ __forceinline__ uint32_t as_u(__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t*>(&v); }
template <bool THIRD>
__device__ __forceinline__ void split3(uint32_t y, const uint4& w, uint32_t& a, uint32_t& b, uint32_t& c) {
  const __nv_bfloat162 y2 = as_b2(y), wx = as_b2(w.x), wy = as_b2(w.y), wz = as_b2(w.z);
  const __nv_bfloat162 hi = __hmul2(y2, wx), rem = __hfma2(y2, wx, __hneg2(hi));
  const __nv_bfloat162 mid = __hfma2(y2, wy, rem);
  a = as_u(hi);
  b = as_u(mid);
  if (THIRD) c = as_u(__hfma2(y2, wz, __hfma2(y2, wy, __hsub2(rem, mid))));
}
// four vectors of a thread, RS rows apart (a multiple of 8: the same place in the swizzle), each part PART bytes on
template <bool THIRD, int RS, int PART>
__device__ __forceinline__ void split_rows(const uint4 (&v)[4], const uint4 (&w)[4], unsigned char* d) {
  uint4 o[4][3];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    split3<THIRD>(v[e].x, w[e], o[e][0].x, o[e][1].x, o[e][2].x);
    split3<THIRD>(v[e].y, w[e], o[e][0].y, o[e][1].y, o[e][2].y);
    split3<THIRD>(v[e].z, w[e], o[e][0].z, o[e][1].z, o[e][2].z);
    split3<THIRD>(v[e].w, w[e], o[e][0].w, o[e][1].w, o[e][2].w);
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
#pragma unroll
    for (int p = 0; p < (THIRD ? 3 : 2); ++p) *reinterpret_cast<uint4*>(d + e * RS * 128 + p * PART) = o[e][p];
}

// one 32-byte store (a whole sector)
__device__ __forceinline__ void st_global_32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ uint32_t packf2(uint64_t v) { return pack2(f2_lo(v), f2_hi(v)); }
__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }

// The P warps of a run of n chunks: P = c_intra l^|i-j| S on the causal side, in bf16, over S's own columns
// (thread = token row i; block cb of S's columns is read before P's block cb goes over columns read earlier).
// l^|i-j| is l^(distance of i to the block) pb[c] beside the diagonal block. nv0: valid tokens of the first chunk,
// where a reverse run finds its sequence's ragged end (forwards, columns behind the end are above the diagonal).
template <bool REV>
__device__ __forceinline__ void weights(int n, const Waiter& wait, uint64_t* bars, uint32_t ts, const float* pw,
                                        const float* pb, int nv0) {
  const int lane = threadIdx.x & 31, q = (threadIdx.x >> 5) & 3, i = 32 * q + lane;
  const uint32_t srow = ts + ((uint32_t)(32 * q) << 16);
  const float* pd = pw + (REV ? -lane : lane);   // pw is zero for 31 exponents below 0
  for (int k = 0; k < n; ++k) {
    wait(kSFull, k);
    tc_fence_after();
#pragma unroll 1
    for (int cb = 0; cb < 4; ++cb) {
      uint32_t w[16];
      if (REV ? cb >= q : cb <= q) {
        uint32_t v[32];
        tmem_ld32_async(srow + 32 * cb, v);
        if (cb == q) {
          float p[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) p[c] = pd[REV ? c : -c];
          tmem_wait_ld(v);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float x = __uint_as_float(v[c]) * p[c];
            v[c] = (REV ? c >= lane : c <= lane) ? __float_as_uint(x) : 0u;
          }
        } else {
          const float f = pw[REV ? 32 * cb - i : i - 32 * cb - 31];
          const uint64_t ff = f2(f, f);
          tmem_wait_ld(v);
#pragma unroll
          for (int c = 0; c < 32; c += 4) {
            const ulonglong2 p = *reinterpret_cast<const ulonglong2*>(pb + c);
            const uint64_t x = mul2(f2(v[c], v[c + 1]), mul2(ff, p.x)), y = mul2(f2(v[c + 2], v[c + 3]), mul2(ff, p.y));
            v[c] = (uint32_t)x;
            v[c + 1] = (uint32_t)(x >> 32);
            v[c + 2] = (uint32_t)y;
            v[c + 3] = (uint32_t)(y >> 32);
          }
        }
        if (REV && k == 0 && nv0 < 32 * cb + 32) {   // columns of tokens behind the end may hold anything
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (32 * cb + c >= nv0) v[c] = 0;
        }
#pragma unroll
        for (int c = 0; c < 16; ++c) w[c] = pack2(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1]));
      } else {   // the other side of the diagonal
#pragma unroll
        for (int c = 0; c < 16; ++c) w[c] = 0;
      }
      tmem_st16(srow + 16 * cb, w);
    }
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + kPReady);
  }
}

template <int DP, bool STATE>
__global__ void __launch_bounds__(Cfg<DP, STATE>::kThreads, 1) k_decay_tc(const __grid_constant__ TcArgs a) {
  using C = Cfg<DP, STATE>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  const TcJob& jb = a.job[blockIdx.z];
  const int u = blockIdx.x, seg = blockIdx.y, b = u / a.heads, h = u % a.heads;
  const int L = unit_length(a.lengths, b, a.N), nch = (L + kC - 1) / kC;
  const int c_lo = seg * a.seg_chunks, c_hi = min(c_lo + a.seg_chunks, nch), n = c_hi - c_lo;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int da = jb.da, db = jb.db;
  const bool rev = jb.rev;
  const size_t dd = (size_t)da * db;
  if (n <= 0) {
    if (!STATE && L == 0 && seg == 0 && jb.fin)
      for (size_t e = t; e < dd; e += C::kThreads) jb.fin[u * dd + e] = jb.init ? jb.init[u * dd + e] : 0.f;
    return;
  }
  if (STATE && (rev ? seg == 0 : c_hi == nch)) return;   // nothing follows this segment
  const bool ends = !STATE && jb.fin && (rev ? seg == 0 : c_hi == nch);

  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::kOffBar + 304);
  volatile int* gave_up = reinterpret_cast<volatile int*>(sm + C::kOffBar + 308);
  float* pw = reinterpret_cast<float*>(sm + C::kOffPw);   // l^0 .. l^128
  float* pb = pw + kC + 4;                                 // rev: l^c, else l^(31-c), c = 0 .. 31
  float* pi = pb + 32 + 32;                                // c_intra l^0 .. c_intra l^127 after 32 zeros
  uint4* wt = reinterpret_cast<uint4*>(sm + C::kOffWt);   // c_state l^n as three bf16 parts, each twice in a word
  const float ld = decay_log(a.log_decay[h]);
  const Waiter wait{bars, gave_up};
  if (t == 0) {
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(bars + i, i >= kEmpty && i < kSFull                                            ? (STATE ? 1 : 2)
                          : i == kPReady || (i >= kYdReady && i < kPartFree) || i == kZClean ? 4
                          : i == kDRead || i == kRbReady || i == kOFree                      ? 8
                                                                                             : 1);
    mbar_init_fence();
    *gave_up = 0;
  }
  if (warp == C::kMma) tmem_alloc(tmem_slot, C::kTmem);
  for (int i = t; i <= kC; i += C::kThreads) {
    const float w = expf(ld * i);
    pw[i] = w;
    if (i < 32) {
      pb[rev ? i : 31 - i] = w;
      pi[i - 32] = 0.f;
    }
    if (i < kC) pi[i] = jb.c_intra * w;
    const float f = jb.c_state * w, f1 = f - bf_lo(pack2(f, f)), f2 = f1 - bf_lo(pack2(f1, f1));
    wt[i] = make_uint4(pack2(f, f), pack2(f1, f1), pack2(f2, f2), 0u);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // chunk of step k, and its valid tokens
  auto chunk = [&](int k) { return rev ? c_hi - 1 - k : c_lo + k; };
  auto valid = [&](int c) { return min(kC, L - c * kC); };

  if (warp == C::kLoad) {
    if (lane == 0) {
      const int total = n * C::kPer;
      int g = 0;
      for (; g < total; ++g) {   // y, [x], z of every chunk in turn, one ring slot each
        const int s = g % C::kSlots, w = g % C::kPer;
        if (g >= C::kSlots) wait(kEmpty + s, g / C::kSlots - 1);
        if (*gave_up) break;
        const CUtensorMap* m = w == 0 ? &jb.y : w == C::kPer - 1 ? &jb.z : &jb.x;
        mbar_expect_tx(bars + kFull + s, C::kTile);
        for (int p = 0; p < DP / 64; ++p)
          tma_load_4d(sm + s * C::kTile + p * kPanelB, m, 64 * p, chunk(g / C::kPer) * kC, h, b, bars + kFull + s);
      }
      for (int i = max(0, g - C::kSlots); i < g; ++i) wait.drain(kFull + i % C::kSlots, i / C::kSlots);
    }
  } else if (!STATE && warp == C::kMmaO) {
    if (lane == 0) {
      // S, Ox, Oz of every chunk in turn. Descriptors of the ring's first slot and R; b bytes further is + b / 16
      const uint32_t base = smem_u32(sm);
      const uint64_t d_k = desc_sw128(base, 16, 1024), d_mn = desc_sw128(base, kPanelB, 1024),
                     d_rb = desc_sw128(base + C::kOffR, DP * 128, 1024);
      constexpr uint32_t id_s = idesc(1, kC, kC, 0, 0), id_o = idesc(1, kC, DP, 0, 1);
      for (int k = 0; k < n; ++k) {
        const int gy = k * C::kPer, gx = gy + 1, gz = gy + C::kPer - 1;
        const int sy = gy % C::kSlots, sx = gx % C::kSlots, sz = gz % C::kSlots;
        const uint64_t y = d_k + sy * (C::kTile / 16), x = d_k + sx * (C::kTile / 16), z = d_mn + sz * (C::kTile / 16);
        wait(kFull + sy, gy / C::kSlots);
        wait(kFull + sx, gx / C::kSlots);
        if (k > 0) wait(kOFull, k - 1);   // P of the chunk before has been used
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk) {
          const int off = ((kk >> 2) * kPanelB + (kk & 3) * 32) / 16;
          mma_bf16(tmem + C::kTs, x + off, y + off, id_s, kk > 0);
        }
        mma_commit(bars + kSFull);
        mma_commit(bars + kEmpty + sy);
        wait(kRbReady, k);
        if (k > 0) wait(kOFree, k - 1);
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk)
          mma_bf16(tmem + C::kTox, x + ((kk >> 2) * kPanelB + (kk & 3) * 32) / 16, d_rb + kk * 128, id_o, kk > 0);
        mma_commit(bars + kXDone);
        mma_commit(bars + kEmpty + sx);
        mma_commit(bars + kEmpty + sx);
        wait(kFull + sz, gz / C::kSlots);
        if (valid(chunk(k)) < kC) wait(kZClean, 0);
        wait(kPReady, k);
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kC / 16; ++kk)
          mma_bf16_ta(tmem + C::kToz, tmem + C::kTs + 8 * kk, z + kk * 128, id_o, kk > 0);
        mma_commit(bars + kOFull);
        mma_commit(bars + kEmpty + sz);
      }
      mma_commit(bars + kFin);
      wait.drain(kFin, 0);
    }
  } else if (warp == C::kMma) {
    if (lane == 0) {
      // D of every chunk: its own thread, so that the state runs ahead of the outputs
      const uint32_t base = smem_u32(sm);
      const uint64_t d_mn = desc_sw128(base, kPanelB, 1024), d_part = desc_sw128(base + C::kOffPart, C::kStep * 128, 1024);
      constexpr uint32_t id_d = idesc(1, DP, DP, 1, 1);
      const bool third = jb.parts == 3;
      for (int k = 0; k < n; ++k) {
        const int gy = k * C::kPer, gz = gy + C::kPer - 1, sy = gy % C::kSlots, sz = gz % C::kSlots;
        const uint64_t z = d_mn + sz * (C::kTile / 16);
        const bool carry = STATE || ends || k < n - 1;
        wait(kFull + sz, gz / C::kSlots);
        if (k > 0) wait(kDRead, k - 1);
#pragma unroll 1
        for (int s = 0; s < C::kSteps; ++s) {
          const int g = k * C::kSteps + s, buf = g & 1;
          wait(kYdReady + buf, g >> 1);
          tc_fence_after();
          if (carry) {
#pragma unroll
            for (int p = 0; p < 3; ++p)
              if (p < 2 || third) {
#pragma unroll
                for (int kk = 0; kk < C::kStep / 16; ++kk)
                  mma_bf16(tmem + C::kTd, d_part + (3 * buf + p) * (C::kPart / 16) + kk * 128,
                           z + (s * C::kStep + 16 * kk) * 8, id_d, s + p + kk > 0);
              }
          }
          mma_commit(bars + kPartFree + buf);
        }
        if (carry) mma_commit(bars + kDFull);
        mma_commit(bars + kEmpty + sy);
        mma_commit(bars + kEmpty + sz);
      }
      mma_commit(bars + kFin + 1);
      wait.drain(kFin + 1, 0);
    }
  } else if (!STATE && warp < C::kY0) {
    if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (rev)
      weights<true>(n, wait, bars, tmem + C::kTs, pi, pb, L - (c_hi - 1) * kC);
    else
      weights<false>(n, wait, bars, tmem + C::kTs, pi, pb, kC);
  } else if (warp < C::kR0) {
    // y's decayed rows, in steps of kStep tokens into one of two buffers
    if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    const int ty = t - 32 * C::kY0;
    constexpr int CH = DP / 8, RS = 128 / CH;   // 16-byte vectors of a row, rows per pass
    const int ch = ty % CH, rr = ty / CH;
    const bool third = jb.parts == 3;
    for (int k = 0; k < n; ++k) {
      const int c = chunk(k), nv = valid(c), sub = (!STATE && c == nch - 1) ? jb.fin_sub : 0;
      const int gy = k * C::kPer, gz = gy + C::kPer - 1;
      const unsigned char* y = sm + (gy % C::kSlots) * C::kTile + (ch >> 3) * kPanelB;
      unsigned char* z = sm + (gz % C::kSlots) * C::kTile + (ch >> 3) * kPanelB;
      const uint4* w0 = wt + (rev ? 1 : nv) - sub;   // row r has weight w0[r] (rev) or w0[-r]
      wait(kFull + gy % C::kSlots, gy / C::kSlots);
      if (nv < kC) wait(kFull + gz % C::kSlots, gz / C::kSlots);
#pragma unroll 1
      for (int st = 0; st < C::kSteps; ++st) {
        const int g = k * C::kSteps + st, buf = g & 1;
        uint4 v[4], w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = st * C::kStep + rr + e * RS;
          v[e] = *reinterpret_cast<const uint4*>(y + sw128(r, ch & 7));
          w[e] = w0[r < nv ? (rev ? r : -r) : 0];
        }
        if (nv < kC) {   // rows behind the sequence's end may hold anything
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = st * C::kStep + rr + e * RS;
            if (r >= nv) {
              v[e] = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(z + sw128(r, ch & 7)) = v[e];
            }
          }
        }
        if (g >= 2) wait(kPartFree + buf, (g >> 1) - 1);
        unsigned char* d = sm + C::kOffPart + 3 * buf * C::kPart + (ch >> 3) * (C::kStep * 128) + sw128(rr, ch & 7);
        if (third)
          split_rows<true, RS, C::kPart>(v, w, d);
        else
          split_rows<false, RS, C::kPart>(v, w, d);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + kYdReady + buf);
      }
      if (!STATE && nv < kC && lane == 0) mbar_arrive(bars + kZClean);
    }
  } else if (warp < C::kLoad) {
    if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 120;");
    // state and epilogue: R row and half of its columns per thread (DP 64: M = 64 puts row 16 q + lane in
    // lane < 16); in the epilogue thread = token row, the same half of O's columns
    constexpr int NR = DP / 2;
    const int q = warp & 3, half = (warp - C::kR0) >> 2, i = 32 * q + lane;
    const bool live = DP == 128 || lane < 16, trans = jb.trans;
    const int row = DP == 128 ? i : 16 * q + lane, col = half * NR;
    const uint32_t quad = tmem + ((uint32_t)(32 * q) << 16) + col;
    uint64_t R[NR / 2];   // pairs of columns
    {
      const float* src = STATE ? nullptr : a.segs > 1 ? jb.seg_init : jb.init;
      const float f0 = (a.segs > 1 || !jb.init_decays) ? 1.f : expf(ld);
      const size_t at = (a.segs > 1 ? (size_t)u * a.segs + seg : (size_t)u) * dd;
#pragma unroll
      for (int c = 0; c < NR; c += 2) {   // da and db are even
        float r0 = 0.f, r1 = 0.f;
        if (src && live && row < da && col + c < db) {
          r0 = f0 * src[at + (trans ? (size_t)(col + c) * da + row : (size_t)row * db + col + c)];
          r1 = f0 * src[at + (trans ? (size_t)(col + c + 1) * da + row : (size_t)row * db + col + c + 1)];
        }
        R[c / 2] = f2(r0, r1);
      }
    }
    auto update = [&](int k) {   // R after the chunk of step k
      const int c = chunk(k);
      const Decay dec(ld * (valid(c) - (!STATE && c == nch - 1 ? jb.fin_sub : 0)));
      const uint64_t em = f2(dec.em, dec.em), mu = f2(dec.mul, dec.mul);
      wait(kDFull, k);
      tc_fence_after();
#pragma unroll
      for (int c0 = 0; c0 < NR; c0 += 16) {
        uint32_t d[16];
        tmem_ld16_async(quad + C::kTd + c0, d);
        tmem_wait_ld16(d);
        if (c0 + 16 == NR) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars + kDRead);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint64_t r = R[c0 / 2 + e];
          R[c0 / 2 + e] = add2(fma2(em, r, mul2(mu, r)), f2(d[2 * e], d[2 * e + 1]));
        }
      }
    };
    const long long ts = jb.os[2];
    __nv_bfloat16* O = STATE ? nullptr : jb.O + b * jb.os[0] + h * jb.os[1] + col;
    const bool wide = jb.wide;
    const float c_inter = jb.c_inter;
    auto epilogue = [&](int k) {
      const int c = chunk(k), nv = valid(c), e = rev ? nv - 1 - i : i;
      const float f = e >= 0 ? c_inter * pw[e] : 0.f;
      const uint64_t ff = f2(f, f);
      wait(kOFull, k);
      tc_fence_after();
      __nv_bfloat16* o = O + (long long)(c * kC + i) * ts;
#pragma unroll 1
      for (int c0 = 0; c0 < NR; c0 += 16) {
        uint32_t z[16], x[16];
        tmem_ld16_async(quad + C::kToz + c0, z);
        tmem_ld16_async(quad + C::kTox + c0, x);
        tmem_wait_ld16(z);
        tmem_wait_ld16(x);
        if (c0 + 16 == NR) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars + kOFree);
        }
        uint32_t w[8];
#pragma unroll
        for (int g = 0; g < 8; ++g)
          w[g] = packf2(fma2(ff, f2(x[2 * g], x[2 * g + 1]), f2(z[2 * g], z[2 * g + 1])));
        if (i < nv) {
          const int left = db - col - c0;
          if (wide && left > 0) {
            st_global_32(o + c0, w);
          } else {
            if (left > 0) *reinterpret_cast<uint4*>(o + c0) = make_uint4(w[0], w[1], w[2], w[3]);
            if (left > 8) *reinterpret_cast<uint4*>(o + c0 + 8) = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
      }
    };
    for (int k = 0; k < n; ++k) {
      if (k > 0) update(k - 1);
      if (!STATE) {
        if (k > 0) wait(kXDone, k - 1);
        if (live) {
#pragma unroll
          for (int g = 0; g < NR; g += 8) {
            const int cc = col + g;
            *reinterpret_cast<uint4*>(sm + C::kOffR + (cc >> 6) * (DP * 128) + sw128(row, (cc & 63) >> 3)) =
                make_uint4(packf2(R[g / 2]), packf2(R[g / 2 + 1]), packf2(R[g / 2 + 2]), packf2(R[g / 2 + 3]));
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + kRbReady);
        if (k > 0) epilogue(k - 1);
      }
    }
    if (!STATE) epilogue(n - 1);
    if (STATE || ends) {
      update(n - 1);
      float* dst = STATE ? jb.local + ((size_t)u * a.segs + seg) * dd : jb.fin + u * dd;
      if (live && row < da) {
#pragma unroll
        for (int c = 0; c < NR; c += 2)
          if (col + c < db) {
            dst[!STATE && trans ? (size_t)(col + c) * da + row : (size_t)row * db + col + c] = f2_lo(R[c / 2]);
            dst[!STATE && trans ? (size_t)(col + c + 1) * da + row : (size_t)row * db + col + c + 1] = f2_hi(R[c / 2]);
          }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == C::kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmem);
    tmem_relinquish();
  }
}

// States before each segment from the segments' own sums, in place: st [jobs][units][segs][dd].
struct PrefixArgs {
  float* st;
  const float* init[2];   // state before the run (the forward's S0, the reverse run's dS_out), or null
  int rev[2], init_decays[2];
  const float* log_decay;
  const int* lengths;
  int heads, N, segs, seg_chunks, dd;
};
__global__ void __launch_bounds__(256) k_decay_prefix(const __grid_constant__ PrefixArgs a) {
  const int u = blockIdx.x, j = blockIdx.z, e = (blockIdx.y * 256 + threadIdx.x) * 4;
  if (e >= a.dd) return;
  const int L = unit_length(a.lengths, u / a.heads, a.N), nch = (L + kC - 1) / kC;
  const int segs = (nch + a.seg_chunks - 1) / a.seg_chunks, span = a.seg_chunks * kC;
  if (segs == 0) return;
  const float ld = decay_log(a.log_decay[u % a.heads]);
  float* st = a.st + ((size_t)j * gridDim.x + u) * a.segs * a.dd + e;
  float4 r = make_float4(0, 0, 0, 0);
  if (a.init[j]) {
    const float f = a.init_decays[j] ? expf(ld) : 1.f;
    r = *reinterpret_cast<const float4*>(a.init[j] + (size_t)u * a.dd + e);
    r.x *= f; r.y *= f; r.z *= f; r.w *= f;
  }
  for (int i = 0; i < segs; ++i) {
    const int p = a.rev[j] ? segs - 1 - i : i;
    float4* at = reinterpret_cast<float4*>(st + (size_t)p * a.dd);
    const bool more = i + 1 < segs;
    const float4 own = more ? *at : r;
    *at = r;
    if (more) {
      const Decay dec(ld * min(span, L - p * span));
      r.x = dec(r.x) + own.x;
      r.y = dec(r.y) + own.y;
      r.z = dec(r.z) + own.z;
      r.w = dec(r.w) + own.w;
    }
  }
}

bool maps(TcJob* t, const DecayArgs& a, const DecayJob& j, bool with_x) {
  if (with_x && !make_tmap_tokens_bf16(&t->x, j.X, j.da, a.N, a.heads, a.B, j.xs, kC)) return false;
  return make_tmap_tokens_bf16(&t->y, j.Y, j.da, a.N, a.heads, a.B, j.ys, kC) &&
         make_tmap_tokens_bf16(&t->z, j.Z, j.db, a.N, a.heads, a.B, j.zs, kC);
}

template <int DP, bool STATE>
cudaError_t run(const TcArgs& a, int units, int njobs, cudaStream_t st) {
  using C = Cfg<DP, STATE>;
  cudaError_t e = cudaFuncSetAttribute(k_decay_tc<DP, STATE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  k_decay_tc<DP, STATE><<<dim3(units, a.segs, njobs), C::kThreads, C::kSmem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

// One CTA fills an SM. With fewer than 148 of them the sequences are cut so that about 148 run at once, in
// segments of at least 4 chunks (below that the extra launches and the second reading of y and z cost more).
DecaySplit decay_split(int B, int heads, int N, int njobs, int dtype) {
  const int nch = ceil_div(N, kC);
  const long long ctas = (long long)B * heads * njobs;
  int segs = dtype == LFA_BF16 && ctas < 148 ? (int)(148 / ctas) : 1;
  if (segs > nch / 4) segs = nch / 4;
  if (segs < 1) segs = 1;
  DecaySplit s;
  s.seg_chunks = ceil_div(nch, segs);
  s.segs = ceil_div(nch, s.seg_chunks);
  return s;
}

size_t decay_workspace_floats(int B, int heads, int N, int dk, int dv, int njobs, int dtype) {
  const DecaySplit s = decay_split(B, heads, N, njobs, dtype);
  return s.segs > 1 ? (size_t)(njobs > 1 ? 2 : 1) * B * heads * s.segs * dk * dv : 0;
}

cudaError_t decay_take_status(int* out, cudaStream_t st) {
  void* p = nullptr;
  cudaError_t e = cudaGetSymbolAddress(&p, g_decay_status);
  if (e == cudaSuccess) e = cudaMemcpyAsync(out, p, sizeof(int), cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && *out) {
    e = cudaMemsetAsync(p, 0, sizeof(int), st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  return e;
}

cudaError_t launch_decay_tc(const DecayArgs& a, cudaStream_t st) {
  const DecaySplit sp = decay_split(a.B, a.heads, a.N, a.njobs, LFA_BF16);
  const int units = a.B * a.heads;
  TcArgs t;
  memset(&t, 0, sizeof(t));
  t.log_decay = a.log_decay;
  t.lengths = a.lengths;
  t.heads = a.heads;
  t.N = a.N;
  t.segs = sp.segs;
  t.seg_chunks = sp.seg_chunks;
  int dp = 64;
  for (int i = 0; i < a.njobs; ++i) {
    const DecayJob& j = a.job[i];
    if (j.da > 64 || j.db > 64) dp = 128;
  }
  const int dd = a.job[0].da * a.job[0].db;
  // states before the segments: run 0 forwards, and for the backward its last run (y = q, z = dO)
  const size_t states = (size_t)units * sp.segs * dd;
  if (sp.segs > 1) {
    const int ns = a.njobs > 1 ? 2 : 1;
    PrefixArgs p;
    memset(&p, 0, sizeof(p));
    p.st = a.ws;
    for (int i = 0; i < ns; ++i) {
      // the state as [dk][dv]: forwards y = k, z = v (the backward's run 0 has it transposed)
      DecayJob j = a.job[i == 0 ? 0 : 2];
      if (j.trans) {
        DecayJob s = j;
        s.Y = j.Z; s.Z = j.Y;
        memcpy(s.ys, j.zs, sizeof(s.ys));
        memcpy(s.zs, j.ys, sizeof(s.zs));
        s.da = j.db; s.db = j.da;
        j = s;
      }
      TcJob& o = t.job[i];
      if (!maps(&o, a, j, false)) return cudaErrorInvalidValue;
      o.da = j.da;
      o.db = j.db;
      o.rev = j.rev;
      o.c_state = j.c_state;
      o.local = a.ws + i * states;
      o.parts = j.fin ? 3 : 2;
      p.init[i] = j.init;
      p.rev[i] = j.rev;
      p.init_decays[i] = j.init_decays;
    }
    const cudaError_t e = dp == 64 ? run<64, true>(t, units, ns, st) : run<128, true>(t, units, ns, st);
    if (e != cudaSuccess) return e;
    p.log_decay = a.log_decay;
    p.lengths = a.lengths;
    p.heads = a.heads;
    p.N = a.N;
    p.segs = sp.segs;
    p.seg_chunks = sp.seg_chunks;
    p.dd = dd;
    k_decay_prefix<<<dim3(units, ceil_div(dd, 1024), ns), 256, 0, st>>>(p);
    const cudaError_t e2 = cudaGetLastError();
    if (e2 != cudaSuccess) return e2;
  }
  for (int i = 0; i < a.njobs; ++i) {
    const DecayJob& j = a.job[i];
    TcJob& o = t.job[i];
    if (!maps(&o, a, j, true)) return cudaErrorInvalidValue;
    o.O = static_cast<__nv_bfloat16*>(j.O);
    memcpy(o.os, j.os, sizeof(o.os));
    o.init = j.init;
    o.seg_init = a.ws + (i == 0 ? 0 : states);
    o.fin = j.fin;
    o.wide = j.db % 16 == 0 && (reinterpret_cast<uintptr_t>(j.O) & 31u) == 0 && (j.os[0] | j.os[1] | j.os[2]) % 16 == 0;
    o.da = j.da;
    o.db = j.db;
    o.rev = j.rev;
    o.trans = j.trans;
    o.init_decays = j.init_decays;
    o.fin_sub = j.fin_sub;
    o.parts = j.fin ? 3 : 2;
    o.c_inter = j.c_inter;
    o.c_intra = j.c_intra;
    o.c_state = j.c_state;
  }
  return dp == 64 ? run<64, false>(t, units, a.njobs, st) : run<128, false>(t, units, a.njobs, st);
}

}  // namespace lfa
