// Decay attention on bf16 tensors: the chunked run of lfa_decay.cu on tcgen05 tensor cores.
//
// A CTA takes one segment of one unit's tokens (one run: DecayJob) and walks its chunks of 128 tokens. Per chunk,
// with x, y, z tiles brought in by TMA and the carried state R [da][db] held in fp32 registers:
//   S  = x y^T                              (M 128 tokens, N 128 tokens, K da)
//   P  = c_intra l^(i-j) S, j <= i, in bf16   (P warps; the only rounding of the weights)
//   Oz = P z,  Ox = x bf16(R)               (M 128, N db; K 128 and K da)
//   O  = Oz + c_inter l^i Ox                (epilogue warps, fp32, rounded once)
//   D  = (y c_state l^(n-j))^T z            (M da, N db, K 128 tokens), R' = l^n R + D   (state warps)
// The decayed rows of y enter as three bf16 parts (value and remainders, three products), which hold all 24 bits
// of them; D starts from zero in every chunk and is added to R by CUDA cores, since tensor-core accumulation
// truncates and would drift over thousands of chunks. All widths are padded to DP = 64 or 128 by TMA's zero fill.
//
// Warps: 4 for P, 8 for the state (thread = one row of R, half the columns), 4 for the epilogue, one thread each
// to issue TMA loads and tensor-core products. Every hand-over is an mbarrier; every wait is bounded (on expiry
// the device's status word is set, the CTA stops waiting for anything and drains what it has in flight).
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
  static constexpr int kSlots = DP == 64 ? (STATE ? 6 : 12) : (STATE ? 6 : 5);
  // y's decayed rows are formed in steps of kStep tokens, one 16-byte vector per state thread and part
  static constexpr int kStep = 2048 / DP;
  static constexpr int kSteps = kC / kStep;
  static constexpr int kPart = kStep * DP * 2;             // bytes of one part of a step
  static constexpr int kOffPart = kSlots * kTile;          // 2 buffers of 3 parts
  static constexpr int kOffR = kOffPart + 6 * kPart;
  static constexpr int kOffBar = kOffR + (STATE ? 0 : DP * DP * 2);
  static constexpr int kOffPw = kOffBar + 320;
  static constexpr int kSmem = kOffPw + 4 * (kC + 4) + 1024;   // + alignment of the base to 1024
  static_assert(kSmem <= 232448, "shared memory over the sm_100 per-block limit");
  // warps
  static constexpr int kS0 = STATE ? 0 : 4;   // state warps (the P warps come before them)
  static constexpr int kE0 = kS0 + 8;
  static constexpr int kLoad = STATE ? 8 : 16;
  static constexpr int kMma = kLoad + 1;
  static constexpr int kThreads = 32 * (kMma + 1);
  // tensor memory columns; P (bf16 pairs) takes the first half of S's columns, row by row as S is read
  static constexpr int kTs = 0, kToz = STATE ? 0 : kC, kTox = kToz + (STATE ? 0 : DP), kTd = kTox + (STATE ? 0 : DP);
  static constexpr int kTmem = STATE ? DP : 512;
};
enum Bar {
  kFull = 0, kEmpty = 12, kSFull = 24, kPReady, kKdReady, kPartFree = kKdReady + 2, kDFull = kPartFree + 2, kRbReady,
  kXDone, kOFull, kOFree, kFin, kNumBars
};
static_assert(kNumBars * 8 <= 304, "barriers overlap the TMEM slot");

struct Waiter {
  uint64_t* bars;
  volatile int* gave_up;
  __device__ __forceinline__ void operator()(int bar, uint32_t phase) const {
    if (mbar_try_wait(bars + bar, phase & 1)) return;
    const long long t0 = clock64();
    while (!mbar_try_wait(bars + bar, phase & 1)) {
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
// one 32-byte store (a whole sector)
__device__ __forceinline__ void st_global_32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

template <int DP, bool STATE>
__global__ void __launch_bounds__(Cfg<DP, STATE>::kThreads, 1) k_decay_tc(const __grid_constant__ TcArgs a) {
  using C = Cfg<DP, STATE>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  const TcJob& jb = a.job[blockIdx.z];
  const int u = blockIdx.x, seg = blockIdx.y, b = u / a.heads, h = u % a.heads;
  const int L = unit_length(a.lengths, b, a.N), nch = (L + kC - 1) / kC;
  const int c_lo = seg * a.seg_chunks, c_hi = min(c_lo + a.seg_chunks, nch), n = c_hi - c_lo;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const size_t dd = (size_t)jb.da * jb.db;
  if (n <= 0) {
    if (!STATE && L == 0 && seg == 0 && jb.fin)
      for (size_t e = t; e < dd; e += C::kThreads) jb.fin[u * dd + e] = jb.init ? jb.init[u * dd + e] : 0.f;
    return;
  }
  if (STATE && (jb.rev ? seg == 0 : c_hi == nch)) return;   // nothing follows this segment
  const bool ends = !STATE && jb.fin && (jb.rev ? seg == 0 : c_hi == nch);

  unsigned char* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::kOffBar + 304);
  volatile int* gave_up = reinterpret_cast<volatile int*>(sm + C::kOffBar + 308);
  float* pw = reinterpret_cast<float*>(sm + C::kOffPw);   // l^0 .. l^128
  const float ld = decay_log(a.log_decay[h]);
  const Waiter wait{bars, gave_up};
  if (t == 0) {
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(bars + i, i == kPReady || i == kOFree ? 4 : (i >= kKdReady && i < kPartFree) || i == kRbReady ? 8 : 1);
    mbar_init_fence();
    *gave_up = 0;
  }
  if (warp == C::kMma) tmem_alloc(tmem_slot, C::kTmem);
  for (int i = t; i <= kC; i += C::kThreads) pw[i] = expf(ld * i);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // chunk of step k, and its valid tokens
  auto chunk = [&](int k) { return jb.rev ? c_hi - 1 - k : c_lo + k; };
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
  } else if (warp == C::kMma) {
    if (lane == 0) {
      const uint32_t base = smem_u32(sm), parts = base + C::kOffPart, rb = base + C::kOffR;
      constexpr uint32_t id_s = idesc(1, kC, kC, 0, 0), id_o = idesc(1, kC, DP, 0, 1), id_d = idesc(1, DP, DP, 1, 1);
      for (int k = 0; k < n; ++k) {
        const int gy = k * C::kPer, gx = gy + 1, gz = gy + C::kPer - 1;
        const int sy = gy % C::kSlots, sx = gx % C::kSlots, sz = gz % C::kSlots;
        const uint32_t y = base + sy * C::kTile, x = base + sx * C::kTile, z = base + sz * C::kTile;
        const bool carry = STATE || ends || k < n - 1;
        if (!STATE) {
          wait(kFull + sy, gy / C::kSlots);
          wait(kFull + sx, gx / C::kSlots);
          if (k > 0) wait(kOFull, k - 1);   // P of the chunk before has been used
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < DP / 16; ++kk) {
            const uint32_t off = (kk >> 2) * kPanelB + (kk & 3) * 32;
            mma_bf16(tmem + C::kTs, desc_sw128(x + off, 16, 1024), desc_sw128(y + off, 16, 1024), id_s, kk > 0);
          }
          mma_commit(bars + kSFull);
          wait(kRbReady, k);
          if (k > 0) wait(kOFree, k - 1);
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < DP / 16; ++kk)
            mma_bf16(tmem + C::kTox, desc_sw128(x + (kk >> 2) * kPanelB + (kk & 3) * 32, 16, 1024),
                     desc_sw128(rb + kk * 2048, DP * 128, 1024), id_o, kk > 0);
          mma_commit(bars + kXDone);
          mma_commit(bars + kEmpty + sx);
        }
        wait(kFull + sz, gz / C::kSlots);
        for (int s = 0; s < C::kSteps; ++s) {
          const int g = k * C::kSteps + s, buf = g & 1;
          wait(kKdReady + buf, g >> 1);
          tc_fence_after();
          if (carry) {
#pragma unroll
            for (int p = 0; p < 3; ++p)
#pragma unroll
              for (int kk = 0; kk < C::kStep / 16; ++kk)
                mma_bf16(tmem + C::kTd, desc_sw128(parts + (3 * buf + p) * C::kPart + kk * 2048, C::kStep * 128, 1024),
                         desc_sw128(z + (s * C::kStep + 16 * kk) * 128, kPanelB, 1024), id_d, s + p + kk > 0);
          }
          mma_commit(bars + kPartFree + buf);
        }
        if (carry) mma_commit(bars + kDFull);
        mma_commit(bars + kEmpty + sy);
        if (!STATE) {
          wait(kPReady, k);
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < kC / 16; ++kk)
            mma_bf16_ta(tmem + C::kToz, tmem + C::kTs + 8 * kk, desc_sw128(z + kk * 2048, kPanelB, 1024), id_o, kk > 0);
          mma_commit(bars + kOFull);
        }
        mma_commit(bars + kEmpty + sz);
      }
      mma_commit(bars + kFin);
      wait.drain(kFin, 0);
    }
  } else if (!STATE && warp < C::kS0) {
    // P warps: thread = token row i of the chunk
    const int q = warp & 3, i = 32 * q + lane;
    const uint32_t srow = tmem + C::kTs + ((uint32_t)(32 * q) << 16);
    for (int k = 0; k < n; ++k) {
      const int nv = valid(chunk(k));
      wait(kSFull, k);
      tc_fence_after();
#pragma unroll 1
      for (int cb = 0; cb < 4; ++cb) {
        uint32_t w[16];
        if (jb.rev ? cb >= q : cb <= q) {
          float v[32];
          tmem_ld32(srow + 32 * cb, v);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const int j = 32 * cb + c, e = jb.rev ? j - i : i - j;
            v[c] = (e >= 0 && j < nv) ? v[c] * (jb.c_intra * pw[e & 127]) : 0.f;
          }
#pragma unroll
          for (int c = 0; c < 16; ++c) w[c] = pack2(v[2 * c], v[2 * c + 1]);
        } else {   // the other side of the diagonal
#pragma unroll
          for (int c = 0; c < 16; ++c) w[c] = 0;
        }
        tmem_st16(srow + 16 * cb, w);   // columns of S that this warp has read
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + kPReady);
    }
  } else if (!STATE && warp >= C::kE0) {
    // epilogue: thread = token row
    const int q = warp & 3, i = 32 * q + lane;
    __nv_bfloat16* O = jb.O + b * jb.os[0] + h * jb.os[1];
    for (int k = 0; k < n; ++k) {
      const int c = chunk(k), nv = valid(c), e = jb.rev ? nv - 1 - i : i;
      const float f = e >= 0 ? jb.c_inter * pw[e] : 0.f;
      wait(kOFull, k);
      tc_fence_after();
      __nv_bfloat16* row = O + (long long)(c * kC + i) * jb.os[2];
#pragma unroll 1
      for (int c0 = 0; c0 < DP; c0 += 32) {
        float z[32], x[32];
        tmem_ld32(tmem + C::kToz + c0 + ((uint32_t)(32 * q) << 16), z);
        tmem_ld32(tmem + C::kTox + c0 + ((uint32_t)(32 * q) << 16), x);
        if (c0 + 32 >= DP) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars + kOFree);
        }
        uint32_t w[16];
#pragma unroll
        for (int e2 = 0; e2 < 16; ++e2) w[e2] = pack2(fmaf(f, x[2 * e2], z[2 * e2]), fmaf(f, x[2 * e2 + 1], z[2 * e2 + 1]));
        if (i < nv) {
#pragma unroll
          for (int g = 0; g < 32; g += 16) {
            if (jb.wide && c0 + g < jb.db) {
              st_global_32(row + c0 + g, w + g / 2);
            } else {
              if (c0 + g < jb.db) *reinterpret_cast<uint4*>(row + c0 + g) = make_uint4(w[g / 2], w[g / 2 + 1], w[g / 2 + 2], w[g / 2 + 3]);
              if (c0 + g + 8 < jb.db)
                *reinterpret_cast<uint4*>(row + c0 + g + 8) = make_uint4(w[g / 2 + 4], w[g / 2 + 5], w[g / 2 + 6], w[g / 2 + 7]);
            }
          }
        }
      }
    }
  } else if (warp >= C::kS0 && warp < C::kE0) {
    // state warps: R row and half of its columns per thread (DP 64: M = 64 puts row 16 q + lane in lane < 16)
    constexpr int NR = DP / 2;
    const int ts = t - 32 * C::kS0, q = warp & 3, half = (warp - C::kS0) >> 2;
    const bool live = DP == 128 || lane < 16;
    const int row = DP == 128 ? 32 * q + lane : 16 * q + lane, col = half * NR;
    float R[NR];
    {
      const float* src = a.segs > 1 ? jb.seg_init : jb.init;
      if (STATE) src = nullptr;
      const float f0 = (a.segs > 1 || !jb.init_decays) ? 1.f : expf(ld);
      const size_t at = (a.segs > 1 ? (size_t)u * a.segs + seg : (size_t)u) * dd;
#pragma unroll
      for (int c = 0; c < NR; ++c) {
        R[c] = 0.f;
        if (src && live && row < jb.da && col + c < jb.db)
          R[c] = f0 * src[at + (jb.trans ? (size_t)(col + c) * jb.da + row : (size_t)row * jb.db + col + c)];
      }
    }
    auto update = [&](int k) {   // R after the chunk of step k
      const int c = chunk(k);
      const Decay dec(ld * (valid(c) - (!STATE && c == nch - 1 ? jb.fin_sub : 0)));
      wait(kDFull, k);
      tc_fence_after();
#pragma unroll
      for (int c0 = 0; c0 < NR; c0 += 32) {
        float d[32];
        tmem_ld32(tmem + C::kTd + col + c0 + ((uint32_t)(32 * q) << 16), d);
#pragma unroll
        for (int e = 0; e < 32; ++e) R[c0 + e] = dec(R[c0 + e]) + d[e];
      }
      tc_fence_before();
    };
    for (int k = 0; k < n; ++k) {
      const int c = chunk(k), nv = valid(c), sub = (!STATE && c == nch - 1) ? jb.fin_sub : 0;
      if (k > 0) update(k - 1);
      if (!STATE) {
        if (k > 0) wait(kXDone, k - 1);
        if (live) {
#pragma unroll
          for (int g = 0; g < NR; g += 8) {
            const int cc = col + g;
            *reinterpret_cast<uint4*>(sm + C::kOffR + (cc >> 6) * (DP * 128) + sw128(row, (cc & 63) >> 3)) =
                make_uint4(pack2(R[g], R[g + 1]), pack2(R[g + 2], R[g + 3]), pack2(R[g + 4], R[g + 5]), pack2(R[g + 6], R[g + 7]));
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + kRbReady);
      }
      const int gy = k * C::kPer, gz = gy + C::kPer - 1;
      unsigned char* y = sm + (gy % C::kSlots) * C::kTile;
      unsigned char* z = sm + (gz % C::kSlots) * C::kTile;
      wait(kFull + gy % C::kSlots, gy / C::kSlots);
      if (nv < kC) wait(kFull + gz % C::kSlots, gz / C::kSlots);
      constexpr int CH = DP / 8;   // 16-byte vectors of a row
      const int ch = ts % CH, rr = ts / CH;
      for (int st = 0; st < C::kSteps; ++st) {
        const int g = k * C::kSteps + st, buf = g & 1, r = st * C::kStep + rr;
        const uint32_t off = (ch >> 3) * kPanelB + sw128(r, ch & 7);
        const uint4 v = *reinterpret_cast<const uint4*>(y + off);
        uint32_t o[3][4] = {};
        if (r < nv) {
          const float w = jb.c_state * pw[(jb.rev ? r + 1 : nv - r) - sub];
          const uint32_t in[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float f0 = bf_lo(in[e]) * w, f1 = bf_hi(in[e]) * w;
#pragma unroll
            for (int p = 0; p < 3; ++p) {
              o[p][e] = pack2(f0, f1);
              f0 -= bf_lo(o[p][e]);
              f1 -= bf_hi(o[p][e]);
            }
          }
        } else {   // rows behind the sequence's end may hold anything
          *reinterpret_cast<uint4*>(z + off) = make_uint4(0, 0, 0, 0);
        }
        if (g >= 2) wait(kPartFree + buf, (g >> 1) - 1);
        unsigned char* d = sm + C::kOffPart + 3 * buf * C::kPart + (ch >> 3) * (C::kStep * 128) + sw128(rr, ch & 7);
#pragma unroll
        for (int p = 0; p < 3; ++p) *reinterpret_cast<uint4*>(d + p * C::kPart) = make_uint4(o[p][0], o[p][1], o[p][2], o[p][3]);
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + kKdReady + buf);
      }
    }
    if (STATE || ends) {
      update(n - 1);
      float* dst = STATE ? jb.local + ((size_t)u * a.segs + seg) * dd : jb.fin + u * dd;
      const bool tr = !STATE && jb.trans;
      if (live && row < jb.da) {
#pragma unroll
        for (int c = 0; c < NR; ++c)
          if (col + c < jb.db) dst[tr ? (size_t)(col + c) * jb.da + row : (size_t)row * jb.db + col + c] = R[c];
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
    o.c_inter = j.c_inter;
    o.c_intra = j.c_intra;
    o.c_state = j.c_state;
  }
  return dp == 64 ? run<64, false>(t, units, a.njobs, st) : run<128, false>(t, units, a.njobs, st);
}

}  // namespace lfa
