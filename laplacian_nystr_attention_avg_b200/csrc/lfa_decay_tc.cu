// Decay attention on bf16 tensors: the chunked run of lfa_decay.cu on tcgen05 tensor cores.
//
// A CTA takes one segment of one unit's tokens (one run: DecayJob) and walks its chunks of 128 tokens. Per chunk,
// with x, y, z tiles brought in by TMA and the carried state R [da][db] held in fp32 registers:
//   S  = x y^T                              (M 128 tokens, N 128 tokens, K da)
//   P  = c_intra l^(i-j) S, j <= i, in bf16   (P warps; the only rounding of the weights)
//   Oz = P z,  Ox = x bf16(R)               (M 128, N db; K 128 and K da)
//   O  = Oz + c_inter l^i Ox                (epilogue warps, fp32, rounded once)
//   D  = (y c_state l^(n-j))^T z            (M da, N db, K 128 tokens), R' = l^n R + D   (state warps)
// The decayed rows of y enter as bf16 parts, one product each. Where R only meets x, which rounds it to bf16, two parts
// leave 4e-6 of its norm. Runs that return a state take three, the 24 bits of an fp32 product: such a state is 0.5e-6
// off, after 8 tokens as after 4096, of which the tensor cores' own sums are the most. (8 x 16 x 4096 tokens x 128: 140
// us with a state, 118 without; at 64 channels 94 and 72, where the third product has zeros in half of its rows; of
// segments only the states' kernel has it: 1 x 8 x 65536 x 64 112 and 107.) An infinity has a NaN as its remainder:
// states and outputs that the formula makes infinite may be NaN. D starts from zero in every chunk and is added to R by
// CUDA cores: tensor-core accumulation truncates and would drift over thousands of chunks.
// All widths are padded to DP = 64 or 128 by TMA's zero fill.
//
// Warps: 4 or 8 for P, 4 or 8 for y's decayed rows, 8 for R and the epilogue, one each to issue TMA loads, the
// products of the state and those of the output. Every hand-over is an mbarrier; every wait is bounded (on expiry
// the device's status word is set, the CTA stops waiting for anything and drains what it has in flight).
//
// What bounds it: 128 units x 4096 tokens take 115 us at 128 channels (83 at the copy bandwidth, with 128 of 148 SMs
// at work; 144 units 116 of 94) and 64 us at 64 channels (42): there a chunk takes 3.0 k cycles, in which issue slots
// are half full, shared memory 65 % busy and the tensor pipe 32 %, the longest chains being P's warps and D -> R -> D.
// Not taken: 8 P warps at 128 channels, their registers from the others (117 us); a second set of O instead of the
// second set of S at 64; a unit's three backward runs on neighbouring SMs (they read the same tiles at the same time:
// 188 instead of 178 us for 128 units x 2048 tokens x 128, 120 instead of 104 at 64).
//
// Few units over long sequences: segments run at once. k_decay_tc<.., true, ..> sums up each segment's own
// state, k_decay_prefix carries them over the segments and writes the state after the last, and the main kernel starts
// every segment from its state.
#include <string.h>

#include <type_traits>

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
  int third;              // y's decayed rows in three parts (PARTS 3)
  int wide;               // O's rows are whole, aligned 32-byte sectors
  const __nv_bfloat16 *X, *Y, *Z;   // what the maps read, for before_odd
  long long xs[3], ys[3], zs[3];
  float c_inter, c_intra, c_state;
};
struct TcArgs {
  TcJob job[3];
  const float* log_decay;
  const int* lengths;
  int heads, N, segs, seg_chunks;
};

template <int DP, bool STATE, int PARTS>
struct Cfg {
  static constexpr int kTile = DP / 64 * kPanelB;   // bytes of a token tile
  // rings of tiles. At 128 channels five fit: x is done with first (S, then Ox), y and z are held longer
  static constexpr int kNY = DP == 64 ? 3 : 2;
  static constexpr int kNX = STATE ? 0 : DP == 64 ? 4 : 1;
  static constexpr int kNZ = DP == 64 ? 4 : 2;
  static constexpr int kOffX = kNY * kTile;
  static constexpr int kOffZ = kOffX + kNX * kTile;
  static constexpr int kOffPart = kOffZ + kNZ * kTile;
  // y's decayed rows are formed in steps of kStep tokens, kVec 16-byte vectors per thread, in two buffers of PARTS parts
  static constexpr int kStep = (PARTS == 3 && !STATE ? 2048 : 4096) / DP;
  static constexpr int kSteps = kC / kStep;
  static constexpr int kYW = STATE && DP == 64 ? 8 : 4;   // warps that form them
  static constexpr int kVec = kStep * DP / 8 / (32 * kYW);
  static constexpr int kPart = kStep * DP * 2;             // bytes of one part of a step
  // DP 64: the two parts share the product's 128 rows (M = 64 runs at half the speed): rows 64 .. 127 of D, and of R
  // with it, are the second part's. Their sum is formed in x R's product (two tiles of R) and where a state is written.
  // A third part has 16 tokens of zeros for company.
  static constexpr bool kStack = DP == 64;
  static constexpr int kOffZero = kOffPart + 2 * PARTS * kPart;
  static constexpr int kOffR = kOffZero + (kStack && PARTS == 3 ? 16 * 128 : 0);
  static constexpr int kOffBar = kOffR + (STATE ? 0 : DP * DP * 2 * (kStack ? 2 : 1));
  static constexpr int kOffPb = kOffBar + 384;
  static constexpr int kOffPi = kOffPb + 4 * 32;
  static constexpr int kOffWt = kOffPi + 4 * (32 + kC);
  static constexpr int kSmem = kOffWt + 8 * (kC + 1);
  static_assert(kSmem <= 232448, "shared memory over the sm_100 per-block limit");
  // warps: P (not STATE), y's decayed rows, 8 for the state and the epilogue, loads, products (two)
  static constexpr int kPW = STATE ? 0 : DP == 64 ? 8 : 4;
  static constexpr int kY0 = kPW;
  static constexpr int kR0 = kY0 + kYW;
  static constexpr int kLoad = kR0 + 8;
  static constexpr int kMma = kLoad + 1;      // products of the state
  static constexpr int kMmaO = kMma + 1;      // products of the output (not STATE)
  static constexpr int kThreads = 32 * (STATE ? kMma + 1 : kMmaO + 1);
  // DP 64: 736 threads have 80 registers each; the state warps take 16 more from the P warps (8 each) and the y warps
  // (16 each): 256 72 + 128 64 + 256 96 + 96 80 = 736 80. DP 128: 608 threads with 96; the state warps, R being 64 of
  // theirs, take 16 more from the P and y warps (16 each): 128 80 + 128 80 + 256 112 + 96 96 = 608 96
  static constexpr int kRegsP = DP == 64 ? 72 : 80, kRegsY = DP == 64 ? 64 : 80, kRegsR = DP == 64 ? 96 : 112;
  static constexpr bool kSplitRegs = !STATE;
  // tensor memory columns. DP 64: two sets of S, so that the next scores are there when the P warps, its longest
  // chain, are; P (bf16 pairs), Oz, Ox, D. DP 128: no room for that; P goes over the first half of S's columns, row
  // by row as S is read
  static constexpr bool kOwnP = DP == 64;
  static constexpr int kNS = kOwnP ? 2 : 1;   // sets of S
  static constexpr int kTs = 0, kTp = kOwnP ? 2 * kC : 0, kToz = STATE ? 0 : kOwnP ? 2 * kC + kC / 2 : kC;
  static constexpr int kTd = STATE ? 0 : kToz + 2 * DP;
  static constexpr int kTmem = STATE ? DP : 512;
  static_assert(kTd + DP <= kTmem, "tensor memory");
};
enum Bar {
  kFullY = 0, kFullX = 4, kFullZ = 8, kEmptyY = 12, kEmptyX = 16, kEmptyZ = 20, kSFull = 24, kSRead = 26,
  kPReady = 28, kYdReady, kPartFree = kYdReady + 2, kDFull = kPartFree + 2, kDRead, kRbReady, kXDone, kOFull, kOFree,
  kZClean, kFin, kNumBars = kFin + 2
};
static_assert(kNumBars * 8 <= 368, "barriers overlap the TMEM slot");

// The products are issued by one lane of a warp whose lanes stay together, so that descriptors and loop counters are
// uniform over the warp (in a branch of one lane each product spent about 80 cycles on moving them there).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}\n" : "=r"(p));
  return p;
}
__device__ __forceinline__ void mma_by(uint32_t lead, uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc), "r"(lead));
}
// A in tensor memory: lane = row, 16-bit K elements 2c, 2c + 1 in column c
__device__ __forceinline__ void mma_ta_by(uint32_t lead, uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc), "r"(lead));
}
__device__ __forceinline__ void commit_by(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}\n" ::"r"(smem_u32(bar)),
      "r"(lead)
      : "memory");
}

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
__device__ __forceinline__ uint32_t packf2(uint64_t v) { return pack2(f2_lo(v), f2_hi(v)); }
// y w for a pair y of bf16 as a sum of bf16 parts. Two: w = w.x + w.y in bf16 parts; a = y w.x rounded, its remainder
// y w.x - a is a bf16 itself (8 by 8 bits make 16), and about 2^-17 of y w is left out. Three: w in fp32, the
// product's 24 bits in turn.
__device__ __forceinline__ __nv_bfloat162 as_b2(uint32_t v) { return *reinterpret_cast<const __nv_bfloat162*>(&v); }
__device__ __forceinline__ uint32_t as_u(__nv_bfloat162 v) { return *reinterpret_cast<const uint32_t*>(&v); }
__device__ __forceinline__ void split(uint32_t y, uint2 w, uint32_t& a, uint32_t& b) {
  const __nv_bfloat162 y2 = as_b2(y), wx = as_b2(w.x), wy = as_b2(w.y);
  const __nv_bfloat162 hi = __hmul2(y2, wx);
  a = as_u(hi);
  b = as_u(__hfma2(y2, wy, __hfma2(y2, wx, __hneg2(hi))));
}
__device__ __forceinline__ void split3(uint32_t y, uint2 w, uint32_t& a, uint32_t& b, uint32_t& c) {
  const uint64_t less = f2(-1.f, -1.f);
  uint64_t v = mul2(f2(y << 16, y & 0xffff0000u), f2(w.x, w.y));
  a = packf2(v);
  v = fma2(f2(a << 16, a & 0xffff0000u), less, v);
  b = packf2(v);
  v = fma2(f2(b << 16, b & 0xffff0000u), less, v);
  c = packf2(v);
}

// one 32-byte store (a whole sector)
__device__ __forceinline__ void st_global_32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ float bf_lo(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float bf_hi(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

// The P warps of a run of n chunks: P = c_intra l^|i-j| S on the causal side, in bf16 (thread = token row i; with
// two warps for a quarter of the rows, they take its blocks of 32 columns in turn). pi holds c_intra l^n after 32
// zeros; beside the diagonal block l^|i-j| is l^(distance of i to the block) pb[c]. nv0: valid tokens of the first
// chunk, where a reverse run finds its sequence's ragged end (forwards, columns behind the end are above the
// diagonal).
template <class C, bool REV>
__device__ __forceinline__ void weights(int n, const Waiter& wait, uint64_t* bars, uint32_t tmem, const float* pi,
                                        const float* pb, int nv0) {
  const int lane = threadIdx.x & 31, q = (threadIdx.x >> 5) & 3, i = 32 * q + lane, first = threadIdx.x >> 7;
  const uint32_t quad = tmem + ((uint32_t)(32 * q) << 16), srow = quad + C::kTs, prow = quad + C::kTp;
  const float* pd = pi + (REV ? -lane : lane);
  // the other side of the diagonal is zero: once where P has its own columns, else in every chunk
  auto zeros = [&]() {
    uint32_t w[16] = {};
    for (int cb = 0; cb < 4; ++cb)
      if (REV ? cb < q : cb > q) tmem_st16(prow + 16 * cb, w);
  };
  if (C::kOwnP) {
    if (q == (REV ? 3 : 0) && first == (REV ? 0 : 1)) return;   // the one of eight that has no block at all
    zeros();
  }
  for (int k = 0; k < n; ++k) {
    const bool ragged = REV && k == 0 && nv0 < kC;
    wait(kSFull + k % C::kNS, k / C::kNS);
    const uint32_t sk = srow + k % C::kNS * kC;
    tc_fence_after();
    bool used = !C::kOwnP || k == 0;   // P's columns are free
#pragma unroll 1
    for (int cb = first; cb < 4; cb += C::kPW / 4) {
      if (REV ? cb < q : cb > q) continue;
      uint32_t v[32];
      tmem_ld32_async(sk + 32 * cb, v);
      if (cb == q) {
        tmem_wait_ld(v);
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          const float x = __uint_as_float(v[c]) * pd[REV ? c : -c];
          v[c] = (REV ? c >= lane : c <= lane) ? __float_as_uint(x) : 0u;
        }
      } else {
        const float f = pi[REV ? 32 * cb - i : i - 32 * cb - 31];
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
      if (ragged && nv0 < 32 * cb + 32) {   // columns of tokens behind the end may hold anything
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (32 * cb + c >= nv0) v[c] = 0;
      }
      uint32_t w[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) w[c] = pack2(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1]));
      if (!used) {
        wait(kOFull, k - 1);
        tc_fence_after();
        used = true;
      }
      tmem_st16(prow + 16 * cb, w);   // on S's columns where it has none of its own: on those read before
    }
    if (C::kOwnP) {   // S has been read
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bars + kSRead + k % C::kNS);
    } else {
      zeros();
    }
    tmem_wait_st();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + kPReady);
  }
}

__device__ __forceinline__ void unpack8(const void* p, float* v) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[2 * e] = bf_lo(w[e]);
    v[2 * e + 1] = bf_hi(w[e]);
  }
}

// P is zero on the other side of the diagonal, but a z there that is not finite makes 0 z a NaN in its column, for all
// rows of its chunk; from the next chunk on the state carries it, as the recurrence does. So the rows that must not see
// it are those of the same chunk before the run comes to a column's first such z. They are formed again here, in fp32
// from the tensors themselves, at the end of a segment whose last row is not finite (which both ways make it). One of
// `warps` warps takes every so many sets of 8 columns: the state before the chunk, then the chunk's rows, a row a lane.
// Looking at the last row alone keeps this out of the chunks (a check in every epilogue cost them 12 %); the barrier
// at the end costs 1 x 8 x 65536 tokens 3 us of 103, the other listed sizes nothing that shows. A NaN in one channel of
// the last of 4096 tokens takes 2.6 ms, tensors that are not finite from the run's start the time of a look.
__device__ __forceinline__ void before_odd(const TcArgs& a, int warp, int warps, unsigned char* mem) {
  const TcJob& jb = a.job[blockIdx.z];
  const int u = blockIdx.x, seg = blockIdx.y, b = u / a.heads, h = u % a.heads, lane = threadIdx.x & 31;
  const int L = unit_length(a.lengths, b, a.N), da = jb.da, db = jb.db;
  const int t_lo = seg * a.seg_chunks * kC, t_hi = min(L, t_lo + a.seg_chunks * kC), T = t_hi - t_lo;
  const bool rev = jb.rev;
  const float ld = decay_log(a.log_decay[h]);
  auto tok = [&](int p) { return rev ? t_hi - 1 - p : t_lo + p; };   // of place p in the run
  const __nv_bfloat16* X = jb.X + b * jb.xs[0] + h * jb.xs[1];
  const __nv_bfloat16* Y = jb.Y + b * jb.ys[0] + h * jb.ys[1];
  for (int c0 = 8 * warp; c0 < db; c0 += 8 * warps) {
    const __nv_bfloat16* Z = jb.Z + b * jb.zs[0] + h * jb.zs[1] + c0;
    auto z_row = [&](int p) { return *reinterpret_cast<const uint4*>(Z + tok(p) * jb.zs[2]); };
    // y and the columns of z of 32 places, in this warp's memory
    unsigned char* ym = mem + warp * 32 * (2 * kDecayMaxD + 16);
    unsigned char* zm = ym + 32 * 2 * kDecayMaxD;
    auto stage = [&](int p, int n) {
      __syncwarp();
      for (int e = lane; e < n * (da / 8); e += 32) {
        const int r = e / (da / 8), c = e % (da / 8) * 8;
        *reinterpret_cast<uint4*>(ym + 2 * (r * kDecayMaxD + c)) = *reinterpret_cast<const uint4*>(Y + tok(p + r) * jb.ys[2] + c);
      }
      if (lane < n) *reinterpret_cast<uint4*>(zm + 16 * lane) = z_row(p + lane);
      __syncwarp();
    };
    int first[8];   // the columns' first such places
#pragma unroll
    for (int e = 0; e < 8; ++e) first[e] = T;
    uint32_t found = 0;
    for (int p = 0; p < T && found != 255u; p += 32) {
      uint32_t m = 0;
      if (p + lane < T) {
        const uint4 v = z_row(p + lane);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int e = 0; e < 4; ++e)
          m |= ((w[e] & 0x7f80u) == 0x7f80u ? 1u << 2 * e : 0u) | ((w[e] & 0x7f800000u) == 0x7f800000u ? 2u << 2 * e : 0u);
      }
      if (__any_sync(0xffffffffu, m != 0)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t lanes = __ballot_sync(0xffffffffu, m >> e & 1);
          if (lanes && first[e] == T) {
            first[e] = p + __ffs(lanes) - 1;
            found |= 1u << e;
          }
        }
      }
    }
    // where their chunks begin, in the run
    int from[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      from[e] = first[e] == T ? T : rev ? t_hi - min((tok(first[e]) / kC + 1) * kC, t_hi) : first[e] / kC * kC;
    for (;;) {   // the columns of one chunk at a time
      int start = T, end = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (from[e] < first[e]) start = min(start, from[e]);
      if (start == T) break;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (from[e] == start) end = max(end, first[e]);
      float R[4][8];   // rows lane, lane + 32, ..
      const float* src = a.segs > 1 ? jb.seg_init : jb.init;
      const size_t at = (a.segs > 1 ? (size_t)u * a.segs + seg : (size_t)u) * da * db;
      const float f0 = a.segs > 1 || !jb.init_decays ? 1.f : expf(ld);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int r = lane + 32 * i;
          R[i][e] = src && r < da ? f0 * src[at + (jb.trans ? (size_t)(c0 + e) * da + r : (size_t)r * db + c0 + e)] : 0.f;
        }
      for (int p0 = 0; p0 < start; p0 += kC) {
        const int n = min(kC, start - p0);
        const Decay dec(ld * n);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) R[i][e] = dec(R[i][e]);
        for (int m0 = 0; m0 < n; m0 += 32) {
          const int nm = min(32, n - m0);
          stage(p0 + m0, nm);
          for (int m = 0; m < nm; ++m) {
            const float w = jb.c_state * expf(ld * (n - m0 - m));
            float z[8];
            unpack8(zm + 16 * m, z);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = lane + 32 * i;
              const float y = r < da ? w * __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(ym)[m * kDecayMaxD + r]) : 0.f;
#pragma unroll
              for (int e = 0; e < 8; ++e) R[i][e] = fmaf(y, z[e], R[i][e]);
            }
          }
        }
      }
      for (int p0 = start; p0 < end; p0 += 32) {
        const int pr = p0 + lane;
        const __nv_bfloat16* x = X + tok(min(pr, end - 1)) * jb.xs[2];
        float acc[8] = {}, o[8] = {};
        for (int q0 = start; q0 < min(p0 + 32, end); q0 += 32) {
          const int nq = min(32, end - q0);
          stage(q0, nq);
          for (int m = 0; m < nq; ++m) {
            float s = 0.f;
            for (int k = 0; k < da; k += 8) {
              float xv[8], yv[8];
              unpack8(x + k, xv);
              unpack8(ym + 2 * (m * kDecayMaxD + k), yv);
#pragma unroll
              for (int e = 0; e < 8; ++e) s = fmaf(xv[e], yv[e], s);
            }
            if (q0 + m <= pr) {
              const float w = jb.c_intra * expf(ld * (pr - q0 - m)) * s;
              float z[8];
              unpack8(zm + 16 * m, z);
#pragma unroll
              for (int e = 0; e < 8; ++e) acc[e] = fmaf(w, z[e], acc[e]);
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          for (int r = 0; r < min(32, da - 32 * i); ++r) {
            const float xr = __bfloat162float(x[32 * i + r]);
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = fmaf(xr, __shfl_sync(0xffffffffu, R[i][e], r), o[e]);
          }
        const float f = jb.c_inter * expf(ld * (pr - start));
        __nv_bfloat16* O = jb.O + b * jb.os[0] + h * jb.os[1] + tok(min(pr, end - 1)) * jb.os[2] + c0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (from[e] == start && pr < first[e]) O[e] = __float2bfloat16_rn(fmaf(f, o[e], acc[e]));
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (from[e] == start) from[e] = first[e];
    }
  }
}

template <int DP, bool STATE, int PARTS>
__global__ void __launch_bounds__(Cfg<DP, STATE, PARTS>::kThreads, 1) k_decay_tc(const __grid_constant__ TcArgs a) {
  using C = Cfg<DP, STATE, PARTS>;
  extern __shared__ __align__(1024) unsigned char sm[];
  const TcJob& jb = a.job[blockIdx.z];
  const int u = blockIdx.x, seg = blockIdx.y, b = u / a.heads, h = u % a.heads;
  const int L = unit_length(a.lengths, b, a.N), nch = (L + kC - 1) / kC;
  const int c_lo = seg * a.seg_chunks, c_hi = min(c_lo + a.seg_chunks, nch), n = c_hi - c_lo;
  const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
  const int da = jb.da, db = jb.db;
  const bool rev = jb.rev;
  const size_t dd = (size_t)da * db;
  if (STATE) let_next_start();
  const bool third = PARTS == 3 && jb.third;
  if (n <= 0) {
    if (!STATE) wait_for_previous();   // a call is over when all its launches are
    if (!STATE && L == 0 && seg == 0 && jb.fin)
      for (size_t e = t; e < dd; e += C::kThreads) jb.fin[u * dd + e] = jb.init ? jb.init[u * dd + e] : 0.f;
    return;
  }
  if (STATE && !jb.fin && (rev ? seg == 0 : c_hi == nch)) return;   // nothing follows this segment
  const bool ends = !STATE && jb.fin && (rev ? seg == 0 : c_hi == nch);

  if ((smem_u32(sm) & 1023u) != 0) {   // the swizzle needs it; the declaration asks for it
    if (t == 0) atomicOr(&g_decay_status, 1);
    return;
  }
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + C::kOffBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sm + C::kOffBar + 368);
  volatile int* gave_up = reinterpret_cast<volatile int*>(sm + C::kOffBar + 372);
  volatile int* odd = gave_up + 1;   // the segment's last row is not finite
  float* pb = reinterpret_cast<float*>(sm + C::kOffPb);        // rev: l^c, else l^(31-c), c = 0 .. 31
  float* pi = reinterpret_cast<float*>(sm + C::kOffPi) + 32;   // c_intra l^0 .. c_intra l^127 after 32 zeros
  uint2* wt = reinterpret_cast<uint2*>(sm + C::kOffWt);        // c_state l^n: two bf16 parts, each twice in a word; or fp32 twice
  const float ld = decay_log(a.log_decay[h]);
  const Waiter wait{bars, gave_up};
  // chunk of step k, and its valid tokens
  auto chunk = [&](int k) { return rev ? c_hi - 1 - k : c_lo + k; };
  auto valid = [&](int c) { return min(kC, L - c * kC); };
  // tile k of a tensor into its ring
  auto load = [&](const CUtensorMap* m, int off, int ring, int full, int empty, int k) {
    const int s = k % ring;
    if (k >= ring) wait(empty + s, k / ring - 1);
    if (*gave_up) return false;
    mbar_expect_tx(bars + full + s, C::kTile);
    for (int p = 0; p < DP / 64; ++p)
      tma_load_4d(sm + off + s * C::kTile + p * kPanelB, m, 64 * p, chunk(k) * kC, h, b, bars + full + s);
    return true;
  };
  if (t == 32 * C::kLoad) {
    for (int i = 0; i < kNumBars; ++i)
      mbar_init(bars + i, i >= kEmptyY && i < kEmptyX                                    ? C::kYW + (STATE ? 0 : 1)
                          : i >= kEmptyZ && i < kSFull                                   ? (STATE ? 1 : 2)
                          : (i >= kYdReady && i < kPartFree) || i == kZClean             ? C::kYW
                          : i >= kSRead && i <= kPReady                                  ? (C::kPW ? C::kPW - C::kOwnP : 1)
                          : i == kDRead || i == kRbReady || i == kOFree                  ? 8
                                                                                         : 1);
    mbar_init_fence();
    *gave_up = 0;
    *odd = 0;
    // the first chunk is under way while the rest is set up
    load(&jb.y, 0, C::kNY, kFullY, kEmptyY, 0);
    load(&jb.z, C::kOffZ, C::kNZ, kFullZ, kEmptyZ, 0);
    if (!STATE) load(&jb.x, C::kOffX, 1 > C::kNX ? 1 : C::kNX, kFullX, kEmptyX, 0);
  }
  if (warp == C::kMma) tmem_alloc(tmem_slot, C::kTmem);
  for (int i = t; i <= kC; i += C::kThreads) {
    const float w = expf(ld * i);
    if (i < 32) {
      pb[rev ? i : 31 - i] = w;
      pi[i - 32] = 0.f;
    }
    if (i < kC) pi[i] = jb.c_intra * w;
    const float f = jb.c_state * w, f1 = f - bf_lo(pack2(f, f));
    wt[i] = third ? make_uint2(__float_as_uint(f), __float_as_uint(f)) : make_uint2(pack2(f, f), pack2(f1, f1));
  }
  if (C::kStack && PARTS == 3) {
    for (int i = t; i < 16 * 128 / 16; i += C::kThreads) *reinterpret_cast<uint4*>(sm + C::kOffZero + 16 * i) = make_uint4(0, 0, 0, 0);
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // the two warps that issue the products, at their end: they have the registers
  auto mend = [&](int which) {
    __syncwarp();
    named_bar_sync(2, 320);
    if (*odd) {
      if (!*gave_up) before_odd(a, which, 2, sm);   // the tiles are done with
      named_bar_sync(2, 320);
    }
  };
  if (warp == C::kLoad) {
    if (lane == 0) {
      // y, z, x of every chunk in turn, each tensor in a ring of its own
      int ny = 1, nx = 1, nz = 1;   // loads issued
      for (int k = 1; k < n; ++k) {
        if (!load(&jb.y, 0, C::kNY, kFullY, kEmptyY, k)) break;
        ++ny;
        // x before z where its ring is as deep: its slot is free sooner, and S needs it sooner than P z needs z
        if constexpr (C::kNX > 1) {
          if (!load(&jb.x, C::kOffX, C::kNX, kFullX, kEmptyX, k)) break;
          ++nx;
        }
        if (!load(&jb.z, C::kOffZ, C::kNZ, kFullZ, kEmptyZ, k)) break;
        ++nz;
        if constexpr (C::kNX == 1) {
          if (!load(&jb.x, C::kOffX, C::kNX, kFullX, kEmptyX, k)) break;
          ++nx;
        }
      }
      for (int i = max(0, ny - C::kNY); i < ny; ++i) wait.drain(kFullY + i % C::kNY, i / C::kNY);
      for (int i = max(0, nz - C::kNZ); i < nz; ++i) wait.drain(kFullZ + i % C::kNZ, i / C::kNZ);
      if constexpr (!STATE)
        for (int i = max(0, nx - C::kNX); i < nx; ++i) wait.drain(kFullX + i % C::kNX, i / C::kNX);
    }
  } else if (!STATE && warp == C::kMmaO) {
    if constexpr (!STATE) {
      const uint32_t lead = elect_one(), tm = __shfl_sync(0xffffffffu, tmem, 0);
      const int steps = __shfl_sync(0xffffffffu, n, 0);
      // S, Ox, Oz of every chunk in turn. Descriptors of a ring's first tile; b bytes further is + b / 16
      const uint32_t base = smem_u32(sm);
      const uint64_t d_y = desc_sw128(base, 16, 1024), d_x = desc_sw128(base + C::kOffX, 16, 1024),
                     d_z = desc_sw128(base + C::kOffZ, kPanelB, 1024), d_rb = desc_sw128(base + C::kOffR, DP * 128, 1024);
      constexpr uint32_t id_s = idesc(1, kC, kC, 0, 0), id_o = idesc(1, kC, DP, 0, 1);
      auto scores = [&](int k) {
        const int sy = k % C::kNY, sx = k % C::kNX;
        const uint64_t y = d_y + sy * (C::kTile / 16), x = d_x + sx * (C::kTile / 16);
        wait(kFullY + sy, k / C::kNY);
        wait(kFullX + sx, k / C::kNX);
        if (k >= C::kNS) C::kOwnP ? wait(kSRead + k % C::kNS, k / C::kNS - 1) : wait(kOFull, k - 1);   // S (and P over it) used
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < DP / 16; ++kk) {
          const int off = ((kk >> 2) * kPanelB + (kk & 3) * 32) / 16;
          mma_by(lead, tm + C::kTs + k % C::kNS * kC, x + off, y + off, id_s, kk > 0);
        }
        commit_by(lead, bars + kSFull + k % C::kNS);
        commit_by(lead, bars + kEmptyY + sy);
      };
      scores(0);
      for (int k = 0; k < steps; ++k) {
        const int sx = k % C::kNX, sz = k % C::kNZ;
        const uint64_t x = d_x + sx * (C::kTile / 16), z = d_z + sz * (C::kTile / 16);
        const uint32_t oz = tm + C::kToz, ox = oz + DP;
        if (C::kOwnP && k + 1 < steps) scores(k + 1);
        wait(kRbReady, k);
        if (k > 0) wait(kOFree, k - 1);
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < (C::kStack ? 2 : 1) * DP / 16; ++kk) {   // stacked: x again, times the second tile of R
          const int kx = kk % (DP / 16);
          mma_by(lead, ox, x + ((kx >> 2) * kPanelB + (kx & 3) * 32) / 16, d_rb + kk * 128, id_o, kk > 0);
        }
        commit_by(lead, bars + kXDone);
        commit_by(lead, bars + kEmptyX + sx);
        wait(kFullZ + sz, k / C::kNZ);
        if (valid(chunk(k)) < kC) wait(kZClean, 0);
        wait(kPReady, k);
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kC / 16; ++kk) mma_ta_by(lead, oz, tm + C::kTp + 8 * kk, z + kk * 128, id_o, kk > 0);
        commit_by(lead, bars + kOFull);
        commit_by(lead, bars + kEmptyZ + sz);
        if (!C::kOwnP && k + 1 < steps) scores(k + 1);
      }
      commit_by(lead, bars + kFin);
      wait.drain(kFin, 0);
      mend(0);
    }
  } else if (warp == C::kMma) {
    const uint32_t lead = elect_one(), tm = __shfl_sync(0xffffffffu, tmem, 0);
    const int steps = __shfl_sync(0xffffffffu, n, 0);
    // D of every chunk: its own thread, so that the state runs ahead of the outputs
    const uint32_t base = smem_u32(sm);
    const uint64_t d_z = desc_sw128(base + C::kOffZ, kPanelB, 1024),
                   d_part = desc_sw128(base + C::kOffPart, C::kStack ? C::kPart : C::kStep * 128, 1024);
    constexpr uint32_t id_d = idesc(1, 128, DP, 1, 1);
    for (int k = 0; k < steps; ++k) {
      const int sz = k % C::kNZ;
      const uint64_t z = d_z + sz * (C::kTile / 16);
      const bool carry = STATE || ends || k < n - 1;
      wait(kFullZ + sz, k / C::kNZ);
      if (k > 0) wait(kDRead, k - 1);
#pragma unroll 1
      for (int s = 0; s < C::kSteps; ++s) {
        const int g = k * C::kSteps + s, buf = g & 1;
        wait(kYdReady + buf, g >> 1);
        tc_fence_after();
        if (carry) {
#pragma unroll
          for (int p = 0; p < PARTS; p += C::kStack ? 2 : 1) {
            if (p == 2 && !third) break;
#pragma unroll
            for (int kk = 0; kk < C::kStep / 16; ++kk) {
              const int at = (PARTS * buf + p) * C::kPart + kk * 2048;
              uint64_t part = d_part + at / 16;
              if (C::kStack && p == 2) part = desc_sw128(base + C::kOffPart + at, C::kOffZero - C::kOffPart - at, 1024);
              mma_by(lead, tm + C::kTd, part, z + (s * C::kStep + 16 * kk) * 8, id_d, s + p + kk > 0);
            }
          }
        }
        commit_by(lead, bars + kPartFree + buf);
      }
      if (carry) commit_by(lead, bars + kDFull);
      commit_by(lead, bars + kEmptyZ + sz);
    }
    commit_by(lead, bars + kFin + 1);
    wait.drain(kFin + 1, 0);
    if (!STATE) mend(1);
  } else if (!STATE && warp < C::kY0) {
    if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsP));
    if (rev)
      weights<C, true>(n, wait, bars, tmem, pi, pb, L - (c_hi - 1) * kC);
    else
      weights<C, false>(n, wait, bars, tmem, pi, pb, kC);
  } else if (warp < C::kR0) {
    // y's decayed rows, in steps of kStep tokens into one of two buffers
    if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsY));
    const int ty = t - 32 * C::kY0;
    constexpr int CH = DP / 8, RS = 32 * C::kYW / CH;   // 16-byte vectors of a row, rows per pass (a multiple of 8)
    const int ch = ty % CH, rr = ty / CH;
    const uint32_t at = (ch >> 3) * kPanelB + sw128(rr, ch & 7);   // rows RS apart have the same place in the swizzle
    unsigned char* d0 = sm + C::kOffPart + (ch >> 3) * (C::kStep * 128) + sw128(rr, ch & 7);
    for (int k = 0; k < n; ++k) {
      const int c = chunk(k), nv = valid(c), sub = c == nch - 1 ? jb.fin_sub : 0;
      const unsigned char* y = sm + (k % C::kNY) * C::kTile + at;
      unsigned char* z = sm + C::kOffZ + (k % C::kNZ) * C::kTile + at;
      const uint2* w0 = wt + (rev ? 1 : nv) - sub;   // row r: r weights on (rev) or back
      const int ws = rev ? 1 : -1;
      wait(kFullY + k % C::kNY, k / C::kNY);
      if (nv < kC) wait(kFullZ + k % C::kNZ, k / C::kNZ);
#pragma unroll 1
      for (int st = 0; st < C::kSteps; ++st) {
        const int g = k * C::kSteps + st, buf = g & 1;
        uint4 v[C::kVec];
        uint2 w[C::kVec];
#pragma unroll
        for (int e = 0; e < C::kVec; ++e) {
          const int r = st * C::kStep + rr + e * RS;
          v[e] = *reinterpret_cast<const uint4*>(y + (st * C::kStep + e * RS) * 128);
          w[e] = w0[(r < nv ? r : 0) * ws];
        }
        if (nv < kC) {   // rows behind the sequence's end may hold anything
#pragma unroll
          for (int e = 0; e < C::kVec; ++e)
            if (st * C::kStep + rr + e * RS >= nv) {
              v[e] = make_uint4(0, 0, 0, 0);
              *reinterpret_cast<uint4*>(z + (st * C::kStep + e * RS) * 128) = v[e];
            }
        }
        if (g >= 2) wait(kPartFree + buf, (g >> 1) - 1);
        unsigned char* d = d0 + PARTS * buf * C::kPart;
#pragma unroll
        for (int e = 0; e < C::kVec; ++e) {
          uint4 hi, lo;
          if (third) {
            uint4 rest;
            split3(v[e].x, w[e], hi.x, lo.x, rest.x);
            split3(v[e].y, w[e], hi.y, lo.y, rest.y);
            split3(v[e].z, w[e], hi.z, lo.z, rest.z);
            split3(v[e].w, w[e], hi.w, lo.w, rest.w);
            *reinterpret_cast<uint4*>(d + e * RS * 128 + 2 * C::kPart) = rest;
          } else {
            split(v[e].x, w[e], hi.x, lo.x);
            split(v[e].y, w[e], hi.y, lo.y);
            split(v[e].z, w[e], hi.z, lo.z);
            split(v[e].w, w[e], hi.w, lo.w);
          }
          *reinterpret_cast<uint4*>(d + e * RS * 128) = hi;
          *reinterpret_cast<uint4*>(d + e * RS * 128 + C::kPart) = lo;
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + kYdReady + buf);
      }
      if (lane == 0) {
        mbar_arrive(bars + kEmptyY + k % C::kNY);
        if (!STATE && nv < kC) mbar_arrive(bars + kZClean);
      }
    }
  } else if (warp < C::kLoad) {
    if constexpr (C::kSplitRegs) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsR));
    // state and epilogue: a row of R and half of its columns per thread (stacked: rows 64 .. 127 are the second
    // part's share of rows 0 .. 63); in the epilogue thread = token row, the same half of O's columns
    constexpr int NR = DP / 2, NT = 16;   // columns of R, columns read at once
    const int q = warp & 3, half = (warp - C::kR0) >> 2, i = 32 * q + lane;
    const bool trans = jb.trans, second = C::kStack && i >= DP;
    const int row = i % DP, col = half * NR;
    const uint32_t quad = tmem + ((uint32_t)(32 * q) << 16) + col;
    uint64_t R[NR / 2];   // pairs of columns
    {
      const float* src = STATE ? nullptr : a.segs > 1 ? jb.seg_init : jb.init;
      if (!STATE) wait_for_previous();   // for the segments' states; q, k, v, ... were there before them
      const float f0 = (a.segs > 1 || !jb.init_decays) ? 1.f : expf(ld);
      const size_t at = (a.segs > 1 ? (size_t)u * a.segs + seg : (size_t)u) * dd;
#pragma unroll
      for (int c = 0; c < NR; c += 4) {   // da and db are multiples of 8
        float4 r = make_float4(0, 0, 0, 0);
        if (src && !second && row < da && col + c < db) {
          const float* p = src + at + (trans ? (size_t)(col + c) * da + row : (size_t)row * db + col + c);
          r = trans ? make_float4(p[0], p[da], p[2 * da], p[3 * da]) : *reinterpret_cast<const float4*>(p);
        }
        R[c / 2] = f2(f0 * r.x, f0 * r.y);
        R[c / 2 + 1] = f2(f0 * r.z, f0 * r.w);
      }
    }
    Decay dec(ld * kC);
    auto update = [&](int k) {   // R after the chunk of step k
      const int c = chunk(k), tokens = valid(c) - (c == nch - 1 ? jb.fin_sub : 0);
      if (tokens < kC || k == 1) dec = Decay(ld * tokens);   // step 0 may have been the ragged one
      const uint64_t em = f2(dec.em, dec.em), mu = f2(dec.mul, dec.mul);
      wait(kDFull, k);
      tc_fence_after();
#pragma unroll
      for (int c0 = 0; c0 < NR; c0 += NT) {
        uint32_t d[NT];
        tmem_ld16_async(quad + C::kTd + c0, d);
        tmem_wait_ld16(d);
        if (c0 + NT == NR) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars + kDRead);
        }
#pragma unroll
        for (int e = 0; e < NT / 2; ++e) {
          const uint64_t r = R[c0 / 2 + e];
          R[c0 / 2 + e] = add2(fma2(em, r, mul2(mu, r)), f2(d[2 * e], d[2 * e + 1]));
        }
      }
    };
    const long long ts = jb.os[2];
    const bool wide = jb.wide;
    const float c_inter = jb.c_inter;
    const int left = db - col;
    __nv_bfloat16* o = STATE ? nullptr : jb.O + b * jb.os[0] + h * jb.os[1] + col + (long long)(chunk(0) * kC + i) * ts;
    const long long o_step = (rev ? -kC : kC) * ts;
    float f = STATE ? 0.f : c_inter * expf(ld * (rev ? kC - 1 - i : i));
    auto epilogue = [&](int k, auto last) {
      const int nv = valid(chunk(k));
      float fk = f;
      if (rev && nv < kC) fk = i < nv ? c_inter * expf(ld * (nv - 1 - i)) : 0.f;
      const uint64_t ff = f2(fk, fk);
      const uint32_t oz = quad + C::kToz, ox = oz + DP;
      wait(kOFull, k);
      tc_fence_after();
#pragma unroll
      for (int c0 = 0; c0 < NR; c0 += NT) {
        uint32_t z[NT], x[NT];
        tmem_ld16_async(oz + c0, z);
        tmem_ld16_async(ox + c0, x);
        tmem_wait_ld16(z);
        tmem_wait_ld16(x);
        if (c0 + NT == NR) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(bars + kOFree);
        }
#pragma unroll
        for (int g = 0; g < NT; g += 16) {
          uint32_t w[8];
          uint64_t nan = 0;   // stays zero unless an output is not finite
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint64_t v = fma2(ff, f2(x[g + 2 * e], x[g + 2 * e + 1]), f2(z[g + 2 * e], z[g + 2 * e + 1]));
            if (decltype(last)::value) nan = fma2(v, 0ull, nan);
            w[e] = packf2(v);
          }
          if (decltype(last)::value && i < nv && f2_lo(nan) + f2_hi(nan) != 0.f) *odd = 1;
          if (i < nv && c0 + g < left) {
            if (wide) {
              st_global_32(o + c0 + g, w);
            } else {
              *reinterpret_cast<uint4*>(o + c0 + g) = make_uint4(w[0], w[1], w[2], w[3]);
              if (c0 + g + 8 < left) *reinterpret_cast<uint4*>(o + c0 + g + 8) = make_uint4(w[4], w[5], w[6], w[7]);
            }
          }
        }
      }
      o += o_step;
    };
    for (int k = 0; k < n; ++k) {
      if (k > 0) update(k - 1);
      if (!STATE) {
        if (k > 0) wait(kXDone, k - 1);
#pragma unroll
        for (int g = 0; g < NR; g += 8) {
          const int cc = col + g;
          *reinterpret_cast<uint4*>(sm + C::kOffR + (second ? DP : cc >> 6 << 7) * 128 + sw128(row, (cc & 63) >> 3)) =
              make_uint4(packf2(R[g / 2]), packf2(R[g / 2 + 1]), packf2(R[g / 2 + 2]), packf2(R[g / 2 + 3]));
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bars + kRbReady);
        if (k > 0) epilogue(k - 1, std::false_type());
      }
    }
    if (!STATE) {
      epilogue(n - 1, std::true_type());
      named_bar_sync(2, 320);
      if (*odd) named_bar_sync(2, 320);   // before_odd needs the state that may be written in place
    }
    if (STATE || ends) {
      update(n - 1);
      float* dst = STATE ? jb.local + ((size_t)u * a.segs + seg) * dd : jb.fin + u * dd;
      if constexpr (C::kStack) {   // the second part's share, through the parts' memory: their last product is done
        float4* share = reinterpret_cast<float4*>(sm + C::kOffPart) + half * (DP * NR / 4) + row;
        if (second)
#pragma unroll
          for (int c = 0; c < NR; c += 4)
            share[c / 4 * DP] = make_float4(f2_lo(R[c / 2]), f2_hi(R[c / 2]), f2_lo(R[c / 2 + 1]), f2_hi(R[c / 2 + 1]));
        named_bar_sync(1, 256);
        if (!second)
#pragma unroll
          for (int c = 0; c < NR; c += 4) {
            const float4 v = share[c / 4 * DP];
            R[c / 2] = add2(R[c / 2], f2(v.x, v.y));
            R[c / 2 + 1] = add2(R[c / 2 + 1], f2(v.z, v.w));
          }
      }
      if (!second && row < da) {
#pragma unroll
        for (int c = 0; c < NR; c += 4)
          if (col + c < db)   // a returned state is never a transposed one
            *reinterpret_cast<float4*>(dst + (size_t)row * db + col + c) =
                make_float4(f2_lo(R[c / 2]), f2_hi(R[c / 2]), f2_lo(R[c / 2 + 1]), f2_hi(R[c / 2 + 1]));
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

// States before each segment from the segments' own sums, in place: st [jobs][units][segs][dd]. Reads and writes every
// state once; a few microseconds of launch and latency (8 units x 18 segments of 64 x 64: 7.7 us, 2.4 MB each way).
struct PrefixArgs {
  float* st;
  const float* init[2];   // state before the run (the forward's S0, the reverse run's dS_out), or null
  float* fin[2];          // state after it, from the last segment's own too, or null
  int fin_sub[2];
  int rev[2], init_decays[2];
  const float* log_decay;
  const int* lengths;
  int heads, N, segs, seg_chunks, dd;
};
__global__ void __launch_bounds__(64) k_decay_prefix(const __grid_constant__ PrefixArgs a) {
  const int u = blockIdx.x, j = blockIdx.z, e = (blockIdx.y * 64 + threadIdx.x) * 4;
  let_next_start();
  wait_for_previous();
  if (e >= a.dd) return;
  const int L = unit_length(a.lengths, u / a.heads, a.N), nch = (L + kC - 1) / kC;
  const int segs = (nch + a.seg_chunks - 1) / a.seg_chunks, span = a.seg_chunks * kC;
  const float ld = decay_log(a.log_decay[u % a.heads]);
  float* st = a.st + ((size_t)j * gridDim.x + u) * a.segs * a.dd + e;
  float4 r = make_float4(0, 0, 0, 0);
  if (a.init[j]) r = *reinterpret_cast<const float4*>(a.init[j] + (size_t)u * a.dd + e);
  if (a.init_decays[j] && segs > 0) {
    const float f = expf(ld);
    r.x *= f; r.y *= f; r.z *= f; r.w *= f;
  }
  const int sums = a.fin[j] ? segs : segs - 1;   // the run's last segment has a sum only for a state after it
  const long long step = a.rev[j] ? -(long long)a.dd : a.dd;
  float* from = a.rev[j] ? st + (size_t)(segs > 0 ? segs - 1 : 0) * a.dd : st;
  constexpr int kAhead = 8;   // segments read at once: the chain over them is arithmetic only
  for (int i0 = 0; i0 < segs; i0 += kAhead) {
    float4 own[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i0 + i < sums) own[i] = *reinterpret_cast<const float4*>(from + (i0 + i) * step);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i0 + i < segs) {
        const int p = a.rev[j] ? segs - 1 - i0 - i : i0 + i;
        *reinterpret_cast<float4*>(from + (i0 + i) * step) = r;
        if (i0 + i < sums) {
          const Decay dec(ld * (min(span, L - p * span) - (p == segs - 1 ? a.fin_sub[j] : 0)));
          r.x = dec(r.x) + own[i].x;
          r.y = dec(r.y) + own[i].y;
          r.z = dec(r.z) + own[i].z;
          r.w = dec(r.w) + own[i].w;
        }
      }
  }
  if (a.fin[j]) *reinterpret_cast<float4*>(a.fin[j] + (size_t)u * a.dd + e) = r;
}

bool maps(TcJob* t, const DecayArgs& a, const DecayJob& j, bool with_x) {
  if (with_x && !make_tmap_tokens_bf16(&t->x, j.X, j.da, a.N, a.heads, a.B, j.xs, kC)) return false;
  return make_tmap_tokens_bf16(&t->y, j.Y, j.da, a.N, a.heads, a.B, j.ys, kC) &&
         make_tmap_tokens_bf16(&t->z, j.Z, j.db, a.N, a.heads, a.B, j.zs, kC);
}

template <int DP, bool STATE, int PARTS>
cudaError_t run(const TcArgs& a, int units, int njobs, cudaStream_t st) {
  using C = Cfg<DP, STATE, PARTS>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = raise_smem(k_decay_tc<DP, STATE, PARTS>, C::kSmem, done);
  if (e != cudaSuccess) return e;
  const dim3 grid(units, a.segs, njobs);
  // A forward's blocks set up and read their first tokens while the states are joined (1 x 8 x 65536 tokens: 108 ->
  // 103 us). Not a backward's: three runs have more blocks than the states' two, and those that come up early on the
  // SMs left free cost more than they win (289 us, 253 one after the other).
  if (!STATE && a.segs > 1 && njobs == 1) return launch_next(k_decay_tc<DP, STATE, PARTS>, grid, C::kThreads, C::kSmem, st, a);
  k_decay_tc<DP, STATE, PARTS><<<grid, C::kThreads, C::kSmem, st>>>(a);
  return cudaGetLastError();
}
template <bool STATE>
cudaError_t run(const TcArgs& a, int dp, int parts, int units, int njobs, cudaStream_t st) {
  if (dp == 64) return parts == 2 ? run<64, STATE, 2>(a, units, njobs, st) : run<64, STATE, 3>(a, units, njobs, st);
  return parts == 2 ? run<128, STATE, 2>(a, units, njobs, st) : run<128, STATE, 3>(a, units, njobs, st);
}

}  // namespace

// How the sequences are cut. bf16: one CTA fills an SM, and fewer than 148 of them (units x runs) are cut so that about
// 148 run at once. A cut call takes 1.4 times as long for the chunks of its longest segment (the states' pass reads y and
// z too) and about five chunks more for two launches and the join: it has to win more than that. Forward, 1024 tokens:
// 8 units of 128 channels in 8 segments 23 us, uncut 29; 24 units in 4 segments 29.5 both; 40 units in 3 40, uncut 31;
// 512 tokens 22 and 18. 8 units of 2048 tokens x 64 in 16 segments 18 us, in 4 22, uncut 31; 70 units of 2048 x 64 in 2
// 35.5, uncut 32; 40 units of 2048 x 128 in 3 51, uncut 56.
// fp32: blocks (64 columns of a unit's run) are bound by arithmetic, and the states take it to 1.5 (backward 1.3) times.
// So fewer than 148 runs are cut, into about 592 segments in all, if uncut blocks would leave more than
// that idle. At more than 64 rows of the state one block fills an SM (dk = dv = 128, forward, 1024 tokens: 147 units
// uncut 652 us, cut 852; 64 units 328 and 415; 36 units x 2048 cut 476, uncut 647; backward 24 units x 2048 uncut 648,
// cut 815, 36 units 1150 cut, 1287 uncut). Below, two share one, and both together do a third more (64 units x 784
// tokens, dk = dv = 64: cut 94 us, uncut 151; 147 units of dk 32 uncut 102, cut 118).
DecaySplit decay_split(int B, int heads, int N, int dk, int dv, int njobs, int dtype) {
  const int nch = ceil_div(N, kC);
  const long long units = (long long)B * heads, runs = units * njobs;
  long long segs = 1;
  if (dtype == LFA_BF16) {
    if (runs < 148) segs = 148 / runs;
    segs = segs < nch ? segs : nch;
    if (7 * ceil_div(nch, (int)segs) + 25 >= 5 * nch) segs = 1;
  } else if (runs < 148) {
    // a forward's run has dk rows and dv columns; a backward's have dv, dv, dk rows and dk, dk, dv columns
    const bool bwd = njobs > 1;
    const int rows = bwd && dv > dk ? dv : dk, ck = ceil_div(dk, 64), cv = ceil_div(dv, 64);
    const long long blocks = units * (bwd ? 2 * ck + cv : cv);
    const long long whole = bwd ? units * (2 * ck * dv + cv * dk) / rows : blocks;   // as many of `rows` rows
    const long long full = rows > 64 ? (blocks + 147) / 148 * 148 : 196;
    if (bwd ? 13 * whole < 10 * full : 3 * whole < 2 * full) segs = 592 / runs;
    segs = segs < nch ? segs : nch;
  }
  if (segs < 1) segs = 1;
  DecaySplit s;
  s.seg_chunks = ceil_div(nch, (int)segs);
  s.segs = ceil_div(nch, s.seg_chunks);
  return s;
}
DecaySplit decay_split(const DecayArgs& a, int dtype) {
  const DecayJob& j = a.job[0];   // the forward's run, or dQ's with k in z's place
  return a.njobs > 1 ? decay_split(a.B, a.heads, a.N, j.db, j.da, a.njobs, dtype)
                     : decay_split(a.B, a.heads, a.N, j.da, j.db, a.njobs, dtype);
}

cudaError_t launch_prefix(const DecayArgs& a, const DecaySplit& sp, const PrefixRun* r, int n, cudaStream_t st) {
  PrefixArgs p;
  memset(&p, 0, sizeof(p));
  p.st = a.ws;
  for (int i = 0; i < n; ++i) {
    p.init[i] = r[i].init;
    p.rev[i] = r[i].rev;
    p.init_decays[i] = r[i].init_decays;
    p.fin[i] = r[i].fin;
    p.fin_sub[i] = r[i].fin_sub;
  }
  p.log_decay = a.log_decay;
  p.lengths = a.lengths;
  p.heads = a.heads;
  p.N = a.N;
  p.segs = sp.segs;
  p.seg_chunks = sp.seg_chunks;
  p.dd = a.job[0].da * a.job[0].db;
  return launch_next(k_decay_prefix, dim3(a.B * a.heads, ceil_div(p.dd, 256), n), 64, 0, st, p);
}

size_t decay_workspace_floats(int B, int heads, int N, int dk, int dv, int njobs, int dtype) {
  const DecaySplit s = decay_split(B, heads, N, dk, dv, njobs, dtype);
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
  const DecaySplit sp = decay_split(a, LFA_BF16);
  const int units = a.B * a.heads;
  TcArgs t;
  memset(&t, 0, sizeof(t));
  t.log_decay = a.log_decay;
  t.lengths = a.lengths;
  t.heads = a.heads;
  t.N = a.N;
  t.segs = sp.segs;
  t.seg_chunks = sp.seg_chunks;
  int dp = 64, parts = 2;   // three parts of y's decayed rows where a state is returned
  for (int i = 0; i < a.njobs; ++i) {
    const DecayJob& j = a.job[i];
    if (j.da > 64 || j.db > 64) dp = 128;
    if (j.fin) parts = 3;
  }
  const int dd = a.job[0].da * a.job[0].db;
  // states before the segments: run 0 forwards, and for the backward its last run (y = q, z = dO)
  const size_t states = (size_t)units * sp.segs * dd;
  if (sp.segs > 1) {
    DecayJob jobs[2];
    PrefixRun p[2];
    const int ns = state_runs(a, jobs, p);
    for (int i = 0; i < ns; ++i) {
      TcJob& o = t.job[i];
      if (!maps(&o, a, jobs[i], false)) return cudaErrorInvalidValue;
      o.da = jobs[i].da;
      o.db = jobs[i].db;
      o.rev = jobs[i].rev;
      o.c_state = jobs[i].c_state;
      o.local = a.ws + i * states;
      o.fin = p[i].fin = jobs[i].fin;
      o.fin_sub = jobs[i].fin ? jobs[i].fin_sub : 0;
      p[i].fin_sub = o.fin_sub;
      o.third = jobs[i].fin != nullptr;
    }
    cudaError_t e = run<true>(t, dp, parts, units, ns, st);
    if (e != cudaSuccess) return e;
    e = launch_prefix(a, sp, p, ns, st);
    if (e != cudaSuccess) return e;
  }
  for (int i = 0; i < a.njobs; ++i) {
    const DecayJob& j = a.job[i];
    TcJob& o = t.job[i];
    if (!maps(&o, a, j, true)) return cudaErrorInvalidValue;
    o.O = static_cast<__nv_bfloat16*>(j.O);
    memcpy(o.os, j.os, sizeof(o.os));
    o.X = static_cast<const __nv_bfloat16*>(j.X);
    o.Y = static_cast<const __nv_bfloat16*>(j.Y);
    o.Z = static_cast<const __nv_bfloat16*>(j.Z);
    memcpy(o.xs, j.xs, sizeof(o.xs));
    memcpy(o.ys, j.ys, sizeof(o.ys));
    memcpy(o.zs, j.zs, sizeof(o.zs));
    o.init = j.init;
    o.seg_init = a.ws + (i == 0 ? 0 : states);
    o.fin = sp.segs > 1 ? nullptr : j.fin;   // the join writes it
    o.third = o.fin != nullptr;
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
  return run<false>(t, dp, sp.segs > 1 ? 2 : parts, units, a.njobs, st);
}

}  // namespace lfa
