// Rotary positions (lfa_rotary) and group norm with an activation (lfa_group_norm and its backward).
#include <string.h>

#include <type_traits>

#include "lfa_internal.h"
#include "lfa_sm100.cuh"
#include "lfa_token.h"

namespace lfa {
namespace {

using sm100::add2;
using sm100::f2;
using sm100::f2_hi;
using sm100::f2_lo;
using sm100::fma2;
using sm100::mul2;

// Channels go in pairs: the packed fp32 instructions take two at a time.
__device__ __forceinline__ uint64_t both(float v) { return f2(v, v); }
// VB bytes of a row, and its elements in fp32
template <int VB>
struct Raw {
  uint32_t w[(VB + 3) / 4];
};
template <int VB>
__device__ __forceinline__ Raw<VB> raw_load(const void* p) {
  Raw<VB> r;
  if constexpr (VB == 16) *reinterpret_cast<uint4*>(r.w) = *reinterpret_cast<const uint4*>(p);
  if constexpr (VB == 8) *reinterpret_cast<uint2*>(r.w) = *reinterpret_cast<const uint2*>(p);
  if constexpr (VB == 4) r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  if constexpr (VB == 2) r.w[0] = *reinterpret_cast<const uint16_t*>(p);
  return r;
}
template <int VB>
__device__ __forceinline__ void raw_store(void* p, const Raw<VB>& r) {
  if constexpr (VB == 16) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(r.w);
  if constexpr (VB == 8) *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(r.w);
  if constexpr (VB == 4) *reinterpret_cast<uint32_t*>(p) = r.w[0];
  if constexpr (VB == 2) *reinterpret_cast<uint16_t*>(p) = (uint16_t)r.w[0];
}
template <typename T, int VB>
__device__ __forceinline__ float raw_get(const Raw<VB>& r, int i) {
  if constexpr (sizeof(T) == 4) return __uint_as_float(r.w[i]);
  return __uint_as_float((i & 1) ? (r.w[i >> 1] & 0xffff0000u) : (r.w[i >> 1] << 16));
}
// elements 2 i, 2 i + 1 (a single element has a zero beside it), and back
template <typename T, int VB>
__device__ __forceinline__ uint64_t raw_pair(const Raw<VB>& r, int i) {
  if constexpr (sizeof(T) == 4) return f2(r.w[2 * i], VB == 4 ? 0u : r.w[(2 * i + 1) % ((VB + 3) / 4)]);
  return f2(r.w[i] << 16, VB == 2 ? 0u : r.w[i] & 0xffff0000u);
}
template <typename T, int VB>
__device__ __forceinline__ Raw<VB> raw_make(const uint64_t* v) {
  Raw<VB> r;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < VB / 4; ++i) r.w[i] = (uint32_t)(v[i / 2] >> (32 * (i & 1)));
  } else if constexpr (VB == 2) {
    const __nv_bfloat16 b = __float2bfloat16_rn(f2_lo(v[0]));
    r.w[0] = *reinterpret_cast<const uint16_t*>(&b);
  } else {
#pragma unroll
    for (int i = 0; i < VB / 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f2_lo(v[i]), f2_hi(v[i]));
      r.w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
  }
  return r;
}
// ---- rotary positions -------------------------------------------------------------------------------
// Pair i of a token at position p turns by th = p f_i: (a, b) -> mscale (a cos th - b sin th, a sin th + b cos th).
// th is reduced in turns in 64 bits (p f / 2 pi minus its nearest whole number), so that far positions keep their
// angle; the rest is fp32. A thread has one token and one unit of a head's channels (V pairs in two 16-byte vectors,
// V / 2 pairs in one, or a single pair), forms their cosines and sines once, and goes over the heads.
// Bound by the bytes: 4 x 4096 tokens, 2 x 16 heads of 128 (268 MB) in 50 us, 5.4 TB/s, whether 64, 96 or 128 channels
// turn, in either layout; a plain copy of them takes 47. A half layout whose rot / 2 is no whole number of vectors goes
// element by element: 142 us (20 of 128 channels, bf16), 83 in fp32.
constexpr int kRThreads = 256;
constexpr int rotary_blocks(int mode) { return mode == 0 ? 3 : 5; }   // an SM at a time: 80 registers a thread, or 48
constexpr int kRHeads = 2;   // heads read at once, one such group ahead

__device__ __forceinline__ float2 turn(const RotaryArgs& a, double pos, int i) {
  const double turns = pos * (a.freqs[i] * 0.15915494309189533577);
  float sn, c;
  sincospif(2.f * (float)(turns - rint(turns)), &sn, &c);
  return make_float2(a.mscale * c, a.inverse ? -a.mscale * sn : a.mscale * sn);
}

// Units of a head's row. MODE 0: half layout, rot / 2 a whole number of vectors: the two vectors of V pairs, or two
// vectors to copy; 1: interleaved, a vector; 2: half layout, any even rot: a pair, or a channel to copy
template <typename T, int MODE>
__host__ __device__ __forceinline__ int rotary_units(int d, int rot) {
  constexpr int V = 16 / sizeof(T);
  return MODE == 0 ? rot / 2 / V + ((d - rot) / V + 1) / 2 : MODE == 1 ? d / V : rot / 2 + d - rot;
}

template <typename T, int MODE>
__global__ void __launch_bounds__(kRThreads, rotary_blocks(MODE)) k_rotary(const __grid_constant__ RotaryArgs a, int units, int tokens,
                                                      int heads_each) {
  constexpr int V = 16 / sizeof(T), NP = MODE == 0 ? V : MODE == 1 ? V / 2 : 1;   // pairs of a unit
  const int tl = threadIdx.x / units, unit = threadIdx.x - tl * units, tok = blockIdx.x * tokens + tl;
  if (tl >= tokens || tok >= a.B * a.N) return;
  const int half = a.rot >> 1;
  const int b = tok / a.N, n = tok - b * a.N;
  const int pair = unit * NP;   // the unit's first
  const bool turns = pair < half;
  // channels of the unit's first and second part
  const int cp = MODE == 1 ? unit * V : turns ? pair : MODE == 0 ? a.rot + (2 * unit - a.rot / V) * V : half + unit;
  const int cq = turns ? cp + half : cp + V;
  const bool two = MODE == 1 ? false : turns || (MODE == 0 && cq < a.d);
  const int all = a.heads + a.heads2;
  const int h0 = blockIdx.y * heads_each, h1 = min(h0 + heads_each, all);
  const T* const x1 = static_cast<const T*>(a.x) + b * a.xs[0] + n * a.xs[2];
  const T* const x2 = static_cast<const T*>(a.x2) + b * a.x2s[0] + n * a.x2s[2];
  T* const y1 = static_cast<T*>(a.y) + b * a.ys[0] + n * a.ys[2];
  T* const y2 = static_cast<T*>(a.y2) + b * a.y2s[0] + n * a.y2s[2];
  struct Group {
    Raw<16> p[kRHeads], q[kRHeads];
    T sp[kRHeads], sq[kRHeads];
  };
  auto load = [&](Group& g, int h) {
#pragma unroll
    for (int e = 0; e < kRHeads; ++e)
      if (h + e < h1) {
        const int k = h + e - a.heads;
        const T* x = k >= 0 ? x2 + k * a.x2s[1] : x1 + (h + e) * a.xs[1];
        if constexpr (MODE == 2) {
          g.sp[e] = x[cp];
          if (two) g.sq[e] = x[cq];
        } else {
          g.p[e] = raw_load<16>(x + cp);
          if (MODE == 0 && two) g.q[e] = raw_load<16>(x + cq);
        }
      }
  };
  Group cur, next;
  load(cur, h0);   // under way while the angles are formed
  float2 w[NP];
  if (turns) {
    const double pos = (double)a.positions[tok];
#pragma unroll
    for (int i = 0; i < NP; ++i) w[i] = pair + i < half ? turn(a, pos, pair + i) : make_float2(1.f, 0.f);
  }
  for (int h = h0; h < h1; h += kRHeads) {
    if (h + kRHeads < h1) load(next, h + kRHeads);
#pragma unroll
    for (int e = 0; e < kRHeads; ++e) {
      if (h + e >= h1) break;
      const int k = h + e - a.heads;
      T* y = k >= 0 ? y2 + k * a.y2s[1] : y1 + (h + e) * a.ys[1];
      if constexpr (MODE == 0) {
        if (turns) {
          uint64_t o[V / 2], r[V / 2];
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {
            const uint64_t u = raw_pair<T>(cur.p[e], i), v = raw_pair<T>(cur.q[e], i);
            const uint64_t cs = f2(w[2 * i].x, w[2 * i + 1].x), sn = f2(w[2 * i].y, w[2 * i + 1].y);
            o[i] = fma2(mul2(v, sn), both(-1.f), mul2(u, cs));
            r[i] = fma2(v, cs, mul2(u, sn));
          }
          cur.p[e] = raw_make<T, 16>(o);
          cur.q[e] = raw_make<T, 16>(r);
        }
        raw_store<16>(y + cp, cur.p[e]);
        if (two) raw_store<16>(y + cq, cur.q[e]);
      } else if constexpr (MODE == 1) {
        if (turns) {
          uint64_t o[V / 2];
#pragma unroll
          for (int i = 0; i < V / 2; ++i) {   // channels behind rot stay as they are, bit by bit
            const uint64_t u = raw_pair<T>(cur.p[e], i);
            o[i] = pair + i < half ? fma2(u, both(w[i].x), mul2(f2(f2_hi(u), f2_lo(u)), f2(-w[i].y, w[i].y))) : u;
          }
          cur.p[e] = raw_make<T, 16>(o);
        }
        raw_store<16>(y + cp, cur.p[e]);
      } else {
        if (turns) {
          const float u = to_f<T>(cur.sp[e]), v = to_f<T>(cur.sq[e]);
          y[cp] = from_f<T>(u * w[0].x - v * w[0].y);
          y[cq] = from_f<T>(u * w[0].y + v * w[0].x);
        } else {
          y[cp] = cur.sp[e];
        }
      }
    }
    cur = next;
  }
}

template <typename T, int MODE>
void rotary_launch(const RotaryArgs& a, cudaStream_t st) {
  const int units = rotary_units<T, MODE>(a.d, a.rot), tokens = kRThreads / units;   // units <= 256
  const int tiles = ceil_div(a.B * a.N, tokens), all = a.heads + a.heads2;
  // Heads are split over blocks, which form the angles once each (worth about three heads): as many parts as give
  // the shortest run of whole waves (half layout, 4 x 4096 tokens, 32 heads: one part 57 us in 1.5 waves, two 51 us
  // in 3).
  constexpr int kWave = rotary_blocks(MODE) * 148;
  int each = all;
  long long best = 0;
  for (int parts = 1; parts <= all; ++parts) {
    const int e = ceil_div(all, parts);
    const long long waves = ((long long)tiles * ceil_div(all, e) + kWave - 1) / kWave, cost = waves * (e + 3);
    if (best == 0 || cost < best) {
      best = cost;
      each = e;
    }
  }
  k_rotary<T, MODE><<<dim3(tiles, ceil_div(all, each)), kRThreads, 0, st>>>(a, units, tokens, each);
}
template <typename T>
void run_rotary(const RotaryArgs& a, cudaStream_t st) {
  if (a.interleaved)
    rotary_launch<T, 1>(a, st);
  else if ((a.rot / 2) % (16 / (int)sizeof(T)) == 0)
    rotary_launch<T, 0>(a, st);
  else
    rotary_launch<T, 2>(a, st);
}

// ---- group norm ---------------------------------------------------------------------------------------
// Two ways through the data. Small groups (N C/G elements that one warp or one block holds in registers) are read
// once: a team of threads per (sample, group) forms the mean, the variance about it and the output. Larger ones
// take three launches: per-channel sums of row chunks, their combination per group, and the output; the second
// reading comes from the 126 MB L2 as far as the tensor fits there. All sums are joined in a fixed order.
// Measured, bf16 with silu: 8192 x 1024 in 16 groups (33.6 MB) 13 us, of which a launch and four dependent rounds a
// warp are most; 65536 rows 56 us, 4.8 TB/s, where exponentials and reciprocals alone take 30 (without silu 46 us,
// the copy bandwidth), and backward 91 us (402 MB: 62; with the sums of dgamma and dbeta in a launch before: 169).
// Large, 32 x 3136 x 256 in 32 groups (51 MB a tensor): forward 42 us, sums 19 and output 20 of it; backward 56 us,
// sums 26, output 24. These wait for memory latency and the activation's two special-function instructions per element
// (half their pipe) in turn; the join is a few microseconds of latency, most of it under the neighbours (three launches
// apart: 49 and 64 us).
constexpr int kNT = 256;         // threads per block
constexpr int kNRows = 8;        // rows a thread has in flight
constexpr int kNormWave = 4 * 148;   // blocks that run at once
constexpr int kMaxChunks = 64;   // row chunks per sample (large groups)

// The activations, in pairs. p = 1 / (1 + exp(-z)) and q = 1 - p are formed from exp(-|z|), so that neither loses its
// small end, and p is within 2^-20 of itself down to fp32's last number. bf16 tensors, whose output keeps 2^-8, take p
// alone as ex2 of z log2 e rounded once, |z| 2^-24 relative, 0 below z = -87: two special-function instructions an
// element, which is what their rows wait for.
__device__ __forceinline__ float rcp_approx(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
// exp(-x) for x >= 0, within 2^-20: the square of ex2 of t = -x log2 e / 2, rounded, so that results below 2^-126 are
// left (the instruction has none), times exp of what t's rounding cut off. (0 from x = 104 on; x may be infinite.)
__device__ __forceinline__ uint64_t exp_minus2(uint64_t x) {
  x = f2(fminf(f2_lo(x), 200.f), fminf(f2_hi(x), 200.f));
  constexpr float kHalf = 0.72134752044448170f;   // log2 e / 2, and what fp32 leaves of it
  constexpr float kRest = (float)(0.72134752044448170 - (double)kHalf);
  const uint64_t t = mul2(x, both(-kHalf));
  const uint64_t cut = fma2(x, both(kRest), fma2(x, both(kHalf), t));   // minus what t lacks
  const uint64_t h = f2(sm100::ex2_approx(f2_lo(t)), sm100::ex2_approx(f2_hi(t)));
  return mul2(mul2(h, fma2(cut, both(-1.3862943611198906f), both(1.f))), h);
}
struct Pq {
  uint64_t p, q;
};
__device__ __forceinline__ Pq sigmoid_full2(uint64_t z) {
  const float a = f2_lo(z), b = f2_hi(z);
  const uint64_t e = exp_minus2(f2(fabsf(a), fabsf(b))), d = add2(e, both(1.f));
  const uint64_t r = f2(rcp_approx(f2_lo(d)), rcp_approx(f2_hi(d))), s = mul2(e, r);   // r in [1/2, 1]
  return Pq{f2(a < 0.f ? f2_lo(s) : f2_lo(r), b < 0.f ? f2_hi(s) : f2_hi(r)),
            f2(a < 0.f ? f2_lo(r) : f2_lo(s), b < 0.f ? f2_hi(r) : f2_hi(s))};
}
__device__ __forceinline__ uint64_t sigmoid2(uint64_t z) {
  const uint64_t t = mul2(z, both(-1.4426950408889634f));
  const uint64_t d = add2(f2(sm100::ex2_approx(f2_lo(t)), sm100::ex2_approx(f2_hi(t))), both(1.f));
  return f2(rcp_approx(f2_lo(d)), rcp_approx(f2_hi(d)));
}
// The normal distribution's integral and exp(-z^2 / 2). With a = |z|, the tail beyond a is m(a) exp(-a^2 / 2) with a
// smooth m, so it keeps its relative accuracy at any a (0.5 + 0.5 erf(z / sqrt 2) is off by more than half a step of
// bf16 from z = -4.3 on, of fp32 from z = -2.2). m = t (c0 + c1 t + ..), t = 1 / (1 + s a): the coefficients of least
// relative deviation for a <= 15, behind which the exponential is zero; degree 5 leaves 2^-16.6, degree 8 in fp32
// arithmetic 2^-21.5. 65536 x 1024 bf16 in 16 groups: 74 us; with erff 98, with erfcf 148.
struct Normal {
  uint64_t cdf, e;
};
template <typename T>
__device__ __forceinline__ Normal normal2(uint64_t z) {
  constexpr bool kFull = sizeof(T) == 4;
  constexpr int D = kFull ? 8 : 5;
  constexpr float c[2][9] = {{0.120041706f, 0.11409373f, 0.14278448f, -0.0143023f, 0.21370372f, -0.07631655f},
                             {0.13962126f, 0.13986428f, 0.119816035f, 0.10557231f, -0.0232571f, 0.1593819f, -0.2558912f,
                              0.14405517f, -0.029162677f}};
  const float zl = f2_lo(z), zh = f2_hi(z);
  const uint64_t d = fma2(f2(fabsf(zl), fabsf(zh)), both(kFull ? 0.35f : 0.3f), both(1.f));
  const uint64_t t = f2(rcp_approx(f2_lo(d)), rcp_approx(f2_hi(d)));
  Normal n;
  if constexpr (kFull) {
    n.e = exp_minus2(mul2(mul2(z, both(0.5f)), z));
  } else {
    const uint64_t w = mul2(mul2(z, z), both(-0.72134752044448170f));
    n.e = f2(sm100::ex2_approx(f2_lo(w)), sm100::ex2_approx(f2_hi(w)));
  }
  uint64_t m = both(c[kFull][D]);
#pragma unroll
  for (int i = D - 1; i >= 0; --i) m = fma2(m, t, both(c[kFull][i]));
  const uint64_t tail = mul2(mul2(m, t), n.e), rest = fma2(tail, both(-1.f), both(1.f));
  n.cdf = f2(zl < 0.f ? f2_lo(tail) : f2_lo(rest), zh < 0.f ? f2_hi(tail) : f2_hi(rest));
  return n;
}
template <typename T, int ACT>
__device__ __forceinline__ uint64_t act2(uint64_t z) {
  if (ACT == LFA_ACT_SILU) {
    if constexpr (sizeof(T) == 4) return mul2(z, sigmoid_full2(z).p);
    return mul2(z, sigmoid2(z));
  }
  if (ACT == LFA_ACT_GELU) return mul2(z, normal2<T>(z).cdf);
  return z;
}
template <typename T, int ACT>
__device__ __forceinline__ uint64_t slope2(uint64_t z) {
  if (ACT == LFA_ACT_SILU) {   // p + z p q
    if constexpr (sizeof(T) == 4) {
      const Pq s = sigmoid_full2(z);
      return fma2(mul2(z, s.q), s.p, s.p);
    }
    const uint64_t p = sigmoid2(z);
    return fma2(mul2(z, p), fma2(p, both(-1.f), both(1.f)), p);
  }
  if (ACT == LFA_ACT_GELU) {   // the integral and z times the density
    const Normal n = normal2<T>(z);
    return fma2(mul2(z, both(0.3989422804014327f)), n.e, n.cdf);
  }
  return both(1.f);
}

// V values from channel c on of an fp32 array (`none` without one), in pairs; a single one has a zero beside it
template <int V>
__device__ __forceinline__ void load_pairs(const float* p, int c, float none, uint64_t* o) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < (V + 1) / 2; ++i) o[i] = both(none);
    return;
  }
  p += c;
  if constexpr (V % 4 == 0) {
    if ((reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
#pragma unroll
      for (int i = 0; i < V / 4; ++i) {
        const float4 t = reinterpret_cast<const float4*>(p)[i];
        o[2 * i] = f2(t.x, t.y);
        o[2 * i + 1] = f2(t.z, t.w);
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < (V + 1) / 2; ++i) o[i] = f2(p[2 * i], 2 * i + 1 < V ? p[2 * i + 1] : 0.f);
}

// sum over a team of T lanes (a power of two up to 32), or with T = 0 over the block
template <bool BLOCK>
__device__ __forceinline__ float team_sum(float v, int T, float* s) {
  if constexpr (!BLOCK) {
    for (int o = T >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  } else {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    float r = 0.f;
#pragma unroll
    for (int i = 0; i < kNT / 32; ++i) r += s[i];
    return r;
  }
}

struct SmallArgs {
  NormArgs a;
  int T, dv, nvec;     // threads of a team (0: the block), vectors of a group in a row and in all
  uint32_t magic;      // j / dv = umulhi(j, magic) for dv > 1
  int blocks;          // of k_norm_rows (one vector a thread)
  float* part;         // its backward: channel sums [team / G][row of the group][2][C], or null
};

// Where a team's vector j lies: element offset from the group's first element, and its first channel in the group
template <typename T, int VB>
__device__ __forceinline__ void place(const SmallArgs& s, int j, long long& off, int& c) {
  constexpr int V = VB / sizeof(T);
  const int n = s.dv > 1 ? (int)__umulhi((uint32_t)j, s.magic) : j;
  c = (j - n * s.dv) * V;
  off = (long long)n * s.a.C + c;
}

template <typename T, int VB, int E, bool BLOCK, int ACT>
__global__ void __launch_bounds__(kNT) k_norm_small(const __grid_constant__ SmallArgs s) {
  __shared__ float red[kNT / 32];
  constexpr int V = VB / sizeof(T);
  const NormArgs& a = s.a;
  const int team = BLOCK ? kNT : s.T, tl = threadIdx.x & (team - 1);
  const long long id = BLOCK ? blockIdx.x : (long long)blockIdx.x * (kNT / s.T) + threadIdx.x / s.T;
  const bool on = id < (long long)a.B * a.G;
  const int b = on ? (int)(id / a.G) : 0, g = on ? (int)(id % a.G) : 0, dg = a.C / a.G;
  const size_t base = (size_t)b * a.N * a.C + g * dg;
  const T* x = static_cast<const T*>(a.x) + base;
  Raw<VB> v[E];
  float sum = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int j = tl + e * team;
    if (on && j < s.nvec) {
      long long off;
      int c;
      place<T, VB>(s, j, off, c);
      v[e] = raw_load<VB>(x + off);
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (on && tl + e * team < s.nvec)
#pragma unroll
      for (int i = 0; i < V; ++i) sum += raw_get<T>(v[e], i);
  const float n = (float)(s.nvec * V), mean = team_sum<BLOCK>(sum, s.T, red) / n;
  sum = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e)
    if (on && tl + e * team < s.nvec)
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const float d = raw_get<T>(v[e], i) - mean;
        sum = fmaf(d, d, sum);
      }
  const float rstd = rsqrtf(team_sum<BLOCK>(sum, s.T, red) / n + a.eps);
  if (!on) return;
  if (tl == 0 && a.mean) {
    a.mean[id] = mean;
    a.rstd[id] = rstd;
  }
  T* y = static_cast<T*>(a.y) + base;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int j = tl + e * team;
    if (j >= s.nvec) break;
    long long off;
    int c;
    place<T, VB>(s, j, off, c);
    constexpr int NP = (V + 1) / 2;
    uint64_t o[NP], ga[NP], be[NP];
    load_pairs<V>(a.gamma, g * dg + c, 1.f, ga);
    load_pairs<V>(a.beta, g * dg + c, 0.f, be);
#pragma unroll
    for (int i = 0; i < NP; ++i)
      o[i] = act2<T, ACT>(fma2(mul2(add2(raw_pair<T>(v[e], i), both(-mean)), both(rstd)), ga[i], be[i]));
    raw_store<VB>(y + off, raw_make<T, VB>(o));
  }
}

// The same for groups of one vector per thread (T a power of two): a thread keeps its channels over all the samples it
// takes (every teams-th (sample, group); teams is a multiple of G), U at once and the next U on their way; backward it
// sums its channels' dgamma and dbeta as it goes. (Twice the blocks, or U = 4 on three a SM, were slower: 8192 x 1024
// 16.6 and 17.3 us when this took 15.1, now 13.)
template <typename T, int VB, int ACT, bool BACKWARD>
__global__ void __launch_bounds__(kNT, BACKWARD ? 2 : 4) k_norm_rows(const __grid_constant__ SmallArgs s, int teams) {
  constexpr int V = VB / sizeof(T), U = 2;
  const NormArgs& a = s.a;
  const int shift = __ffs(s.T) - 1, tl = threadIdx.x & (s.T - 1), team = (int)((blockIdx.x * kNT + threadIdx.x) >> shift);
  const int total = a.B * a.G;   // up to 2^30, and teams up to 2^28
  const int b0 = team / a.G, g = team - b0 * a.G, dg = a.C / a.G;
  const bool has = tl < s.nvec;
  long long off;
  int c;
  place<T, VB>(s, has ? tl : 0, off, c);
  constexpr int NP = (V + 1) / 2;
  uint64_t ga[NP], be[NP];
  load_pairs<V>(a.gamma, g * dg + c, 1.f, ga);
  load_pairs<V>(a.beta, g * dg + c, 0.f, be);
  const float n = (float)(s.nvec * V), inv = 1.f / n;
  const bool two_power = (s.nvec * V & (s.nvec * V - 1)) == 0;   // 1 / n is exact
  const long long step = (long long)(teams / a.G) * a.N * a.C;   // elements from one sample of this thread to its next
  const long long at = (long long)b0 * a.N * a.C + g * dg + off;
  const T* x = static_cast<const T*>(a.x) + at;
  const T* dy = static_cast<const T*>(a.dy) + at;
  T* y = static_cast<T*>(a.y) + at;
  // lanes of the team (uniform: a block's threads stay together, whatever teams still have a sample)
  auto join = [&](float (&v)[U]) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      if (o < s.T)
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] += __shfl_xor_sync(0xffffffffu, v[u], o);
  };
  uint64_t sb[NP] = {}, sg[NP] = {};   // backward: this thread's share of dbeta and dgamma
  if (BACKWARD) let_next_start();
  Raw<VB> nv[U], nw[U];
  float nm[U], nr[U];
  auto load = [&](int id) {   // U samples, and on to the next; zeros where there is none
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int iu = id + u * teams;
      const bool on = iu < total;
#pragma unroll
      for (int i = 0; i < (VB + 3) / 4; ++i) nv[u].w[i] = nw[u].w[i] = 0u;
      if (on && has) {
        nv[u] = raw_load<VB>(x);
        if (BACKWARD) nw[u] = raw_load<VB>(dy);
      }
      if (BACKWARD) {
        nm[u] = on ? a.mean[iu] : 0.f;
        nr[u] = on ? a.rstd[iu] : 0.f;
      }
      x += step;
      dy += step;
    }
  };
  load(team);
  int id = team;
  for (int id0 = (int)(blockIdx.x * kNT) >> shift; id0 < total; id0 += U * teams, id += U * teams, y += U * step) {
    Raw<VB> v[U], w[U];
    float m[U], rs[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v[u] = nv[u];
      w[u] = nw[u];
      m[u] = nm[u];
      rs[u] = nr[u];
    }
    load(id + U * teams);   // the next ones, meanwhile
    if constexpr (!BACKWARD) {
      uint64_t d[U][NP];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint64_t t = 0;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          d[u][i] = raw_pair<T>(v[u], i);
          t = add2(t, d[u][i]);   // threads without a vector hold zeros
        }
        m[u] = f2_lo(t) + f2_hi(t);
      }
      join(m);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        m[u] = two_power ? m[u] * inv : __fdiv_rn(m[u], n);   // exact for constant groups
        uint64_t t = 0;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          d[u][i] = add2(d[u][i], V == 1 ? f2(-m[u], 0.f) : both(-m[u]));
          t = fma2(d[u][i], d[u][i], t);
        }
        rs[u] = has ? f2_lo(t) + f2_hi(t) : 0.f;
      }
      join(rs);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        rs[u] = rsqrtf(fmaf(rs[u], inv, a.eps));
        const int iu = id + u * teams;
        if (iu < total) {
          if (tl == 0 && a.mean) {
            a.mean[iu] = m[u];
            a.rstd[iu] = rs[u];
          }
          if (has) {
#pragma unroll
            for (int i = 0; i < NP; ++i) d[u][i] = act2<T, ACT>(fma2(mul2(d[u][i], both(rs[u])), ga[i], be[i]));
            raw_store<VB>(y + u * step, raw_make<T, VB>(d[u]));
          }
        }
      }
    } else {
      uint64_t d[U][NP], xh[U][NP];
      float s1[U], s2[U];
      // (samples there are none of have x = dy = 0, and so have threads without a vector)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        uint64_t t1 = 0, t2 = 0;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
          xh[u][i] = mul2(add2(raw_pair<T>(v[u], i), both(-m[u])), both(rs[u]));
          const uint64_t dz = mul2(raw_pair<T>(w[u], i), slope2<T, ACT>(fma2(xh[u][i], ga[i], be[i])));
          sb[i] = add2(sb[i], dz);
          sg[i] = fma2(dz, xh[u][i], sg[i]);
          d[u][i] = mul2(ga[i], dz);
          t1 = add2(t1, d[u][i]);   // dy is zero in threads without a vector and beside a lone channel
          t2 = fma2(d[u][i], xh[u][i], t2);
        }
        s1[u] = f2_lo(t1) + f2_hi(t1);
        s2[u] = f2_lo(t2) + f2_hi(t2);
      }
      join(s1);
      join(s2);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (has && id + u * teams < total) {
          const uint64_t m1 = both(-s1[u] * inv), m2 = both(-s2[u] * inv);
#pragma unroll
          for (int i = 0; i < NP; ++i) d[u][i] = mul2(both(rs[u]), fma2(xh[u][i], m2, add2(d[u][i], m1)));
          raw_store<VB>(y + u * step, raw_make<T, VB>(d[u]));
        }
    }
  }
  if (BACKWARD && s.part && has) {
    const int row = s.dv > 1 ? (int)__umulhi((uint32_t)tl, s.magic) : tl;
    float* o = s.part + ((size_t)b0 * a.N + row) * 2 * a.C + g * dg + c;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      o[i] = (i & 1) ? f2_hi(sb[i / 2]) : f2_lo(sb[i / 2]);
      o[a.C + i] = (i & 1) ? f2_hi(sg[i / 2]) : f2_lo(sg[i / 2]);
    }
  }
}

template <typename T, int VB, int E, bool BLOCK, int ACT>
__global__ void __launch_bounds__(kNT) k_norm_small_dx(const __grid_constant__ SmallArgs s) {
  __shared__ float red[kNT / 32];
  constexpr int V = VB / sizeof(T), NP = (V + 1) / 2;
  const NormArgs& a = s.a;
  const int team = BLOCK ? kNT : s.T, tl = threadIdx.x & (team - 1);
  const long long id = BLOCK ? blockIdx.x : (long long)blockIdx.x * (kNT / s.T) + threadIdx.x / s.T;
  const bool on = id < (long long)a.B * a.G;
  const int b = on ? (int)(id / a.G) : 0, g = on ? (int)(id % a.G) : 0, dg = a.C / a.G;
  const size_t base = (size_t)b * a.N * a.C + g * dg;
  const T* x = static_cast<const T*>(a.x) + base;
  const T* dy = static_cast<const T*>(a.dy) + base;
  const float mean = on ? a.mean[id] : 0.f, rstd = on ? a.rstd[id] : 0.f;
  Raw<VB> v[E], w[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int j = tl + e * team;
    if (on && j < s.nvec) {
      long long off;
      int c;
      place<T, VB>(s, j, off, c);
      v[e] = raw_load<VB>(x + off);
      w[e] = raw_load<VB>(dy + off);
    }
  }
  uint64_t t1 = 0, t2 = 0;
  auto grads = [&](int e, int c, uint64_t* d, uint64_t* xh) {
    uint64_t ga[NP], be[NP];
    load_pairs<V>(a.gamma, g * dg + c, 1.f, ga);
    load_pairs<V>(a.beta, g * dg + c, 0.f, be);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      xh[i] = mul2(add2(raw_pair<T>(v[e], i), both(-mean)), both(rstd));
      d[i] = mul2(mul2(ga[i], raw_pair<T>(w[e], i)), slope2<T, ACT>(fma2(xh[i], ga[i], be[i])));
    }
  };
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int j = tl + e * team;
    if (on && j < s.nvec) {
      long long off;
      int c;
      place<T, VB>(s, j, off, c);
      uint64_t d[NP], xh[NP];
      grads(e, c, d, xh);
#pragma unroll
      for (int i = 0; i < NP; ++i) {   // a lone channel's neighbour has dy = 0
        t1 = add2(t1, d[i]);
        t2 = fma2(d[i], xh[i], t2);
      }
    }
  }
  const float n = (float)(s.nvec * V);
  const float m1 = team_sum<BLOCK>(f2_lo(t1) + f2_hi(t1), s.T, red) / n;
  const float m2 = team_sum<BLOCK>(f2_lo(t2) + f2_hi(t2), s.T, red) / n;
  if (!on) return;
  T* dx = static_cast<T*>(a.y) + base;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int j = tl + e * team;
    if (j >= s.nvec) break;
    long long off;
    int c;
    place<T, VB>(s, j, off, c);
    uint64_t d[NP], xh[NP];
    grads(e, c, d, xh);
#pragma unroll
    for (int i = 0; i < NP; ++i) d[i] = mul2(both(rstd), fma2(xh[i], both(-m2), add2(d[i], both(-m1))));
    raw_store<VB>(dx + off, raw_make<T, VB>(d));
  }
}

// ---- large groups: rows in chunks, a thread takes the same V channels of every rl-th row -------------------
struct RowArgs {
  NormArgs a;
  int cw, rl, colblocks;     // vector columns and row lanes of a block, blocks side by side
  int chunks, chunk_rows;    // per sample, or over all rows (flat)
  float* part;               // [B or 1][chunks][2][C]
};
struct Lane {   // this thread's place
  int c, ty, b, r0, r1;
  bool on;
};
template <int V>
__device__ __forceinline__ Lane lane_of(const RowArgs& p, int rows) {
  Lane l;
  const int tx = threadIdx.x % p.cw, col = blockIdx.y * p.cw + tx;
  l.ty = threadIdx.x / p.cw;
  l.c = col * V;
  l.on = l.ty < p.rl && l.c < p.a.C;
  l.b = blockIdx.x / p.chunks;
  l.r0 = (blockIdx.x - l.b * p.chunks) * p.chunk_rows;
  l.r1 = min(l.r0 + p.chunk_rows, rows);
  return l;
}

// per-channel mean and sum of squares about it of a chunk's rows
template <typename T, int VB>
__global__ void __launch_bounds__(kNT) k_norm_stats(const __grid_constant__ RowArgs p) {
  constexpr int V = VB / sizeof(T);
  extern __shared__ float sm[];   // [rl][cw V] means, the same of squares
  const NormArgs& a = p.a;
  const Lane l = lane_of<V>(p, a.N);
  float m[V] = {}, q[V] = {};
  int cnt = 0;
  let_next_start();
  if (l.on) {
    const T* x = static_cast<const T*>(a.x) + (size_t)l.b * a.N * a.C + l.c;
    for (int r = l.r0 + l.ty; r < l.r1; r += p.rl * kNRows) {
      Raw<VB> v[kNRows];
      int k = 0;
#pragma unroll
      for (int e = 0; e < kNRows; ++e)
        if (r + e * p.rl < l.r1) {
          v[e] = raw_load<VB>(x + (size_t)(r + e * p.rl) * a.C);
          ++k;
        }
      // the block's mean and squares, joined to those so far (parallel form of the running variance)
      const float inv = 1.f / (float)k, fr = (float)k / (float)(cnt + k), wt = (float)cnt * fr;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < kNRows; ++e)
          if (e < k) s += raw_get<T>(v[e], i);
        s *= inv;
        float d2 = 0.f;
#pragma unroll
        for (int e = 0; e < kNRows; ++e)
          if (e < k) {
            const float d = raw_get<T>(v[e], i) - s;
            d2 = fmaf(d, d, d2);
          }
        const float d = s - m[i];
        q[i] += fmaf(d * d, wt, d2);
        m[i] = fmaf(d, fr, m[i]);
      }
      cnt += k;
    }
  }
  const int width = p.cw * V, at = l.ty * width + (threadIdx.x % p.cw) * V;
  float* sq = sm + p.rl * width;
  if (l.ty < p.rl)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      sm[at + i] = m[i];
      sq[at + i] = q[i];
    }
  __syncthreads();
  const int rows = l.r1 - l.r0;
  float* out = p.part + (size_t)blockIdx.x * 2 * a.C;
  for (int c = threadIdx.x; c < width; c += kNT) {
    const int ch = blockIdx.y * width + c;
    if (ch >= a.C) continue;
    float mean = 0.f, sqs = 0.f;
    int n = 0;
    for (int y = 0; y < p.rl && y < rows; ++y) {
      const int k = (rows - y + p.rl - 1) / p.rl;   // rows of lane y
      const float d = sm[y * width + c] - mean, fr = (float)k / (float)(n + k);
      sqs += sq[y * width + c] + d * d * (float)n * fr;
      mean = fmaf(d, fr, mean);
      n += k;
    }
    out[ch] = mean;
    out[a.C + ch] = sqs;
  }
}

// one block per (sample, group): mean and 1 / deviation from the chunks' channels
__global__ void __launch_bounds__(kNT) k_norm_group(const __grid_constant__ RowArgs p) {
  __shared__ float red[kNT / 32];
  const NormArgs& a = p.a;
  const int b = blockIdx.x / a.G, g = blockIdx.x % a.G, dg = a.C / a.G, cells = p.chunks * dg;
  const float* part = p.part + (size_t)b * p.chunks * 2 * a.C + g * dg;
  const float total = (float)a.N * (float)dg;
  let_next_start();
  wait_for_previous();
  float s = 0.f;
  for (int e = threadIdx.x; e < cells; e += kNT) {
    const int k = e / dg;
    s = fmaf(part[(size_t)k * 2 * a.C + e % dg], (float)(min(a.N, (k + 1) * p.chunk_rows) - k * p.chunk_rows), s);
  }
  const float mean = team_sum<true>(s, 0, red) / total;
  s = 0.f;
  for (int e = threadIdx.x; e < cells; e += kNT) {
    const int k = e / dg;
    const float* at = part + (size_t)k * 2 * a.C + e % dg;
    const float d = at[0] - mean;
    s += fmaf(d * d, (float)(min(a.N, (k + 1) * p.chunk_rows) - k * p.chunk_rows), at[a.C]);
  }
  s = team_sum<true>(s, 0, red);
  if (threadIdx.x == 0) {
    a.mean[blockIdx.x] = mean;
    a.rstd[blockIdx.x] = rsqrtf(s / total + a.eps);
  }
}

// the channels' constants of a thread, in pairs: minus the mean, 1 / deviation, gamma, beta
template <int V>
struct Chan {
  static constexpr int NP = (V + 1) / 2;
  uint64_t nm[NP], rs[NP], ga[NP], be[NP];
};
template <int V>
__device__ __forceinline__ void chan_affine(const NormArgs& a, int c, Chan<V>& k) {
  load_pairs<V>(a.gamma, c, 1.f, k.ga);
  load_pairs<V>(a.beta, c, 0.f, k.be);
}
// ONE: the V channels are of one group
template <int V, bool ONE>
__device__ __forceinline__ void chan_stats(const NormArgs& a, int b, int c, int dg, Chan<V>& k) {
  const size_t at = (size_t)b * a.G;
  if constexpr (ONE) {
    const uint64_t m = both(-a.mean[at + c / dg]), r = both(a.rstd[at + c / dg]);
#pragma unroll
    for (int i = 0; i < Chan<V>::NP; ++i) {
      k.nm[i] = m;
      k.rs[i] = r;
    }
  } else
#pragma unroll
  for (int i = 0; i < Chan<V>::NP; ++i) {
    const size_t g0 = at + (c + 2 * i) / dg, g1 = 2 * i + 1 < V ? at + (c + 2 * i + 1) / dg : g0;
    k.nm[i] = f2(-a.mean[g0], -a.mean[g1]);
    k.rs[i] = f2(a.rstd[g0], a.rstd[g1]);
  }
}

// A thread's next rows, kAhead of one or two tensors, on their way into slots of its own in shared memory: registers
// for them would cost blocks on the SM (32 x 3136 x 256, 32 groups: a backward with two rows of both tensors in
// registers 69.5 us, so 63.7; forward 51 and 49).
constexpr int kAhead = 4;
template <int VB>
__device__ __forceinline__ void stage_row(void* slot, const void* from) {
  if constexpr (VB == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sm100::smem_u32(slot)), "l"(from) : "memory");
  else if constexpr (VB >= 4)
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(sm100::smem_u32(slot)), "l"(from), "n"(VB) : "memory");
  else
    *reinterpret_cast<uint16_t*>(slot) = *reinterpret_cast<const uint16_t*>(from);
}
__device__ __forceinline__ void stage_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void stage_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// f(row, a's raw vector, b's) for the rows of this thread, in order (NB 1: a alone)
template <int VB, int NB, typename F>
__device__ __forceinline__ void for_rows(const Lane& l, int rl, int C, int es, const void* a, const void* b, float* sm, F f) {
  char* slots = reinterpret_cast<char*>(sm) + threadIdx.x * VB;
  const int first = l.r0 + l.ty;
  const size_t step = (size_t)rl * C * es;
  const char* pa = static_cast<const char*>(a) + (size_t)first * C * es;
  const char* pb = static_cast<const char*>(b) + (size_t)first * C * es;
  int ahead = first, in = 0, out = 0;   // next row to fetch, and the slots of fetching and reading
  auto fetch = [&]() {
    if (ahead < l.r1) {
      stage_row<VB>(slots + in * kNT * VB, pa);
      if (NB == 2) stage_row<VB>(slots + (kAhead + in) * kNT * VB, pb);
      pa += step;
      pb += step;
      ahead += rl;
    }
    stage_commit();
    in = (in + 1) % kAhead;
  };
#pragma unroll
  for (int i = 0; i < kAhead - 1; ++i) fetch();
  for (int r = first; r < l.r1; r += rl) {
    fetch();
    stage_wait<kAhead - 1>();
    const Raw<VB> va = raw_load<VB>(slots + out * kNT * VB);
    Raw<VB> vb = va;
    if (NB == 2) vb = raw_load<VB>(slots + (kAhead + out) * kNT * VB);
    out = (out + 1) % kAhead;
    f(r, va, vb);
  }
  stage_wait<0>();
}

template <typename T, int VB, int ACT, bool ONE>
__global__ void __launch_bounds__(kNT, ONE && ACT != LFA_ACT_GELU ? 4 : 2) k_norm_apply(const __grid_constant__ RowArgs p) {
  constexpr int V = VB / sizeof(T), NP = (V + 1) / 2;
  extern __shared__ float sm[];
  const NormArgs& a = p.a;
  const Lane l = lane_of<V>(p, a.N);
  if (!l.on) return;
  Chan<V> k;
  chan_affine(a, l.c, k);
  wait_for_previous();
  chan_stats<V, ONE>(a, l.b, l.c, a.C / a.G, k);
#pragma unroll
  for (int i = 0; i < NP; ++i) k.ga[i] = mul2(k.ga[i], k.rs[i]);
  const size_t base = (size_t)l.b * a.N * a.C + l.c;
  const T* x = static_cast<const T*>(a.x) + base;
  T* y = static_cast<T*>(a.y) + base;
  for_rows<VB, 1>(l, p.rl, a.C, sizeof(T), x, x, sm, [&](int r, const Raw<VB>& v, const Raw<VB>&) {
    uint64_t o[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) o[i] = act2<T, ACT>(fma2(add2(raw_pair<T>(v, i), k.nm[i]), k.ga[i], k.be[i]));
    raw_store<VB>(y + (size_t)r * a.C, raw_make<T, VB>(o));
  });
}

// per-channel sums of dz and dz xhat over a chunk's rows: of one sample, or (FLAT) of all samples' rows in turn
template <typename T, int VB, int ACT, bool ONE, bool FLAT>
__global__ void __launch_bounds__(kNT, ONE && ACT != LFA_ACT_GELU ? 4 : 2) k_norm_bsum(const __grid_constant__ RowArgs p) {
  constexpr int V = VB / sizeof(T);
  extern __shared__ float sm[];
  const NormArgs& a = p.a;
  const int dg = a.C / a.G;
  const Lane l = lane_of<V>(p, FLAT ? a.B * a.N : a.N);
  constexpr int NP = (V + 1) / 2;
  uint64_t s1[NP] = {}, s2[NP] = {};   // of dz, and of dz (x - mean) (FLAT: dz xhat)
  let_next_start();
  if (l.on) {
    Chan<V> k;
    chan_affine(a, l.c, k);
    if (!FLAT) {
      chan_stats<V, ONE>(a, l.b, l.c, dg, k);
#pragma unroll
      for (int i = 0; i < NP; ++i) k.ga[i] = mul2(k.ga[i], k.rs[i]);
    }
    const size_t base = (size_t)l.b * a.N * a.C + l.c;
    const T* x = static_cast<const T*>(a.x) + base;
    const T* dy = static_cast<const T*>(a.dy) + base;
    for_rows<VB, 2>(l, p.rl, a.C, sizeof(T), x, dy, sm, [&](int r, const Raw<VB>& v, const Raw<VB>& w) {
      if (FLAT) chan_stats<V, ONE>(a, r / a.N, l.c, dg, k);
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        uint64_t d = add2(raw_pair<T>(v, i), k.nm[i]);
        if (FLAT) d = mul2(d, k.rs[i]);
        const uint64_t dz = mul2(raw_pair<T>(w, i), slope2<T, ACT>(fma2(d, k.ga[i], k.be[i])));
        s1[i] = add2(s1[i], dz);
        s2[i] = fma2(dz, d, s2[i]);
      }
    });
    if (!FLAT)
#pragma unroll
      for (int i = 0; i < NP; ++i) s2[i] = mul2(s2[i], k.rs[i]);
  }
  const int width = p.cw * V, at = l.ty * width + (threadIdx.x % p.cw) * V;
  float* sq = sm + p.rl * width;
  __syncthreads();   // the rows' slots are done with
  if (l.ty < p.rl)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      sm[at + i] = (i & 1) ? f2_hi(s1[i / 2]) : f2_lo(s1[i / 2]);
      sq[at + i] = (i & 1) ? f2_hi(s2[i / 2]) : f2_lo(s2[i / 2]);
    }
  __syncthreads();
  float* out = p.part + (size_t)blockIdx.x * 2 * a.C;
  for (int c = threadIdx.x; c < width; c += kNT) {
    const int ch = blockIdx.y * width + c;
    if (ch >= a.C) continue;
    float t1 = 0.f, t2 = 0.f;
    for (int y = 0; y < p.rl; ++y) {
      t1 += sm[y * width + c];
      t2 += sq[y * width + c];
    }
    out[ch] = t1;
    out[a.C + ch] = t2;
  }
}

// Blocks below groups: m1, m2 of one (sample, group) from its channels' sums. The rest: dbeta, dgamma of 8
// channels, 32 lanes over the records.
__global__ void __launch_bounds__(kNT) k_norm_bjoin(const __grid_constant__ RowArgs p, int groups, int records,
                                                     float* m12) {
  __shared__ float red[2][kNT];
  const NormArgs& a = p.a;
  let_next_start();
  wait_for_previous();
  if ((int)blockIdx.x < groups) {
    const int b = blockIdx.x / a.G, g = blockIdx.x % a.G, dg = a.C / a.G, cells = p.chunks * dg;
    const float* part = p.part + (size_t)b * p.chunks * 2 * a.C + g * dg;
    float s1 = 0.f, s2 = 0.f;
    for (int e = threadIdx.x; e < cells; e += kNT) {
      const int k = e / dg, c = e % dg;
      const float ga = a.gamma ? a.gamma[g * dg + c] : 1.f;
      s1 = fmaf(ga, part[(size_t)k * 2 * a.C + c], s1);
      s2 = fmaf(ga, part[(size_t)k * 2 * a.C + a.C + c], s2);
    }
    const float n = (float)a.N * (float)dg;
    s1 = team_sum<true>(s1, 0, red[0]);
    s2 = team_sum<true>(s2, 0, red[1]);
    if (threadIdx.x == 0) {
      m12[2 * blockIdx.x] = s1 / n;
      m12[2 * blockIdx.x + 1] = s2 / n;
    }
  } else {
    const int cl = threadIdx.x & 7, c = ((int)blockIdx.x - groups) * 8 + cl, y = threadIdx.x >> 3;
    float s1 = 0.f, s2 = 0.f;
    if (c < a.C) {
#pragma unroll 8
      for (int r = y; r < records; r += kNT / 8) {
        s1 += p.part[(size_t)r * 2 * a.C + c];
        s2 += p.part[(size_t)r * 2 * a.C + a.C + c];
      }
    }
    red[0][threadIdx.x] = s1;
    red[1][threadIdx.x] = s2;
    __syncthreads();
    if (y == 0 && c < a.C) {
      for (int i = 1; i < kNT / 8; ++i) {
        s1 += red[0][8 * i + cl];
        s2 += red[1][8 * i + cl];
      }
      a.dbeta[c] = s1;
      a.dgamma[c] = s2;
    }
  }
}

template <typename T, int VB, int ACT, bool ONE>
__global__ void __launch_bounds__(kNT, ONE && ACT != LFA_ACT_GELU ? 4 : 2) k_norm_dx(const __grid_constant__ RowArgs p, const float* m12) {
  constexpr int V = VB / sizeof(T), NP = (V + 1) / 2;
  extern __shared__ float sm[];
  const NormArgs& a = p.a;
  const int dg = a.C / a.G;
  const Lane l = lane_of<V>(p, a.N);
  if (!l.on) return;
  Chan<V> k;
  chan_affine(a, l.c, k);
  chan_stats<V, ONE>(a, l.b, l.c, dg, k);
  wait_for_previous();
  uint64_t m1[NP], m2[NP];   // minus the group's means of gamma dz and of gamma dz xhat
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const size_t at = (size_t)l.b * a.G, g0 = 2 * (at + (l.c + (ONE ? 0 : 2 * i)) / dg),
                 g1 = ONE || 2 * i + 1 >= V ? g0 : 2 * (at + (l.c + 2 * i + 1) / dg);
    m1[i] = f2(-m12[g0], -m12[g1]);
    m2[i] = f2(-m12[g0 + 1], -m12[g1 + 1]);
  }
  const size_t base = (size_t)l.b * a.N * a.C + l.c;
  const T* x = static_cast<const T*>(a.x) + base;
  const T* dy = static_cast<const T*>(a.dy) + base;
  T* dx = static_cast<T*>(a.y) + base;
  for_rows<VB, 2>(l, p.rl, a.C, sizeof(T), x, dy, sm, [&](int r, const Raw<VB>& v, const Raw<VB>& w) {
    uint64_t o[NP];
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const uint64_t xh = mul2(add2(raw_pair<T>(v, i), k.nm[i]), k.rs[i]);
      const uint64_t d = mul2(mul2(k.ga[i], raw_pair<T>(w, i)), slope2<T, ACT>(fma2(xh, k.ga[i], k.be[i])));
      o[i] = mul2(k.rs[i], fma2(xh, m2[i], add2(d, m1[i])));
    }
    raw_store<VB>(dx + (size_t)r * a.C, raw_make<T, VB>(o));
  });
}

// ---- choice of the way, by sizes alone -----------------------------------------------------------------
// bytes of a vector: the widest power of two up to 16 that divides n elements
int vec_bytes(int n, int es) {
  int v = es;
  while (v < 16 && n % (2 * v / es) == 0) v *= 2;
  return v;
}

struct Plan {
  bool small;
  int VB, E;
  SmallArgs s;
  RowArgs r;           // large groups; small ones: the flat sums of the backward
  size_t floats;       // workspace
  size_t m12, stats;   // offsets in it
};

// Registers or three launches, by whether a warp's or block's team holds a group. Registers win forward wherever they
// hold it (2000 x 16 x 512 in 8 groups, bf16: 29 us, 81 in three launches; 500 x 64 x 512 in 16: 25 and 46). A backward
// with gamma has to read its rows again for the channels' sums, where dgamma and dbeta do not come from k_norm_rows.
// With samples of 64 bytes a channel and groups of 1.5 KB the three launches are the shorter way: bf16, N = 64 in 16
// groups 54 us, from registers 83, and N = 16 77 and 68; fp32, N = 16 in 8 groups 93 and 119, N = 4 138 and 118 (all
// 8.2 M elements); 1000 x 32 x 256 in 32 groups of 1 KB 79 and 62. Without gamma registers take 52 for the first.
Plan plan_norm(int B, int N, int C, int G, int es, bool backward, bool affine) {
  Plan p;
  memset(&p, 0, sizeof(p));
  const int dg = C / G;
  p.VB = vec_bytes(dg, es);
  const long long nvec = (long long)N * dg * es / p.VB;
  // a warp's team holds up to 8 vectors a thread (2 tensors: 4), a block's as well
  const int cap = backward ? 4 : 8;
  p.small = nvec <= (long long)kNT * cap;
  if (p.small) {
    p.s.dv = dg * es / p.VB;
    p.s.nvec = (int)nvec;
    p.s.magic = p.s.dv > 1 ? (uint32_t)(((1ull << 32) + p.s.dv - 1) / p.s.dv) : 0;
    if (nvec <= 32 * cap) {
      p.s.T = 1;
      while (p.s.T < 32 && p.s.T < nvec) p.s.T *= 2;
      p.E = nvec <= p.s.T ? 1 : cap;
    } else {
      p.s.T = 0;
      p.E = cap;
    }
  }
  RowArgs& r = p.r;
  if (p.small && p.E == 1) {   // k_norm_rows: at most one wave of blocks, with a number of teams that G divides
    const int per = kNT / p.s.T, wave = backward ? 2 * 148 : kNormWave;
    int unit = G;   // G / gcd(G, per)
    for (int d = per; d > 1; d /= 2)
      if (unit % 2 == 0) unit /= 2;
    const long long need = ((long long)B * G + per - 1) / per;
    // Many groups with few factors of two: more than a wave, or (backward) mostly records of channels that no sample
    // filled. These take the teams that know nothing of each other.
    if (unit <= wave && (!backward || unit <= need)) {
      const long long up = (need + unit - 1) / unit * unit;
      p.s.blocks = (int)(up <= wave ? up : wave / unit * unit);
      r.chunks = (int)((long long)p.s.blocks * per / G) * N;   // records of channel sums
      if (backward) p.floats = (size_t)r.chunks * 2 * C;
      return p;
    }
    p.E = cap;
  }
  if (p.small && backward && affine && N * es >= 64 && N * dg * es >= 1536) p.small = false;   // (p.small bounds N dg)
  // rows in chunks
  const int VB = p.small ? vec_bytes(C, es) : (p.VB = vec_bytes(C, es)), cv = C * es / VB;
  r.cw = cv <= 256 ? cv : 128;
  r.rl = kNT / r.cw;
  r.colblocks = ceil_div(cv, r.cw);
  const long long rows = p.small ? (long long)B * N : N;
  const int samples = p.small ? 1 : B;
  long long want = kNormWave / ((long long)samples * r.colblocks < kNormWave ? samples * r.colblocks : kNormWave);   // one wave
  const long long most = (rows + r.rl * kNRows - 1) / (r.rl * kNRows);
  if (want > most) want = most;
  if (want < 1) want = 1;
  if (!p.small && want > kMaxChunks) want = kMaxChunks;
  r.chunk_rows = (int)((rows + want - 1) / want);
  r.chunks = (int)((rows + r.chunk_rows - 1) / r.chunk_rows);
  if (!p.small || backward) p.floats = (size_t)samples * r.chunks * 2 * C;
  p.m12 = p.floats;
  if (!p.small && backward) p.floats += 2 * (size_t)B * G;
  p.stats = p.floats;
  if (!p.small && !backward) p.floats += 2 * (size_t)B * G;
  return p;
}

template <typename T, int VB, int ACT, bool BACKWARD>
void rows_launch(const Plan& p, cudaStream_t st) {
  k_norm_rows<T, VB, ACT, BACKWARD><<<p.s.blocks, kNT, 0, st>>>(p.s, p.s.blocks * (kNT / p.s.T));
}
template <typename T, int VB, int ACT>
void small_forward(const Plan& p, cudaStream_t st) {
  const long long teams = (long long)p.s.a.B * p.s.a.G;
  if (p.s.T == 0) {
    k_norm_small<T, VB, 8, true, ACT><<<(unsigned)teams, kNT, 0, st>>>(p.s);
  } else {
    const unsigned grid = (unsigned)((teams + kNT / p.s.T - 1) / (kNT / p.s.T));
    if (p.E == 1)
      rows_launch<T, VB, ACT, false>(p, st);
    else
      k_norm_small<T, VB, 8, false, ACT><<<grid, kNT, 0, st>>>(p.s);
  }
}
template <typename T, int VB, int ACT>
void small_backward(const Plan& p, cudaStream_t st) {
  const long long teams = (long long)p.s.a.B * p.s.a.G;
  if (p.s.T == 0) {
    k_norm_small_dx<T, VB, 4, true, ACT><<<(unsigned)teams, kNT, 0, st>>>(p.s);
  } else {
    const unsigned grid = (unsigned)((teams + kNT / p.s.T - 1) / (kNT / p.s.T));
    if (p.E == 1)
      rows_launch<T, VB, ACT, true>(p, st);
    else
      k_norm_small_dx<T, VB, 4, false, ACT><<<grid, kNT, 0, st>>>(p.s);
  }
}
template <typename T, int VB>
size_t row_smem(const RowArgs& r) { return 2 * sizeof(float) * r.rl * r.cw * (VB / sizeof(T)); }
template <typename T, int VB>
size_t ahead_smem(const RowArgs& r) {   // the rows' slots, and the sums that follow there
  const size_t slots = 2 * kAhead * kNT * VB, sums = row_smem<T, VB>(r);
  return slots > sums ? slots : sums;
}

template <typename T, int VB, int ACT>
void large_forward(const Plan& p, cudaStream_t st) {
  const RowArgs& r = p.r;
  const dim3 grid(r.chunks * r.a.B, r.colblocks);
  k_norm_stats<T, VB><<<grid, kNT, row_smem<T, VB>(r), st>>>(r);
  launch_next(k_norm_group, r.a.B * r.a.G, kNT, 0, st, r);
  if (r.a.C / r.a.G % (VB / sizeof(T)) == 0)
    launch_next(k_norm_apply<T, VB, ACT, true>, grid, kNT, kAhead * kNT * VB, st, r);
  else
    launch_next(k_norm_apply<T, VB, ACT, false>, grid, kNT, kAhead * kNT * VB, st, r);
}
template <typename T, int VB, int ACT, bool FLAT>
void channel_sums(const Plan& p, cudaStream_t st) {
  const RowArgs& r = p.r;
  const dim3 grid(r.chunks * (FLAT ? 1 : r.a.B), r.colblocks);
  if (r.a.C / r.a.G % (VB / sizeof(T)) == 0)
    k_norm_bsum<T, VB, ACT, true, FLAT><<<grid, kNT, ahead_smem<T, VB>(r), st>>>(r);
  else
    k_norm_bsum<T, VB, ACT, false, FLAT><<<grid, kNT, ahead_smem<T, VB>(r), st>>>(r);
  const int groups = FLAT ? 0 : r.a.B * r.a.G, chan = r.a.dgamma ? ceil_div(r.a.C, 8) : 0;
  launch_next(k_norm_bjoin, groups + chan, kNT, 0, st, r, groups, (FLAT ? 1 : r.a.B) * r.chunks, r.a.ws + p.m12);
}
template <typename T, int VB, int ACT>
void large_backward(const Plan& p, cudaStream_t st) {
  channel_sums<T, VB, ACT, false>(p, st);
  const dim3 grid(p.r.chunks * p.r.a.B, p.r.colblocks);
  if (p.r.a.C / p.r.a.G % (VB / sizeof(T)) == 0)
    launch_next(k_norm_dx<T, VB, ACT, true>, grid, kNT, ahead_smem<T, VB>(p.r), st, p.r, p.r.a.ws + p.m12);
  else
    launch_next(k_norm_dx<T, VB, ACT, false>, grid, kNT, ahead_smem<T, VB>(p.r), st, p.r, p.r.a.ws + p.m12);
}

// f.template operator()<T, VB, ACT>() for the vector's bytes and the activation
template <typename T, typename F>
void by_vec(int VB, int act, F f) {
  auto go = [&](auto vb) {
    constexpr int N = decltype(vb)::value;
    if constexpr (N >= (int)sizeof(T)) {
      if (act == LFA_ACT_SILU) f.template operator()<N, LFA_ACT_SILU>();
      else if (act == LFA_ACT_GELU) f.template operator()<N, LFA_ACT_GELU>();
      else f.template operator()<N, LFA_ACT_NONE>();
    }
  };
  if (VB == 16) go(std::integral_constant<int, 16>{});
  else if (VB == 8) go(std::integral_constant<int, 8>{});
  else if (VB == 4) go(std::integral_constant<int, 4>{});
  else go(std::integral_constant<int, 2>{});
}

template <typename T>
struct Forward {
  const Plan& p;
  cudaStream_t st;
  template <int VB, int ACT>
  void operator()() const {
    if (p.small) small_forward<T, VB, ACT>(p, st);
    else large_forward<T, VB, ACT>(p, st);
  }
};
template <typename T>
struct SmallDx {
  const Plan& p;
  cudaStream_t st;
  template <int VB, int ACT>
  void operator()() const { small_backward<T, VB, ACT>(p, st); }
};
template <typename T>
struct FlatSums {
  const Plan& p;
  cudaStream_t st;
  template <int VB, int ACT>
  void operator()() const { channel_sums<T, VB, ACT, true>(p, st); }
};
template <typename T>
struct LargeBackward {
  const Plan& p;
  cudaStream_t st;
  template <int VB, int ACT>
  void operator()() const { large_backward<T, VB, ACT>(p, st); }
};

template <typename T>
void run_norm(const NormArgs& a, cudaStream_t st) {
  Plan p = plan_norm(a.B, a.N, a.C, a.G, sizeof(T), false, a.gamma != nullptr);
  p.s.a = p.r.a = a;
  p.r.part = a.ws;
  if (!p.small && !a.mean) {
    p.r.a.mean = a.ws + p.stats;
    p.r.a.rstd = p.r.a.mean + (size_t)a.B * a.G;
  }
  by_vec<T>(p.VB, a.act, Forward<T>{p, st});
}
template <typename T>
void run_norm_backward(const NormArgs& a, cudaStream_t st) {
  Plan p = plan_norm(a.B, a.N, a.C, a.G, sizeof(T), true, a.gamma != nullptr);
  p.s.a = p.r.a = a;
  p.r.part = a.ws;
  if (!p.small) {
    by_vec<T>(p.VB, a.act, LargeBackward<T>{p, st});
    return;
  }
  if (p.E == 1) {   // dx's threads keep their channels over all samples, and sum dgamma and dbeta on the way
    if (a.dgamma) p.s.part = a.ws;
    by_vec<T>(p.VB, a.act, SmallDx<T>{p, st});
    if (a.dgamma) launch_next(k_norm_bjoin, ceil_div(a.C, 8), kNT, 0, st, p.r, 0, p.r.chunks, (float*)nullptr);
    return;
  }
  if (a.dgamma) by_vec<T>(vec_bytes(a.C, sizeof(T)), a.act, FlatSums<T>{p, st});   // before dx, which may overwrite dy
  by_vec<T>(p.VB, a.act, SmallDx<T>{p, st});
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int dtype, cudaStream_t st) {
  if (dtype == LFA_BF16)
    run_rotary<__nv_bfloat16>(a, st);
  else
    run_rotary<float>(a, st);
  return cudaGetLastError();
}

size_t norm_workspace_floats(int B, int N, int C, int G, int dtype, int backward) {
  const int es = dtype == LFA_BF16 ? 2 : 4;
  const size_t with = plan_norm(B, N, C, G, es, backward != 0, true).floats;
  const size_t without = plan_norm(B, N, C, G, es, backward != 0, false).floats;
  return with > without ? with : without;
}

cudaError_t launch_norm(const NormArgs& a, int dtype, cudaStream_t st) {
  if (dtype == LFA_BF16)
    run_norm<__nv_bfloat16>(a, st);
  else
    run_norm<float>(a, st);
  return cudaGetLastError();
}

cudaError_t launch_norm_backward(const NormArgs& a, int dtype, cudaStream_t st) {
  if (dtype == LFA_BF16)
    run_norm_backward<__nv_bfloat16>(a, st);
  else
    run_norm_backward<float>(a, st);
  return cudaGetLastError();
}

}  // namespace lfa
