// Rotary positions (lfa_rotary) and group norm with an activation (lfa_group_norm and its backward).
#include "lfa_internal.h"
#include "lfa_token.h"

namespace lfa {
namespace {

// ---- rotary positions -------------------------------------------------------------------------------
// Pair i of a token at position p turns by th = p f_i: (a, b) -> mscale (a cos th - b sin th, a sin th + b cos th).
// th is reduced in turns in 64 bits (p f / 2 pi minus its nearest whole number), so that far positions keep
// their angle; the rest is fp32. A CTA takes kRT tokens: their cosines and sines are formed once in shared
// memory and serve every head.
constexpr int kRT = 16;        // tokens per CTA
constexpr int kRThreads = 256;
constexpr int kRMaxPairs = 64;

template <typename T>
struct Vec {
  static constexpr int n = 16 / sizeof(T);
  T v[n];
};
template <typename T>
__device__ __forceinline__ Vec<T> vload(const T* p) {
  Vec<T> r;
  *reinterpret_cast<uint4*>(r.v) = *reinterpret_cast<const uint4*>(p);
  return r;
}
template <typename T>
__device__ __forceinline__ void vstore(T* p, const Vec<T>& r) {
  *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(r.v);
}

// MODE 0: half layout, rot / 2 a whole number of 16-byte vectors; 1: interleaved; 2: half layout, any even rot
template <typename T, int MODE>
__global__ void __launch_bounds__(kRThreads) k_rotary(const __grid_constant__ RotaryArgs a) {
  __shared__ float2 cs[kRT][kRMaxPairs];
  constexpr int V = Vec<T>::n;
  const int tiles = (a.N + kRT - 1) / kRT;
  const int b = blockIdx.x / tiles, n0 = (blockIdx.x % tiles) * kRT, nt = min(kRT, a.N - n0);
  const int half = a.rot >> 1;
  for (int e = threadIdx.x; e < nt * half; e += kRThreads) {
    const int n = e / half, i = e % half;
    const double turns = (double)a.positions[(size_t)b * a.N + n0 + n] * (a.freqs[i] * 0.15915494309189533577);
    float sn, c;
    sincospif(2.f * (float)(turns - rint(turns)), &sn, &c);
    cs[n][i] = make_float2(a.mscale * c, a.inverse ? -a.mscale * sn : a.mscale * sn);
  }
  __syncthreads();
  const int rest = a.d - a.rot;
  const int units = MODE == 0 ? half / V + rest / V : (MODE == 1 ? a.d / V : half + rest);
  const int all = a.heads + a.heads2;
  for (int e = threadIdx.x; e < units * nt * all; e += kRThreads) {
    const int unit = e % units, n = (e / units) % nt, h = e / (units * nt);
    const bool second = h >= a.heads;
    const long long* si = second ? a.x2s : a.xs;
    const long long* so = second ? a.y2s : a.ys;
    const int hh = second ? h - a.heads : h;
    const T* x = static_cast<const T*>(second ? a.x2 : a.x) + b * si[0] + hh * si[1] + (n0 + n) * si[2];
    T* y = static_cast<T*>(second ? a.y2 : a.y) + b * so[0] + hh * so[1] + (n0 + n) * so[2];
    if (MODE == 0) {
      if (unit < half / V) {
        const Vec<T> p = vload(x + unit * V), q = vload(x + half + unit * V);
        Vec<T> po, qo;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const float2 w = cs[n][unit * V + i];
          const float u = to_f<T>(p.v[i]), v = to_f<T>(q.v[i]);
          po.v[i] = from_f<T>(u * w.x - v * w.y);
          qo.v[i] = from_f<T>(u * w.y + v * w.x);
        }
        vstore(y + unit * V, po);
        vstore(y + half + unit * V, qo);
      } else {
        const int c = a.rot + (unit - half / V) * V;
        vstore(y + c, vload(x + c));
      }
    } else if (MODE == 1) {
      Vec<T> p = vload(x + unit * V);
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const int c = unit * V + i;
        if (c < a.rot) {
          const float2 w = cs[n][c >> 1];
          const float u = to_f<T>(p.v[i]), v = to_f<T>(p.v[i + 1]);
          p.v[i] = from_f<T>(u * w.x - v * w.y);
          p.v[i + 1] = from_f<T>(u * w.y + v * w.x);
        }
      }
      vstore(y + unit * V, p);
    } else {
      if (unit < half) {
        const float2 w = cs[n][unit];
        const float u = to_f<T>(x[unit]), v = to_f<T>(x[unit + half]);
        y[unit] = from_f<T>(u * w.x - v * w.y);
        y[unit + half] = from_f<T>(u * w.y + v * w.x);
      } else {
        y[half + unit] = x[half + unit];
      }
    }
  }
}

template <typename T>
void run_rotary(const RotaryArgs& a, cudaStream_t st) {
  const int grid = a.B * ceil_div(a.N, kRT);
  if (a.interleaved)
    k_rotary<T, 1><<<grid, kRThreads, 0, st>>>(a);
  else if ((a.rot / 2) % Vec<T>::n == 0)
    k_rotary<T, 0><<<grid, kRThreads, 0, st>>>(a);
  else
    k_rotary<T, 2><<<grid, kRThreads, 0, st>>>(a);
}

// ---- group norm ---------------------------------------------------------------------------------------
constexpr int kNT = 256;

__device__ __forceinline__ float act_f(float z, int act) {
  if (act == LFA_ACT_SILU) return z / (1.f + expf(-z));
  if (act == LFA_ACT_GELU) return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
  return z;
}
__device__ __forceinline__ float act_slope(float z, int act) {
  if (act == LFA_ACT_SILU) {
    const float p = 1.f / (1.f + expf(-z));
    return p * fmaf(z, 1.f - p, 1.f);
  }
  if (act == LFA_ACT_GELU)
    return 0.5f * (1.f + erff(z * 0.70710678118654752f)) + z * 0.3989422804014327f * expf(-0.5f * z * z);
  return 1.f;
}

__device__ __forceinline__ float block_sum(float v) {
  __shared__ float s[kNT / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  float r = 0.f;
  for (int i = 0; i < kNT / 32; ++i) r += s[i];
  return r;
}

// one CTA per (sample, group): mean, then the variance about it, then the output
template <typename T>
__global__ void __launch_bounds__(kNT) k_norm(const __grid_constant__ NormArgs a) {
  const int b = blockIdx.x / a.G, g = blockIdx.x % a.G, dg = a.C / a.G;
  const long long n = (long long)a.N * dg;
  const T* x = static_cast<const T*>(a.x) + (size_t)b * a.N * a.C + g * dg;
  T* y = static_cast<T*>(a.y) + (size_t)b * a.N * a.C + g * dg;
  float s = 0.f;
  for (long long e = threadIdx.x; e < n; e += kNT) s += to_f<T>(x[e / dg * a.C + e % dg]);
  const float mean = block_sum(s) / (float)n;
  s = 0.f;
  for (long long e = threadIdx.x; e < n; e += kNT) {
    const float d = to_f<T>(x[e / dg * a.C + e % dg]) - mean;
    s = fmaf(d, d, s);
  }
  const float rstd = rsqrtf(block_sum(s) / (float)n + a.eps);
  for (long long e = threadIdx.x; e < n; e += kNT) {
    const int c = (int)(e % dg);
    const size_t at = (size_t)(e / dg) * a.C + c;
    float z = (to_f<T>(x[at]) - mean) * rstd;
    z = z * (a.gamma ? a.gamma[g * dg + c] : 1.f) + (a.beta ? a.beta[g * dg + c] : 0.f);
    y[at] = from_f<T>(act_f(z, a.act));
  }
  if (threadIdx.x == 0 && a.mean) {
    a.mean[blockIdx.x] = mean;
    a.rstd[blockIdx.x] = rstd;
  }
}

template <typename T>
__global__ void __launch_bounds__(kNT) k_norm_dx(const __grid_constant__ NormArgs a) {
  const int b = blockIdx.x / a.G, g = blockIdx.x % a.G, dg = a.C / a.G;
  const long long n = (long long)a.N * dg;
  const size_t base = (size_t)b * a.N * a.C + g * dg;
  const T* x = static_cast<const T*>(a.x) + base;
  const T* dy = static_cast<const T*>(a.dy) + base;
  T* dx = static_cast<T*>(a.y) + base;
  const float mean = a.mean[blockIdx.x], rstd = a.rstd[blockIdx.x];
  float s1 = 0.f, s2 = 0.f;
  for (int pass = 0; pass < 2; ++pass) {
    const float m1 = pass ? block_sum(s1) / (float)n : 0.f, m2 = pass ? block_sum(s2) / (float)n : 0.f;
    for (long long e = threadIdx.x; e < n; e += kNT) {
      const int c = (int)(e % dg);
      const size_t at = (size_t)(e / dg) * a.C + c;
      const float ga = a.gamma ? a.gamma[g * dg + c] : 1.f, be = a.beta ? a.beta[g * dg + c] : 0.f;
      const float xh = (to_f<T>(x[at]) - mean) * rstd;
      const float gz = ga * to_f<T>(dy[at]) * act_slope(fmaf(xh, ga, be), a.act);
      if (pass) {
        dx[at] = from_f<T>(rstd * (gz - m1 - xh * m2));
      } else {
        s1 += gz;
        s2 = fmaf(gz, xh, s2);
      }
    }
  }
}

// one CTA per channel
template <typename T>
__global__ void __launch_bounds__(kNT) k_norm_dparam(const __grid_constant__ NormArgs a) {
  const int c = blockIdx.x, g = c / (a.C / a.G);
  const float ga = a.gamma ? a.gamma[c] : 1.f, be = a.beta ? a.beta[c] : 0.f;
  float s1 = 0.f, s2 = 0.f;
  for (long long r = threadIdx.x; r < (long long)a.B * a.N; r += kNT) {
    const int b = (int)(r / a.N);
    const float xh = (to_f<T>(static_cast<const T*>(a.x)[r * a.C + c]) - a.mean[b * a.G + g]) * a.rstd[b * a.G + g];
    const float dz = to_f<T>(static_cast<const T*>(a.dy)[r * a.C + c]) * act_slope(fmaf(xh, ga, be), a.act);
    s1 += dz;
    s2 = fmaf(dz, xh, s2);
  }
  s1 = block_sum(s1);
  s2 = block_sum(s2);
  if (threadIdx.x == 0) {
    a.dbeta[c] = s1;
    a.dgamma[c] = s2;
  }
}

template <typename T>
void run_norm(const NormArgs& a, cudaStream_t st) {
  k_norm<T><<<a.B * a.G, kNT, 0, st>>>(a);
}
template <typename T>
void run_norm_backward(const NormArgs& a, cudaStream_t st) {
  if (a.dgamma) k_norm_dparam<T><<<a.C, kNT, 0, st>>>(a);   // first: dx may overwrite dy
  k_norm_dx<T><<<a.B * a.G, kNT, 0, st>>>(a);
}

}  // namespace

cudaError_t launch_rotary(const RotaryArgs& a, int dtype, cudaStream_t st) {
  if (dtype == LFA_BF16)
    run_rotary<__nv_bfloat16>(a, st);
  else
    run_rotary<float>(a, st);
  return cudaGetLastError();
}

size_t norm_workspace_floats(int, int, int, int, int) { return 64; }

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
