// Linear attention with a decay per head (lfa_decay_forward, lfa_decay_backward, lfa_decay_step).
//
// Per (batch, head) unit, S_t = l S_{t-1} + k_t v_t^T and o_t = scale q_t S_t with l = exp(log_decay). All of
// the prompt form and its backward are the same run (DecayJob) over other tensors:
//   o    : x = q,  y = k,  z = v,  first to last token, state [dk][dv]
//   dq   : x = dO, y = v,  z = k,  first to last, state transposed
//   dk   : x = v,  y = dO, z = q,  last to first, state G transposed
//   dv   : x = k,  y = q,  z = dO, last to first, state G [dk][dv] (its end is dS0)
// A run walks chunks of tokens: with R the carried state (already decayed to the chunk's first token),
//   O_i = c_inter l^i x_i R + c_intra sum_{j<=i} l^(i-j) (x_i . y_j) z_j,
//   R'  = l^n R + c_state sum_j l^(n-j) y_j z_j^T.
// Every power of l in use has an exponent >= 0, so nothing overflows however small l is. R is carried in fp32;
// with l near 1 the rounding of l^n would bias every chunk alike, so there l^n R is R + expm1(n log l) R.
#include "lfa_token.h"

#include "lfa_internal.h"

namespace lfa {
namespace {

// ---- CUDA-core run (fp32 arithmetic throughout) ------------------------------------------------------
constexpr int kCC = 32;          // tokens per step
constexpr int kCB = 64;          // columns of Z a CTA takes
constexpr int kCT = 256;
constexpr int kCStride = kDecayMaxD + 4;

struct CoreSmem {
  float X[kCC][kCStride];
  float Y[kCC][kCStride];
  float Z[kCC][kCB + 4];
  float P[kCC][kCC + 4];
  float R[kDecayMaxD][kCB + 4];
  float pw[kCC + 1];
};

template <typename T>
__device__ __forceinline__ float4 load4(const T* p);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p) { return *reinterpret_cast<const float4*>(p); }
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ void store4(T* p, float4 v);
template <>
__device__ __forceinline__ void store4<float>(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
template <>
__device__ __forceinline__ void store4<__nv_bfloat16>(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// grid: (units, column slices, jobs)
template <typename T>
__global__ void __launch_bounds__(kCT) k_decay_core(const __grid_constant__ DecayArgs a) {
  extern __shared__ float4 smem_f4[];
  CoreSmem& s = *reinterpret_cast<CoreSmem*>(smem_f4);
  const DecayJob& jb = a.job[blockIdx.z];
  const int c0 = blockIdx.y * kCB, u = blockIdx.x, b = u / a.heads, h = u % a.heads, t = threadIdx.x;
  if (c0 >= jb.db) return;
  const int da = jb.da, nb = min(kCB, jb.db - c0);
  const float ld = decay_log(a.log_decay[h]);
  const int L = unit_length(a.lengths, b, a.N);
  const T* X = static_cast<const T*>(jb.X) + b * jb.xs[0] + h * jb.xs[1];
  const T* Y = static_cast<const T*>(jb.Y) + b * jb.ys[0] + h * jb.ys[1];
  const T* Z = static_cast<const T*>(jb.Z) + b * jb.zs[0] + h * jb.zs[1] + c0;
  T* O = static_cast<T*>(jb.O) + b * jb.os[0] + h * jb.os[1] + c0;
  const size_t st0 = (size_t)u * da * jb.db;
  for (int n = t; n <= kCC; n += kCT) s.pw[n] = expf(ld * n);
  const float f0 = (L > 0 && jb.init_decays) ? expf(ld) : 1.f;
  for (int e = t; e < da * kCB; e += kCT) {
    const int r = e / kCB, c = e % kCB;
    float v = 0.f;
    if (jb.init && c < nb)
      v = f0 * jb.init[st0 + (jb.trans ? (size_t)(c0 + c) * da + r : (size_t)r * jb.db + c0 + c)];
    s.R[r][c] = v;
  }
  const int nch = (L + kCC - 1) / kCC;
  for (int ci = 0; ci < nch; ++ci) {
    const int t0 = (jb.rev ? nch - 1 - ci : ci) * kCC, nv = min(kCC, L - t0);
    __syncthreads();
    for (int e = t; e < kCC * (da >> 2); e += kCT) {
      const int r = e / (da >> 2), c = (e % (da >> 2)) * 4;
      const bool on = r < nv;
      *reinterpret_cast<float4*>(&s.X[r][c]) = on ? load4(X + (t0 + r) * jb.xs[2] + c) : make_float4(0, 0, 0, 0);
      *reinterpret_cast<float4*>(&s.Y[r][c]) = on ? load4(Y + (t0 + r) * jb.ys[2] + c) : make_float4(0, 0, 0, 0);
    }
    for (int e = t; e < kCC * (kCB / 4); e += kCT) {
      const int r = e / (kCB / 4), c = (e % (kCB / 4)) * 4;
      *reinterpret_cast<float4*>(&s.Z[r][c]) =
          (r < nv && c < nb) ? load4(Z + (t0 + r) * jb.zs[2] + c) : make_float4(0, 0, 0, 0);
    }
    __syncthreads();
    {   // P = c_intra decay^|i-j| x_i . y_j on the causal side
      const int i = t >> 3;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      for (int k = 0; k < da; k += 4) {
        const float4 x = *reinterpret_cast<const float4*>(&s.X[i][k]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 y = *reinterpret_cast<const float4*>(&s.Y[(t & 7) + 8 * q][k]);
          acc[q] = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, acc[q]))));
        }
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int j = (t & 7) + 8 * q, n = jb.rev ? j - i : i - j;
        s.P[i][j] = n >= 0 ? jb.c_intra * s.pw[n] * acc[q] : 0.f;
      }
    }
    __syncthreads();
    {
      const int i0 = 2 * (t >> 4), c = 4 * (t & 15);
      float4 acc[2] = {make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0)};
      for (int k = 0; k < da; k += 4) {
        const float4 x0 = *reinterpret_cast<const float4*>(&s.X[i0][k]), x1 = *reinterpret_cast<const float4*>(&s.X[i0 + 1][k]);
        const float xa[2][4] = {{x0.x, x0.y, x0.z, x0.w}, {x1.x, x1.y, x1.z, x1.w}};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 r = *reinterpret_cast<const float4*>(&s.R[k + q][c]);
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            acc[p].x = fmaf(xa[p][q], r.x, acc[p].x);
            acc[p].y = fmaf(xa[p][q], r.y, acc[p].y);
            acc[p].z = fmaf(xa[p][q], r.z, acc[p].z);
            acc[p].w = fmaf(xa[p][q], r.w, acc[p].w);
          }
        }
      }
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int n = jb.rev ? nv - 1 - (i0 + p) : i0 + p;
        const float f = n >= 0 ? jb.c_inter * s.pw[n] : 0.f;
        acc[p].x *= f; acc[p].y *= f; acc[p].z *= f; acc[p].w *= f;
      }
      for (int j = 0; j < kCC; ++j) {
        const float4 z = *reinterpret_cast<const float4*>(&s.Z[j][c]);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const float w = s.P[i0 + p][j];
          acc[p].x = fmaf(w, z.x, acc[p].x);
          acc[p].y = fmaf(w, z.y, acc[p].y);
          acc[p].z = fmaf(w, z.z, acc[p].z);
          acc[p].w = fmaf(w, z.w, acc[p].w);
        }
      }
#pragma unroll
      for (int p = 0; p < 2; ++p)
        if (i0 + p < nv && c < nb) store4(O + (t0 + i0 + p) * jb.os[2] + c, acc[p]);
    }
    __syncthreads();
    {   // R' = l^n R + c_state sum_j l^(n-j) y_j z_j^T (the run's last chunk: l^-fin_sub of that)
      const int sub = ci == nch - 1 ? jb.fin_sub : 0, c = 4 * (t & 15);
      const Decay dec(ld * (nv - sub));
      for (int r0 = 4 * (t >> 4); r0 < da; r0 += 64) {
        float acc[4][4] = {};
        for (int j = 0; j < nv; ++j) {
          const float w = jb.c_state * s.pw[(jb.rev ? j + 1 : nv - j) - sub];
          const float4 y = *reinterpret_cast<const float4*>(&s.Y[j][r0]);
          float4 z = *reinterpret_cast<const float4*>(&s.Z[j][c]);
          z.x *= w; z.y *= w; z.z *= w; z.w *= w;
          const float ya[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            acc[q][0] = fmaf(ya[q], z.x, acc[q][0]);
            acc[q][1] = fmaf(ya[q], z.y, acc[q][1]);
            acc[q][2] = fmaf(ya[q], z.z, acc[q][2]);
            acc[q][3] = fmaf(ya[q], z.w, acc[q][3]);
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float4* rp = reinterpret_cast<float4*>(&s.R[r0 + q][c]);
          float4 r = *rp;
          r.x = dec(r.x) + acc[q][0];
          r.y = dec(r.y) + acc[q][1];
          r.z = dec(r.z) + acc[q][2];
          r.w = dec(r.w) + acc[q][3];
          *rp = r;
        }
      }
    }
  }
  __syncthreads();
  if (jb.fin)
    for (int e = t; e < da * kCB; e += kCT) {
      const int r = e / kCB, c = e % kCB;
      if (c < nb) jb.fin[st0 + (jb.trans ? (size_t)(c0 + c) * da + r : (size_t)r * jb.db + c0 + c)] = s.R[r][c];
    }
}

// ---- one token --------------------------------------------------------------------------------------
// One CTA per (row, head): S [dk][dv] is read and written once, columns across the lanes (float4), rows across
// the warps; o = scale q S' from the warps' partial sums, joined in shared memory in a fixed order.
constexpr int kStepT = 256;

template <typename T>
__global__ void __launch_bounds__(kStepT) k_decay_step(const __grid_constant__ DecayStepArgs a) {
  __shared__ float q[kDecayMaxD], k[kDecayMaxD];
  __shared__ float4 part[kStepT / 32][32];
  __shared__ int dup;
  const int b = blockIdx.x / a.heads, h = blockIdx.x % a.heads, t = threadIdx.x, lane = t & 31, w = t >> 5;
  if (t == 0) dup = 0;
  __syncthreads();
  int slot = b;
  if (a.slots) {
    slot = a.slots[b];
    for (int i = t; i < b; i += kStepT)
      if (a.slots[i] == slot) dup = 1;
  }
  const T* qp = static_cast<const T*>(a.q) + b * a.qs[0] + h * a.qs[1];
  const T* kp = static_cast<const T*>(a.k) + b * a.ks[0] + h * a.ks[1];
  const T* vp = static_cast<const T*>(a.v) + b * a.vs[0] + h * a.vs[1];
  T* op = static_cast<T*>(a.o) + b * a.os[0] + h * a.os[1];
  for (int i = t; i < a.dk; i += kStepT) {
    q[i] = to_f<T>(qp[i]);
    k[i] = to_f<T>(kp[i]);
  }
  __syncthreads();
  const int c = 4 * lane;
  float4 o = make_float4(0, 0, 0, 0);
  if (slot >= 0 && slot < a.n_slots && !dup && c < a.dv) {
    const float l = expf(decay_log(a.log_decay[h]));
    const float4 v = load4(vp + c);
    float* S = a.S + ((size_t)slot * a.heads + h) * a.dk * a.dv + c;
    constexpr int W = kStepT / 32, U = 8;   // warps; rows a thread has in flight
    for (int r0 = w; r0 < a.dk; r0 += W * U) {
      float4 s[U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (r0 + i * W < a.dk) s[i] = *reinterpret_cast<const float4*>(S + (size_t)(r0 + i * W) * a.dv);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int r = r0 + i * W;
        if (r < a.dk) {
          s[i].x = fmaf(l, s[i].x, k[r] * v.x);
          s[i].y = fmaf(l, s[i].y, k[r] * v.y);
          s[i].z = fmaf(l, s[i].z, k[r] * v.z);
          s[i].w = fmaf(l, s[i].w, k[r] * v.w);
          *reinterpret_cast<float4*>(S + (size_t)r * a.dv) = s[i];
          o.x = fmaf(q[r], s[i].x, o.x);
          o.y = fmaf(q[r], s[i].y, o.y);
          o.z = fmaf(q[r], s[i].z, o.z);
          o.w = fmaf(q[r], s[i].w, o.w);
        }
      }
    }
  }
  part[w][lane] = o;
  __syncthreads();
  if (w == 0 && c < a.dv) {
    float4 r = part[0][lane];
    for (int i = 1; i < kStepT / 32; ++i) {
      r.x += part[i][lane].x;
      r.y += part[i][lane].y;
      r.z += part[i][lane].z;
      r.w += part[i][lane].w;
    }
    store4(op + c, make_float4(a.scale * r.x, a.scale * r.y, a.scale * r.z, a.scale * r.w));
  }
}

template <typename T>
cudaError_t run_core(const DecayArgs& a, cudaStream_t st) {
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = raise_smem(k_decay_core<T>, (int)sizeof(CoreSmem), done);
  if (e != cudaSuccess) return e;
  int db = 0;
  for (int j = 0; j < a.njobs; ++j) db = a.job[j].db > db ? a.job[j].db : db;
  k_decay_core<T><<<dim3(a.B * a.heads, ceil_div(db, kCB), a.njobs), kCT, sizeof(CoreSmem), st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decay(const DecayArgs& a, int dtype, cudaStream_t st) {
  return dtype == LFA_BF16 ? launch_decay_tc(a, st) : run_core<float>(a, st);
}

cudaError_t launch_decay_step(const DecayStepArgs& a, int dtype, cudaStream_t st) {
  if (dtype == LFA_BF16)
    k_decay_step<__nv_bfloat16><<<a.B * a.heads, kStepT, 0, st>>>(a);
  else
    k_decay_step<float><<<a.B * a.heads, kStepT, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace lfa
