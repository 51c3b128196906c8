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
#include <string.h>

#include "lfa_internal.h"
#include "lfa_token.h"

namespace lfa {
namespace {

// ---- fp32 tensors: the run on CUDA cores --------------------------------------------------------------
// A block takes CB columns of one segment of a unit's tokens and walks it 64 tokens at a time, everything staged in
// shared memory; the state R [da][CB] lives there. A thread has a 4 x 4 tile of each product, which makes 64
// multiply-adds per eight 16-byte reads; above the diagonal nothing is computed, by the rows of a warp.
// STATE: the segment's own state only. Bound by the fp32 multiply-adds and the shared-memory reads that feed them
// (64 units x 784 tokens, dk 32, dv 64: 65 us in three launches, issue slots half full, two blocks an SM; with three,
// at 80 registers, the backward took 245 instead of 192). Not taken: 32 columns a block (174 us), operands transposed
// for packed multiply-adds (75 us beside 58 in the main launch alone, when that was written).
constexpr int kCC = 64;   // tokens per step
constexpr int CB = 64;    // columns of z a block takes

template <int DA>
struct CoreSmem {
  float X[kCC][DA + 4];
  float Y[kCC][DA + 4];
  float Z[kCC][CB + 4];
  float P[kCC][kCC + 4];
  float R[DA][CB + 4];
  float pw[kCC + 1];
};

__device__ __forceinline__ void fma4(float4& a, float s, const float4& v) {
  a.x = fmaf(s, v.x, a.x);
  a.y = fmaf(s, v.y, a.y);
  a.z = fmaf(s, v.z, a.z);
  a.w = fmaf(s, v.w, a.w);
}
__device__ __forceinline__ float dot4(const float4& a, const float4& b, float c) {
  return fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, c))));
}
__device__ __forceinline__ float part(const float4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }

struct CoreArgs {
  DecayArgs a;
  int segs, seg_chunks;        // chunks of kDecayChunk tokens
  const float* seg_init[3];    // segs > 1: R at each segment's start, [units][segs]
  float* local[2];             // STATE: where the segments' own states go
};

template <int DA, bool STATE>
__global__ void __launch_bounds__(4 * CB, DA == 128 ? 1 : 2) k_decay_core(const __grid_constant__ CoreArgs ca) {
  extern __shared__ float4 smem_f4[];
  CoreSmem<DA>& s = *reinterpret_cast<CoreSmem<DA>*>(smem_f4);
  constexpr int NT = 4 * CB, TJ = CB / 4, NQ = kCC / TJ;
  const DecayArgs& a = ca.a;
  const int jx = blockIdx.z % a.njobs, seg = blockIdx.z / a.njobs;
  if (STATE) let_next_start();
  const DecayJob& jb = a.job[jx];
  const int c0 = blockIdx.y * CB, u = blockIdx.x, b = u / a.heads, h = u % a.heads, t = threadIdx.x;
  if (c0 >= jb.db) return;
  const int da = jb.da, nb = min(CB, jb.db - c0), L = unit_length(a.lengths, b, a.N);
  const bool rev = jb.rev;
  const int nch = (L + kDecayChunk - 1) / kDecayChunk;   // the sequence's chunks, in whole segments
  const int lo = seg * ca.seg_chunks, hi = min(lo + ca.seg_chunks, nch);
  if (hi <= lo && !(L == 0 && seg == 0 && !STATE)) return;
  if (STATE && (rev ? seg == 0 : hi == nch)) return;     // nothing follows this segment
  const bool ends = !STATE && jb.fin && (L == 0 || (rev ? seg == 0 : hi == nch));
  const int t_lo = lo * kDecayChunk, t_hi = min(L, hi * kDecayChunk), steps = (t_hi - t_lo + kCC - 1) / kCC;
  const float ld = decay_log(a.log_decay[h]);
  const float* X = static_cast<const float*>(jb.X) + b * jb.xs[0] + h * jb.xs[1];
  const float* Y = static_cast<const float*>(jb.Y) + b * jb.ys[0] + h * jb.ys[1];
  const float* Z = static_cast<const float*>(jb.Z) + b * jb.zs[0] + h * jb.zs[1] + c0;
  float* O = static_cast<float*>(jb.O) + b * jb.os[0] + h * jb.os[1] + c0;
  const size_t dd = (size_t)da * jb.db;
  for (int n = t; n <= kCC; n += NT) s.pw[n] = expf(ld * n);
  {
    const bool split = ca.segs > 1 && L > 0;
    const float* src = STATE ? nullptr : split ? ca.seg_init[jx] : jb.init;
    const size_t at = split ? ((size_t)u * ca.segs + seg) * dd : u * dd;
    const float f0 = L > 0 && !split && jb.init_decays ? expf(ld) : 1.f;
    if (!STATE) wait_for_previous();
    float4 v[DA * TJ / NT];   // read together
#pragma unroll
    for (int i = 0; i < DA * TJ / NT; ++i) {
      const int e = t + i * NT, r = e / TJ, c = e % TJ * 4;
      v[i] = make_float4(0, 0, 0, 0);
      if (src && r < da && c < nb) {
        const float* p = src + at + (jb.trans ? (size_t)(c0 + c) * da + r : (size_t)r * jb.db + c0 + c);
        v[i] = jb.trans ? make_float4(p[0], p[da], p[2 * da], p[3 * da]) : *reinterpret_cast<const float4*>(p);
      }
    }
#pragma unroll
    for (int i = 0; i < DA * TJ / NT; ++i) {
      const int e = t + i * NT;
      *reinterpret_cast<float4*>(&s.R[e / TJ][e % TJ * 4]) = make_float4(v[i].x * f0, v[i].y * f0, v[i].z * f0, v[i].w * f0);
    }
  }
  const int ti = t / TJ, tj = t % TJ, i0 = 4 * ti, cc = 4 * tj;
  const int w0 = (t & ~31) / TJ * 4, w1 = w0 + 128 / TJ;   // rows of this thread's warp
  constexpr int NX = kCC * DA / 4 / NT, NZ = kCC * CB / 4 / NT;   // 16-byte vectors of a thread
  float4 xr[STATE ? 1 : NX], yr[NX], zr[NZ];                      // the next step's, on their way
  auto start = [&](int si) { return t_lo + (rev ? steps - 1 - si : si) * kCC; };
  auto fetch = [&](int si) {
    const int t0 = start(si), nv = min(kCC, t_hi - t0);
    const float4 zero = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int e = t + i * NT, r = e / (DA / 4), c = e % (DA / 4) * 4;
      const bool on = r < nv && c < da;
      if (!STATE) xr[STATE ? 0 : i] = zero;
      yr[i] = zero;
      if (on) {
        if (!STATE) xr[STATE ? 0 : i] = *reinterpret_cast<const float4*>(X + (t0 + r) * jb.xs[2] + c);
        yr[i] = *reinterpret_cast<const float4*>(Y + (t0 + r) * jb.ys[2] + c);
      }
    }
#pragma unroll
    for (int i = 0; i < NZ; ++i) {
      const int e = t + i * NT, r = e / TJ, c = e % TJ * 4;
      zr[i] = zero;
      if (r < nv && c < nb) zr[i] = *reinterpret_cast<const float4*>(Z + (t0 + r) * jb.zs[2] + c);
    }
  };
  if (steps > 0) fetch(0);
  for (int si = 0; si < steps; ++si) {
    const int t0 = start(si), nv = min(kCC, t_hi - t0);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int e = t + i * NT, r = e / (DA / 4), c = e % (DA / 4) * 4;
      if (!STATE) *reinterpret_cast<float4*>(&s.X[r][c]) = xr[STATE ? 0 : i];
      *reinterpret_cast<float4*>(&s.Y[r][c]) = yr[i];
    }
#pragma unroll
    for (int i = 0; i < NZ; ++i) {
      const int e = t + i * NT, r = e / TJ, c = e % TJ * 4;
      *reinterpret_cast<float4*>(&s.Z[r][c]) = zr[i];
    }
    __syncthreads();
    if (si + 1 < steps) fetch(si + 1);
    if constexpr (!STATE) {
      if (w0 < nv) {   // (a warp's rows may all lie behind the end)
        {   // P = c_intra decay^|i-j| x_i . y_j on the causal side
          float acc[4][NQ] = {};
          for (int k = 0; k < da; k += 4) {
            float4 x[4];
#pragma unroll
            for (int p = 0; p < 4; ++p) x[p] = *reinterpret_cast<const float4*>(&s.X[i0 + p][k]);
#pragma unroll
            for (int q = 0; q < NQ; ++q) {
              if (rev ? TJ * q + TJ <= w0 : TJ * q >= w1) continue;   // wholly on the other side, for the warp
              const float4 y = *reinterpret_cast<const float4*>(&s.Y[tj + TJ * q][k]);
#pragma unroll
              for (int p = 0; p < 4; ++p) acc[p][q] = dot4(x[p], y, acc[p][q]);
            }
          }
#pragma unroll
          for (int q = 0; q < NQ; ++q) {
            if (rev ? TJ * q + TJ <= w0 : TJ * q >= w1) continue;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
              const int j = tj + TJ * q, n = rev ? j - i0 - p : i0 + p - j;
              s.P[i0 + p][j] = n >= 0 ? jb.c_intra * s.pw[n] * acc[p][q] : 0.f;
            }
          }
        }
        float4 acc[4] = {};
        for (int k = 0; k < da; k += 4) {
          float4 x[4], r[4];
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            x[p] = *reinterpret_cast<const float4*>(&s.X[i0 + p][k]);
            r[p] = *reinterpret_cast<const float4*>(&s.R[k + p][cc]);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int p = 0; p < 4; ++p) fma4(acc[p], part(x[p], q), r[q]);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const int n = rev ? nv - 1 - i0 - p : i0 + p;
          const float f = n >= 0 ? jb.c_inter * s.pw[n] : 0.f;
          acc[p] = make_float4(acc[p].x * f, acc[p].y * f, acc[p].z * f, acc[p].w * f);
        }
        __syncwarp();   // P's rows are used by the warp that wrote them
        // tokens j .. j + 3; z is zero behind the end. On the diagonal (j = i0) the other side's z is left out, not
        // multiplied by zero: it need not be finite
        auto add = [&](int j, auto on) {
          float4 w[4], z[4];
#pragma unroll
          for (int p = 0; p < 4; ++p) {
            w[p] = *reinterpret_cast<const float4*>(&s.P[i0 + p][j]);
            z[p] = *reinterpret_cast<const float4*>(&s.Z[j + p][cc]);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int p = 0; p < 4; ++p)
              if (on(p, q)) fma4(acc[p], part(w[p], q), z[q]);
        };
        const auto all = [](int, int) { return true; };
        static_assert(TJ == 16, "a warp has eight rows, two tiles of four");
        if (!rev) {
          for (int j = 0; j < w0; j += 4) add(j, all);
          if (i0 > w0) add(w0, all);
          add(i0, [](int p, int q) { return q <= p; });
        } else {
          add(i0, [](int p, int q) { return q >= p; });
          if (i0 == w0) add(w0 + 4, all);
          for (int j = w1; j < nv; j += 4) add(j, all);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p)
          if (i0 + p < nv && cc < nb) *reinterpret_cast<float4*>(O + (t0 + i0 + p) * jb.os[2] + cc) = acc[p];
      }
      __syncthreads();   // R has been read
    }
    {   // R' = l^n R + c_state sum_j l^(n-j) y_j z_j^T (the run's last step: l^-fin_sub of that)
      const int sub = !STATE && ends && !rev && si == steps - 1 ? jb.fin_sub : 0;
      const Decay dec(ld * (nv - sub));
      for (int r0 = 4 * ti; r0 < da; r0 += 64) {
        float4 acc[4] = {};
#pragma unroll 4
        for (int j = 0; j < nv; ++j) {
          const float w = jb.c_state * s.pw[(rev ? j + 1 : nv - j) - sub];
          const float4 y = *reinterpret_cast<const float4*>(&s.Y[j][r0]);
          float4 z = *reinterpret_cast<const float4*>(&s.Z[j][cc]);
          z = make_float4(z.x * w, z.y * w, z.z * w, z.w * w);
#pragma unroll
          for (int p = 0; p < 4; ++p) fma4(acc[p], part(y, p), z);
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          float4* rp = reinterpret_cast<float4*>(&s.R[r0 + p][cc]);
          const float4 r = *rp;
          *rp = make_float4(dec(r.x) + acc[p].x, dec(r.y) + acc[p].y, dec(r.z) + acc[p].z, dec(r.w) + acc[p].w);
        }
      }
    }
  }
  __syncthreads();
  if (STATE || ends) {
    float* dst = STATE ? ca.local[jx] + ((size_t)u * ca.segs + seg) * dd : jb.fin + u * dd;
    for (int e = t; e < da * TJ; e += NT) {
      const int r = e / TJ, c = e % TJ * 4;
      if (c < nb)   // a returned state is never a transposed one
        *reinterpret_cast<float4*>(dst + (size_t)r * jb.db + c0 + c) = *reinterpret_cast<const float4*>(&s.R[r][c]);
    }
  }
}

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

// ---- one token --------------------------------------------------------------------------------------
// One CTA per (row, head): S [dk][dv] is read and written once, columns across the lanes (float4), rows across
// the warps; o = scale q S' from the warps' partial sums, joined in shared memory in a fixed order. Bound by the
// state's bytes: 192 rows x 16 heads of 128 x 128 (406 MB) in 62.5 us, 6.5 TB/s, the copy bandwidth. A row's slot is
// compared with those of all rows before it, so that two rows never write one state.
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

template <int DA, bool STATE>
cudaError_t run_core(const CoreArgs& c, int db, cudaStream_t st) {
  constexpr int bytes = (int)sizeof(CoreSmem<DA>);
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = raise_smem(k_decay_core<DA, STATE>, bytes, done);
  if (e != cudaSuccess) return e;
  const dim3 grid(c.a.B * c.a.heads, ceil_div(db, CB), c.a.njobs * c.segs);
  if (!STATE && c.segs > 1) return launch_next(k_decay_core<DA, STATE>, grid, 4 * CB, bytes, st, c);
  k_decay_core<DA, STATE><<<grid, 4 * CB, bytes, st>>>(c);
  return cudaGetLastError();
}
template <bool STATE>
cudaError_t run_core(const CoreArgs& c, cudaStream_t st) {
  int da = 0, db = 0;
  for (int j = 0; j < c.a.njobs; ++j) {
    da = c.a.job[j].da > da ? c.a.job[j].da : da;
    db = c.a.job[j].db > db ? c.a.job[j].db : db;
  }
  return da <= 32 ? run_core<32, STATE>(c, db, st) : da <= 64 ? run_core<64, STATE>(c, db, st) : run_core<128, STATE>(c, db, st);
}

cudaError_t launch_core(const DecayArgs& a, cudaStream_t st) {
  const DecaySplit sp = decay_split(a, LFA_F32);
  CoreArgs c;
  memset(&c, 0, sizeof(c));
  c.a = a;
  c.segs = sp.segs;
  c.seg_chunks = sp.seg_chunks;
  if (sp.segs > 1) {
    CoreArgs s = c;
    PrefixRun p[2];
    s.a.njobs = state_runs(a, s.a.job, p);
    const size_t states = (size_t)a.B * a.heads * sp.segs * a.job[0].da * a.job[0].db;
    for (int i = 0; i < s.a.njobs; ++i) s.local[i] = a.ws + i * states;
    cudaError_t e = run_core<true>(s, st);
    if (e != cudaSuccess) return e;
    e = launch_prefix(a, sp, p, s.a.njobs, st);
    if (e != cudaSuccess) return e;
    for (int i = 0; i < a.njobs; ++i) c.seg_init[i] = a.ws + (i == 0 ? 0 : states);
  }
  return run_core<false>(c, st);
}

}  // namespace

// Runs whose end states are wanted segment by segment: the first one's and, in the backward, the last one's
// (y = q, z = dO; the other reverse run has the same state transposed). States are [dk][dv].
int state_runs(const DecayArgs& a, DecayJob* jobs, PrefixRun* p) {
  const int n = a.njobs > 1 ? 2 : 1;
  DecayJob run[2] = {a.job[0], a.job[a.njobs - 1]};
  for (int i = 0; i < n; ++i) {
    DecayJob j = run[i];
    if (j.trans) {   // the same sums with y and z exchanged
      const DecayJob o = j;
      j.Y = o.Z;
      j.Z = o.Y;
      memcpy(j.ys, o.zs, sizeof(j.ys));
      memcpy(j.zs, o.ys, sizeof(j.zs));
      j.da = o.db;
      j.db = o.da;
      j.trans = 0;
    }
    p[i].init = j.init;
    p[i].rev = j.rev;
    p[i].init_decays = j.init_decays;
    p[i].fin = nullptr;
    p[i].fin_sub = 0;
    jobs[i] = j;
  }
  return n;
}

cudaError_t launch_decay(const DecayArgs& a, int dtype, cudaStream_t st) {
  return dtype == LFA_BF16 ? launch_decay_tc(a, st) : launch_core(a, st);
}

cudaError_t launch_decay_step(const DecayStepArgs& a, int dtype, cudaStream_t st) {
  if (dtype == LFA_BF16)
    k_decay_step<__nv_bfloat16><<<a.B * a.heads, kStepT, 0, st>>>(a);
  else
    k_decay_step<float><<<a.B * a.heads, kStepT, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace lfa
