// Internal declarations of the token operators (decay attention, rotary positions, group norm): kernel
// argument blocks, filled by lfa_token_api.cu, and the launchers of lfa_decay.cu and lfa_token_ops.cu.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>

#include "lfa.h"

namespace lfa {

constexpr int kDecayChunk = 128;   // tokens per chunk of the prompt form; segments are whole chunks
constexpr int kDecayMaxD = 128;    // largest dk, dv

// One causal run over a unit's tokens: O_i = sum over j up to i of decay^(i-j) (x_i . y_j) z_j plus what the
// state from before contributes (rev: from the last token backwards). The carried state R is the sum of
// y_j z_j^T already decayed up to the token at hand: R = decay S_{t-1} (rev: decay G_{t+1}).
struct DecayJob {
  const void* X;
  const void* Y;
  const void* Z;
  void* O;
  long long xs[3], ys[3], zs[3], os[3];   // strides in elements: batch, head, token
  const float* init;    // [units][..] state before the run, or null (zero)
  float* fin;           // state after the run, or null
  int da, db;           // channels of X, Y and of Z, O
  int rev;              // runs from the last token to the first
  int trans;            // the state is stored [db][da] instead of [da][db]
  int init_decays;      // R_0 = decay^init_decays * init
  int fin_sub;          // fin is decay^-fin_sub times the R after the last token
  float c_inter, c_intra, c_state;   // factors of the state's part, of the chunk's own, of y z^T in the state
};

struct DecayArgs {
  int B, heads, N;
  const float* log_decay;   // [heads]
  const int* lengths;       // [B] or null
  float* ws;                // device workspace
  int njobs;
  DecayJob job[3];
};

// How a call's units are cut along the sequence: segs segments of seg_chunks chunks.
struct DecaySplit {
  int segs, seg_chunks;
};
DecaySplit decay_split(int B, int heads, int N, int dk, int dv, int njobs, int dtype);
DecaySplit decay_split(const DecayArgs& a, int dtype);
size_t decay_workspace_floats(int B, int heads, int N, int dk, int dv, int njobs, int dtype);

struct DecayStepArgs {
  int B, heads, dk, dv;
  const void* q;
  const void* k;
  const void* v;
  void* o;
  long long qs[2], ks[2], vs[2], os[2];   // batch, head
  const float* log_decay;
  float* S;
  const int* slots;
  int n_slots;
  float scale;
};

struct RotaryArgs {
  int B, N, d, rot, heads, heads2, interleaved, inverse;
  const void* x;
  const void* x2;
  void* y;
  void* y2;
  long long xs[3], x2s[3], ys[3], y2s[3];
  const int* positions;
  const double* freqs;
  float mscale;
};

struct NormArgs {
  int B, N, C, G, act;
  float eps;
  const void* x;
  const void* dy;
  void* y;          // forward output, or dx
  const float* gamma;
  const float* beta;
  float* mean;      // [B][G]
  float* rstd;
  float* dgamma;
  float* dbeta;
  float* ws;        // backward: channel sums
};

cudaError_t launch_decay(const DecayArgs& a, int dtype, cudaStream_t st);
// The end states of a call's segments, carried over the segments (in place in a.ws): initial state, direction, and
// where the state after the run goes, if the last segment's own state is there too.
struct PrefixRun {
  const float* init;
  float* fin;
  int rev, init_decays, fin_sub;
};
int state_runs(const DecayArgs& a, DecayJob* jobs, PrefixRun* p);
cudaError_t launch_prefix(const DecayArgs& a, const DecaySplit& sp, const PrefixRun* p, int n, cudaStream_t st);
cudaError_t launch_decay_tc(const DecayArgs& a, cudaStream_t st);
cudaError_t decay_take_status(int* out, cudaStream_t st);
cudaError_t launch_decay_step(const DecayStepArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_rotary(const RotaryArgs& a, int dtype, cudaStream_t st);
size_t norm_workspace_floats(int B, int N, int C, int G, int dtype, int backward);
cudaError_t launch_norm(const NormArgs& a, int dtype, cudaStream_t st);
cudaError_t launch_norm_backward(const NormArgs& a, int dtype, cudaStream_t st);

// the dynamic shared memory limit of a kernel, raised once per device; `done` is that kernel's own
template <typename K>
inline cudaError_t raise_smem(K kernel, int bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Kernels of one call that follow one another: the next one's blocks come up while the last of the one before run
// (which says when, with let_next_start) and wait for its end and its results in wait_for_previous.
template <typename... P, typename... A>
inline cudaError_t launch_next(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t c = {};
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  c.gridDim = grid;
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  c.attrs = &at;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, P(args)...);
}
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---- small device helpers shared by the two files -------------------------------------------------
// decays below exp(-1e4) are zero to every power but 0; the bound keeps 0 * inf out of exp(n ld)
__device__ __forceinline__ float decay_log(float ld) { return ld < -1e4f ? -1e4f : ld; }

// r exp(x), rounded once for x near 0 and to a relative few 2^-24 everywhere
struct Decay {
  float em, mul;
  __device__ explicit Decay(float x) : em(x > -0.5f ? expm1f(x) : 0.f), mul(x > -0.5f ? 1.f : expf(x)) {}
  __device__ __forceinline__ float operator()(float r) const { return fmaf(em, r, mul * r); }
};

__device__ __forceinline__ int unit_length(const int* lengths, int b, int N) {
  if (!lengths) return N;
  const int l = lengths[b];
  return l < 0 ? 0 : (l > N ? N : l);
}

template <typename T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ float from_f<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

}  // namespace lfa
