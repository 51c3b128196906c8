// C-ABI entry points of the token operators (declared in include/lfa.h): validation and argument blocks.
#include <math.h>
#include <string.h>

#include "lfa_internal.h"
#include "lfa_token.h"

namespace {

using lfa::DecayArgs;
using lfa::DecayJob;

bool ok16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool ok16_or_null(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// What the size calls answer: 256 says that none is used, so a used one is larger however little it holds
size_t ws_bytes(size_t used) { return used == 0 ? 256 : 256 + (used + 255) / 256 * 256; }
bool ok_ws(const void* p, size_t bytes, size_t need) {
  return need <= 256 || (p && (reinterpret_cast<uintptr_t>(p) & 255u) == 0 && bytes >= need);
}
int elem(int dtype) { return dtype == LFA_BF16 ? 2 : 4; }

// Strides of a [B][heads][N][d] tensor: the caller's, or contiguous for three zeros. Dimensions of size 1 get
// a legal stride of their own. `out`: distinct elements must not share memory.
bool strides(const long long (&in)[3], int B, int heads, int N, int d, int dtype, bool out, long long* s) {
  const long long size[3] = {B, heads, N};
  if (in[0] == 0 && in[1] == 0 && in[2] == 0) {
    s[2] = d;
    s[1] = (long long)N * d;
    s[0] = s[1] * heads;
    return true;
  }
  const int v = 16 / elem(dtype);
  for (int i = 0; i < 3; ++i) {
    s[i] = size[i] == 1 ? (long long)(d + v - 1) / v * v : in[i];
    if (s[i] <= 0 || s[i] % v != 0 || s[i] >= (1ll << 37)) return false;
  }
  if (out) {   // from the smallest stride on, each must step over all that lies below it
    int o[3] = {0, 1, 2};
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2 - i; ++j)
        if (s[o[j]] > s[o[j + 1]]) { const int x = o[j]; o[j] = o[j + 1]; o[j + 1] = x; }
    long long span = d;
    for (int i = 0; i < 3; ++i) {
      if (size[o[i]] == 1) continue;
      if (s[o[i]] < span) return false;
      span += s[o[i]] * (size[o[i]] - 1);
    }
  }
  return true;
}

lfa_status check(const lfa_decay_config* c) {
  if (!c || c->B < 1 || c->heads < 1 || c->N < 1 || !isfinite(c->scale)) return LFA_ERR_INVALID_ARG;
  if (c->dtype != LFA_F32 && c->dtype != LFA_BF16) return LFA_ERR_UNSUPPORTED;
  const int v = 16 / elem(c->dtype);
  if (c->dk < 8 || c->dv < 8 || c->dk > lfa::kDecayMaxD || c->dv > lfa::kDecayMaxD) return LFA_ERR_UNSUPPORTED;
  if (c->dk % v != 0 || c->dv % v != 0) return LFA_ERR_UNSUPPORTED;
  if ((long long)c->B * c->heads > (1 << 24) || c->N > (1 << 28)) return LFA_ERR_UNSUPPORTED;
  return LFA_OK;
}

void set3(long long* to, const long long* from) { memcpy(to, from, 3 * sizeof(long long)); }

}  // namespace

extern "C" {

size_t lfa_decay_workspace_size(const lfa_decay_config* cfg, int backward) {
  if (check(cfg) != LFA_OK) return 0;
  const size_t n = 4 * lfa::decay_workspace_floats(cfg->B, cfg->heads, cfg->N, cfg->dk, cfg->dv, backward ? 3 : 1, cfg->dtype);
  return ws_bytes(n);
}

lfa_status lfa_decay_forward(const lfa_decay_config* c, const void* Q, const void* K, const void* V,
                             const float* log_decay, const float* S0, const int* lengths, void* O, float* S_out,
                             void* workspace, size_t workspace_bytes, void* stream) {
  const lfa_status st = check(c);
  if (st != LFA_OK) return st;
  if (!ok16(Q) || !ok16(K) || !ok16(V) || !ok16(O) || !log_decay || !ok16_or_null(S0) || !ok16_or_null(S_out))
    return LFA_ERR_INVALID_ARG;
  if (O == Q || O == K || O == V) return LFA_ERR_INVALID_ARG;
  if (!ok_ws(workspace, workspace_bytes, lfa_decay_workspace_size(c, 0))) return LFA_ERR_INVALID_ARG;
  DecayArgs a;
  memset(&a, 0, sizeof(a));
  DecayJob& j = a.job[0];
  if (!strides(c->q_stride, c->B, c->heads, c->N, c->dk, c->dtype, false, j.xs) ||
      !strides(c->k_stride, c->B, c->heads, c->N, c->dk, c->dtype, false, j.ys) ||
      !strides(c->v_stride, c->B, c->heads, c->N, c->dv, c->dtype, false, j.zs) ||
      !strides(c->o_stride, c->B, c->heads, c->N, c->dv, c->dtype, true, j.os))
    return LFA_ERR_INVALID_ARG;
  a.B = c->B;
  a.heads = c->heads;
  a.N = c->N;
  a.log_decay = log_decay;
  a.lengths = lengths;
  a.njobs = 1;
  a.ws = static_cast<float*>(workspace);
  j.X = Q;
  j.Y = K;
  j.Z = V;
  j.O = O;
  j.init = S0;
  j.fin = S_out;
  j.da = c->dk;
  j.db = c->dv;
  j.init_decays = 1;
  j.fin_sub = 1;
  j.c_inter = j.c_intra = c->scale;
  j.c_state = 1.f;
  return lfa::launch_decay(a, c->dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? LFA_OK : LFA_ERR_CUDA;
}

lfa_status lfa_decay_backward(const lfa_decay_config* c, const void* Q, const void* K, const void* V,
                              const float* log_decay, const float* S0, const int* lengths, const void* dO,
                              const float* dS_out, void* dQ, void* dK, void* dV, float* dS0, void* workspace,
                              size_t workspace_bytes, void* stream) {
  const lfa_status st = check(c);
  if (st != LFA_OK) return st;
  if (!ok16(Q) || !ok16(K) || !ok16(V) || !ok16(dO) || !ok16(dQ) || !ok16(dK) || !ok16(dV) || !log_decay ||
      !ok16_or_null(S0) || !ok16_or_null(dS_out) || !ok16_or_null(dS0))
    return LFA_ERR_INVALID_ARG;
  const void* ins[4] = {Q, K, V, dO};
  void* outs[3] = {dQ, dK, dV};
  for (int i = 0; i < 3; ++i) {
    for (int j = 0; j < 4; ++j)
      if (outs[i] == ins[j]) return LFA_ERR_INVALID_ARG;
    if (outs[i] == outs[(i + 1) % 3]) return LFA_ERR_INVALID_ARG;
  }
  if (dS0 && (dS0 == S0 || dS0 == dS_out)) return LFA_ERR_INVALID_ARG;
  if (!ok_ws(workspace, workspace_bytes, lfa_decay_workspace_size(c, 1))) return LFA_ERR_INVALID_ARG;
  long long qs[3], ks[3], vs[3], os[3];
  if (!strides(c->q_stride, c->B, c->heads, c->N, c->dk, c->dtype, true, qs) ||
      !strides(c->k_stride, c->B, c->heads, c->N, c->dk, c->dtype, true, ks) ||
      !strides(c->v_stride, c->B, c->heads, c->N, c->dv, c->dtype, true, vs) ||
      !strides(c->o_stride, c->B, c->heads, c->N, c->dv, c->dtype, false, os))
    return LFA_ERR_INVALID_ARG;
  DecayArgs a;
  memset(&a, 0, sizeof(a));
  a.B = c->B;
  a.heads = c->heads;
  a.N = c->N;
  a.log_decay = log_decay;
  a.lengths = lengths;
  a.njobs = 3;
  a.ws = static_cast<float*>(workspace);
  for (int i = 0; i < 3; ++i) {   // dQ, dK, dV
    DecayJob& j = a.job[i];
    j.X = i == 0 ? dO : i == 1 ? V : K;
    j.Y = i == 0 ? V : i == 1 ? dO : Q;
    j.Z = i == 0 ? K : i == 1 ? Q : dO;
    j.O = i == 0 ? dQ : i == 1 ? dK : dV;
    set3(j.xs, i == 0 ? os : i == 1 ? vs : ks);
    set3(j.ys, i == 0 ? vs : i == 1 ? os : qs);
    set3(j.zs, i == 0 ? ks : i == 1 ? qs : os);
    set3(j.os, i == 0 ? qs : i == 1 ? ks : vs);
    j.da = i == 2 ? c->dk : c->dv;
    j.db = i == 2 ? c->dv : c->dk;
    j.rev = i != 0;
    j.trans = i != 2;
    j.init = i == 0 ? S0 : dS_out;
    j.fin = i == 2 ? dS0 : nullptr;
    j.init_decays = i == 0;
    j.c_inter = i == 0 ? c->scale : 1.f;
    j.c_intra = c->scale;
    j.c_state = i == 0 ? 1.f : c->scale;
  }
  return lfa::launch_decay(a, c->dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? LFA_OK : LFA_ERR_CUDA;
}

lfa_status lfa_decay_step(const lfa_decay_config* c, const void* q, const void* k, const void* v,
                          const float* log_decay, float* S, const int* slots, int n_slots, void* o, void* stream) {
  const lfa_status st = check(c);
  if (st != LFA_OK) return st;
  if (c->N != 1 || n_slots < 1 || (!slots && n_slots < c->B)) return LFA_ERR_INVALID_ARG;
  if (!ok16(q) || !ok16(k) || !ok16(v) || !ok16(o) || !ok16(S) || !log_decay) return LFA_ERR_INVALID_ARG;
  long long s[4][3];
  if (!strides(c->q_stride, c->B, c->heads, 1, c->dk, c->dtype, false, s[0]) ||
      !strides(c->k_stride, c->B, c->heads, 1, c->dk, c->dtype, false, s[1]) ||
      !strides(c->v_stride, c->B, c->heads, 1, c->dv, c->dtype, false, s[2]) ||
      !strides(c->o_stride, c->B, c->heads, 1, c->dv, c->dtype, true, s[3]))
    return LFA_ERR_INVALID_ARG;
  lfa::DecayStepArgs a;
  memset(&a, 0, sizeof(a));
  a.B = c->B;
  a.heads = c->heads;
  a.dk = c->dk;
  a.dv = c->dv;
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  for (int i = 0; i < 2; ++i) {
    a.qs[i] = s[0][i];
    a.ks[i] = s[1][i];
    a.vs[i] = s[2][i];
    a.os[i] = s[3][i];
  }
  a.log_decay = log_decay;
  a.S = S;
  a.slots = slots;
  a.n_slots = n_slots;
  a.scale = c->scale;
  return lfa::launch_decay_step(a, c->dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? LFA_OK : LFA_ERR_CUDA;
}

lfa_status lfa_decay_status(void* stream) {
  int status = 0;
  if (lfa::decay_take_status(&status, static_cast<cudaStream_t>(stream)) != cudaSuccess) return LFA_ERR_CUDA;
  return status ? LFA_ERR_TIMEOUT : LFA_OK;
}

lfa_status lfa_rotary(const lfa_rotary_config* c, const void* x, const void* x2, const int* positions,
                      const double* freqs, void* y, void* y2, void* stream) {
  if (!c || c->B < 1 || c->N < 1 || c->heads < 1 || c->heads2 < 0 || !isfinite(c->mscale)) return LFA_ERR_INVALID_ARG;
  if (c->dtype != LFA_F32 && c->dtype != LFA_BF16) return LFA_ERR_UNSUPPORTED;
  if (c->d < 8 || c->d > 256 || c->d % (16 / elem(c->dtype)) != 0) return LFA_ERR_UNSUPPORTED;
  if (c->rot < 2 || c->rot % 2 != 0 || c->rot > c->d) return LFA_ERR_INVALID_ARG;
  if (c->rot > 128 || c->heads > 4096 || c->heads2 > 4096 || c->N > (1 << 28)) return LFA_ERR_UNSUPPORTED;
  if ((long long)c->B * c->N > (1ll << 30)) return LFA_ERR_UNSUPPORTED;
  if (!ok16(x) || !ok16(y) || !positions || !freqs) return LFA_ERR_INVALID_ARG;
  if (c->heads2 > 0 ? (!ok16(x2) || !ok16(y2)) : (x2 || y2)) return LFA_ERR_INVALID_ARG;
  lfa::RotaryArgs a;
  memset(&a, 0, sizeof(a));
  if (!strides(c->x_stride, c->B, c->heads, c->N, c->d, c->dtype, false, a.xs) ||
      !strides(c->y_stride, c->B, c->heads, c->N, c->d, c->dtype, true, a.ys))
    return LFA_ERR_INVALID_ARG;
  if (c->heads2 > 0 && (!strides(c->x2_stride, c->B, c->heads2, c->N, c->d, c->dtype, false, a.x2s) ||
                        !strides(c->y2_stride, c->B, c->heads2, c->N, c->d, c->dtype, true, a.y2s)))
    return LFA_ERR_INVALID_ARG;
  if (x == y && memcmp(a.xs, a.ys, sizeof(a.xs)) != 0) return LFA_ERR_INVALID_ARG;
  if (x2 && (y == y2 || y == x2 || y2 == x)) return LFA_ERR_INVALID_ARG;
  if (x2 && x2 == y2 && memcmp(a.x2s, a.y2s, sizeof(a.x2s)) != 0) return LFA_ERR_INVALID_ARG;
  a.B = c->B;
  a.N = c->N;
  a.d = c->d;
  a.rot = c->rot;
  a.heads = c->heads;
  a.heads2 = c->heads2;
  a.interleaved = c->interleaved != 0;
  a.inverse = c->inverse != 0;
  a.mscale = c->mscale;
  a.x = x;
  a.x2 = x2;
  a.y = y;
  a.y2 = y2;
  a.positions = positions;
  a.freqs = freqs;
  return lfa::launch_rotary(a, c->dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? LFA_OK : LFA_ERR_CUDA;
}

static lfa_status check_norm(const lfa_norm_config* c) {
  if (!c || c->B < 1 || c->N < 1 || c->C < 1 || c->groups < 1 || c->C % c->groups != 0) return LFA_ERR_INVALID_ARG;
  if (!(c->eps > 0.f) || !isfinite(c->eps)) return LFA_ERR_INVALID_ARG;
  if (c->act < LFA_ACT_NONE || c->act > LFA_ACT_GELU) return LFA_ERR_INVALID_ARG;
  if (c->dtype != LFA_F32 && c->dtype != LFA_BF16) return LFA_ERR_UNSUPPORTED;
  // row and (sample, group) counts, and one sample's elements, fit 30 bits
  if (c->C > (1 << 20)) return LFA_ERR_UNSUPPORTED;
  if ((long long)c->B * c->N > (1ll << 30) || (long long)c->B * c->groups > (1ll << 30) ||
      (long long)c->N * c->C > (1ll << 30))
    return LFA_ERR_UNSUPPORTED;
  return LFA_OK;
}

size_t lfa_group_norm_workspace_size(const lfa_norm_config* cfg, int backward) {
  if (check_norm(cfg) != LFA_OK) return 0;
  const size_t n = lfa::norm_workspace_floats(cfg->B, cfg->N, cfg->C, cfg->groups, cfg->dtype, backward) * sizeof(float);
  return ws_bytes(n);
}

lfa_status lfa_group_norm(const lfa_norm_config* c, const void* x, const float* gamma, const float* beta, void* y,
                          float* mean, float* rstd, void* workspace, size_t workspace_bytes, void* stream) {
  const lfa_status st = check_norm(c);
  if (st != LFA_OK) return st;
  if (!ok16(x) || !ok16(y) || (gamma == nullptr) != (beta == nullptr) || (mean == nullptr) != (rstd == nullptr))
    return LFA_ERR_INVALID_ARG;
  if (!ok_ws(workspace, workspace_bytes, lfa_group_norm_workspace_size(c, 0))) return LFA_ERR_INVALID_ARG;
  lfa::NormArgs a;
  memset(&a, 0, sizeof(a));
  a.B = c->B;
  a.N = c->N;
  a.C = c->C;
  a.G = c->groups;
  a.act = c->act;
  a.eps = c->eps;
  a.x = x;
  a.y = y;
  a.gamma = gamma;
  a.beta = beta;
  a.mean = mean;
  a.rstd = rstd;
  a.ws = static_cast<float*>(workspace);
  return lfa::launch_norm(a, c->dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? LFA_OK : LFA_ERR_CUDA;
}

lfa_status lfa_group_norm_backward(const lfa_norm_config* c, const void* x, const void* dy, const float* mean,
                                   const float* rstd, const float* gamma, const float* beta, void* dx, float* dgamma,
                                   float* dbeta, void* workspace, size_t workspace_bytes, void* stream) {
  const lfa_status st = check_norm(c);
  if (st != LFA_OK) return st;
  if (!ok16(x) || !ok16(dy) || !ok16(dx) || !mean || !rstd || (gamma == nullptr) != (beta == nullptr))
    return LFA_ERR_INVALID_ARG;
  if ((dgamma == nullptr) != (gamma == nullptr) || (dbeta == nullptr) != (gamma == nullptr)) return LFA_ERR_INVALID_ARG;
  if (!ok_ws(workspace, workspace_bytes, lfa_group_norm_workspace_size(c, 1))) return LFA_ERR_INVALID_ARG;
  lfa::NormArgs a;
  memset(&a, 0, sizeof(a));
  a.B = c->B;
  a.N = c->N;
  a.C = c->C;
  a.G = c->groups;
  a.act = c->act;
  a.eps = c->eps;
  a.x = x;
  a.dy = dy;
  a.y = dx;
  a.gamma = gamma;
  a.beta = beta;
  a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd);
  a.dgamma = dgamma;
  a.dbeta = dbeta;
  a.ws = static_cast<float*>(workspace);
  return lfa::launch_norm_backward(a, c->dtype, static_cast<cudaStream_t>(stream)) == cudaSuccess ? LFA_OK
                                                                                                  : LFA_ERR_CUDA;
}

}  // extern "C"
