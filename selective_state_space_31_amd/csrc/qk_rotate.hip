// qk_rotate.hip -- the norm of queries and keys for each head with the
// position rotation in the same pass, and its gradients, behind the C ABI in
// include/ssm_recurrent.h.
//
//   n = v rstd w, rstd = 1 / sqrt(mean(v^2) + eps); pairs (p, q) of n turn by
//   theta = position * inv_freq.  Backward, with g the gradient turned back:
//   dv = rstd (g w - vhat mean(g w vhat)), vhat = v rstd;  dw = sum g vhat.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ssm_recurrent.h"

#include "host_util.hpp"
#include "kernels.hpp"

namespace ssm {

// sin and cos of pos * freq.  The product is exact to 2^-53 in float64 (31 and
// 24 bits), is reduced there to a quarter turn, and what is left (|r| <= 1/8
// turn) goes through float32 Taylor polynomials: sin to x^9, cos to x^10 at
// |x| <= pi/4 (next terms 1.8e-9 and 1.2e-10).
__device__ __forceinline__ void turn_f32(int32_t pos, float freq, float& sn, float& cs) {
  double t = static_cast<double>(pos) * static_cast<double>(freq) * 0.15915494309189535;
  t -= __builtin_rint(t);  // turns, [-1/2, 1/2]
  const double q = __builtin_rint(t * 4.0);
  const float x = static_cast<float>((t - q * 0.25) * 6.283185307179586);
  const float x2 = x * x;
  float s = __builtin_fmaf(x2, 2.75573192e-6f, -1.98412698e-4f);
  s = __builtin_fmaf(x2, s, 8.33333333e-3f);
  s = __builtin_fmaf(x2, s, -1.66666667e-1f);
  s = __builtin_fmaf(x2 * x, s, x);
  float c = __builtin_fmaf(x2, -2.75573192e-7f, 2.48015873e-5f);
  c = __builtin_fmaf(x2, c, -1.38888889e-3f);
  c = __builtin_fmaf(x2, c, 4.16666667e-2f);
  c = __builtin_fmaf(x2, c, -0.5f);
  c = __builtin_fmaf(x2, c, 1.0f);
  const int k = static_cast<int>(q) & 3;  // quarter turns, mod 4
  const float ss = (k & 1) ? c : s, cc = (k & 1) ? s : c;
  sn = (k & 2) ? -ss : ss;
  cs = (k == 1 || k == 2) ? -cc : cc;
}

template <typename TA>
struct RotArgs {
  const TA *q, *k;             // inputs, tokens qs / ks values apart
  const float *qw, *kw, *freq;
  const int32_t* pos;
  const TA *dqo, *dko;         // backward: gradients of the outputs
  TA *qo, *ko;                 // outputs (forward) or dq, dk (backward)
  float* part;                 // backward: (waves, 2, D) partial weight gradients
  float eps;
  int64_t tokens, L, qs, ks;
  int Hq, Hk, D, R;            // R = rotary_dim
};

constexpr int kRotWaves = 4;     // waves of a workgroup
constexpr int kRotElems = 4;     // elements of a row per lane (headdim <= 256)

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// One wave per row (token, head); lane l holds elements l, l + 64, ...
template <typename TA, bool INTER, bool BWD>
__global__ void __launch_bounds__(64 * kRotWaves) rotate_kernel(RotArgs<TA> p) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = static_cast<int64_t>(blockIdx.x) * kRotWaves + (threadIdx.x >> 6);
  const int64_t nwaves = static_cast<int64_t>(gridDim.x) * kRotWaves;
  const int heads = p.Hq + p.Hk, half = p.R / 2;
  float wq[kRotElems] = {}, wk[kRotElems] = {};
  for (int64_t row = wave; row < p.tokens * heads; row += nwaves) {
    const int64_t tok = row / heads;
    const int hd = static_cast<int>(row % heads);
    const bool isq = hd < p.Hq;
    const TA* in = isq ? p.q + tok * p.qs + hd * p.D : p.k + tok * p.ks + (hd - p.Hq) * p.D;
    const int64_t oo = isq ? (tok * p.Hq + hd) * p.D : (tok * p.Hk + hd - p.Hq) * p.D;
    const TA* go = isq ? p.dqo : p.dko;
    const float* w = isq ? p.qw : p.kw;
    const int32_t pos = p.pos ? p.pos[tok] : static_cast<int32_t>(tok % p.L);
    float v[kRotElems], u[kRotElems], ss = 0.0f;  // own and partner's values
#pragma unroll
    for (int n = 0; n < kRotElems; ++n) {
      const int e = lane + 64 * n;
      v[n] = u[n] = 0.0f;
      if (e < p.D) {
        v[n] = to_f32(in[e]);
        if (e < p.R) {
          const int o = INTER ? (e ^ 1) : (e < half ? e + half : e - half);
          u[n] = to_f32(BWD ? go[oo + o] : in[o]) * (!BWD && w ? w[o] : 1.0f);
        }
      }
      ss += v[n] * v[n];
    }
    const float rstd = 1.0f / __builtin_sqrtf(wave_sum(ss) / static_cast<float>(p.D) + p.eps);
    float res[kRotElems], dot = 0.0f;
#pragma unroll
    for (int n = 0; n < kRotElems; ++n) {
      const int e = lane + 64 * n;
      res[n] = 0.0f;
      if (e >= p.D) continue;
      const float we = w ? w[e] : 1.0f;
      float sn = 0.0f, cs = 1.0f;
      bool first = true;
      if (e < p.R) {
        first = INTER ? !(e & 1) : e < half;
        turn_f32(pos, p.freq[INTER ? e >> 1 : (e < half ? e : e - half)], sn, cs);
      }
      if (!BWD) {
        const float side = first ? -sn : sn;
        res[n] = rstd * (v[n] * we * cs + u[n] * side);
      } else {
        const float side = first ? sn : -sn;
        const float g = to_f32(go[oo + e]) * cs + u[n] * side;
        const float vh = v[n] * rstd;
        (isq ? wq : wk)[n] += g * vh;
        res[n] = g * we;
        dot += res[n] * vh;
      }
    }
    if (BWD) dot = wave_sum(dot) / static_cast<float>(p.D);
    TA* out = (isq ? p.qo : p.ko) + oo;
#pragma unroll
    for (int n = 0; n < kRotElems; ++n) {
      const int e = lane + 64 * n;
      if (e < p.D) store_act(out + e, BWD ? rstd * (res[n] - v[n] * rstd * dot) : res[n]);
    }
  }
  if (BWD) {
#pragma unroll
    for (int n = 0; n < kRotElems; ++n) {
      const int e = lane + 64 * n;
      if (e < p.D) {
        p.part[(wave * 2) * p.D + e] = wq[n];
        p.part[(wave * 2 + 1) * p.D + e] = wk[n];
      }
    }
  }
}

// Sum of the partial weight gradients, in wave order: one lane per element.
__global__ void __launch_bounds__(64) rotate_sum_kernel(const float* part, int n, int D, float* dqw,
                                                        float* dkw) {
  const int e = blockIdx.x * 64 + threadIdx.x;
  float* to = blockIdx.y == 0 ? dqw : dkw;
  if (e >= D || !to) return;
  float v = 0.0f;
  for (int k = 0; k < n; ++k) v += part[(k * 2 + blockIdx.y) * static_cast<int64_t>(D) + e];
  to[e] = v;
}

namespace {

constexpr int64_t kRotMaxTokens = int64_t{1} << 31;

bool rot_sizes_ok(int64_t batch, int64_t L, int64_t Hq, int64_t Hk, int64_t D) {
  return batch >= 1 && L >= 0 && batch < kRotMaxTokens && L < kRotMaxTokens &&
         batch * L < kRotMaxTokens && Hq >= 1 && Hq <= 65536 && Hk >= 0 && Hk <= 65536 && D >= 2 &&
         D <= 256 && D % 2 == 0;
}

// Workgroups of the backward: each wave leaves one partial row of weight
// gradients, so their number is bounded.
int64_t rot_bwd_blocks(int64_t rows) {
  const int64_t want = (rows + kRotWaves * 4 - 1) / (kRotWaves * 4);
  return want < 1 ? 1 : want > 1024 ? 1024 : want;
}

struct RotCall {
  const char* fn;
  const void *q, *k;
  const float *qw, *kw, *freq;
  const int32_t* pos;
  float eps;
  int interleaved;
  const void *dqo, *dko;
  void *qo, *ko;
  float *dqw, *dkw;
  int64_t batch, L, Hq, Hk, D, R, qs, ks;
  int dtype;
  void* ws;
  size_t ws_bytes;
  hipStream_t stream;
  bool bwd;
};

template <typename TA>
int rot_launch(const RotCall& c) {
  RotArgs<TA> a{static_cast<const TA*>(c.q), static_cast<const TA*>(c.k), c.qw, c.kw, c.freq, c.pos,
                static_cast<const TA*>(c.dqo), static_cast<const TA*>(c.dko), static_cast<TA*>(c.qo),
                static_cast<TA*>(c.ko), static_cast<float*>(c.ws), c.eps, c.batch * c.L, c.L, c.qs,
                c.ks, static_cast<int>(c.Hq), static_cast<int>(c.Hk), static_cast<int>(c.D),
                static_cast<int>(c.R)};
  const int64_t rows = c.batch * c.L * (c.Hq + c.Hk);
  const int64_t want = (rows + kRotWaves - 1) / kRotWaves;
  const int64_t blocks = c.bwd ? rot_bwd_blocks(rows) : want > (1 << 20) ? (1 << 20) : want;
  const dim3 grid(static_cast<unsigned>(blocks)), block(64 * kRotWaves);
  if (c.bwd) {
    if (c.interleaved)
      hipLaunchKernelGGL((rotate_kernel<TA, true, true>), grid, block, 0, c.stream, a);
    else
      hipLaunchKernelGGL((rotate_kernel<TA, false, true>), grid, block, 0, c.stream, a);
    if (c.dqw || c.dkw)
      hipLaunchKernelGGL(rotate_sum_kernel, dim3((a.D + 63) / 64, 2), dim3(64), 0, c.stream, a.part,
                         static_cast<int>(blocks * kRotWaves), a.D, c.dqw, c.dkw);
  } else if (c.interleaved) {
    hipLaunchKernelGGL((rotate_kernel<TA, true, false>), grid, block, 0, c.stream, a);
  } else {
    hipLaunchKernelGGL((rotate_kernel<TA, false, false>), grid, block, 0, c.stream, a);
  }
  return launch_status(c.fn);
}

int rot_call(const RotCall& c) {
  clear_error();
  if (c.dtype != SSM_DTYPE_F32 && c.dtype != SSM_DTYPE_BF16)
    return fail(SSM_ERR_UNSUPPORTED, "%s: unknown dtype %d", c.fn, c.dtype);
  if (c.interleaved != 0 && c.interleaved != 1)
    return fail(SSM_ERR_UNSUPPORTED, "%s: interleaved must be 0 or 1, got %d", c.fn, c.interleaved);
  if (!(c.eps >= 0.0f)) return fail(SSM_ERR_UNSUPPORTED, "%s: eps must be at least 0", c.fn);
  if (c.D < 2 || c.D > 256 || c.D % 2 || c.R < 0 || c.R > c.D || c.R % 2)
    return fail(SSM_ERR_UNSUPPORTED,
                "%s: headdim must be even, 2..256, rotary_dim even, 0..headdim; got %lld, %lld", c.fn,
                (long long)c.D, (long long)c.R);
  if (!rot_sizes_ok(c.batch, c.L, c.Hq, c.Hk, c.D))
    return fail(SSM_ERR_SHAPE, "%s: bad sizes batch %lld, seqlen %lld, heads %lld and %lld", c.fn,
                (long long)c.batch, (long long)c.L, (long long)c.Hq, (long long)c.Hk);
  constexpr int64_t kMaxStride = int64_t{1} << 31;
  if (c.qs < c.Hq * c.D || c.qs > kMaxStride || (c.Hk > 0 && (c.ks < c.Hk * c.D || c.ks > kMaxStride)))
    return fail(SSM_ERR_SHAPE, "%s: a token stride (%lld, %lld) is shorter than its heads", c.fn,
                (long long)c.qs, (long long)c.ks);
  const int64_t tokens = c.batch * c.L;
  const bool any = tokens > 0;
  if (c.R > 0 && !c.freq) return fail(SSM_ERR_NULL, "%s: inv_freq is required with rotary_dim > 0", c.fn);
  if (any && (!c.q || !c.qo || (c.bwd && !c.dqo)))
    return fail(SSM_ERR_NULL, "%s: a query tensor is missing", c.fn);
  if (any && c.Hk > 0 && (!c.k || !c.ko || (c.bwd && !c.dko)))
    return fail(SSM_ERR_NULL, "%s: a key tensor is missing", c.fn);
  if (c.Hk == 0 && (c.k || c.ko || c.kw || c.dko || c.dkw))
    return fail(SSM_ERR_NULL, "%s: a key tensor is given with nheads_k = 0", c.fn);
  const size_t es = c.dtype == SSM_DTYPE_F32 ? 4 : 2;
  const char* const oq = c.bwd ? "dq" : "q_out";
  const char* const ok = c.bwd ? "dk" : "k_out";
  const struct { const void* p; size_t k; const char* n; } al[] = {
      {c.q, es, "q"}, {c.k, es, "k"}, {c.qo, es, oq}, {c.ko, es, ok}, {c.dqo, es, "dq_out"},
      {c.dko, es, "dk_out"}, {c.qw, 4, "q_weight"}, {c.kw, 4, "k_weight"}, {c.freq, 4, "inv_freq"},
      {c.pos, 4, "positions"}, {c.dqw, 4, "dq_weight"}, {c.dkw, 4, "dk_weight"}};
  for (const auto& e : al)
    if (e.p && !aligned(e.p, e.k))
      return fail(SSM_ERR_ALIGN, "%s: %s is not %zu-byte aligned", c.fn, e.n, e.k);
  const size_t nq = static_cast<size_t>(tokens) * c.Hq * c.D * es;
  const size_t nk = static_cast<size_t>(tokens) * c.Hk * c.D * es;
  const size_t eq = any ? (static_cast<size_t>(tokens - 1) * c.qs + c.Hq * c.D) * es : 0;
  const size_t ek = any && c.Hk ? (static_cast<size_t>(tokens - 1) * c.ks + c.Hk * c.D) * es : 0;
  const size_t wd = static_cast<size_t>(c.D) * 4;
  const size_t need = c.bwd ? ssm_qk_norm_rotate_bwd_workspace_bytes(c.batch, c.L, c.Hq, c.Hk, c.D) : 0;
  const Span ins[] = {{c.q, eq, "q"}, {c.k, ek, "k"}, {c.dqo, c.dqo ? nq : 0, "dq_out"},
                      {c.dko, c.dko ? nk : 0, "dk_out"}, {c.qw, c.qw ? wd : 0, "q_weight"},
                      {c.kw, c.kw ? wd : 0, "k_weight"},
                      {c.freq, c.freq ? static_cast<size_t>(c.R) * 2 : 0, "inv_freq"},
                      {c.pos, c.pos ? static_cast<size_t>(tokens) * 4 : 0, "positions"}};
  const Span outs[] = {{c.qo, nq, oq}, {c.ko, nk, ok}, {c.dqw, c.dqw ? wd : 0, "dq_weight"},
                       {c.dkw, c.dkw ? wd : 0, "dk_weight"}, {c.ws, c.ws ? need : 0, "workspace"}};
  for (const auto& o : outs)
    for (const auto& n : ins) {
      // a contiguous input may be normalised where it is (forward)
      const bool here = !c.bwd && o.p == n.p &&
                        ((o.p == c.qo && n.p == c.q && c.qs == c.Hq * c.D) ||
                         (o.p == c.ko && n.p == c.k && c.ks == c.Hk * c.D));
      if (overlap(o, n) && !here)
        return fail(SSM_ERR_ALIAS, "%s: output %s overlaps input %s", c.fn, o.name, n.name);
    }
  for (int x = 0; x < 5; ++x)
    for (int y = x + 1; y < 5; ++y)
      if (overlap(outs[x], outs[y]))
        return fail(SSM_ERR_ALIAS, "%s: %s overlaps %s", c.fn, outs[x].name, outs[y].name);
  if (need > 0 && (!c.ws || c.ws_bytes < need))
    return fail(SSM_ERR_WORKSPACE, "%s: workspace of %zu bytes given, %zu needed", c.fn,
                c.ws ? c.ws_bytes : 0, need);
  if (need > 0 && !aligned(c.ws, 256))
    return fail(SSM_ERR_ALIGN, "%s: workspace is not 256-byte aligned", c.fn);
  if (!any && !c.bwd) return SSM_OK;  // (the backward of no tokens leaves zero weight gradients)
  return c.dtype == SSM_DTYPE_F32 ? rot_launch<float>(c) : rot_launch<bf16_t>(c);
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" {

int ssm_qk_norm_rotate_fwd(const void* q, const void* k, const float* q_weight,
                           const float* k_weight, const float* inv_freq, const int32_t* positions,
                           float eps, int interleaved, void* q_out, void* k_out, int64_t batch,
                           int64_t seqlen, int64_t nheads_q, int64_t nheads_k, int64_t headdim,
                           int64_t rotary_dim, int64_t q_token_stride, int64_t k_token_stride,
                           int dtype, hipStream_t stream) {
  return rot_call(RotCall{"ssm_qk_norm_rotate_fwd", q, k, q_weight, k_weight, inv_freq, positions,
                          eps, interleaved, nullptr, nullptr, q_out, k_out, nullptr, nullptr, batch,
                          seqlen, nheads_q, nheads_k, headdim, rotary_dim, q_token_stride,
                          k_token_stride, dtype, nullptr, 0, stream, false});
}

int ssm_qk_norm_rotate_bwd(const void* q, const void* k, const float* q_weight,
                           const float* k_weight, const float* inv_freq, const int32_t* positions,
                           float eps, int interleaved, const void* dq_out, const void* dk_out,
                           void* dq, void* dk, float* dq_weight, float* dk_weight, int64_t batch,
                           int64_t seqlen, int64_t nheads_q, int64_t nheads_k, int64_t headdim,
                           int64_t rotary_dim, int64_t q_token_stride, int64_t k_token_stride,
                           int dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return rot_call(RotCall{"ssm_qk_norm_rotate_bwd", q, k, q_weight, k_weight, inv_freq, positions,
                          eps, interleaved, dq_out, dk_out, dq, dk, dq_weight, dk_weight, batch,
                          seqlen, nheads_q, nheads_k, headdim, rotary_dim, q_token_stride,
                          k_token_stride, dtype, workspace, workspace_bytes, stream, true});
}

size_t ssm_qk_norm_rotate_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads_q,
                                              int64_t nheads_k, int64_t headdim) {
  if (!rot_sizes_ok(batch, seqlen, nheads_q, nheads_k, headdim)) return 0;
  const int64_t rows = batch * seqlen * (nheads_q + nheads_k);
  return static_cast<size_t>(rot_bwd_blocks(rows)) * kRotWaves * 2 * headdim * sizeof(float);
}

}  // extern "C"
