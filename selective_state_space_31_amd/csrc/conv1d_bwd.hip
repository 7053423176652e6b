// conv1d_bwd.hip -- the gradients of the causal depthwise convolution (+ SiLU)
// of conv1d.hip, behind the C ABI in include/ssm_recurrent.h.
//
// With xx the input extended to the left by the conv state,
//   pre_t = bias + sum_k w_k xx_{t-(W-1)+k},  d_t = dout_t silu'(pre_t)
//   dxx_s = sum_k w_k d_{s+(W-1)-k}   (d = 0 outside the sequence)
//           (+ dfinal for the last W-1 inputs)
//   dw_k = sum_t d_t xx_{t-(W-1)+k};  dbias = sum_t d_t
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ssm_recurrent.h"

#include "host_util.hpp"
#include "kernels.hpp"

namespace ssm {

template <typename TA>
struct ConvBwdArgs {
  const TA* x;
  const float *w, *bias;
  const TA *state0, *dout, *dstate1;  // state0, dstate1: (batch, dim, W-1) or NULL
  TA* dx;
  TA* dstate0;
  float* part;  // (W + 1, batch, dim)
  int64_t batch, L;
  int dim;
};

// One lane per (sequence, channel) walks the tokens with the last W - 1
// inputs and gradients in registers.
template <typename TA, int W, bool SILU>
__global__ void __launch_bounds__(64) conv_bwd_kernel(ConvBwdArgs<TA> a) {
  const int c = blockIdx.x * 64 + threadIdx.x;
  const int64_t b = blockIdx.y;
  if (c >= a.dim) return;
  const int64_t row = b * a.dim + c, L = a.L;
  float w[W], xw[W], dw[W] = {}, db = 0.0f;
  float dd[W] = {};  // dd[j]: gradient so far of the input j steps back
#pragma unroll
  for (int k = 0; k < W; ++k) w[k] = a.w[static_cast<size_t>(c) * W + k];
#pragma unroll
  for (int k = 0; k + 1 < W; ++k)
    xw[k + 1] = a.state0 ? to_f32(a.state0[row * (W - 1) + k]) : 0.0f;
  const float bias = a.bias ? a.bias[c] : 0.0f;
  // after the last token the window still holds W - 1 inputs
  for (int64_t t = 0; t < L + W - 1; ++t) {
    float d = 0.0f, x = 0.0f;
    if (t < L) {
      x = to_f32(a.x[(b * L + t) * a.dim + c]);
      d = to_f32(a.dout[(b * L + t) * a.dim + c]);
    }
#pragma unroll
    for (int k = 0; k + 1 < W; ++k) xw[k] = xw[k + 1];
    xw[W - 1] = x;
    if (SILU && t < L) {
      float pre = bias;
#pragma unroll
      for (int k = 0; k < W; ++k) pre = __builtin_fmaf(w[k], xw[k], pre);
      const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-pre * kLog2e));
      d *= s * (1.0f + pre * (1.0f - s));
    }
#pragma unroll
    for (int k = 0; k < W; ++k) {
      dw[k] = __builtin_fmaf(d, xw[k], dw[k]);
      dd[W - 1 - k] = __builtin_fmaf(d, w[k], dd[W - 1 - k]);
    }
    db += d;
    // the input W - 1 steps back is done
    const int64_t s = t - (W - 1);
    float g = dd[W - 1];
    if (a.dstate1 && s >= L - (W - 1))
      g += to_f32(a.dstate1[row * (W - 1) + (s - (L - (W - 1)))]);
    if (s >= 0)
      store_act(a.dx + (b * L + s) * a.dim + c, g);
    else if (a.dstate0)
      store_act(a.dstate0 + row * (W - 1) + (s + W - 1), g);
#pragma unroll
    for (int k = W - 1; k > 0; --k) dd[k] = dd[k - 1];
    dd[0] = 0.0f;
  }
#pragma unroll
  for (int k = 0; k < W; ++k) a.part[(k * a.batch + b) * a.dim + c] = dw[k];
  a.part[(W * a.batch + b) * a.dim + c] = db;
}

// Sums of the partials, in sequence order: one lane per channel, a row of
// workgroups per tap (the last one the bias).
__global__ void __launch_bounds__(64) conv_bwd_sum_kernel(const float* part, int64_t n, int dim, int W,
                                                          float* dweight, float* dbias) {
  const int c = blockIdx.x * 64 + threadIdx.x, k = blockIdx.y;
  if (c >= dim || (k == W && !dbias)) return;
  float v = 0.0f;
  for (int64_t j = 0; j < n; ++j) v += part[(k * n + j) * dim + c];
  if (k == W)
    dbias[c] = v;
  else
    dweight[static_cast<size_t>(c) * W + k] = v;
}

namespace {

constexpr int64_t kConvBwdMaxDim = int64_t{1} << 24;

bool conv_bwd_sizes_ok(int64_t batch, int64_t L, int64_t dim) {
  return batch >= 1 && dim >= 1 && L >= 0 && dim <= kConvBwdMaxDim && batch <= 65535 &&
         L <= (int64_t{1} << 40) / dim &&
         batch * ((L + 15) / 16) * ((dim + 63) / 64) < (int64_t{1} << 25);
}

template <typename TA>
int conv_bwd_launch(const ConvBwdArgs<TA>& a, int W, bool silu, float* dweight, float* dbias,
                    hipStream_t s) {
  const dim3 grid((a.dim + 63) / 64, static_cast<unsigned>(a.batch)), block(64);
#define SSM_CONV_BWD_CASE(WW)                                                            \
  case WW:                                                                               \
    if (silu)                                                                            \
      hipLaunchKernelGGL((conv_bwd_kernel<TA, WW, true>), grid, block, 0, s, a);         \
    else                                                                                 \
      hipLaunchKernelGGL((conv_bwd_kernel<TA, WW, false>), grid, block, 0, s, a);        \
    break;
  switch (W) {
    SSM_CONV_BWD_CASE(2)
    SSM_CONV_BWD_CASE(3)
    SSM_CONV_BWD_CASE(4)
    default: break;
  }
#undef SSM_CONV_BWD_CASE
  hipLaunchKernelGGL(conv_bwd_sum_kernel, dim3((a.dim + 63) / 64, W + 1), block, 0, s, a.part, a.batch,
                     a.dim, W, dweight, dbias);
  return launch_status("ssm_causal_conv1d_bwd");
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" {

size_t ssm_causal_conv1d_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim,
                                             int64_t width) {
  if (!conv_bwd_sizes_ok(batch, seqlen, dim) || width < 2 || width > 4) return 0;
  return static_cast<size_t>(width + 1) * batch * dim * sizeof(float);
}

int ssm_causal_conv1d_bwd(const void* x, const float* weight, const float* bias,
                          const void* initial_conv_state, const void* dout,
                          const void* dfinal_conv_state, void* dx, float* dweight, float* dbias,
                          void* dinitial_conv_state, int64_t batch, int64_t seqlen, int64_t dim,
                          int64_t width, int silu, int dtype, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  const char* fn = "ssm_causal_conv1d_bwd";
  if (dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16)
    return fail(SSM_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, dtype);
  if (silu != 0 && silu != 1)
    return fail(SSM_ERR_UNSUPPORTED, "%s: silu must be 0 or 1, got %d", fn, silu);
  if (width < 2 || width > 4)
    return fail(SSM_ERR_UNSUPPORTED, "%s: width must be 2, 3 or 4, got %lld", fn, (long long)width);
  if (!conv_bwd_sizes_ok(batch, seqlen, dim))
    return fail(SSM_ERR_SHAPE, "%s: bad sizes batch %lld, seqlen %lld, dim %lld", fn,
                (long long)batch, (long long)seqlen, (long long)dim);
  if (!weight || !dweight || (seqlen > 0 && (!x || !dout || !dx)))
    return fail(SSM_ERR_NULL, "%s: weight, dweight, x, dout and dx are required", fn);
  const size_t es = dtype == SSM_DTYPE_F32 ? 4 : 2;
  const struct { const void* p; size_t k; const char* n; } al[] = {
      {x, es, "x"}, {dout, es, "dout"}, {dx, es, "dx"}, {weight, 4, "weight"}, {bias, 4, "bias"},
      {initial_conv_state, es, "initial_conv_state"}, {dfinal_conv_state, es, "dfinal_conv_state"},
      {dinitial_conv_state, es, "dinitial_conv_state"}, {dweight, 4, "dweight"}, {dbias, 4, "dbias"}};
  for (const auto& e : al)
    if (e.p && !aligned(e.p, e.k))
      return fail(SSM_ERR_ALIGN, "%s: %s is not %zu-byte aligned", fn, e.n, e.k);
  const size_t tok = static_cast<size_t>(batch) * seqlen * dim * es;
  const size_t st = static_cast<size_t>(batch) * dim * (width - 1) * es;
  const size_t wt = static_cast<size_t>(dim) * width * 4, pd = static_cast<size_t>(dim) * 4;
  const size_t need = ssm_causal_conv1d_bwd_workspace_bytes(batch, seqlen, dim, width);
  const Span ins[] = {{x, tok, "x"}, {dout, tok, "dout"}, {weight, wt, "weight"},
                      {bias, bias ? pd : 0, "bias"},
                      {initial_conv_state, initial_conv_state ? st : 0, "initial_conv_state"},
                      {dfinal_conv_state, dfinal_conv_state ? st : 0, "dfinal_conv_state"}};
  const Span outs[] = {{dx, tok, "dx"}, {dweight, wt, "dweight"}, {dbias, dbias ? pd : 0, "dbias"},
                       {dinitial_conv_state, dinitial_conv_state ? st : 0, "dinitial_conv_state"},
                       {workspace, workspace ? need : 0, "workspace"}};
  for (const auto& o : outs)
    for (const auto& i : ins)
      if (overlap(o, i))
        return fail(SSM_ERR_ALIAS, "%s: output %s overlaps input %s", fn, o.name, i.name);
  for (int p = 0; p < 5; ++p)
    for (int q = p + 1; q < 5; ++q)
      if (overlap(outs[p], outs[q]))
        return fail(SSM_ERR_ALIAS, "%s: %s overlaps %s", fn, outs[p].name, outs[q].name);
  if (!workspace || workspace_bytes < need)
    return fail(SSM_ERR_WORKSPACE, "%s: workspace of %zu bytes given, %zu needed", fn,
                workspace ? workspace_bytes : 0, need);
  if (!aligned(workspace, 256))
    return fail(SSM_ERR_ALIGN, "%s: workspace is not 256-byte aligned", fn);
  const auto go = [&](auto tag) {
    using TA = decltype(tag);
    ConvBwdArgs<TA> a{static_cast<const TA*>(x), weight, bias,
                      static_cast<const TA*>(initial_conv_state), static_cast<const TA*>(dout),
                      static_cast<const TA*>(dfinal_conv_state), static_cast<TA*>(dx),
                      static_cast<TA*>(dinitial_conv_state), static_cast<float*>(workspace), batch,
                      seqlen, static_cast<int>(dim)};
    return conv_bwd_launch(a, static_cast<int>(width), silu != 0, dweight, dbias, stream);
  };
  return dtype == SSM_DTYPE_F32 ? go(float{}) : go(bf16_t{});
}

}  // extern "C"
