// gated.hip -- the gated linear recurrence, forward and decode step, behind
// the C ABI in include/ssm_recurrent.h.
//
//   a_t = e^(A sigma(r_t + rb)),  h_t = a_t h_{t-1} + m_t sigma(i_t + ib) x_t
//   out_t = h_t silu(z_t)
//
#include "gated.hpp"
#include "host_util.hpp"

namespace ssm {

// One lane per (sequence, channel) walks the tokens.
template <typename TA, bool NORM>
__global__ void __launch_bounds__(64) gated_fwd_kernel(GatedFwdArgs<TA> p) {
  const int c = blockIdx.x * 64 + threadIdx.x;
  const int64_t s = blockIdx.y + static_cast<int64_t>(blockIdx.z) * gridDim.y;
  const int64_t nseq = p.cu ? p.nseq : p.rows;
  if (c >= p.dim || s >= nseq) return;
  int64_t t0, t1;
  seq_range(p.cu, s, p.L, t0, t1);
  const float A = p.A[c], rb = p.rb ? p.rb[c] : 0.0f, ib = p.ib ? p.ib[c] : 0.0f;
  const int64_t nch = (p.L + SSM_GATED_CHUNK - 1) / SSM_GATED_CHUNK;
  float h = p.h0 ? p.h0[s * p.dim + c] : 0.0f;
  for (int64_t t = t0; t < t1; ++t) {
    const int64_t tr = p.cu ? t : t - t0;  // token in its row
    if (p.chunk_states && tr % SSM_GATED_CHUNK == 0)
      p.chunk_states[((p.cu ? 0 : s) * nch + tr / SSM_GATED_CHUNK) * p.dim + c] = h;
    const int64_t o = t * p.dim + c;
    float a, m;
    decay<NORM>(A * sigmoid_f32(to_f32(p.r[o]) + rb), a, m);
    h = __builtin_fmaf(a, h, m * sigmoid_f32(to_f32(p.i[o]) + ib) * to_f32(p.x[o]));
    store_act(p.out + o, p.z ? h * silu_f32(to_f32(p.z[o])) : h);
  }
  if (p.last) p.last[s * p.dim + c] = h;
}

template <typename TA, bool NORM>
int launch_gated_fwd(const GatedFwdArgs<TA>& a, const char* fn, hipStream_t s) {
  const int64_t nseq = a.cu ? a.nseq : a.rows;
  const unsigned gy = static_cast<unsigned>(nseq < 65535 ? nseq : 65535);
  const dim3 grid((a.dim + 63) / 64, gy, static_cast<unsigned>((nseq + gy - 1) / gy));
  hipLaunchKernelGGL((gated_fwd_kernel<TA, NORM>), grid, dim3(64), 0, s, a);
  return launch_status(fn);
}

template <typename TA>
struct GatedStepArgs {
  float* state;
  const TA *x, *r, *i, *z;
  const float *A, *rb, *ib;
  TA* out;
  int64_t n;
  int dim;
};

// One lane per (sequence, channel).
template <typename TA, bool NORM>
__global__ void __launch_bounds__(256) gated_step_kernel(GatedStepArgs<TA> p) {
  const int64_t o = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (o >= p.n) return;
  const int c = static_cast<int>(o % p.dim);
  float a, m;
  decay<NORM>(p.A[c] * sigmoid_f32(to_f32(p.r[o]) + (p.rb ? p.rb[c] : 0.0f)), a, m);
  const float u = sigmoid_f32(to_f32(p.i[o]) + (p.ib ? p.ib[c] : 0.0f));
  const float h = __builtin_fmaf(a, p.state[o], m * u * to_f32(p.x[o]));
  p.state[o] = h;
  store_act(p.out + o, p.z ? h * silu_f32(to_f32(p.z[o])) : h);
}

constexpr int64_t kGatedMaxDim = int64_t{1} << 24;
constexpr int64_t kGatedMaxSeqs = int64_t{1} << 24;

// Whether batch, seqlen (or nseq, total_len) and dim can be launched.
bool gated_sizes_ok(int64_t rows, int64_t L, int64_t nseq, int64_t dim, bool packed) {
  if (dim < 1 || dim > kGatedMaxDim || L < 0 || L > (int64_t{1} << 40) / dim) return false;
  return packed ? (nseq >= 1 && nseq < kGatedMaxSeqs) : (rows >= 1 && rows <= 65535);
}

namespace {

int gated_fwd(const char* fn, const void* x, const void* r, const void* i, const float* A,
              const float* rb, const float* ib, int normalize, const void* z, void* out,
              float* last, const float* h0, float* chunk_states, const int32_t* cu, int64_t nseq,
              int64_t rows, int64_t L, int64_t dim, int dtype, bool packed, void* ws,
              size_t ws_bytes, hipStream_t stream) {
  clear_error();
  if (dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16)
    return fail(SSM_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, dtype);
  if (normalize != 0 && normalize != 1)
    return fail(SSM_ERR_UNSUPPORTED, "%s: normalize must be 0 or 1, got %d", fn, normalize);
  if (!gated_sizes_ok(rows, L, nseq, dim, packed))
    return fail(SSM_ERR_SHAPE, "%s: bad sizes: %lld sequence(s), %lld tokens, dim %lld", fn,
                (long long)(packed ? nseq : rows), (long long)L, (long long)dim);
  if (!A || (packed && !cu)) return fail(SSM_ERR_NULL, "%s: A%s required", fn, packed ? " and cu_seqlens are" : " is");
  if (L > 0 && (!x || !r || !i || !out))
    return fail(SSM_ERR_NULL, "%s: x, rgate, igate and out are required", fn);
  const size_t es = dtype == SSM_DTYPE_F32 ? 4 : 2;
  const struct { const void* p; size_t k; const char* n; } al[] = {
      {x, es, "x"}, {r, es, "rgate"}, {i, es, "igate"}, {z, es, "z"}, {out, es, "out"}, {A, 4, "A"},
      {rb, 4, "rgate_bias"}, {ib, 4, "igate_bias"}, {h0, 4, "initial_state"},
      {last, 4, "last_state"}, {chunk_states, 4, "chunk_states"}, {cu, 4, "cu_seqlens"}};
  for (const auto& e : al)
    if (e.p && !aligned(e.p, e.k))
      return fail(SSM_ERR_ALIGN, "%s: %s is not %zu-byte aligned", fn, e.n, e.k);
  const size_t tok = static_cast<size_t>(rows) * L * dim * es;
  const size_t st = static_cast<size_t>(packed ? nseq : rows) * dim * 4;
  const size_t cst = static_cast<size_t>(rows) * ((L + SSM_GATED_CHUNK - 1) / SSM_GATED_CHUNK) * dim * 4;
  const size_t pd = static_cast<size_t>(dim) * 4;
  const Span ins[] = {{x, tok, "x"}, {r, tok, "rgate"}, {i, tok, "igate"}, {z, z ? tok : 0, "z"},
                      {A, pd, "A"}, {rb, rb ? pd : 0, "rgate_bias"}, {ib, ib ? pd : 0, "igate_bias"},
                      {cu, packed ? static_cast<size_t>(nseq + 1) * 4 : 0, "cu_seqlens"},
                      {h0, h0 ? st : 0, "initial_state"}};
  const Span outs[] = {{out, tok, "out"}, {last, last ? st : 0, "last_state"},
                       {chunk_states, chunk_states ? cst : 0, "chunk_states"}};
  for (const auto& o : outs)
    for (const auto& n : ins)
      if (overlap(o, n) && !(o.p == last && n.p == h0 && last == h0 && !packed))
        return fail(SSM_ERR_ALIAS, "%s: output %s overlaps input %s", fn, o.name, n.name);
  for (int a = 0; a < 3; ++a)
    for (int b = a + 1; b < 3; ++b)
      if (overlap(outs[a], outs[b]))
        return fail(SSM_ERR_ALIAS, "%s: %s overlaps %s", fn, outs[a].name, outs[b].name);
  (void)ws;
  (void)ws_bytes;
  if (dtype == SSM_DTYPE_F32) {
    GatedFwdArgs<float> a{static_cast<const float*>(x), static_cast<const float*>(r),
                          static_cast<const float*>(i), static_cast<const float*>(z), A, rb, ib,
                          static_cast<float*>(out), last, h0, chunk_states, cu, rows, L, nseq,
                          static_cast<int>(dim), ws};
    return normalize ? launch_gated_fwd<float, true>(a, fn, stream)
                     : launch_gated_fwd<float, false>(a, fn, stream);
  }
  GatedFwdArgs<bf16_t> a{static_cast<const bf16_t*>(x), static_cast<const bf16_t*>(r),
                         static_cast<const bf16_t*>(i), static_cast<const bf16_t*>(z), A, rb, ib,
                         static_cast<bf16_t*>(out), last, h0, chunk_states, cu, rows, L, nseq,
                         static_cast<int>(dim), ws};
  return normalize ? launch_gated_fwd<bf16_t, true>(a, fn, stream)
                   : launch_gated_fwd<bf16_t, false>(a, fn, stream);
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" {

int ssm_gated_scan_fwd(const void* x, const void* rgate, const void* igate, const float* A,
                       const float* rgate_bias, const float* igate_bias, int normalize,
                       const void* z, void* out, float* last_state, const float* initial_state,
                       float* chunk_states, int64_t batch, int64_t seqlen, int64_t dim, int dtype,
                       void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return gated_fwd("ssm_gated_scan_fwd", x, rgate, igate, A, rgate_bias, igate_bias, normalize, z,
                   out, last_state, initial_state, chunk_states, nullptr, batch, batch, seqlen, dim,
                   dtype, false, workspace, workspace_bytes, stream);
}

size_t ssm_gated_scan_fwd_workspace_bytes(int64_t, int64_t, int64_t, int) { return 0; }

int ssm_gated_scan_fwd_varlen(const void* x, const void* rgate, const void* igate, const float* A,
                              const float* rgate_bias, const float* igate_bias, int normalize,
                              const void* z, void* out, float* last_state,
                              const float* initial_state, float* chunk_states,
                              const int32_t* cu_seqlens, int64_t nseq, int64_t total_len,
                              int64_t dim, int dtype, void* workspace, size_t workspace_bytes,
                              hipStream_t stream) {
  return gated_fwd("ssm_gated_scan_fwd_varlen", x, rgate, igate, A, rgate_bias, igate_bias,
                   normalize, z, out, last_state, initial_state, chunk_states, cu_seqlens, nseq, 1,
                   total_len, dim, dtype, true, workspace, workspace_bytes, stream);
}

size_t ssm_gated_scan_fwd_varlen_workspace_bytes(int64_t, int64_t, int64_t, int) { return 0; }

int ssm_gated_state_update(float* state, const void* x, const void* rgate, const void* igate,
                           const float* A, const float* rgate_bias, const float* igate_bias,
                           int normalize, const void* z, void* out, int64_t batch, int64_t dim,
                           int dtype, hipStream_t stream) {
  clear_error();
  const char* fn = "ssm_gated_state_update";
  if (dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16)
    return fail(SSM_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, dtype);
  if (normalize != 0 && normalize != 1)
    return fail(SSM_ERR_UNSUPPORTED, "%s: normalize must be 0 or 1, got %d", fn, normalize);
  if (batch < 1 || dim < 1 || dim > kGatedMaxDim || batch > (int64_t{1} << 31) ||
      batch * dim > (int64_t{1} << 31) - 2048)  // (batch bounded first: no overflow)
    return fail(SSM_ERR_SHAPE, "%s: bad sizes batch %lld, dim %lld", fn, (long long)batch,
                (long long)dim);
  if (!state || !x || !rgate || !igate || !A || !out)
    return fail(SSM_ERR_NULL, "%s: state, x, rgate, igate, A and out are required", fn);
  const size_t es = dtype == SSM_DTYPE_F32 ? 4 : 2;
  const struct { const void* p; size_t k; const char* n; } al[] = {
      {state, 4, "state"}, {x, es, "x"}, {rgate, es, "rgate"}, {igate, es, "igate"}, {z, es, "z"},
      {out, es, "out"}, {A, 4, "A"}, {rgate_bias, 4, "rgate_bias"}, {igate_bias, 4, "igate_bias"}};
  for (const auto& e : al)
    if (e.p && !aligned(e.p, e.k))
      return fail(SSM_ERR_ALIGN, "%s: %s is not %zu-byte aligned", fn, e.n, e.k);
  const size_t tok = static_cast<size_t>(batch) * dim * es, pd = static_cast<size_t>(dim) * 4;
  const Span ins[] = {{x, tok, "x"}, {rgate, tok, "rgate"}, {igate, tok, "igate"},
                      {z, z ? tok : 0, "z"}, {A, pd, "A"},
                      {rgate_bias, rgate_bias ? pd : 0, "rgate_bias"},
                      {igate_bias, igate_bias ? pd : 0, "igate_bias"}};
  const Span outs[] = {{out, tok, "out"}, {state, static_cast<size_t>(batch) * dim * 4, "state"}};
  for (const auto& o : outs)
    for (const auto& n : ins)
      if (overlap(o, n))
        return fail(SSM_ERR_ALIAS, "%s: %s overlaps input %s", fn, o.name, n.name);
  if (overlap(outs[0], outs[1])) return fail(SSM_ERR_ALIAS, "%s: out overlaps state", fn);
  const int64_t n = batch * dim;
  const dim3 grid(static_cast<unsigned>((n + 255) / 256)), block(256);
  const auto go = [&](auto tag) {
    using TA = decltype(tag);
    GatedStepArgs<TA> a{state, static_cast<const TA*>(x), static_cast<const TA*>(rgate),
                        static_cast<const TA*>(igate), static_cast<const TA*>(z), A, rgate_bias,
                        igate_bias, static_cast<TA*>(out), n, static_cast<int>(dim)};
    if (normalize)
      hipLaunchKernelGGL((gated_step_kernel<TA, true>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((gated_step_kernel<TA, false>), grid, block, 0, stream, a);
  };
  if (dtype == SSM_DTYPE_F32)
    go(float{});
  else
    go(bf16_t{});
  return launch_status(fn);
}

}  // extern "C"
