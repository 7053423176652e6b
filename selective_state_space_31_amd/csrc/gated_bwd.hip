// gated_bwd.hip -- the gradients of the gated linear recurrence, behind the C
// ABI in include/ssm_recurrent.h.
//
// With g_t = dout_t silu(z_t), h_t as in the forward:
//   G_t = g_t + a_{t+1} G_{t+1}  (+ dlast at a sequence's last token)
//   dz = dout h silu'(z);  dx = G m u;  di = G m x u (1 - u)
//   dla = G (a h_{t-1} - u x a^2 / m);  dr = dla A s (1 - s)
//   dA = sum dla s;  drb = sum dr;  dib = sum di;  dh0 = a_0 G_0
// (s = sigma(r + rb), u = sigma(i + ib); the a^2 / m term only with normalize.)
#include "gated.hpp"
#include "host_util.hpp"

namespace ssm {

bool gated_sizes_ok(int64_t rows, int64_t L, int64_t nseq, int64_t dim, bool packed);

// Tokens [t0, t1) of sequence s (clamped: offsets that break the rule stay in
// the buffers).
__device__ __forceinline__ void seq_range(const int32_t* cu, int64_t s, int64_t L, int64_t& t0,
                                          int64_t& t1) {
  if (!cu) {
    t0 = s * L;
    t1 = t0 + L;
    return;
  }
  const int64_t a = cu[s], b = cu[s + 1];
  t0 = a < 0 ? 0 : (a > L ? L : a);
  t1 = b < t0 ? t0 : (b > L ? L : b);
}

// One lane per (sequence, channel): a walk forward that leaves every h_{t-1}
// in the workspace, then one back.  Partial sums per sequence, (3, nseq, dim).
template <typename TA, bool NORM>
__global__ void __launch_bounds__(64) gated_bwd_kernel(GatedBwdArgs<TA> p) {
  const int c = blockIdx.x * 64 + threadIdx.x;
  const int64_t s = blockIdx.y + static_cast<int64_t>(blockIdx.z) * gridDim.y;
  const int64_t nseq = p.cu ? p.nseq : p.rows;
  if (c >= p.dim || s >= nseq) return;
  float* hs = static_cast<float*>(p.ws);
  float* part = hs + p.rows * p.L * p.dim;
  int64_t t0, t1;
  seq_range(p.cu, s, p.L, t0, t1);
  const float A = p.A[c], rb = p.rb ? p.rb[c] : 0.0f, ib = p.ib ? p.ib[c] : 0.0f;
  float h = p.h0 ? p.h0[s * p.dim + c] : 0.0f;
  for (int64_t t = t0; t < t1; ++t) {
    const int64_t o = t * p.dim + c;
    float a, m;
    decay<NORM>(A * sigmoid_f32(to_f32(p.r[o]) + rb), a, m);
    hs[o] = h;
    h = __builtin_fmaf(a, h, m * sigmoid_f32(to_f32(p.i[o]) + ib) * to_f32(p.x[o]));
  }
  float k = p.dlast ? p.dlast[s * p.dim + c] : 0.0f;
  float dA = 0.0f, drb = 0.0f, dib = 0.0f;
  for (int64_t t = t1 - 1; t >= t0; --t) {
    const int64_t o = t * p.dim + c;
    float a, m;
    const float sr = sigmoid_f32(to_f32(p.r[o]) + rb), u = sigmoid_f32(to_f32(p.i[o]) + ib);
    const float x = to_f32(p.x[o]), dout = to_f32(p.dout[o]);
    decay<NORM>(A * sr, a, m);
    const float hp = hs[o];
    float g = dout;
    if (p.z) {
      const float z = to_f32(p.z[o]), sz = sigmoid_f32(z);
      const float ht = __builtin_fmaf(a, hp, m * u * x);
      g = dout * z * sz;
      store_act(p.dz + o, dout * ht * sz * (1.0f + z * (1.0f - sz)));
    }
    const float G = g + k;
    float dla = a * hp;
    if (NORM) dla -= u * x * a * a * (m > 0.0f ? __builtin_amdgcn_rcpf(m) : 0.0f);
    dla *= G;
    const float dr = dla * A * sr * (1.0f - sr), di = G * m * x * u * (1.0f - u);
    store_act(p.dx + o, G * m * u);
    store_act(p.dr + o, dr);
    store_act(p.di + o, di);
    dA += dla * sr;
    drb += dr;
    dib += di;
    k = a * G;
  }
  if (p.dh0) p.dh0[s * p.dim + c] = k;
  part[s * p.dim + c] = dA;
  part[(nseq + s) * p.dim + c] = drb;
  part[(2 * nseq + s) * p.dim + c] = dib;
}

__global__ void __launch_bounds__(64) gated_sum_kernel(const float* part, int64_t n, int dim,
                                                       float* dA, float* drb, float* dib) {
  const int c = blockIdx.x * 64 + threadIdx.x;
  float* to = blockIdx.y == 0 ? dA : blockIdx.y == 1 ? drb : dib;
  if (c >= dim || !to) return;
  float v = 0.0f;
  for (int64_t k = 0; k < n; ++k) v += part[(blockIdx.y * n + k) * dim + c];
  to[c] = v;
}

template <typename TA, bool NORM>
int launch_gated_bwd(const GatedBwdArgs<TA>& a, const char* fn, hipStream_t s) {
  const int64_t nseq = a.cu ? a.nseq : a.rows;
  const unsigned gy = static_cast<unsigned>(nseq < 65535 ? nseq : 65535);
  const dim3 grid((a.dim + 63) / 64, gy, static_cast<unsigned>((nseq + gy - 1) / gy));
  hipLaunchKernelGGL((gated_bwd_kernel<TA, NORM>), grid, dim3(64), 0, s, a);
  const float* part = static_cast<const float*>(a.ws) + a.rows * a.L * a.dim;
  hipLaunchKernelGGL(gated_sum_kernel, dim3((a.dim + 63) / 64, 3), dim3(64), 0, s, part, nseq, a.dim,
                     a.dA, a.drb, a.dib);
  return launch_status(fn);
}

namespace {

size_t bwd_ws_bytes(int64_t rows, int64_t L, int64_t nseq, int64_t dim, int dtype, bool packed) {
  if ((dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16) ||
      !gated_sizes_ok(rows, L, nseq, dim, packed))
    return 0;
  return (static_cast<size_t>(rows) * L + 3 * static_cast<size_t>(packed ? nseq : rows)) * dim * 4;
}

int gated_bwd(const char* fn, const void* x, const void* r, const void* i, const float* A,
              const float* rb, const float* ib, int normalize, const void* z, const float* h0,
              const float* chunk_states, const void* dout, const float* dlast, void* dx, void* dr,
              void* di, void* dz, float* dA, float* drb, float* dib, float* dh0, const int32_t* cu,
              int64_t nseq, int64_t rows, int64_t L, int64_t dim, int dtype, bool packed, void* ws,
              size_t ws_bytes, hipStream_t stream) {
  clear_error();
  if (dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16)
    return fail(SSM_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, dtype);
  if (normalize != 0 && normalize != 1)
    return fail(SSM_ERR_UNSUPPORTED, "%s: normalize must be 0 or 1, got %d", fn, normalize);
  if (!gated_sizes_ok(rows, L, nseq, dim, packed))
    return fail(SSM_ERR_SHAPE, "%s: bad sizes: %lld sequence(s), %lld tokens, dim %lld", fn,
                (long long)(packed ? nseq : rows), (long long)L, (long long)dim);
  if (!A || !dA || (packed && !cu))
    return fail(SSM_ERR_NULL, "%s: A, dA%s are required", fn, packed ? " and cu_seqlens" : "");
  if (L > 0 && (!x || !r || !i || !dout || !dx || !dr || !di))
    return fail(SSM_ERR_NULL, "%s: x, rgate, igate, dout, dx, drgate and digate are required", fn);
  if (L > 0 && z && !dz) return fail(SSM_ERR_NULL, "%s: dz is required with z", fn);
  if (!z && dz) return fail(SSM_ERR_NULL, "%s: dz given without z", fn);
  const size_t es = dtype == SSM_DTYPE_F32 ? 4 : 2;
  const struct { const void* p; size_t k; const char* n; } al[] = {
      {x, es, "x"}, {r, es, "rgate"}, {i, es, "igate"}, {z, es, "z"}, {dout, es, "dout"},
      {dx, es, "dx"}, {dr, es, "drgate"}, {di, es, "digate"}, {dz, es, "dz"}, {A, 4, "A"},
      {rb, 4, "rgate_bias"}, {ib, 4, "igate_bias"}, {h0, 4, "initial_state"},
      {chunk_states, 4, "chunk_states"}, {dlast, 4, "dlast_state"}, {dA, 4, "dA"},
      {drb, 4, "drgate_bias"}, {dib, 4, "digate_bias"}, {dh0, 4, "dinitial_state"},
      {cu, 4, "cu_seqlens"}};
  for (const auto& e : al)
    if (e.p && !aligned(e.p, e.k))
      return fail(SSM_ERR_ALIGN, "%s: %s is not %zu-byte aligned", fn, e.n, e.k);
  const size_t tok = static_cast<size_t>(rows) * L * dim * es;
  const size_t st = static_cast<size_t>(packed ? nseq : rows) * dim * 4;
  const size_t cst =
      static_cast<size_t>(rows) * ((L + SSM_GATED_CHUNK - 1) / SSM_GATED_CHUNK) * dim * 4;
  const size_t pd = static_cast<size_t>(dim) * 4;
  const size_t need = bwd_ws_bytes(rows, L, nseq, dim, dtype, packed);
  const Span ins[] = {{x, tok, "x"}, {r, tok, "rgate"}, {i, tok, "igate"}, {z, z ? tok : 0, "z"},
                      {dout, tok, "dout"}, {A, pd, "A"}, {rb, rb ? pd : 0, "rgate_bias"},
                      {ib, ib ? pd : 0, "igate_bias"}, {h0, h0 ? st : 0, "initial_state"},
                      {chunk_states, chunk_states ? cst : 0, "chunk_states"},
                      {dlast, dlast ? st : 0, "dlast_state"},
                      {cu, packed ? static_cast<size_t>(nseq + 1) * 4 : 0, "cu_seqlens"}};
  const Span outs[] = {{dx, tok, "dx"}, {dr, tok, "drgate"}, {di, tok, "digate"},
                       {dz, dz ? tok : 0, "dz"}, {dA, pd, "dA"}, {drb, drb ? pd : 0, "drgate_bias"},
                       {dib, dib ? pd : 0, "digate_bias"}, {dh0, dh0 ? st : 0, "dinitial_state"},
                       {ws, ws ? need : 0, "workspace"}};
  constexpr int kOuts = sizeof(outs) / sizeof(outs[0]);
  for (const auto& o : outs)
    for (const auto& n : ins)
      if (overlap(o, n))
        return fail(SSM_ERR_ALIAS, "%s: output %s overlaps input %s", fn, o.name, n.name);
  for (int a = 0; a < kOuts; ++a)
    for (int b = a + 1; b < kOuts; ++b)
      if (overlap(outs[a], outs[b]))
        return fail(SSM_ERR_ALIAS, "%s: %s overlaps %s", fn, outs[a].name, outs[b].name);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(SSM_ERR_WORKSPACE, "%s: workspace of %zu bytes given, %zu needed", fn,
                ws ? ws_bytes : 0, need);
  if (need > 0 && !aligned(ws, 256))
    return fail(SSM_ERR_ALIGN, "%s: workspace is not 256-byte aligned", fn);
  const auto go = [&](auto tag) {
    using TA = decltype(tag);
    GatedBwdArgs<TA> a{static_cast<const TA*>(x), static_cast<const TA*>(r),
                       static_cast<const TA*>(i), static_cast<const TA*>(z),
                       static_cast<const TA*>(dout), A, rb, ib, h0, chunk_states, dlast,
                       static_cast<TA*>(dx), static_cast<TA*>(dr), static_cast<TA*>(di),
                       static_cast<TA*>(dz), dA, drb, dib, dh0, cu, rows, L, nseq,
                       static_cast<int>(dim), ws};
    return normalize ? launch_gated_bwd<TA, true>(a, fn, stream)
                     : launch_gated_bwd<TA, false>(a, fn, stream);
  };
  return dtype == SSM_DTYPE_F32 ? go(float{}) : go(bf16_t{});
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" {

int ssm_gated_scan_bwd(const void* x, const void* rgate, const void* igate, const float* A,
                       const float* rgate_bias, const float* igate_bias, int normalize,
                       const void* z, const float* initial_state, const float* chunk_states,
                       const void* dout, const float* dlast_state, void* dx, void* drgate,
                       void* digate, void* dz, float* dA, float* drgate_bias, float* digate_bias,
                       float* dinitial_state, int64_t batch, int64_t seqlen, int64_t dim, int dtype,
                       void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return gated_bwd("ssm_gated_scan_bwd", x, rgate, igate, A, rgate_bias, igate_bias, normalize, z,
                   initial_state, chunk_states, dout, dlast_state, dx, drgate, digate, dz, dA,
                   drgate_bias, digate_bias, dinitial_state, nullptr, batch, batch, seqlen, dim,
                   dtype, false, workspace, workspace_bytes, stream);
}

size_t ssm_gated_scan_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int dtype,
                                          int) {
  return bwd_ws_bytes(batch, seqlen, batch, dim, dtype, false);
}

int ssm_gated_scan_bwd_varlen(const void* x, const void* rgate, const void* igate, const float* A,
                              const float* rgate_bias, const float* igate_bias, int normalize,
                              const void* z, const float* initial_state,
                              const float* chunk_states, const void* dout,
                              const float* dlast_state, void* dx, void* drgate, void* digate,
                              void* dz, float* dA, float* drgate_bias, float* digate_bias,
                              float* dinitial_state, const int32_t* cu_seqlens, int64_t nseq,
                              int64_t total_len, int64_t dim, int dtype, void* workspace,
                              size_t workspace_bytes, hipStream_t stream) {
  return gated_bwd("ssm_gated_scan_bwd_varlen", x, rgate, igate, A, rgate_bias, igate_bias,
                   normalize, z, initial_state, chunk_states, dout, dlast_state, dx, drgate, digate,
                   dz, dA, drgate_bias, digate_bias, dinitial_state, cu_seqlens, nseq, 1, total_len,
                   dim, dtype, true, workspace, workspace_bytes, stream);
}

size_t ssm_gated_scan_bwd_varlen_workspace_bytes(int64_t nseq, int64_t total_len, int64_t dim,
                                                 int dtype, int) {
  return bwd_ws_bytes(1, total_len, nseq, dim, dtype, true);
}

}  // extern "C"
