// delta_bwd.hip -- gradients of the gated delta rule, behind
// ssm_delta_rule_bwd and _bwd_varlen of include/ssm_layer.h.
#include "delta.hpp"

namespace ssm {
namespace {

size_t bwd_bytes(const DeltaDims& d, int dtype, bool have) {
  (void)d;
  (void)dtype;
  (void)have;
  return 0;
}

int delta_bwd(const char* fn, const void* q, const void* k, const void* v, const float* beta, const float* g,
              float scale, const float* first, const float* mids, const void* dout, const float* dlast, void* dq,
              void* dk, void* dv, float* dbeta, float* dg, float* dfirst, const int32_t* cu, bool packed,
              int64_t nseq, int64_t L, int64_t hk, int64_t hv, int64_t K, int64_t V, int64_t qs, int64_t ks,
              int64_t vs, int dtype, void* ws, size_t ws_bytes, hipStream_t stream) {
  clear_error();
  if (dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16)
    return fail(SSM_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, dtype);
  if (!delta_sizes_ok(nseq, L, hk, hv, K, V, packed))
    return fail(SSM_ERR_SHAPE, "%s: bad sizes: %lld sequence(s), %lld tokens, heads %lld and %lld, widths %lld and %lld",
                fn, (long long)nseq, (long long)L, (long long)hk, (long long)hv, (long long)K, (long long)V);
  const DeltaDims d{nseq, L, static_cast<int>(hk), static_cast<int>(hv), static_cast<int>(K), static_cast<int>(V),
                    qs, ks, vs, packed};
  if (!delta_strides_ok(d))
    return fail(SSM_ERR_SHAPE, "%s: bad token strides %lld, %lld, %lld", fn, (long long)qs, (long long)ks,
                (long long)vs);
  if (packed && !cu) return fail(SSM_ERR_NULL, "%s: cu_seqlens is required", fn);
  if (L > 0 && (!q || !k || !v || !beta || !dout || !dq || !dk || !dv || !dbeta))
    return fail(SSM_ERR_NULL, "%s: q, k, v, beta, dout, dq, dk, dv and dbeta are required", fn);
  if (dg && !g) return fail(SSM_ERR_NULL, "%s: dg needs g", fn);
  const size_t es = dtype == SSM_DTYPE_F32 ? 4 : 2;
  const struct { const void* p; size_t k; const char* n; } al[] = {
      {q, es, "q"}, {k, es, "k"}, {v, es, "v"}, {dout, es, "dout"}, {dq, es, "dq"}, {dk, es, "dk"}, {dv, es, "dv"},
      {beta, 4, "beta"}, {g, 4, "g"}, {first, 4, "initial_state"}, {mids, 4, "chunk_states"},
      {dlast, 4, "dlast_state"}, {dbeta, 4, "dbeta"}, {dg, 4, "dg"}, {dfirst, 4, "dinitial_state"},
      {cu, 4, "cu_seqlens"}};
  for (const auto& e : al)
    if (e.p && !aligned(e.p, e.k)) return fail(SSM_ERR_ALIGN, "%s: %s is not %zu-byte aligned", fn, e.n, e.k);
  const size_t gate = static_cast<size_t>(d.tokens()) * hv * 4, st = nseq * d.state_values() * 4;
  const size_t key = static_cast<size_t>(d.tokens()) * hk * K * es, val = static_cast<size_t>(d.tokens()) * hv * V * es;
  const size_t need = bwd_bytes(d, dtype, mids != nullptr);
  const Span ins[] = {{q, strided_bytes(d.tokens(), hk * K, qs, es), "q"},
                      {k, strided_bytes(d.tokens(), hk * K, ks, es), "k"},
                      {v, strided_bytes(d.tokens(), hv * V, vs, es), "v"},
                      {beta, gate, "beta"},
                      {g, g ? gate : 0, "g"},
                      {first, first ? st : 0, "initial_state"},
                      {mids, mids ? d.chunks() * d.state_values() * 4 : 0, "chunk_states"},
                      {dout, val, "dout"},
                      {dlast, dlast ? st : 0, "dlast_state"},
                      {cu, packed ? static_cast<size_t>(nseq + 1) * 4 : 0, "cu_seqlens"}};
  const Span outs[] = {{dq, key, "dq"}, {dk, key, "dk"}, {dv, val, "dv"}, {dbeta, gate, "dbeta"},
                       {dg, dg ? gate : 0, "dg"}, {dfirst, dfirst ? st : 0, "dinitial_state"},
                       {ws, ws ? need : 0, "workspace"}};
  constexpr int no = sizeof(outs) / sizeof(outs[0]);
  for (const auto& o : outs)
    for (const auto& n : ins)
      if (overlap(o, n)) return fail(SSM_ERR_ALIAS, "%s: output %s overlaps input %s", fn, o.name, n.name);
  for (int a = 0; a < no; ++a)
    for (int b = a + 1; b < no; ++b)
      if (overlap(outs[a], outs[b]))
        return fail(SSM_ERR_ALIAS, "%s: %s overlaps %s", fn, outs[a].name, outs[b].name);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(SSM_ERR_WORKSPACE, "%s: workspace of %zu bytes given, %zu needed", fn, ws ? ws_bytes : 0, need);
  if (need > 0 && !aligned(ws, 256))
    return fail(SSM_ERR_ALIGN, "%s: workspace is not 256-byte aligned", fn);
  if (L == 0 && !dfirst) return SSM_OK;
  (void)scale;
  (void)stream;
  return fail(SSM_ERR_UNSUPPORTED, "%s: not built yet", fn);
}

size_t query(int64_t nseq, int64_t L, int64_t hk, int64_t hv, int64_t K, int64_t V, bool packed, int dtype, int have) {
  if ((dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16) || !delta_sizes_ok(nseq, L, hk, hv, K, V, packed)) return 0;
  return bwd_bytes(DeltaDims{nseq, L, static_cast<int>(hk), static_cast<int>(hv), static_cast<int>(K),
                             static_cast<int>(V), hk * K, hk * K, hv * V, packed},
                   dtype, have != 0);
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" {

int ssm_delta_rule_bwd(const void* q, const void* k, const void* v, const float* beta, const float* g, float scale,
                       const float* initial_state, const float* chunk_states, const void* dout,
                       const float* dlast_state, void* dq, void* dk, void* dv, float* dbeta, float* dg,
                       float* dinitial_state, int64_t batch, int64_t seqlen, int64_t nheads_k, int64_t nheads_v,
                       int64_t headdim_k, int64_t headdim_v, int64_t q_token_stride, int64_t k_token_stride,
                       int64_t v_token_stride, int dtype, void* workspace, size_t workspace_bytes,
                       hipStream_t stream) {
  return delta_bwd("ssm_delta_rule_bwd", q, k, v, beta, g, scale, initial_state, chunk_states, dout, dlast_state, dq,
                   dk, dv, dbeta, dg, dinitial_state, nullptr, false, batch, seqlen, nheads_k, nheads_v, headdim_k,
                   headdim_v, q_token_stride, k_token_stride, v_token_stride, dtype, workspace, workspace_bytes,
                   stream);
}

size_t ssm_delta_rule_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads_k, int64_t nheads_v,
                                          int64_t headdim_k, int64_t headdim_v, int dtype, int with_chunk_states) {
  return query(batch, seqlen, nheads_k, nheads_v, headdim_k, headdim_v, false, dtype, with_chunk_states);
}

int ssm_delta_rule_bwd_varlen(const void* q, const void* k, const void* v, const float* beta, const float* g,
                              float scale, const float* initial_state, const float* chunk_states, const void* dout,
                              const float* dlast_state, void* dq, void* dk, void* dv, float* dbeta, float* dg,
                              float* dinitial_state, const int32_t* cu_seqlens, int64_t nseq, int64_t total_len,
                              int64_t nheads_k, int64_t nheads_v, int64_t headdim_k, int64_t headdim_v,
                              int64_t q_token_stride, int64_t k_token_stride, int64_t v_token_stride, int dtype,
                              void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return delta_bwd("ssm_delta_rule_bwd_varlen", q, k, v, beta, g, scale, initial_state, chunk_states, dout,
                   dlast_state, dq, dk, dv, dbeta, dg, dinitial_state, cu_seqlens, true, nseq, total_len, nheads_k,
                   nheads_v, headdim_k, headdim_v, q_token_stride, k_token_stride, v_token_stride, dtype, workspace,
                   workspace_bytes, stream);
}

size_t ssm_delta_rule_bwd_varlen_workspace_bytes(int64_t nseq, int64_t total_len, int64_t nheads_k, int64_t nheads_v,
                                                 int64_t headdim_k, int64_t headdim_v, int dtype,
                                                 int with_chunk_states) {
  return query(nseq, total_len, nheads_k, nheads_v, headdim_k, headdim_v, true, dtype, with_chunk_states);
}

}  // extern "C"
