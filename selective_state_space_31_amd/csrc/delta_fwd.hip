// delta_fwd.hip -- the gated delta rule over whole and packed sequences, behind
// ssm_delta_rule_fwd and _fwd_varlen of include/ssm_layer.h.
#include "delta.hpp"

namespace ssm {
namespace {

size_t fwd_bytes(const DeltaDims& d, int dtype) {
  (void)d;
  (void)dtype;
  return 0;
}

int delta_fwd(const char* fn, const void* q, const void* k, const void* v, const float* beta, const float* g,
              float scale, void* out, float* last, const float* first, float* mids, const int32_t* cu, bool packed,
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
  if (L > 0 && (!q || !k || !v || !beta || !out))
    return fail(SSM_ERR_NULL, "%s: q, k, v, beta and out are required", fn);
  const size_t es = dtype == SSM_DTYPE_F32 ? 4 : 2;
  const struct { const void* p; size_t k; const char* n; } al[] = {
      {q, es, "q"}, {k, es, "k"}, {v, es, "v"}, {out, es, "out"}, {beta, 4, "beta"}, {g, 4, "g"},
      {first, 4, "initial_state"}, {last, 4, "last_state"}, {mids, 4, "chunk_states"}, {cu, 4, "cu_seqlens"}};
  for (const auto& e : al)
    if (e.p && !aligned(e.p, e.k)) return fail(SSM_ERR_ALIGN, "%s: %s is not %zu-byte aligned", fn, e.n, e.k);
  const size_t gate = static_cast<size_t>(d.tokens()) * hv * 4, st = nseq * d.state_values() * 4;
  const size_t need = fwd_bytes(d, dtype);
  const Span ins[] = {{q, strided_bytes(d.tokens(), hk * K, qs, es), "q"},
                      {k, strided_bytes(d.tokens(), hk * K, ks, es), "k"},
                      {v, strided_bytes(d.tokens(), hv * V, vs, es), "v"},
                      {beta, gate, "beta"},
                      {g, g ? gate : 0, "g"},
                      {first, first ? st : 0, "initial_state"},
                      {cu, packed ? static_cast<size_t>(nseq + 1) * 4 : 0, "cu_seqlens"}};
  const Span outs[] = {{out, static_cast<size_t>(d.tokens()) * hv * V * es, "out"},
                       {last, last ? st : 0, "last_state"},
                       {mids, mids ? d.chunks() * d.state_values() * 4 : 0, "chunk_states"},
                       {ws, ws ? need : 0, "workspace"}};
  for (const auto& o : outs)
    for (const auto& n : ins)
      if (overlap(o, n) && !(o.p == last && n.p == first && last == first))
        return fail(SSM_ERR_ALIAS, "%s: output %s overlaps input %s", fn, o.name, n.name);
  for (int a = 0; a < 4; ++a)
    for (int b = a + 1; b < 4; ++b)
      if (overlap(outs[a], outs[b]))
        return fail(SSM_ERR_ALIAS, "%s: %s overlaps %s", fn, outs[a].name, outs[b].name);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(SSM_ERR_WORKSPACE, "%s: workspace of %zu bytes given, %zu needed", fn, ws ? ws_bytes : 0, need);
  if (need > 0 && !aligned(ws, 256))
    return fail(SSM_ERR_ALIGN, "%s: workspace is not 256-byte aligned", fn);
  if (L == 0 && !last) return SSM_OK;
  return delta_walk(fn, dtype, q, k, v, beta, g, scale, out, last, first, mids, packed ? cu : nullptr, d, stream);
}

size_t query(int64_t nseq, int64_t L, int64_t hk, int64_t hv, int64_t K, int64_t V, bool packed, int dtype) {
  if ((dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16) || !delta_sizes_ok(nseq, L, hk, hv, K, V, packed)) return 0;
  return fwd_bytes(DeltaDims{nseq, L, static_cast<int>(hk), static_cast<int>(hv), static_cast<int>(K),
                             static_cast<int>(V), hk * K, hk * K, hv * V, packed},
                   dtype);
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" {

int ssm_delta_rule_fwd(const void* q, const void* k, const void* v, const float* beta, const float* g, float scale,
                       void* out, float* last_state, const float* initial_state, float* chunk_states, int64_t batch,
                       int64_t seqlen, int64_t nheads_k, int64_t nheads_v, int64_t headdim_k, int64_t headdim_v,
                       int64_t q_token_stride, int64_t k_token_stride, int64_t v_token_stride, int dtype,
                       void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return delta_fwd("ssm_delta_rule_fwd", q, k, v, beta, g, scale, out, last_state, initial_state, chunk_states,
                   nullptr, false, batch, seqlen, nheads_k, nheads_v, headdim_k, headdim_v, q_token_stride,
                   k_token_stride, v_token_stride, dtype, workspace, workspace_bytes, stream);
}

size_t ssm_delta_rule_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads_k, int64_t nheads_v,
                                          int64_t headdim_k, int64_t headdim_v, int dtype) {
  return query(batch, seqlen, nheads_k, nheads_v, headdim_k, headdim_v, false, dtype);
}

int ssm_delta_rule_fwd_varlen(const void* q, const void* k, const void* v, const float* beta, const float* g,
                              float scale, void* out, float* last_state, const float* initial_state,
                              float* chunk_states, const int32_t* cu_seqlens, int64_t nseq, int64_t total_len,
                              int64_t nheads_k, int64_t nheads_v, int64_t headdim_k, int64_t headdim_v,
                              int64_t q_token_stride, int64_t k_token_stride, int64_t v_token_stride, int dtype,
                              void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return delta_fwd("ssm_delta_rule_fwd_varlen", q, k, v, beta, g, scale, out, last_state, initial_state, chunk_states,
                   cu_seqlens, true, nseq, total_len, nheads_k, nheads_v, headdim_k, headdim_v, q_token_stride,
                   k_token_stride, v_token_stride, dtype, workspace, workspace_bytes, stream);
}

size_t ssm_delta_rule_fwd_varlen_workspace_bytes(int64_t nseq, int64_t total_len, int64_t nheads_k, int64_t nheads_v,
                                                 int64_t headdim_k, int64_t headdim_v, int dtype) {
  return query(nseq, total_len, nheads_k, nheads_v, headdim_k, headdim_v, true, dtype);
}

}  // extern "C"
