// delta_fwd.hip -- the gated delta rule over whole and packed sequences, behind
// ssm_delta_rule_fwd and _fwd_varlen of include/ssm_layer.h.
#include "delta.hpp"

namespace ssm {
namespace {

template <typename TA>
struct RecArgs {
  const TA* v;
  TA* out;
  const float* first;
  float *last, *mids;
  const int32_t* cu;
  ChunkSpace c;
  float scale;
  int64_t nseq, L, vs;
  int hk, hv, K, V, slices;
};

// The chunks one after another.  With S0 the state before a chunk, per column
// block of 16 NC values:
//   X = V - gamma (K S0);  U = T diag(beta) X;  out = scale (gamma (Q S0) + P U)
//   S1 = gamma_C S0 + K^T (d U)
// A workgroup of four waves takes one column block of a head (columns do not
// meet): wave w the tokens 16 w .. + 15 of X, U and out, and every fourth row
// block of S, which stays in its registers.  S, X, U and d U pass through LDS as
// right operands in bf16 parts; the left operands come from memory as fragments,
// each needed by one wave alone, the next chunk's while this one is worked on.
template <typename TA, int KT, int NC, bool MIDS>
__global__ void __launch_bounds__(256) delta_rec_kernel(const RecArgs<TA> p) {
  constexpr int IN = ActParts<TA>::in, OUT = ActParts<TA>::out, TW = (KT + 1) / 2;
  __shared__ u32x4 sS[3][KT][NC][64], sX[3][2][NC][64], sU[OUT][2][NC][64], sD[3][2][NC][64];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  // The workgroups of a head read the same fragments: they go to the same XCD
  // (workgroups are dealt to the eight XCDs in turn).
  const unsigned group = blockIdx.x / (8u * static_cast<unsigned>(p.slices)), in = blockIdx.x % (8u * static_cast<unsigned>(p.slices));
  const int64_t pair = int64_t{group} * 8 + (in & 7);
  if (pair >= p.nseq * p.hv) return;
  const int slice = static_cast<int>(in >> 3), c0 = slice * 16 * NC;
  const int64_t b = pair / p.hv;
  const int h = static_cast<int>(pair - b * p.hv), j = h / (p.hv / p.hk);
  const DeltaSeq q = delta_seq(p.cu, b, p.L);
  const int nc = static_cast<int>((q.hi - q.lo + kDeltaC - 1) / kDeltaC);
  const size_t sv = static_cast<size_t>(p.K) * p.V, mv = sv + static_cast<size_t>(kDeltaC) * p.V;
  const bool tiles = TW > 1 || w < 2 * KT;  // (with 32 rows two waves hold none)

  // state values of this lane: row block t, column block nb
  const auto state_io = [&](auto&& f) {
#pragma unroll
    for (int i = 0; i < TW; ++i)
#pragma unroll
      for (int nb = 0; nb < NC; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * (w + 4 * i) + 4 * g + r, col = c0 + 16 * nb + n;
          if (tiles && row < p.K && col < p.V) f(i, nb, r, static_cast<size_t>(row) * p.V + col);
        }
  };
  f32x4 S[TW][NC];
#pragma unroll
  for (int i = 0; i < TW; ++i)
#pragma unroll
    for (int nb = 0; nb < NC; ++nb) S[i][nb] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (p.first) {
    const float* const src = p.first + pair * sv;
    state_io([&](int i, int nb, int r, size_t at) { S[i][nb][r] = src[at]; });
  }
  const auto put_state = [&]() {
    if (tiles)
#pragma unroll
      for (int i = 0; i < TW; ++i)
#pragma unroll
        for (int nb = 0; nb < NC; ++nb) put_parts<3, NC>(&sS[0][0][0][0], KT, w + 4 * i, nb, lane, S[i][nb]);
  };
  if (nc > 0) put_state();

  // left operands of one chunk
  u32x4 fk[KT][IN], fq[KT][IN], ft[2][3], fp[2][OUT], fkt[TW][2][IN];
  float ga[4], de[4], gC;
  TA rv[NC][4];
  const int kbs = w < 2 ? 1 : 2;
  const auto load_kq = [&](int64_t slot) {
    const size_t at = static_cast<size_t>(slot * p.hk + j) * IN * 4 * KT * 64 + lane;
#pragma unroll
    for (int kb = 0; kb < KT; ++kb)
#pragma unroll
      for (int i = 0; i < IN; ++i) {
        fk[kb][i] = p.c.kf[at + ((i * 4 + w) * KT + kb) * 64];
        fq[kb][i] = p.c.qf[at + ((i * 4 + w) * KT + kb) * 64];
      }
  };
  const auto load_v = [&](int64_t slot, int64_t t0) {
    const float* const vec = p.c.vec + (slot * p.hv + h) * 2 * kDeltaC;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      ga[r] = vec[16 * w + 4 * g + r];
      de[r] = vec[kDeltaC + 16 * w + 4 * g + r];
      const int64_t t = t0 + 16 * w + 4 * g + r;
#pragma unroll
      for (int nb = 0; nb < NC; ++nb) {
        const int col = c0 + 16 * nb + n;
        rv[nb][r] = TA{};
        if (t < q.hi && col < p.V) rv[nb][r] = p.v[t * p.vs + h * p.V + col];
      }
    }
    gC = vec[kDeltaC - 1];
  };
  const auto load_t = [&](int64_t slot) {
    const size_t at = static_cast<size_t>(slot * p.hv + h) * 3 * kTri * 64 + lane;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (kb < kbs) ft[kb][i] = p.c.tf[at + (i * kTri + tri_at(w, kb)) * 64];
  };
  const auto load_pkt = [&](int64_t slot) {
    const size_t at = static_cast<size_t>(slot * p.hv + h) * OUT * kTri * 64 + lane;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < OUT; ++i)
        if (kb < kbs) fp[kb][i] = p.c.pf[at + (i * kTri + tri_at(w, kb)) * 64];
    const size_t kt = static_cast<size_t>(slot * p.hk + j) * IN * 2 * KT * 2 * 64 + lane;
    if (tiles)
#pragma unroll
      for (int x = 0; x < TW; ++x)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int i = 0; i < IN; ++i) fkt[x][kb][i] = p.c.ktf[kt + ((i * 2 * KT + w + 4 * x) * 2 + kb) * 64];
  };
  if (nc > 0) {
    load_kq(q.slot);
    load_v(q.slot, q.lo);
    load_t(q.slot);
    load_pkt(q.slot);
  }
  __syncthreads();
  for (int c = 0; c < nc; ++c) {
    const int64_t slot = q.slot + c, t0 = q.lo + int64_t{c} * kDeltaC;
    const int more = c + 1 < nc ? 1 : 0;  // (the last chunk's loads ahead are its own again)
    if constexpr (MIDS) {
      float* const dst = p.mids + (slot * p.hv + h) * mv;
      state_io([&](int i, int nb, int r, size_t at) { dst[at] = S[i][nb][r]; });
    }
    // ---- X and Q S0 ----
    f32x4 o[NC];
#pragma unroll
    for (int nb = 0; nb < NC; ++nb) {
      f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f}, y = x;
#pragma unroll
      for (int kb = 0; kb < KT; ++kb) {
        u32x4 s[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) s[i] = sS[i][kb][nb][lane];
        x = mul_parts<3>(fk[kb], s, x);
        y = mul_parts<OUT>(fq[kb], s, y);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        o[nb][r] = ga[r] * y[r];
        x[r] = to_f32(rv[nb][r]) - ga[r] * x[r];
      }
      put_parts<3, NC>(&sX[0][0][0][0], 2, w, nb, lane, x);
    }
    load_kq(slot + more);
    float dl[4];
    const float decay = gC;
#pragma unroll
    for (int r = 0; r < 4; ++r) dl[r] = de[r];
    load_v(slot + more, t0 + more * kDeltaC);
    __syncthreads();
    // ---- U ----
#pragma unroll
    for (int nb = 0; nb < NC; ++nb) {
      f32x4 u = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        if (kb >= kbs) break;
        u32x4 x[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) x[i] = sX[i][kb][nb][lane];
        u = mul_parts<3>(ft[kb], x, u);
      }
      put_parts<OUT, NC>(&sU[0][0][0][0], 2, w, nb, lane, u);
      if constexpr (MIDS) {
        const int col = c0 + 16 * nb + n;
        float* const dst = p.mids + (slot * p.hv + h) * mv + sv + col;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (col < p.V) dst[static_cast<size_t>(16 * w + 4 * g + r) * p.V] = u[r];
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) u[r] *= dl[r];
      put_parts<3, NC>(&sD[0][0][0][0], 2, w, nb, lane, u);
    }
    load_t(slot + more);
    __syncthreads();
    // ---- S1, then out ----
    if (tiles) {
#pragma unroll
      for (int nb = 0; nb < NC; ++nb)
#pragma unroll
        for (int i = 0; i < TW; ++i) S[i][nb] *= decay;
#pragma unroll
      for (int nb = 0; nb < NC; ++nb)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          u32x4 u[3];
#pragma unroll
          for (int i = 0; i < 3; ++i) u[i] = sD[i][kb][nb][lane];
#pragma unroll
          for (int i = 0; i < TW; ++i) S[i][nb] = mul_parts<3>(fkt[i][kb], u, S[i][nb]);
        }
      put_state();
    }
#pragma unroll
    for (int nb = 0; nb < NC; ++nb) {
#pragma unroll
      for (int kb = 0; kb < 2; ++kb) {
        if (kb >= kbs) break;
        u32x4 u[OUT];
#pragma unroll
        for (int i = 0; i < OUT; ++i) u[i] = sU[i][kb][nb][lane];
        o[nb] = mul_parts<OUT>(fp[kb], u, o[nb]);
      }
      const int col = c0 + 16 * nb + n;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t t = t0 + 16 * w + 4 * g + r;
        if (p.out && t < q.hi && col < p.V) store_act(p.out + (t * p.hv + h) * p.V + col, p.scale * o[nb][r]);
      }
    }
    load_pkt(slot + more);
    __syncthreads();
  }
  if (p.last) {
    float* const dst = p.last + pair * sv;
    state_io([&](int i, int nb, int r, size_t at) { dst[at] = S[i][nb][r]; });
  }
}

template <typename TA, int KT, int NC>
void launch_rec(const RecArgs<TA>& a, hipStream_t stream) {
  const int64_t pairs = a.nseq * a.hv;
  const dim3 grid(static_cast<unsigned>((pairs + 7) / 8 * 8 * a.slices)), block(256);
  if (a.mids) hipLaunchKernelGGL((delta_rec_kernel<TA, KT, NC, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((delta_rec_kernel<TA, KT, NC, false>), grid, block, 0, stream, a);
}

template <typename TA>
void run_chunks(const void* v, float scale, void* out, float* last, const float* first, float* mids,
                const int32_t* cu, const DeltaDims& d, const ChunkSpace& c, hipStream_t stream) {
  RecArgs<TA> a{static_cast<const TA*>(v), static_cast<TA*>(out), first, last, mids, cu, c, scale, d.nseq, d.L, d.vs,
                d.hk, d.hv, d.K, d.V, (d.V + 15) / 16};
  switch (delta_kt(d.K)) {
    case 1: launch_rec<TA, 1, 1>(a, stream); break;
    case 2: launch_rec<TA, 2, 1>(a, stream); break;
    case 4: launch_rec<TA, 4, 1>(a, stream); break;
    default: launch_rec<TA, 8, 1>(a, stream); break;
  }
}

size_t fwd_bytes(const DeltaDims& d, int dtype) { return chunk_space(d, dtype, false, nullptr, nullptr); }

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
                       {mids, mids ? d.mid_values() * 4 : 0, "chunk_states"},
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
  if (!packed) cu = nullptr;
  ChunkSpace c;
  chunk_space(d, dtype, false, static_cast<char*>(ws), &c);
  if (L > 0) delta_prep(dtype, false, q, k, beta, g, cu, d, c, stream);
  delta_chunks(dtype, v, scale, out, last, first, mids, cu, d, c, stream);
  return launch_status(fn);
}

size_t query(int64_t nseq, int64_t L, int64_t hk, int64_t hv, int64_t K, int64_t V, bool packed, int dtype) {
  if ((dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16) || !delta_sizes_ok(nseq, L, hk, hv, K, V, packed)) return 0;
  return fwd_bytes(DeltaDims{nseq, L, static_cast<int>(hk), static_cast<int>(hv), static_cast<int>(K),
                             static_cast<int>(V), hk * K, hk * K, hv * V, packed},
                   dtype);
}

}  // namespace

void delta_chunks(int dtype, const void* v, float scale, void* out, float* last, const float* first, float* mids,
                  const int32_t* cu, const DeltaDims& d, const ChunkSpace& c, hipStream_t stream) {
  if (dtype == SSM_DTYPE_F32) run_chunks<float>(v, scale, out, last, first, mids, cu, d, c, stream);
  else run_chunks<bf16_t>(v, scale, out, last, first, mids, cu, d, c, stream);
}

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
