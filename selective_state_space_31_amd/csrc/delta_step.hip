// delta_step.hip -- the gated delta rule token by token: one decoding step
// (ssm_delta_state_update of include/ssm_layer.h) and sequences of few tokens.
//
//   S' = e^g S;  u = beta (v - S'^T k);  S = S' + k u^T;
//   out = scale S^T q = scale (e^g S_old^T q + (k.q) u)
// so one sweep over the old state gives both sums (S^T k, S^T q), and the state
// is read once and written once: memory bounds it.  A workgroup holds all rows
// of the columns it takes in registers, over all tokens of its sequence.
#include "delta.hpp"

namespace ssm {
namespace {

template <typename TA>
struct WalkArgs {
  const float* first;  // state before the sequence, or NULL (zeros)
  float* last;         // state behind it, or NULL; may be `first`
  float* mids;         // states before every kDeltaC-th token, or NULL
  const TA *q, *k, *v;
  const float *beta, *g;
  TA* out;
  const int32_t* cu;  // packed: offsets, else NULL
  float scale;
  int hk, hv, K, V, tiles;
  int64_t L, qs, ks, vs;
};

// 256 threads: TPR lanes side by side take VEC columns each, 256 / TPR rows at
// a time, R of them a thread.
template <typename TA, int VEC, int TPR, int R>
__global__ void __launch_bounds__(256) delta_walk_kernel(const WalkArgs<TA> p) {
  constexpr int ROWS = 256 / TPR;
  struct __attribute__((aligned(4 * VEC))) Cols { float x[VEC]; };
  static_assert(ROWS * R <= 256 && kDeltaMaxWidth == 256, "one thread stages one row");
  __shared__ float sk[256], sq[256];
  __shared__ float red[2][4][TPR * VEC], redkq[4];
  const int tid = static_cast<int>(threadIdx.x), w = tid >> 6;
  const int tile = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.tiles));
  const int64_t bh = blockIdx.x / static_cast<unsigned>(p.tiles);
  const int64_t b = bh / p.hv;
  const int h = static_cast<int>(bh - b * p.hv), j = h / (p.hv / p.hk);
  const int col = tid % TPR, c0 = (tile * TPR + col) * VEC, row = tid / TPR;
  const bool mine = c0 < p.V;  // (V is a multiple of VEC)
  const DeltaSeq q = delta_seq(p.cu, b, p.L);
  const size_t sv = static_cast<size_t>(p.K) * p.V, at = static_cast<size_t>(row) * p.V + c0;
  const size_t hop = static_cast<size_t>(ROWS) * p.V, mv = sv + static_cast<size_t>(kDeltaC) * p.V;
  Cols s[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (p.first && mine && row + i * ROWS < p.K)
      s[i] = *reinterpret_cast<const Cols*>(p.first + bh * sv + at + i * hop);
    else
      s[i] = Cols{};
  }
  for (int64_t t = q.lo; t < q.hi; ++t) {
    if (p.mids && (t - q.lo) % kDeltaC == 0 && mine) {
      float* const m = p.mids + ((q.slot + (t - q.lo) / kDeltaC) * p.hv + h) * mv + at;
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (row + i * ROWS < p.K) *reinterpret_cast<Cols*>(m + i * hop) = s[i];
    }
    if (t > q.lo) __syncthreads();  // (the token before is done with LDS)
    sk[tid] = tid < p.K ? to_f32(p.k[t * p.ks + j * p.K + tid]) : 0.0f;  // (rows behind K stay zero)
    sq[tid] = tid < p.K ? to_f32(p.q[t * p.qs + j * p.K + tid]) : 0.0f;
    float vv[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) vv[e] = mine ? to_f32(p.v[t * p.vs + h * p.V + c0 + e]) : 0.0f;
    const float beta = p.beta[t * p.hv + h], decay = p.g ? expf(p.g[t * p.hv + h]) : 1.0f;
    __syncthreads();
    float tk[VEC], tq[VEC], kq = 0.0f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) tk[e] = tq[e] = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float kr = sk[row + i * ROWS], qr = sq[row + i * ROWS];
      kq = __builtin_fmaf(kr, qr, kq);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        tk[e] = __builtin_fmaf(kr, s[i].x[e], tk[e]);
        tq[e] = __builtin_fmaf(qr, s[i].x[e], tq[e]);
      }
    }
#pragma unroll
    for (int m = TPR; m < 64; m <<= 1) {
      kq += __shfl_xor(kq, m);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        tk[e] += __shfl_xor(tk[e], m);
        tq[e] += __shfl_xor(tq[e], m);
      }
    }
    if ((tid & 63) < TPR) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        red[0][w][col * VEC + e] = tk[e];
        red[1][w][col * VEC + e] = tq[e];
      }
      if ((tid & 63) == 0) redkq[w] = kq;
    }
    __syncthreads();
    kq = (redkq[0] + redkq[1]) + (redkq[2] + redkq[3]);
    float u[VEC], miss[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int c = col * VEC + e;
      const float a = (red[0][0][c] + red[0][1][c]) + (red[0][2][c] + red[0][3][c]);
      const float o = (red[1][0][c] + red[1][1][c]) + (red[1][2][c] + red[1][3][c]);
      miss[e] = vv[e] - decay * a;
      u[e] = beta * miss[e];
      vv[e] = p.scale * __builtin_fmaf(kq, u[e], decay * o);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float kr = sk[row + i * ROWS];
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[i].x[e] = __builtin_fmaf(kr, u[e], decay * s[i].x[e]);
    }
    if (p.mids && row == 0 && mine) {  // (behind the last token zeros complete its chunk)
      float* const m = p.mids + ((q.slot + (t - q.lo) / kDeltaC) * p.hv + h) * mv + sv + c0;
      for (int64_t i = (t - q.lo) % kDeltaC; i < (t + 1 < q.hi ? (t - q.lo) % kDeltaC + 1 : kDeltaC); ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) m[i * p.V + e] = i == (t - q.lo) % kDeltaC ? miss[e] : 0.0f;
    }
    if (row == 0 && mine) {
      TA* const o = p.out + (static_cast<size_t>(t) * p.hv + h) * p.V + c0;
#pragma unroll
      for (int e = 0; e < VEC; ++e) store_act(o + e, vv[e]);
    }
  }
  if (!p.last || !mine) return;
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (row + i * ROWS < p.K) *reinterpret_cast<Cols*>(p.last + bh * sv + at + i * hop) = s[i];
}

template <int N>
struct Count {
  static constexpr int value = N;
};

template <typename TA>
int launch_walk(const char* fn, const void* q, const void* k, const void* v, const float* beta, const float* g,
                float scale, void* out, float* last, const float* first, float* mids, const int32_t* cu,
                const DeltaDims& d, hipStream_t stream) {
  WalkArgs<TA> a{first, last, mids, static_cast<const TA*>(q), static_cast<const TA*>(k), static_cast<const TA*>(v),
                 beta, g, static_cast<TA*>(out), cu, scale, d.hk, d.hv, d.K, d.V, 1, d.L, d.qs, d.ks, d.vs};
  const auto go = [&](auto vec, auto tpr, auto rows) {
    constexpr int VEC = decltype(vec)::value, TPR = decltype(tpr)::value, R = decltype(rows)::value;
    a.tiles = (d.V + VEC * TPR - 1) / (VEC * TPR);
    const unsigned grid = static_cast<unsigned>(d.nseq * d.hv * a.tiles);
    hipLaunchKernelGGL((delta_walk_kernel<TA, VEC, TPR, R>), dim3(grid), dim3(256), 0, stream, a);
  };
  const auto deep = [&](auto vec, auto tpr) {
    constexpr int MOST = decltype(tpr)::value;  // rows a thread of 256
    if (d.K <= 64) go(vec, tpr, Count<MOST / 4>{});
    else if (d.K <= 128) go(vec, tpr, Count<MOST / 2>{});
    else go(vec, tpr, Count<MOST>{});
  };
  // Four columns a lane where alignment allows (then eight lanes, 32 columns a
  // workgroup: 1 x 16 heads of 128 4.0 us, with 32 lanes 6.4; 256 x 12 of 128 x 64
  // 35 and 42; 256 x 40 of 128, float32, 264 and 264, 5.1 TB/s).
  const bool quads = d.V % 4 == 0 && aligned(first, 16) && aligned(last, 16) && aligned(mids, 16);
  if (quads) deep(Count<4>{}, Count<8>{});
  else deep(Count<1>{}, Count<32>{});
  return launch_status(fn);
}

}  // namespace

int delta_walk(const char* fn, int dtype, const void* q, const void* k, const void* v, const float* beta,
               const float* g, float scale, void* out, float* last, const float* first, float* mids,
               const int32_t* cu, const DeltaDims& d, hipStream_t stream) {
  return dtype == SSM_DTYPE_F32
             ? launch_walk<float>(fn, q, k, v, beta, g, scale, out, last, first, mids, cu, d, stream)
             : launch_walk<bf16_t>(fn, q, k, v, beta, g, scale, out, last, first, mids, cu, d, stream);
}

}  // namespace ssm

using namespace ssm;

extern "C" int ssm_delta_state_update(float* state, const void* q, const void* k, const void* v, const float* beta,
                                      const float* g, float scale, void* out, int64_t batch, int64_t nheads_k,
                                      int64_t nheads_v, int64_t headdim_k, int64_t headdim_v, int64_t q_stride,
                                      int64_t k_stride, int64_t v_stride, int dtype, hipStream_t stream) {
  clear_error();
  const char* fn = "ssm_delta_state_update";
  if (dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16)
    return fail(SSM_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, dtype);
  if (batch < 1 || batch >= (int64_t{1} << 24) ||
      !delta_sizes_ok(1, 1, nheads_k, nheads_v, headdim_k, headdim_v, false) ||
      batch * nheads_v * ((headdim_v + 31) / 32) >= (int64_t{1} << 24))  // (less than 2^32 threads)
    return fail(SSM_ERR_SHAPE, "%s: bad sizes batch %lld, heads %lld and %lld, widths %lld and %lld", fn,
                (long long)batch, (long long)nheads_k, (long long)nheads_v, (long long)headdim_k,
                (long long)headdim_v);
  const DeltaDims d{batch, 1, static_cast<int>(nheads_k), static_cast<int>(nheads_v), static_cast<int>(headdim_k),
                    static_cast<int>(headdim_v), q_stride, k_stride, v_stride, false};
  if (!delta_strides_ok(d))
    return fail(SSM_ERR_SHAPE, "%s: bad strides %lld, %lld, %lld", fn, (long long)q_stride, (long long)k_stride,
                (long long)v_stride);
  if (!state || !q || !k || !v || !beta || !out)
    return fail(SSM_ERR_NULL, "%s: state, q, k, v, beta and out are required", fn);
  const size_t es = dtype == SSM_DTYPE_F32 ? 4 : 2;
  const struct { const void* p; size_t k; const char* n; } al[] = {
      {state, 4, "state"}, {q, es, "q"}, {k, es, "k"}, {v, es, "v"}, {out, es, "out"}, {beta, 4, "beta"}, {g, 4, "g"}};
  for (const auto& e : al)
    if (e.p && !aligned(e.p, e.k)) return fail(SSM_ERR_ALIGN, "%s: %s is not %zu-byte aligned", fn, e.n, e.k);
  const size_t gate = static_cast<size_t>(batch) * d.hv * 4;
  const Span ins[] = {{q, strided_bytes(batch, int64_t{d.hk} * d.K, d.qs, es), "q"},
                      {k, strided_bytes(batch, int64_t{d.hk} * d.K, d.ks, es), "k"},
                      {v, strided_bytes(batch, int64_t{d.hv} * d.V, d.vs, es), "v"}, {beta, gate, "beta"},
                      {g, g ? gate : 0, "g"}};
  const Span outs[] = {{out, static_cast<size_t>(batch) * d.hv * d.V * es, "out"},
                       {state, static_cast<size_t>(batch) * d.state_values() * 4, "state"}};
  for (const auto& o : outs)
    for (const auto& n : ins)
      if (overlap(o, n)) return fail(SSM_ERR_ALIAS, "%s: %s overlaps input %s", fn, o.name, n.name);
  if (overlap(outs[0], outs[1])) return fail(SSM_ERR_ALIAS, "%s: out overlaps state", fn);
  return delta_walk(fn, dtype, q, k, v, beta, g, scale, out, state, state, nullptr, nullptr, d, stream);
}
