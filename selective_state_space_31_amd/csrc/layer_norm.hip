// layer_norm.hip -- layer norm over the rows of a residual stream with the sum
// in the same pass, and its gradients, behind the C ABI in
// include/ssm_layer.h.
//
//   s = x + residual (rounded), c = s - mean(s), r = 1 / sqrt(mean(c^2) + eps)
//   out = c r w + b
//   with h = c r, y = dout: dx = r (y w - mean(y w) - h mean(y w h)) + dresidual,
//   dw = sum y h, db = sum y.
// A row stays in the registers of one wave (or, wide ones and few ones, of four
// or sixteen waves), so the mean square is taken around the mean itself and
// every value is read once and written once: memory bounds it.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ssm_layer.h"

#include "host_util.hpp"
#include "kernels.hpp"

namespace ssm {
namespace {

constexpr int64_t kNormMaxDim = 16384;
constexpr int kNormWavesPerCu = 32;   // forward: more rows than that go round
constexpr int kNormMaxParts = 512;  // workgroups that leave partial weight gradients

// 16 bytes of a row; rows may start anywhere, so the compiler is told of no
// alignment (the hardware takes unaligned vector accesses)
template <typename TA>
struct Piece {
  static constexpr int n = 16 / static_cast<int>(sizeof(TA));
  TA v[n];
};

template <typename TA, int NV>
struct NormRow {
  static constexpr int VEC = Piece<TA>::n;
  float v[NV][VEC];

  // values `first + i step ..` of the row p of dim values; zeros behind it
  __device__ __forceinline__ void load(const TA* p, int first, int step, int dim) {
    Piece<TA> raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first + i * step;
      if (c + VEC <= dim) {
        __builtin_memcpy(&raw[i], p + c, sizeof(raw[i]));
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          if (c + j < dim) raw[i].v[j] = p[c + j];
          else raw[i].v[j] = TA{};
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) v[i][j] = to_f32(raw[i].v[j]);
  }
  __device__ __forceinline__ void store(TA* p, int first, int step, int dim) const {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first + i * step;
      Piece<TA> raw;
#pragma unroll
      for (int j = 0; j < VEC; ++j) store_act(&raw.v[j], v[i][j]);
      if (c + VEC <= dim) {
        __builtin_memcpy(p + c, &raw, sizeof(raw));
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          if (c + j < dim) p[c + j] = raw.v[j];
      }
    }
  }
  // rounds every value to TA, as a store and a load would
  __device__ __forceinline__ void round() {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        TA t;
        store_act(&t, v[i][j]);
        v[i][j] = to_f32(t);
      }
  }
};

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) x += __shfl_xor(x, m);
  return x;
}

// Sum over the WPR waves of a row (a fixed order).  A slot is written again
// only behind the barrier of another one, so one barrier a sum is enough.
template <int WPR>
__device__ __forceinline__ float row_sum(float x, float* red, int slot) {
  x = wave_sum(x);
  if constexpr (WPR > 1) {
    const int w = static_cast<int>(threadIdx.x >> 6);
    if ((threadIdx.x & 63) == 0) red[slot * WPR + w] = x;
    __syncthreads();
    x = 0.0f;
#pragma unroll
    for (int i = 0; i < WPR; ++i) x += red[slot * WPR + i];
  }
  return x;
}

// Weights of a lane's columns, float32 (`fill` without the array)
template <int NV, int VEC>
__device__ __forceinline__ void load_param(float (&w)[NV][VEC], const float* p, float fill, int first,
                                           int step, int dim) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = first + i * step;
#pragma unroll
    for (int j = 0; j < VEC; ++j) w[i][j] = fill;
    if (!p) continue;
    if (c + VEC <= dim) {
      __builtin_memcpy(&w[i], p + c, sizeof(w[i]));
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (c + j < dim) w[i][j] = p[c + j];
    }
  }
}

template <typename TA>
struct NormArgs {
  const TA *x, *res;  // forward: x and residual; backward: s and dout
  const TA* dres;
  const float *w, *b;
  TA *out, *sum;  // backward: dx in out
  float* part;    // backward: (parts, 2, dim)
  float eps;
  int64_t rows, xs, rs;
  int dim;
};

// c = s - mean(s) in place, and 1 / sqrt(mean(c^2) + eps)
template <int WPR, typename TA, int NV>
__device__ __forceinline__ float centre(NormRow<TA, NV>& s, float* red, int first, int step, int dim,
                                        float eps) {
  constexpr int VEC = NormRow<TA, NV>::VEC;
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) t += s.v[i][j];
  const float inv = 1.0f / static_cast<float>(dim), mean = row_sum<WPR>(t, red, 0) * inv;
  t = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      s.v[i][j] = first + i * step + j < dim ? s.v[i][j] - mean : 0.0f;
      t = __builtin_fmaf(s.v[i][j], s.v[i][j], t);
    }
  return 1.0f / sqrtf(__builtin_fmaf(row_sum<WPR>(t, red, 1), inv, eps));
}

// Each row group (a wave, or WPR of them) goes through every gridDim-th row
// with its columns' weights in registers.
template <typename TA, int NV, int WPR, bool RES>
__global__ void __launch_bounds__(WPR > 4 ? 64 * WPR : 256)
    norm_fwd_kernel(const NormArgs<TA> p) {
  constexpr int VEC = Piece<TA>::n, step = 64 * WPR * VEC, GROUPS = WPR == 1 ? 4 : 1;
  __shared__ float red[2 * WPR];
  const int tid = static_cast<int>(threadIdx.x);
  const int lane = WPR == 1 ? tid & 63 : tid, group = WPR == 1 ? tid >> 6 : 0;
  const int first = lane * VEC, dim = p.dim;
  const int64_t hop = int64_t{gridDim.x} * GROUPS;
  int64_t row = int64_t{blockIdx.x} * GROUPS + group;
  if (row >= p.rows) return;  // (whole waves, and no barrier with one wave a row)
  NormRow<TA, NV> s, r;
  s.load(p.x + row * p.xs, first, step, dim);
  if constexpr (RES) r.load(p.res + row * p.rs, first, step, dim);
  float w[NV][VEC], b[NV][VEC];
  load_param(w, p.w, 1.0f, first, step, dim);
  load_param(b, p.b, 0.0f, first, step, dim);
  for (;;) {
    if constexpr (RES) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) s.v[i][j] += r.v[i][j];
      s.round();
      if (p.sum) s.store(p.sum + row * dim, first, step, dim);
    }
    const float rstd = centre<WPR>(s, red, first, step, dim, p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) s.v[i][j] = __builtin_fmaf(s.v[i][j] * rstd, w[i][j], b[i][j]);
    s.store(p.out + row * dim, first, step, dim);
    row += hop;
    if (row >= p.rows) return;
    s.load(p.x + row * p.xs, first, step, dim);
    if constexpr (RES) r.load(p.res + row * p.rs, first, step, dim);
  }
}

// Gradients: each row group (a wave, or WPR of them) goes through every
// gridDim-th row with its columns' weight gradients in registers; the
// workgroup's groups are added through LDS, and the workgroup leaves one
// partial row.
template <typename TA, int NV, int WPR>
__global__ void __launch_bounds__(WPR > 4 ? 64 * WPR : 256)
    norm_bwd_kernel(const NormArgs<TA> p) {
  constexpr int VEC = Piece<TA>::n, step = 64 * WPR * VEC, GROUPS = WPR == 1 ? 4 : 1;
  __shared__ float red[4 * WPR];
  const int tid = static_cast<int>(threadIdx.x);
  const int lane = WPR == 1 ? tid & 63 : tid, group = WPR == 1 ? tid >> 6 : 0;
  const int first = lane * VEC, dim = p.dim;
  float dw[NV][VEC], db[NV][VEC], w[NV][VEC];
  load_param(w, p.w, 1.0f, first, step, dim);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dw[i][j] = db[i][j] = 0.0f;
  const int64_t hop = int64_t{gridDim.x} * GROUPS;
  for (int64_t row = int64_t{blockIdx.x} * GROUPS + group; row < p.rows; row += hop) {
    NormRow<TA, NV> s, y;
    s.load(p.x + row * p.xs, first, step, dim);
    y.load(p.res + row * dim, first, step, dim);
    const float rstd = centre<WPR>(s, red, first, step, dim, p.eps);
    float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float h = s.v[i][j] * rstd, g = y.v[i][j];
        dw[i][j] = __builtin_fmaf(g, h, dw[i][j]);
        db[i][j] += g;
        s.v[i][j] = h;
        y.v[i][j] = g * w[i][j];
        t0 += y.v[i][j];
        t1 = __builtin_fmaf(y.v[i][j], h, t1);
      }
    const float inv = 1.0f / static_cast<float>(dim);
    t0 = row_sum<WPR>(t0, red, 2) * inv;
    t1 = row_sum<WPR>(t1, red, 3) * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        y.v[i][j] = rstd * (y.v[i][j] - t0 - s.v[i][j] * t1);
    if (p.dres) {
      s.load(p.dres + row * dim, first, step, dim);
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) y.v[i][j] += s.v[i][j];
    }
    y.store(p.out + row * dim, first, step, dim);
  }
  if (!p.part) return;
  if constexpr (GROUPS > 1) {
    __shared__ float fold[2][64 * VEC];
    for (int g = 1; g < GROUPS; ++g)
      for (int i = 0; i < NV; ++i) {
        __syncthreads();
        if (group == g)
          for (int j = 0; j < VEC; ++j) {
            fold[0][j * 64 + lane] = dw[i][j];
            fold[1][j * 64 + lane] = db[i][j];
          }
        __syncthreads();
        if (group == 0)
          for (int j = 0; j < VEC; ++j) {
            dw[i][j] += fold[0][j * 64 + lane];
            db[i][j] += fold[1][j * 64 + lane];
          }
      }
    if (group != 0) return;
  }
  float* const o = p.part + int64_t{blockIdx.x} * 2 * dim;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int c = first + i * step + j;
      if (c < dim) {
        o[c] = dw[i][j];
        o[dim + c] = db[i][j];
      }
    }
}

// The partial rows' sum: a workgroup takes 64 of the 2 dim columns, its four
// waves every fourth row.
__global__ void __launch_bounds__(256)
    norm_reduce_kernel(const float* part, int parts, int dim, float* dw, float* db) {
  __shared__ float red[4][64];
  const int lane = static_cast<int>(threadIdx.x & 63), g = static_cast<int>(threadIdx.x >> 6);
  const int c = static_cast<int>(blockIdx.x) * 64 + lane, n = 2 * dim;
  float t = 0.0f;
  if (c < n)
    for (int i = g; i < parts; i += 4) t += part[static_cast<size_t>(i) * n + c];
  red[g][lane] = t;
  __syncthreads();
  if (g != 0 || c >= n) return;
  t = (red[0][lane] + red[1][lane]) + (red[2][lane] + red[3][lane]);
  if (c < dim) {
    if (dw) dw[c] = t;
  } else if (db) {
    db[c - dim] = t;
  }
}

template <int N>
struct Count {
  static constexpr int value = N;
};

// Calls go(NV, WPR) for the fewest waves a row fits with four pieces a lane;
// with few rows four waves share one.
template <typename TA, typename Go>
void norm_choose(int64_t rows, int dim, Go&& go) {
  constexpr int VEC = Piece<TA>::n;
  const int pieces = (dim + VEC - 1) / VEC;
  const auto with = [&](auto wpr) {
    constexpr int W = decltype(wpr)::value;
    const int nv = (pieces + 64 * W - 1) / (64 * W);
    if (nv <= 1) go(Count<1>{}, wpr);
    else if (nv <= 2) go(Count<2>{}, wpr);
    else if (nv <= 3) go(Count<3>{}, wpr);
    else go(Count<4>{}, wpr);
  };
  const bool few = rows < 4 * device_cus();
  if (pieces <= 64 * 4 && (!few || pieces <= 64)) with(Count<1>{});
  else if (pieces <= 256 * 4) with(Count<4>{});
  else with(Count<16>{});
}

int norm_parts(int64_t rows) {
  const int64_t n = (rows + 3) / 4;
  return static_cast<int>(n < 1 ? 1 : n > kNormMaxParts ? kNormMaxParts : n);
}

bool norm_sizes_ok(int64_t rows, int64_t dim, int64_t s0, int64_t s1) {
  const int64_t most = int64_t{1} << 30;
  return rows >= 0 && rows < (int64_t{1} << 31) && dim >= 1 && dim <= kNormMaxDim && s0 >= dim && s0 <= most &&
         s1 >= dim && s1 <= most;
}

size_t strided(int64_t rows, int64_t dim, int64_t stride, size_t es) {
  return rows > 0 ? (static_cast<size_t>(rows - 1) * stride + dim) * es : 0;
}

template <typename TA>
int launch_norm_fwd(const char* fn, const void* x, const void* res, const float* w, const float* b, float eps,
                    void* out, void* sum, int64_t rows, int dim, int64_t xs, int64_t rs, hipStream_t stream) {
  const NormArgs<TA> a{static_cast<const TA*>(x), static_cast<const TA*>(res), nullptr, w, b,
                       static_cast<TA*>(out), static_cast<TA*>(sum), nullptr, eps, rows, xs, rs, dim};
  norm_choose<TA>(rows, dim, [&](auto nv, auto wpr) {
    constexpr int NV = decltype(nv)::value, W = decltype(wpr)::value;
    const int64_t units = W == 1 ? (rows + 3) / 4 : rows, most = int64_t{device_cus()} * kNormWavesPerCu / (W == 1 ? 4 : W);
    const dim3 grid(static_cast<unsigned>(units < most ? units : most)), block(W == 1 ? 256 : 64 * W);
    if (res) hipLaunchKernelGGL((norm_fwd_kernel<TA, NV, W, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((norm_fwd_kernel<TA, NV, W, false>), grid, block, 0, stream, a);
  });
  return launch_status(fn);
}

template <typename TA>
int launch_norm_bwd(const char* fn, const void* s, const float* w, float eps, const void* dout, const void* dres,
                    void* dx, float* dw, float* db, int64_t rows, int dim, int64_t ss, float* part,
                    hipStream_t stream) {
  const int parts = norm_parts(rows);
  const NormArgs<TA> a{static_cast<const TA*>(s), static_cast<const TA*>(dout), static_cast<const TA*>(dres), w,
                       nullptr, static_cast<TA*>(dx), nullptr, dw || db ? part : nullptr, eps, rows, ss, dim, dim};
  norm_choose<TA>(rows, dim, [&](auto nv, auto wpr) {
    constexpr int NV = decltype(nv)::value, W = decltype(wpr)::value;
    hipLaunchKernelGGL((norm_bwd_kernel<TA, NV, W>), dim3(static_cast<unsigned>(parts)),
                       dim3(W == 1 ? 256 : 64 * W), 0, stream, a);
  });
  if (dw || db)
    hipLaunchKernelGGL(norm_reduce_kernel, dim3(static_cast<unsigned>((2 * dim + 63) / 64)), dim3(256), 0, stream,
                       part, parts, dim, dw, db);
  return launch_status(fn);
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" {

int ssm_layer_norm_fwd(const void* x, const void* residual, const float* weight, const float* bias, float eps,
                       void* out, void* residual_out, int64_t rows, int64_t dim, int64_t x_row_stride,
                       int64_t residual_row_stride, int dtype, hipStream_t stream) {
  clear_error();
  const char* fn = "ssm_layer_norm_fwd";
  if (dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16)
    return fail(SSM_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, dtype);
  if (!(eps >= 0.0f)) return fail(SSM_ERR_UNSUPPORTED, "%s: eps must be at least 0", fn);
  if (!residual) residual_row_stride = dim;
  if (!norm_sizes_ok(rows, dim, x_row_stride, residual_row_stride))
    return fail(SSM_ERR_SHAPE, "%s: bad sizes: %lld rows of %lld, strides %lld and %lld", fn, (long long)rows,
                (long long)dim, (long long)x_row_stride, (long long)residual_row_stride);
  if (residual_out && !residual) return fail(SSM_ERR_NULL, "%s: residual_out needs residual", fn);
  if (rows > 0 && (!x || !out)) return fail(SSM_ERR_NULL, "%s: x and out are required", fn);
  const size_t es = dtype == SSM_DTYPE_F32 ? 4 : 2;
  const struct { const void* p; size_t k; const char* n; } al[] = {
      {x, es, "x"}, {residual, es, "residual"}, {out, es, "out"}, {residual_out, es, "residual_out"},
      {weight, 4, "weight"}, {bias, 4, "bias"}};
  for (const auto& e : al)
    if (e.p && !aligned(e.p, e.k)) return fail(SSM_ERR_ALIGN, "%s: %s is not %zu-byte aligned", fn, e.n, e.k);
  const size_t pd = static_cast<size_t>(dim) * 4;
  const Span ins[] = {{x, strided(rows, dim, x_row_stride, es), "x"},
                      {residual, strided(rows, dim, residual_row_stride, es), "residual"},
                      {weight, weight ? pd : 0, "weight"}, {bias, bias ? pd : 0, "bias"}};
  const size_t whole = strided(rows, dim, dim, es);
  const Span outs[] = {{out, whole, "out"}, {residual_out, residual_out ? whole : 0, "residual_out"}};
  for (const auto& o : outs)
    for (const auto& n : ins)  // (in place: a row is read whole before it is written)
      if (overlap(o, n) && !(o.p == n.p && ((n.p == x && x_row_stride == dim) ||
                                            (n.p == residual && residual_row_stride == dim))))
        return fail(SSM_ERR_ALIAS, "%s: output %s overlaps input %s", fn, o.name, n.name);
  if (overlap(outs[0], outs[1])) return fail(SSM_ERR_ALIAS, "%s: out overlaps residual_out", fn);
  if (rows == 0) return SSM_OK;
  return dtype == SSM_DTYPE_F32
             ? launch_norm_fwd<float>(fn, x, residual, weight, bias, eps, out, residual_out, rows,
                                      static_cast<int>(dim), x_row_stride, residual_row_stride, stream)
             : launch_norm_fwd<bf16_t>(fn, x, residual, weight, bias, eps, out, residual_out, rows,
                                       static_cast<int>(dim), x_row_stride, residual_row_stride, stream);
}

size_t ssm_layer_norm_bwd_workspace_bytes(int64_t rows, int64_t dim, int dtype) {
  if ((dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16) || !norm_sizes_ok(rows, dim, dim, dim)) return 0;
  return static_cast<size_t>(norm_parts(rows)) * 2 * dim * 4;
}

int ssm_layer_norm_bwd(const void* s, const float* weight, float eps, const void* dout, const void* dresidual,
                       void* dx, float* dweight, float* dbias, int64_t rows, int64_t dim, int64_t s_row_stride,
                       int dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  const char* fn = "ssm_layer_norm_bwd";
  if (dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16)
    return fail(SSM_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, dtype);
  if (!(eps >= 0.0f)) return fail(SSM_ERR_UNSUPPORTED, "%s: eps must be at least 0", fn);
  if (!norm_sizes_ok(rows, dim, s_row_stride, dim))
    return fail(SSM_ERR_SHAPE, "%s: bad sizes: %lld rows of %lld, stride %lld", fn, (long long)rows, (long long)dim,
                (long long)s_row_stride);
  if (rows > 0 && (!s || !dout || !dx)) return fail(SSM_ERR_NULL, "%s: s, dout and dx are required", fn);
  const size_t es = dtype == SSM_DTYPE_F32 ? 4 : 2;
  const struct { const void* p; size_t k; const char* n; } al[] = {
      {s, es, "s"}, {dout, es, "dout"}, {dresidual, es, "dresidual"}, {dx, es, "dx"}, {weight, 4, "weight"},
      {dweight, 4, "dweight"}, {dbias, 4, "dbias"}};
  for (const auto& e : al)
    if (e.p && !aligned(e.p, e.k)) return fail(SSM_ERR_ALIGN, "%s: %s is not %zu-byte aligned", fn, e.n, e.k);
  const size_t pd = static_cast<size_t>(dim) * 4, whole = strided(rows, dim, dim, es);
  const size_t need = dweight || dbias ? ssm_layer_norm_bwd_workspace_bytes(rows, dim, dtype) : 0;
  const Span ins[] = {{s, strided(rows, dim, s_row_stride, es), "s"}, {dout, whole, "dout"},
                      {dresidual, dresidual ? whole : 0, "dresidual"}, {weight, weight ? pd : 0, "weight"}};
  const Span outs[] = {{dx, whole, "dx"}, {dweight, dweight ? pd : 0, "dweight"}, {dbias, dbias ? pd : 0, "dbias"},
                       {workspace, workspace ? need : 0, "workspace"}};
  for (const auto& o : outs)
    for (const auto& n : ins)  // (dx in place of a gradient: a row is read whole before it is written)
      if (overlap(o, n) && !(o.p == dx && n.p == dx && (n.p == dout || n.p == dresidual)))
        return fail(SSM_ERR_ALIAS, "%s: output %s overlaps input %s", fn, o.name, n.name);
  for (int a = 0; a < 4; ++a)
    for (int b = a + 1; b < 4; ++b)
      if (overlap(outs[a], outs[b]))
        return fail(SSM_ERR_ALIAS, "%s: %s overlaps %s", fn, outs[a].name, outs[b].name);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(SSM_ERR_WORKSPACE, "%s: workspace of %zu bytes given, %zu needed", fn,
                workspace ? workspace_bytes : 0, need);
  if (need > 0 && !aligned(workspace, 256))
    return fail(SSM_ERR_ALIGN, "%s: workspace is not 256-byte aligned", fn);
  if (rows == 0 && !dweight && !dbias) return SSM_OK;
  float* const part = static_cast<float*>(workspace);
  return dtype == SSM_DTYPE_F32
             ? launch_norm_bwd<float>(fn, s, weight, eps, dout, dresidual, dx, dweight, dbias, rows,
                                      static_cast<int>(dim), s_row_stride, part, stream)
             : launch_norm_bwd<bf16_t>(fn, s, weight, eps, dout, dresidual, dx, dweight, dbias, rows,
                                       static_cast<int>(dim), s_row_stride, part, stream);
}

}  // extern "C"
