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
// every value is read once and written once: memory bounds it (8192 x 2560 bf16 with
// the sum 27.3 us, 6.1 TB/s; 131072 x 2048 187 to 197 us, 5.7 to 5.5; gradients of 8192
// x 1536 25.3 us, 4.0, and 4.1 for the partial rows' sum).
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ssm_layer.h"

#include "host_util.hpp"
#include "kernels.hpp"

namespace ssm {
namespace {

constexpr int64_t kNormMaxDim = 16384;
constexpr int kNormWavesPerCu = 32;  // forward: more rows than that go round

// 16 bytes of a row; rows may start anywhere, so the compiler is told of no
// alignment (the hardware takes unaligned vector accesses)
template <typename TA>
struct Piece {
  static constexpr int n = 16 / static_cast<int>(sizeof(TA));
  TA v[n];
};

// NV pieces of a lane: values first + i step .. of a row of dim values; zeros
// behind its end, and everywhere without the row
template <typename TA, int NV>
struct Raw {
  static constexpr int VEC = Piece<TA>::n;
  Piece<TA> v[NV];
  __device__ __forceinline__ void load(const TA* p, int first, int step, int dim, bool there) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = first + i * step;
      if (there && c + VEC <= dim) {
        __builtin_memcpy(&v[i], p + c, sizeof(v[i]));
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          v[i].v[j] = TA{};
          if (there && c + j < dim) v[i].v[j] = p[c + j];
        }
      }
    }
  }
  __device__ __forceinline__ float at(int i, int j) const { return to_f32(v[i].v[j]); }
};

// (FRESH forms the addresses of a row's last values where they are needed, rather
// than keeping two registers for each from row to row: gradients of 8192 x 8192 bf16
// 142 us, 152 without; the forward is better off keeping them, 65536 x 300 bf16 35
// and 39.)
template <typename TA, int NV, bool FRESH = false>
__device__ __forceinline__ void store_row(const float (&x)[NV][Piece<TA>::n], TA* p, int first, int step, int dim) {
  constexpr int VEC = Piece<TA>::n;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = first + i * step;
    Piece<TA> raw;
#pragma unroll
    for (int j = 0; j < VEC; ++j) store_act(&raw.v[j], x[i][j]);
    if (c + VEC <= dim) {
      __builtin_memcpy(p + c, &raw, sizeof(raw));
    } else {
      int at = c;
      if constexpr (FRESH) asm volatile("" : "+v"(at));
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (at + j < dim) p[at + j] = raw.v[j];
    }
  }
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

// Sums over 16 lanes side by side, in each of them, and over a wave: without LDS,
// whose cross-lane operations the two statistics' sums would wait for (65536 x 300
// bf16 with the sum 35 us, by them 45; gradients of 8192 x 1536 float32 49 and 60).
template <int ROR>
__device__ __forceinline__ float row_add(float x) {
  return x + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x120 + ROR, 0xf, 0xf, false));
}
__device__ __forceinline__ float row_sum16(float x) { return row_add<1>(row_add<2>(row_add<4>(row_add<8>(x)))); }

__device__ __forceinline__ float wave_sum(float x) {
  x = row_sum16(x);
  const auto row = [&](int r) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 16 * r)); };
  return (row(0) + row(1)) + (row(2) + row(3));
}

// A workgroup works on GROUPS rows at a time, `waves` waves each.  Sums over a
// row go through the lanes of its waves and, with MULTI, through LDS in a fixed
// order; a slot is written again only behind the barrier of another one, so one
// barrier a sum is enough (all groups meet there).
template <bool MULTI>
struct RowGroup {
  int lane, group, waves, w;
  float* red;  // [slot][group][2][waves]
  __device__ __forceinline__ RowGroup(int wpr, float* r) {
    const int tid = static_cast<int>(threadIdx.x), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    waves = MULTI ? wpr : 1;
    group = wave / waves;
    w = wave - group * waves;
    lane = w * 64 + (tid & 63);
    red = r;
  }
  __device__ __forceinline__ void sum2(float& a, float& b, int slot) const {
    a = wave_sum(a);
    b = wave_sum(b);
    if constexpr (MULTI) {
      float* const p = red + (slot * 16 + group * waves) * 2;
      if ((lane & 63) == 0) {
        p[2 * w] = a;
        p[2 * w + 1] = b;
      }
      __syncthreads();
      const int i = lane & 15;  // (at most 16 waves)
      a = i < waves ? p[2 * i] : 0.0f;
      b = i < waves ? p[2 * i + 1] : 0.0f;
      a = row_sum16(a);
      b = row_sum16(b);
    }
  }
  __device__ __forceinline__ float sum(float a, int slot) const {
    float none = 0.0f;
    sum2(a, none, slot);
    return a;
  }
};

template <typename TA>
struct NormArgs {
  const TA *x, *res;  // forward: x and residual; backward: s and dout
  const TA* dres;
  const float *w, *b;
  TA *out, *sum;  // backward: dx in out
  float* part;    // backward: (parts, 2, dim)
  float eps;
  int64_t rows, xs, rs;
  int dim, waves, groups;
};

// c = s - mean(s) in place, and 1 / sqrt(mean(c^2) + eps).  The mean is a sum
// rounded at the values' size, which a row far from zero has much of: what c's own
// mean is still off from zero comes with the sum of its squares, and is taken off
// both (values 1000 deviations from zero: out within 3e-7, without it 1.2e-4).
template <bool MULTI, int NV, int VEC>
__device__ __forceinline__ float centre(float (&s)[NV][VEC], const RowGroup<MULTI>& rg, int first, int step, int dim,
                                        float eps) {
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) t += s[i][j];
  const float inv = 1.0f / static_cast<float>(dim), mean = rg.sum(t, 0) * inv;
  float q = 0.0f;
  t = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      s[i][j] = first + i * step + j < dim ? s[i][j] - mean : 0.0f;
      t += s[i][j];
      q = __builtin_fmaf(s[i][j], s[i][j], q);
    }
  rg.sum2(t, q, 1);
  const float off = t * inv;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) s[i][j] -= off;  // (behind the row's end it is not used)
  return 1.0f / sqrtf(__builtin_fmaxf(__builtin_fmaf(q, inv, -off * off), 0.0f) + eps);
}

// Every row group goes through its share of the rows with its columns' weights
// in registers.
// (Two workgroups of sixteen waves a compute unit where one piece a lane allows it:
// 8192 x 8192 bf16 with the sum 108 us, one 123.)
template <typename TA, int NV, bool MULTI, bool RES>
__global__ void __launch_bounds__(MULTI ? 1024 : 256, MULTI && NV == 1 ? 8 : 1) norm_fwd_kernel(const NormArgs<TA> p) {
  constexpr int VEC = Piece<TA>::n;
  __shared__ float red[MULTI ? 64 : 1];
  const RowGroup<MULTI> rg(p.waves, red);
  const int first = rg.lane * VEC, dim = p.dim, step = 64 * rg.waves * VEC;
  const int64_t hop = int64_t{gridDim.x} * p.groups;
  float w[NV][VEC], b[NV][VEC];
  load_param(w, p.w, 1.0f, first, step, dim);
  load_param(b, p.b, 0.0f, first, step, dim);
  for (int64_t base = int64_t{blockIdx.x} * p.groups; base < p.rows; base += hop) {
    const int64_t row = base + rg.group;
    const bool there = row < p.rows;
    Raw<TA, NV> s, r;
    s.load(p.x + row * p.xs, first, step, dim, there);
    if constexpr (RES) r.load(p.res + row * p.rs, first, step, dim, there);
    float x[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        x[i][j] = s.at(i, j);
        if constexpr (RES) {  // rounded, as it is kept
          TA t;
          store_act(&t, x[i][j] + r.at(i, j));
          x[i][j] = to_f32(t);
        }
      }
    if constexpr (RES)
      if (p.sum && there) store_row<TA, NV>(x, p.sum + row * dim, first, step, dim);
    const float rstd = centre<MULTI>(x, rg, first, step, dim, p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) x[i][j] = __builtin_fmaf(x[i][j] * rstd, w[i][j], b[i][j]);
    if (there) store_row<TA, NV>(x, p.out + row * dim, first, step, dim);
  }
}

// Gradients, in the same way, with the columns' weight gradients in registers
// too; the groups' are added through LDS in turn, and the workgroup leaves one
// partial row.
template <typename TA, int NV, bool MULTI>
__global__ void __launch_bounds__(MULTI ? 1024 : 256) norm_bwd_kernel(const NormArgs<TA> p) {
  constexpr int VEC = Piece<TA>::n;
  __shared__ float red[MULTI ? 96 : 1];
  // dresidual is fetched behind the sums where a row's values fill the registers
  // (2048 x 16384 float32 141 us, before them 166)
  constexpr bool LATE = MULTI && NV * VEC > 8;
  extern __shared__ float fold[];  // [2][64 waves VEC], with several groups
  const RowGroup<MULTI> rg(p.waves, red);
  const int first = rg.lane * VEC, dim = p.dim, step = 64 * rg.waves * VEC;
  const int64_t hop = int64_t{gridDim.x} * p.groups;
  float dw[NV][VEC], db[NV][VEC], w[NV][VEC];
  load_param(w, p.w, 1.0f, first, step, dim);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) dw[i][j] = db[i][j] = 0.0f;
  for (int64_t base = int64_t{blockIdx.x} * p.groups; base < p.rows; base += hop) {
    const int64_t row = base + rg.group;
    const bool there = row < p.rows;
    Raw<TA, NV> rs, ry, rd;
    rs.load(p.x + row * p.xs, first, step, dim, there);
    ry.load(p.res + row * dim, first, step, dim, there);
    if (!LATE && p.dres) rd.load(p.dres + row * dim, first, step, dim, there);
    float s[NV][VEC], y[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        s[i][j] = rs.at(i, j);
        y[i][j] = ry.at(i, j);
      }
    float rstd = centre<MULTI>(s, rg, first, step, dim, p.eps);
    if (!there) rstd = 0.0f;  // (1 / 0 with eps = 0: its NaN would reach dw)
    float t0 = 0.0f, t1 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float h = s[i][j] * rstd, g = y[i][j];  // (0 for a row that is not there)
        dw[i][j] = __builtin_fmaf(g, h, dw[i][j]);
        db[i][j] += g;
        s[i][j] = h;
        y[i][j] = g * w[i][j];
        t0 += y[i][j];
        t1 = __builtin_fmaf(y[i][j], h, t1);
      }
    rg.sum2(t0, t1, 2);
    if (LATE && p.dres) rd.load(p.dres + row * dim, first, step, dim, there);
    const float inv = 1.0f / static_cast<float>(dim);
    t0 *= inv;
    t1 *= inv;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        y[i][j] = __builtin_fmaf(rstd, y[i][j] - t0 - s[i][j] * t1, p.dres ? rd.at(i, j) : 0.0f);
    if (there) store_row<TA, NV, NV == 1>(y, p.out + row * dim, first, step, dim);
  }
  if (!p.part) return;
  const int lanes = 64 * rg.waves;
  for (int g = 1; g < p.groups; ++g)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      __syncthreads();
      if (rg.group == g)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          fold[j * lanes + rg.lane] = dw[i][j];
          fold[(VEC + j) * lanes + rg.lane] = db[i][j];
        }
      __syncthreads();
      if (rg.group == 0)
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          dw[i][j] += fold[j * lanes + rg.lane];
          db[i][j] += fold[(VEC + j) * lanes + rg.lane];
        }
    }
  if (rg.group != 0) return;
  float* const o = p.part + int64_t{blockIdx.x} * 2 * dim;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = first + i * step;
    if (c + VEC <= dim) {
      __builtin_memcpy(o + c, dw[i], sizeof(dw[i]));
      __builtin_memcpy(o + dim + c, db[i], sizeof(db[i]));
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        if (c + j < dim) {
          o[c + j] = dw[i][j];
          o[dim + c + j] = db[i][j];
        }
    }
  }
}

// The partial rows' sum: a workgroup takes 64 of the 2 dim columns, each of its
// sixteen waves every sixteenth row, in four sums at a time.
__global__ void __launch_bounds__(1024)
    norm_reduce_kernel(const float* part, int parts, int dim, float* dw, float* db) {
  __shared__ float red[16][64];
  const int lane = static_cast<int>(threadIdx.x & 63), g = static_cast<int>(threadIdx.x >> 6);
  const int c = static_cast<int>(blockIdx.x) * 64 + lane, n = 2 * dim;
  float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < n) {
    int i = g;
    for (; i + 48 < parts; i += 64)
#pragma unroll
      for (int k = 0; k < 4; ++k) t[k] += part[static_cast<size_t>(i + 16 * k) * n + c];
    for (; i < parts; i += 16) t[0] += part[static_cast<size_t>(i) * n + c];
  }
  red[g][lane] = (t[0] + t[1]) + (t[2] + t[3]);
  __syncthreads();
  if (g != 0 || c >= n) return;
  float x = 0.0f;
#pragma unroll
  for (int k = 0; k < 16; ++k) x += red[k][lane];
  if (c < dim) {
    if (dw) dw[c] = x;
  } else if (db) {
    db[c - dim] = x;
  }
}

template <int N>
struct Count {
  static constexpr int value = N;
};

struct NormPlan {
  bool multi;
  int nv, waves, groups;
};

// One wave a row while its share of a row stays within `most` pieces a lane:
// five in the forward (8192 x 2560 bf16 with the sum 27.7 us, shared by five waves
// 30.3; 131072 x 2048 191 and 235 us), three in the backward, which keeps three
// times as many values (both launches, 8192 x 1536 bf16 27.6 us, by three waves
// 34.4; 3001 x 515 float32 11.8 and 14.3 us).  Wider rows, and rows too few to fill
// the device, are shared by waves (1 x 2560 bf16 with the sum 3.3 us, by one wave
// 4.6; 512 rows 4.9 and 5.6, 1000 rows 6.5 and 6.3; gradients of 1000 x 1536 11.4
// and 11.7, of 512 rows 10.4 and 9.4).
NormPlan norm_plan(int64_t rows, int dim, int vec, int most) {
  const int pieces = (dim + vec - 1) / vec, nv = (pieces + 63) / 64;
  const bool few = rows < 4 * device_cus();
  if (nv <= 1 || (nv <= most && !few)) return NormPlan{false, nv, 1, 4};
  NormPlan p{true, 1, nv, 1};
  while (p.nv * 16 < nv) p.nv *= 2;
  p.waves = (nv + p.nv - 1) / p.nv;
  return p;
}

// Calls go(NV, MULTI); ONE and MANY bound what the caller's plans can hold.
template <int ONE, int MANY, typename Go>
void norm_go(const NormPlan& p, Go&& go) {
  if (!p.multi) {
    if (p.nv == 1) go(Count<1>{}, Count<0>{});
    else if (p.nv == 2) go(Count<2>{}, Count<0>{});
    else if (p.nv == 3) go(Count<3>{}, Count<0>{});
    else if constexpr (ONE == 5) {
      if (p.nv == 4) go(Count<4>{}, Count<0>{});
      else go(Count<5>{}, Count<0>{});
    }
  } else if (p.nv == 1) {
    go(Count<1>{}, Count<1>{});
  } else if (p.nv == 2) {
    go(Count<2>{}, Count<1>{});
  } else if constexpr (MANY == 4) {
    go(Count<4>{}, Count<1>{});
  }
}

NormPlan bwd_plan(int64_t rows, int dim, int vec) {
  NormPlan p = norm_plan(rows, dim, vec, 3);
  if (p.multi) p.groups = p.nv == 1 ? 16 / p.waves : 1;  // (more rows to a partial row)
  return p;
}

int norm_parts(const NormPlan& p, int64_t rows) {
  const int64_t n = (rows + p.groups - 1) / p.groups;
  // (two workgroups a compute unit with one wave a row: 8192 x 1536 bf16 27.6 us,
  // one 36.1, three 33.8)
  const int64_t most = device_cus() * (p.multi ? 1 : 2);
  return static_cast<int>(n < 1 ? 1 : n > most ? most : n);
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
  const NormPlan plan = norm_plan(rows, dim, Piece<TA>::n, 5);
  const NormArgs<TA> a{static_cast<const TA*>(x), static_cast<const TA*>(res), nullptr, w, b, static_cast<TA*>(out),
                       static_cast<TA*>(sum), nullptr, eps, rows, xs, rs, dim, plan.waves, plan.groups};
  const int64_t units = (rows + plan.groups - 1) / plan.groups;
  const int64_t most = int64_t{device_cus()} * kNormWavesPerCu / (plan.waves * plan.groups);
  const dim3 grid(static_cast<unsigned>(units < most ? units : most)), block(64 * plan.waves * plan.groups);
  constexpr int most_nv = kNormMaxDim / (16 * 64 * Piece<TA>::n);
  norm_go<5, most_nv>(plan, [&](auto nv, auto multi) {
    constexpr int NV = decltype(nv)::value;
    constexpr bool M = decltype(multi)::value != 0;
    if (res) hipLaunchKernelGGL((norm_fwd_kernel<TA, NV, M, true>), grid, block, 0, stream, a);
    else hipLaunchKernelGGL((norm_fwd_kernel<TA, NV, M, false>), grid, block, 0, stream, a);
  });
  return launch_status(fn);
}

template <typename TA>
int launch_norm_bwd(const char* fn, const void* s, const float* w, float eps, const void* dout, const void* dres,
                    void* dx, float* dw, float* db, int64_t rows, int dim, int64_t ss, float* part,
                    hipStream_t stream) {
  constexpr int VEC = Piece<TA>::n;
  const NormPlan plan = bwd_plan(rows, dim, VEC);
  const int parts = norm_parts(plan, rows);
  const NormArgs<TA> a{static_cast<const TA*>(s), static_cast<const TA*>(dout), static_cast<const TA*>(dres), w,
                       nullptr, static_cast<TA*>(dx), nullptr, dw || db ? part : nullptr, eps, rows, ss, dim, dim,
                       plan.waves, plan.groups};
  const size_t lds = plan.groups > 1 ? sizeof(float) * 2 * 64 * plan.waves * VEC : 0;
  norm_go<3, kNormMaxDim / (16 * 64 * VEC)>(plan, [&](auto nv, auto multi) {
    hipLaunchKernelGGL((norm_bwd_kernel<TA, decltype(nv)::value, decltype(multi)::value != 0>),
                       dim3(static_cast<unsigned>(parts)), dim3(64 * plan.waves * plan.groups), lds, stream, a);
  });
  if (dw || db)
    hipLaunchKernelGGL(norm_reduce_kernel, dim3(static_cast<unsigned>((2 * dim + 63) / 64)), dim3(1024), 0, stream,
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
    for (const auto& n : ins)  // (in place, row on row: a row is read whole before it is written)
      if (overlap(o, n) && !(o.p == n.p && o.bytes == n.bytes && (n.p == x || n.p == residual)))
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
  const NormPlan plan = bwd_plan(rows, static_cast<int>(dim), dtype == SSM_DTYPE_F32 ? 4 : 8);
  return static_cast<size_t>(norm_parts(plan, rows)) * 2 * dim * 4;
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
      if (overlap(o, n) && !(o.p == dx && n.p == dx && o.bytes == n.bytes && (n.p == dout || n.p == dresidual)))
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
