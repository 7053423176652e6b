// gated.hpp -- device code shared by the gated linear recurrence's forward,
// backward and decode kernels (gated.hip, gated_bwd.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "ssm_recurrent.h"

#include "kernels.hpp"

namespace ssm {

// sigma(v) = 1 / (1 + e^-v): one hardware exp2 and one reciprocal (an ulp
// each).  v below -88 gives 0 and v = +-inf its limit.
__device__ __forceinline__ float sigmoid_f32(float v) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-v * kLog2e));
}

// The decay a = e^la and the input's scale m = sqrt(1 - a^2) of one token.
// Both come from E = 1 - a = -expm1(la): next to a = 1, where a long memory
// lives, E has its full precision, so a = 1 - E is rounded to nearest (the
// hardware exp2 rounds low on average, which a memory of thousands of tokens
// adds up) and m = sqrt(E (2 - E)) loses nothing to cancellation.  |la| <
// 1/8: Taylor series of -expm1 to la^5 (the next term is below 2^-24 of it).
// Elsewhere a <= 0.883 and E = 1 - a is exact enough (2^-24 / 0.117).
template <bool NORM>
__device__ __forceinline__ void decay(float la, float& a, float& m) {
  const float ex = __builtin_amdgcn_exp2f(la * kLog2e);
  float q = __builtin_fmaf(la, 1.0f / 120.0f, 1.0f / 24.0f);
  q = __builtin_fmaf(la, q, 1.0f / 6.0f);
  q = __builtin_fmaf(la, q, 0.5f);
  q = __builtin_fmaf(la, q, 1.0f);
  const bool near = __builtin_fabsf(la) < 0.125f;
  const float E = near ? -la * q : 1.0f - ex;
  a = near ? 1.0f - E : ex;
  m = NORM ? __builtin_amdgcn_sqrtf(__builtin_fmaxf(E * (2.0f - E), 0.0f)) : 1.0f;
}

// Arguments of the forward over `rows` rows of `L` tokens (dense: rows = batch;
// packed: one row of total_len tokens, with cu set).
template <typename TA>
struct GatedFwdArgs {
  const TA *x, *r, *i, *z;
  const float *A, *rb, *ib;
  TA* out;
  float* last;
  const float* h0;
  float* chunk_states;
  const int32_t* cu;  // packed: (nseq + 1) offsets; NULL otherwise
  int64_t rows, L, nseq;
  int dim;
  void* ws;
};

template <typename TA>
struct GatedBwdArgs {
  const TA *x, *r, *i, *z, *dout;
  const float *A, *rb, *ib, *h0, *chunk_states, *dlast;
  TA *dx, *dr, *di, *dz;
  float *dA, *drb, *dib, *dh0;
  const int32_t* cu;
  int64_t rows, L, nseq;
  int dim;
  void* ws;
};

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

}  // namespace ssm
