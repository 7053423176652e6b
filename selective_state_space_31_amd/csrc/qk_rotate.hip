// qk_rotate.hip -- the norm of queries and keys for each head with the
// position rotation in the same pass, and its gradients, behind the C ABI in
// include/ssm_recurrent.h.
//
//   n = v rstd w, rstd = 1 / sqrt(mean(v^2) + eps); pairs (p, q) of n turn by
//   theta = position * inv_freq.  Backward, with g the gradient turned back:
//   dv = rstd (g w - vhat mean(g w vhat)), vhat = v rstd;  dw = sum g vhat.
// One read and one write of every value: memory bounds it, then the latency of
// a head's sums.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ssm_recurrent.h"

#include "host_util.hpp"
#include "kernels.hpp"

namespace ssm {

// sin and cos of pos * freq.  The angle in turns is formed in two float64 parts:
// the product of 31 and 24 bits and its rounding, times 1/(2 pi) in two parts;
// at 2^31 the first part alone is off by 4e-7.  It is reduced there to a quarter
// turn, and what is left (|r| <= 1/8 turn) goes through float32 Taylor
// polynomials: sin to x^9, cos to x^10 at |x| <= pi/4 (next terms 1.8e-9 and
// 1.2e-10; with their roundings within 2^-23).
__device__ __forceinline__ void turn_f32(int32_t pos, float freq, float& sn, float& cs) {
#pragma clang fp contract(off)  // (t is the rounded product: fused into the difference below, its rounding would count twice)
  constexpr double kInv = 0.15915494309189535, kInvLow = -9.839338337591243e-18;  // 1/(2 pi)
  const double p = static_cast<double>(pos), f = static_cast<double>(freq), a = p * f;
  double t = a * kInv;
  const double low = __builtin_fma(a, kInv, -t) + __builtin_fma(a, kInvLow, __builtin_fma(p, f, -a) * kInv);
  t = (t - __builtin_rint(t)) + low;  // turns, [-1/2, 1/2]
  const double q = __builtin_rint(t * 4.0);
  const float x = static_cast<float>((t - q * 0.25) * 6.283185307179586);
  const float x2 = x * x;
  float s = __builtin_fmaf(x2, 2.75573192e-6f, -1.98412698e-4f);
  s = __builtin_fmaf(x2, s, 8.33333333e-3f);
  s = __builtin_fmaf(x2, s, -1.66666667e-1f);
  s = __builtin_fmaf(x2 * x, s, x);
  float c = __builtin_fmaf(x2, -2.75573192e-7f, 2.48015873e-5f);
  c = __builtin_fmaf(x2, c, -1.38888889e-3f);
  c = __builtin_fmaf(x2, c, 4.16666667e-2f);
  c = __builtin_fmaf(x2, c, -0.5f);
  c = __builtin_fmaf(x2, c, 1.0f);
  const int k = static_cast<int>(q) & 3;  // quarter turns, mod 4
  const float ss = (k & 1) ? c : s, cc = (k & 1) ? s : c;
  sn = (k & 2) ? -ss : ss;
  cs = (k == 1 || k == 2) ? -cc : cc;
}

template <typename TA>
struct RotArgs {
  const TA *q, *k;             // inputs, tokens qs / ks values apart
  const float *qw, *kw, *freq;
  const int32_t* pos;
  const TA *dqo, *dko;         // backward: gradients of the outputs
  TA *qo, *ko;                 // outputs (forward) or dq, dk (backward)
  float* part;                 // backward: (waves, 2, D) partial weight gradients
  float eps;
  int64_t tokens, L, qs, ks;
  int Hq, Hk, D, R;            // R = rotary_dim
};

constexpr int kRotWaves = 4;     // waves of a workgroup
constexpr int kRotAhead = 4;     // rows of a token in flight (half as many in the backward, two tensors)
constexpr int kRotElems = 4;     // elements of a row per lane (headdim <= 256)

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Head sizes and alignments that no vector access fits: one wave per row
// (token, head); lane l holds elements l, l + 64, ...  Every lane forms its own
// sines, for every head again (16 heads of 128, 8192 tokens, bf16: 62 us where
// the vector kernel takes 12.5): alignment's slow path, not a choice.
template <typename TA, bool INTER, bool BWD>
__global__ void __launch_bounds__(64 * kRotWaves) rotate_any_kernel(RotArgs<TA> p) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = static_cast<int64_t>(blockIdx.x) * kRotWaves + (threadIdx.x >> 6);
  const int64_t nwaves = static_cast<int64_t>(gridDim.x) * kRotWaves;
  const int heads = p.Hq + p.Hk, half = p.R / 2;
  float wq[kRotElems] = {}, wk[kRotElems] = {};
  for (int64_t row = wave; row < p.tokens * heads; row += nwaves) {
    const int64_t tok = row / heads;
    const int hd = static_cast<int>(row % heads);
    const bool isq = hd < p.Hq;
    const TA* in = isq ? p.q + tok * p.qs + hd * p.D : p.k + tok * p.ks + (hd - p.Hq) * p.D;
    const int64_t oo = isq ? (tok * p.Hq + hd) * p.D : (tok * p.Hk + hd - p.Hq) * p.D;
    const TA* go = isq ? p.dqo : p.dko;
    const float* w = isq ? p.qw : p.kw;
    const int32_t pos = p.pos ? p.pos[tok] : static_cast<int32_t>(tok % p.L);
    float v[kRotElems], u[kRotElems], ss = 0.0f;  // own and partner's values
#pragma unroll
    for (int n = 0; n < kRotElems; ++n) {
      const int e = lane + 64 * n;
      v[n] = u[n] = 0.0f;
      if (e < p.D) {
        v[n] = to_f32(in[e]);
        if (e < p.R) {
          const int o = INTER ? (e ^ 1) : (e < half ? e + half : e - half);
          u[n] = to_f32(BWD ? go[oo + o] : in[o]) * (!BWD && w ? w[o] : 1.0f);
        }
      }
      ss += v[n] * v[n];
    }
    const float rstd = __builtin_amdgcn_rsqf(wave_sum(ss) / static_cast<float>(p.D) + p.eps);
    float res[kRotElems], dot = 0.0f;
#pragma unroll
    for (int n = 0; n < kRotElems; ++n) {
      const int e = lane + 64 * n;
      res[n] = 0.0f;
      if (e >= p.D) continue;
      const float we = w ? w[e] : 1.0f;
      float sn = 0.0f, cs = 1.0f;
      bool first = true;
      if (e < p.R) {
        first = INTER ? !(e & 1) : e < half;
        turn_f32(pos, p.freq[INTER ? e >> 1 : (e < half ? e : e - half)], sn, cs);
      }
      if (!BWD) {
        const float side = first ? -sn : sn;
        res[n] = rstd * (v[n] * we * cs + u[n] * side);
      } else {
        const float side = first ? sn : -sn;
        const float g = to_f32(go[oo + e]) * cs + u[n] * side;
        const float vh = v[n] * rstd;
        (isq ? wq : wk)[n] += g * vh;
        res[n] = g * we;
        dot += res[n] * vh;
      }
    }
    if (BWD) dot = wave_sum(dot) / static_cast<float>(p.D);
    TA* out = (isq ? p.qo : p.ko) + oo;
#pragma unroll
    for (int n = 0; n < kRotElems; ++n) {
      const int e = lane + 64 * n;
      if (e < p.D) store_act(out + e, BWD ? rstd * (res[n] - v[n] * rstd * dot) : res[n]);
    }
  }
  if (BWD) {
#pragma unroll
    for (int n = 0; n < kRotElems; ++n) {
      const int e = lane + 64 * n;
      if (e < p.D) {
        p.part[(wave * 2) * p.D + e] = wq[n];
        p.part[(wave * 2 + 1) * p.D + e] = wk[n];
      }
    }
  }
}

// E values moved as one access of 4 (bf16), 8 or 16 bytes.
template <typename TA, int E>
struct RotVec;
template <int E>
struct RotVec<float, E> {
  typedef float vec_t __attribute__((ext_vector_type(E)));
  __device__ static float get(const vec_t& r, int e) { return r[e]; }
  __device__ static void store(float* p, const float (&v)[E]) {
    vec_t r;
#pragma unroll
    for (int e = 0; e < E; ++e) r[e] = v[e];
    __builtin_nontemporal_store(r, reinterpret_cast<vec_t*>(p));
  }
};
template <int E>
struct RotVec<bf16_t, E> {
  typedef uint32_t vec_t __attribute__((ext_vector_type(E / 2)));
  __device__ static float get(const vec_t& r, int e) {
    return __uint_as_float(e & 1 ? r[e / 2] & 0xffff0000u : r[e / 2] << 16);
  }
  __device__ static void store(bf16_t* p, const float (&v)[E]) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    vec_t r;
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      const bf16x2 b = __builtin_convertvector((f32x2{v[2 * e], v[2 * e + 1]}), bf16x2);
      r[e] = __builtin_bit_cast(uint32_t, b);
    }
    __builtin_nontemporal_store(r, reinterpret_cast<vec_t*>(p));
  }
};

// Sum over the lanes of one row (N neighbours, a power of two), in every one
// of them.  Up to 16 lanes by lane moves inside the vector instructions
// (neighbour, pair, half row and row mirrored): a head waits for its sums, and
// exchanges through LDS take ten times as long.
template <int CTRL>
__device__ __forceinline__ float moved(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int N>
__device__ __forceinline__ float row_sum(float v) {
  if constexpr (N > 1) v += moved<0xb1>(v);   // lane ^ 1
  if constexpr (N > 2) v += moved<0x4e>(v);   // lane ^ 2
  if constexpr (N > 4) v += moved<0x141>(v);  // 7 - lane within 8
  if constexpr (N > 8) v += moved<0x140>(v);  // 15 - lane within 16
#pragma unroll
  for (int o = 16; o < N; o <<= 1) v += __shfl_xor(v, o);
  return v;
}

// A row of D values is cut into blocks of E; a lane holds two of them that
// form pairs: block l and the block R/2 values on while l is in the rotated
// part (with interleaved pairs any two), two neighbouring blocks behind it.
// So a rotation needs no other lane, and a row takes N = D / (2 E) lanes,
// rounded up to a power of two; a wave holds 64 / N tokens and goes through
// their heads, forming the sines and cosines once per token.
// Measured (kernel alone): 8192 tokens of 8 + 8 heads of 128 bf16 12.5 us, 5.4
// TB/s; 256 tokens of 1 + 1 heads of 64 3.3 us, a launch and three round trips.
// Gradients: 4002 tokens of 16 + 4 heads of 128 bf16 13.4 us, 4.6 TB/s (rows in
// flight: 2 here; 4 14.1 us).
template <typename TA, int E, int N, bool INTER, bool BWD>
__global__ void __launch_bounds__(64 * kRotWaves) rotate_kernel(RotArgs<TA> p, int head_step) {
  using IO = RotVec<TA, E>;
  constexpr int S = 64 / N;  // tokens of a wave
  __shared__ float s_w[BWD ? kRotWaves : 1][2][BWD ? 2 * E * N : 1];
  const int lane = threadIdx.x & 63, l = lane % N, slot = lane / N;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int heads = p.Hq + p.Hk, half = p.R / 2;
  const bool have = l < p.D / (2 * E);
  const int turned = p.R / (2 * E);  // lanes with rotated values
  // (lanes that pad the row read its first blocks and are left out)
  const int e0 = !have ? 0 : l < turned ? (INTER ? 2 * E * l : E * l) : p.R + 2 * E * (l - turned);
  const int e1 = have && l < turned && !INTER ? E * l + half : e0 + E;
  float dwq[BWD ? 2 * E : 1], dwk[BWD ? 2 * E : 1];
#pragma unroll
  for (int e = 0; e < (BWD ? 2 * E : 1); ++e) dwq[e] = dwk[e] = 0.0f;
  const float mean = 1.0f / static_cast<float>(p.D);
  // (blockIdx.y: a range of heads, where there are few tokens)
  const int h0 = blockIdx.y * head_step, h1 = h0 + head_step < heads ? h0 + head_step : heads;
  for (int64_t g = static_cast<int64_t>(blockIdx.x) * kRotWaves + wave; g * S < p.tokens;
       g += static_cast<int64_t>(gridDim.x) * kRotWaves) {
    const int64_t tok = g * S + slot;
    const bool on = have && tok < p.tokens;
    const int64_t tk = tok < p.tokens ? tok : p.tokens - 1;
    float sn[E], cs[E];
    const int32_t pos = p.pos ? p.pos[tk] : static_cast<int32_t>(tk % p.L);
    // pair i of the lane: values (i, i + E), or (2i, 2i + 1) when interleaved
    const auto rotate = [&](float (&v)[2 * E]) {
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const int a = INTER ? 2 * i : i, b = INTER ? 2 * i + 1 : i + E;
        const float x = v[a], y = v[b];
        v[a] = __builtin_fmaf(x, cs[i], -(y * sn[i]));
        v[b] = __builtin_fmaf(x, sn[i], y * cs[i]);
      }
    };
    typedef typename IO::vec_t vec_t;
    const auto fetch = [&](const TA* r, vec_t (&v)[2]) {
      v[0] = *reinterpret_cast<const vec_t*>(r + e0);
      v[1] = *reinterpret_cast<const vec_t*>(r + e1);
    };
    const auto put = [&](TA* r, const float (&v)[2 * E]) {
      float lo[E], hi[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        lo[e] = v[e];
        hi[e] = v[e + E];
      }
      if (on) {
        IO::store(r + e0, lo);
        IO::store(r + e1, hi);
      }
    };
    // One tensor's heads [b, e), kAhead rows on their way while one is worked
    // on.  Nothing in here depends on a condition but the remainder: behind a
    // branch the wait for a row would be a wait for all of them.
    constexpr int kAhead = BWD ? kRotAhead / 2 : kRotAhead;
    bool turns = false;
    const auto tensor = [&](const TA* in, const TA* dy, TA* to, const float* w, float* dw, int b, int e) {
      if (b >= e) return;
      vec_t vr[kAhead][2], dr[BWD ? kAhead : 1][2];
      const auto ahead = [&](int u, int h) {
        h = h < e ? h : e - 1;
        fetch(in + h * p.D, vr[u]);
        if constexpr (BWD) fetch(dy + h * p.D, dr[u]);
      };
#pragma unroll
      for (int u = 0; u < kAhead; ++u) ahead(u, b + u);
      if (!turns) {  // the first rows are on their way
        turns = true;
#pragma unroll
        for (int i = 0; i < E; ++i) {
          sn[i] = 0.0f;
          cs[i] = 1.0f;
          if (l < turned) turn_f32(pos, p.freq[E * l + i], sn[i], cs[i]);
          if (BWD) sn[i] = -sn[i];
        }
      }
      float wt[2 * E];
#pragma unroll
      for (int i = 0; i < 2 * E; ++i) wt[i] = have && w ? w[i < E ? e0 + i : e1 + i - E] : 1.0f;
      const auto work = [&](int u, int h) {
        float v[2 * E], d[BWD ? 2 * E : 1], ss = 0.0f;
#pragma unroll
        for (int i = 0; i < 2 * E; ++i) {
          v[i] = IO::get(vr[u][i / E], i % E);
          if (BWD) d[i] = IO::get(dr[u][i / E], i % E);
        }
        ahead(u, h + kAhead);
#pragma unroll
        for (int i = 0; i < 2 * E; ++i) ss = __builtin_fmaf(v[i], v[i], ss);
        const float rstd = __builtin_amdgcn_rsqf(__builtin_fmaf(row_sum<N>(have ? ss : 0.0f), mean, p.eps));
        if constexpr (!BWD) {
#pragma unroll
          for (int i = 0; i < 2 * E; ++i) v[i] = v[i] * rstd * wt[i];
          rotate(v);
          put(to + h * p.D, v);
        } else {
          rotate(d);
          float dot = 0.0f;
          const float mine = on ? rstd : 0.0f;  // (a token that is not there adds nothing to the weights' sums)
#pragma unroll
          for (int i = 0; i < 2 * E; ++i) {
            v[i] *= mine;  // vhat
            dw[i] = __builtin_fmaf(d[i], v[i], dw[i]);
            d[i] *= wt[i];
            dot = __builtin_fmaf(d[i], v[i], dot);
          }
          dot = row_sum<N>(have ? dot : 0.0f) * mean;
#pragma unroll
          for (int i = 0; i < 2 * E; ++i) d[i] = rstd * (d[i] - v[i] * dot);
          put(to + h * p.D, d);
        }
      };
      int h = b;
      for (; h + kAhead <= e; h += kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) work(u, h + u);
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (h + u < e) work(u, h + u);
    };
    tensor(p.q + tk * p.qs, BWD ? p.dqo + tk * p.Hq * p.D : nullptr, p.qo + tk * p.Hq * p.D, p.qw, dwq, h0,
           h1 < p.Hq ? h1 : p.Hq);
    tensor(p.k + tk * p.ks, BWD ? p.dko + tk * p.Hk * p.D : nullptr, p.ko + tk * p.Hk * p.D, p.kw, dwk,
           h0 < p.Hq ? 0 : h0 - p.Hq, h1 - p.Hq);
  }
  if constexpr (BWD) {
    // over the wave's tokens, then over the waves, in a fixed order
#pragma unroll
    for (int e = 0; e < 2 * E; ++e) {
#pragma unroll
      for (int o = N; o < 64; o <<= 1) {
        dwq[e] += __shfl_xor(dwq[e], o);
        dwk[e] += __shfl_xor(dwk[e], o);
      }
      if (slot == 0) {
        s_w[wave][0][l * 2 * E + e] = dwq[e];
        s_w[wave][1][l * 2 * E + e] = dwk[e];
      }
    }
    __syncthreads();
    float* const part = p.part + (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 2 * p.D;
    for (int i = threadIdx.x; i < 2 * 2 * E * N; i += 64 * kRotWaves) {
      const int what = i / (2 * E * N), ll = i % (2 * E * N) / (2 * E), e = i % (2 * E);
      if (ll >= p.D / (2 * E)) continue;
      const int b0 = ll < turned ? (INTER ? 2 * E * ll : E * ll) : p.R + 2 * E * (ll - turned);
      const int b1 = ll < turned && !INTER ? E * ll + half : b0 + E;
      float v = 0.0f;
#pragma unroll
      for (int u = 0; u < kRotWaves; ++u) v += s_w[u][what][ll * 2 * E + e];
      part[what * p.D + (e < E ? b0 + e : b1 + e - E)] = v;
    }
  }
}

// Sum of the partial weight gradients: a workgroup takes 16 elements of one of
// the two; wave w and lane quarter t take every 64th row from 4 w + t on, and
// the quarters' and the waves' sums are added in order.
// A launch of its own: the rows are there in no fixed order, and atomics would
// add them in that one, differently from run to run.
// At most 1024 rows of 1 KB (heads of 128): its launch and two round trips, 4.9 us.
constexpr int kRotSumWaves = 16, kRotSumElems = 16;
__global__ void __launch_bounds__(64 * kRotSumWaves) rotate_sum_kernel(const float* part, int n, int D, float* dqw,
                                                                       float* dkw) {
  constexpr int M = kRotSumElems, Q = 64 / M;  // elements, lane quarters
  __shared__ float s_part[kRotSumWaves * Q][M];
  const int m = threadIdx.x % M, t = threadIdx.x / M;
  const int e = blockIdx.x * M + m;
  float* to = blockIdx.y == 0 ? dqw : dkw;
  if (!to) return;
  float v = 0.0f;
  if (e < D) {
    const float* from = part + blockIdx.y * D + e;
#pragma unroll 8
    for (int k = t; k < n; k += kRotSumWaves * Q) v += from[static_cast<int64_t>(k) * 2 * D];
  }
  s_part[t][m] = v;
  __syncthreads();
  if (t == 0 && e < D) {
#pragma unroll
    for (int k = 1; k < kRotSumWaves * Q; ++k) v += s_part[k][m];
    to[e] = v;
  }
}

namespace {

constexpr int64_t kRotMaxTokens = int64_t{1} << 31;

bool rot_sizes_ok(int64_t batch, int64_t L, int64_t Hq, int64_t Hk, int64_t D) {
  return batch >= 1 && L >= 0 && batch < kRotMaxTokens && L < kRotMaxTokens &&
         batch * L < kRotMaxTokens && Hq >= 1 && Hq <= 65536 && Hk >= 0 && Hk <= 65536 && D >= 2 &&
         D <= 256 && D % 2 == 0;
}

// Rows of partial weight gradients the backward may leave at most: as many as
// there are waves (any layout) or workgroups (vectors), bounded so that their
// sum stays short (2048: 14.8 + 6.0 us for the 4002 tokens where 1024 take 13.4
// + 4.9).  Half as many workgroups with four values an access, whose waves hold
// twice the rows (8192 tokens of 16 + 16 heads of 128 float32: 70 us, with all
// of them 74).
constexpr int64_t kRotMaxParts = 1024;
// Workgroups of a forward up to which its heads are spread over more of them
// (twice as many measured 5% slower: the sines are formed once more).
constexpr int64_t kRotFwdBlocks = 512;
int64_t rot_parts(int64_t rows) {
  const int64_t want = (rows + kRotWaves - 1) / kRotWaves * kRotWaves;
  return want < kRotWaves ? kRotWaves : want > kRotMaxParts ? kRotMaxParts : want;
}

struct RotCall {
  const char* fn;
  const void *q, *k;
  const float *qw, *kw, *freq;
  const int32_t* pos;
  float eps;
  int interleaved;
  const void *dqo, *dko;
  void *qo, *ko;
  float *dqw, *dkw;
  int64_t batch, L, Hq, Hk, D, R, qs, ks;
  int dtype;
  void* ws;
  size_t ws_bytes;
  hipStream_t stream;
  bool bwd;
};

// Launch shape of a vector kernel: tokens a wave holds, workgroups over tokens
// (x) and over ranges of heads (y).  Heads stay together, so that a token's
// sines and cosines are formed once, unless there are too few tokens for a
// few waves per SIMD.
template <typename TA, int E, int N>
void rot_launch_vec(const RotCall& c, const RotArgs<TA>& a, int64_t* parts) {
  const int heads = a.Hq + a.Hk;
  const int64_t groups = (a.tokens + 64 / N - 1) / (64 / N);
  int64_t x = (groups + kRotWaves - 1) / kRotWaves;
  x = x < 1 ? 1 : x;
  int step = heads;
  const int64_t most = c.bwd ? (rot_parts(a.tokens * heads) + E / 2 - 1) / (E / 2) : int64_t{1} << 20;
  const int64_t enough = c.bwd ? most : kRotFwdBlocks;
  while (step > 1 && x * ((heads + step - 1) / step) * 2 <= enough) step = (step + 1) / 2;
  const int64_t y = (heads + step - 1) / step;
  x = x * y > most ? (most / y < 1 ? 1 : most / y) : x;
  const dim3 grid(static_cast<unsigned>(x), static_cast<unsigned>(y)), block(64 * kRotWaves);
  *parts = x * y;
#define SSM_ROT_CASE(I, B)                                                                   \
  if ((c.interleaved != 0) == I && c.bwd == B)                                               \
    hipLaunchKernelGGL((rotate_kernel<TA, E, N, I, B>), grid, block, 0, c.stream, a, step);
  SSM_ROT_CASE(false, false)
  SSM_ROT_CASE(true, false)
  SSM_ROT_CASE(false, true)
  SSM_ROT_CASE(true, true)
#undef SSM_ROT_CASE
}

// Whether rows can be moved in vectors of E values, two blocks to a lane.
template <typename TA>
bool rot_fits(const RotCall& c, int E) {
  const size_t bytes = E * sizeof(TA);
  if (c.D % (2 * E) || c.R % (2 * E)) return false;
  if (c.qs % E || !aligned(c.q, bytes) || !aligned(c.qo, bytes) || (c.bwd && !aligned(c.dqo, bytes))) return false;
  return !c.Hk || (c.ks % E == 0 && aligned(c.k, bytes) && aligned(c.ko, bytes) && (!c.bwd || aligned(c.dko, bytes)));
}

template <typename TA, int E>
bool rot_try(const RotCall& c, const RotArgs<TA>& a, int64_t* parts) {
  if (!rot_fits<TA>(c, E)) return false;
  const int lanes = static_cast<int>(c.D / (2 * E));
  if (lanes <= 4) rot_launch_vec<TA, E, 4>(c, a, parts);
  else if (lanes <= 8) rot_launch_vec<TA, E, 8>(c, a, parts);
  else if (lanes <= 16) rot_launch_vec<TA, E, 16>(c, a, parts);
  if constexpr (E == 2) {
    if (lanes > 32) rot_launch_vec<TA, E, 64>(c, a, parts);
    else if (lanes > 16) rot_launch_vec<TA, E, 32>(c, a, parts);
  }
  return true;
}

template <typename TA>
int rot_launch(const RotCall& c) {
  RotArgs<TA> a{static_cast<const TA*>(c.q), static_cast<const TA*>(c.k), c.qw, c.kw, c.freq, c.pos,
                static_cast<const TA*>(c.dqo), static_cast<const TA*>(c.dko), static_cast<TA*>(c.qo),
                static_cast<TA*>(c.ko), static_cast<float*>(c.ws), c.eps, c.batch * c.L, c.L, c.qs,
                c.ks, static_cast<int>(c.Hq), static_cast<int>(c.Hk), static_cast<int>(c.D),
                static_cast<int>(c.R)};
  // Two values an access where the head size, the strides and the addresses
  // allow it, four of float32 up to 128 of them in a head.  8192 tokens,
  // gradients with two | four: 16 + 16 heads of 128 float32 75 | 70 us, 8 + 8 of
  // 256 68 | 78, 4002 tokens of 16 + 4 of 128 bf16 13.4 | 16.8 (half the waves);
  // forward 47 | 45, 40 | 43, 12.5 | 13.8 (8 + 8 of 128 bf16).
  int64_t parts = 0;
  const bool four = sizeof(TA) == 4 && c.D <= 128;
  if (!(four && rot_try<TA, 4>(c, a, &parts)) && !rot_try<TA, 2>(c, a, &parts)) {
    const int64_t rows = c.batch * c.L * (c.Hq + c.Hk);
    const int64_t want = (rows + kRotWaves - 1) / kRotWaves;
    const int64_t blocks = c.bwd ? rot_parts(rows) / kRotWaves : want > (1 << 20) ? (1 << 20) : want;
    const dim3 grid(static_cast<unsigned>(blocks)), block(64 * kRotWaves);
    parts = blocks * kRotWaves;
#define SSM_ROT_CASE(I, B)                                                                   \
  if ((c.interleaved != 0) == I && c.bwd == B)                                               \
    hipLaunchKernelGGL((rotate_any_kernel<TA, I, B>), grid, block, 0, c.stream, a);
    SSM_ROT_CASE(false, false)
    SSM_ROT_CASE(true, false)
    SSM_ROT_CASE(false, true)
    SSM_ROT_CASE(true, true)
#undef SSM_ROT_CASE
  }
  if (c.bwd && (c.dqw || c.dkw))
    hipLaunchKernelGGL(rotate_sum_kernel, dim3((a.D + kRotSumElems - 1) / kRotSumElems, 2), dim3(64 * kRotSumWaves),
                       0, c.stream, a.part, static_cast<int>(parts), a.D, c.dqw, c.dkw);
  return launch_status(c.fn);
}

int rot_call(const RotCall& c) {
  clear_error();
  if (c.dtype != SSM_DTYPE_F32 && c.dtype != SSM_DTYPE_BF16)
    return fail(SSM_ERR_UNSUPPORTED, "%s: unknown dtype %d", c.fn, c.dtype);
  if (c.interleaved != 0 && c.interleaved != 1)
    return fail(SSM_ERR_UNSUPPORTED, "%s: interleaved must be 0 or 1, got %d", c.fn, c.interleaved);
  if (!(c.eps >= 0.0f)) return fail(SSM_ERR_UNSUPPORTED, "%s: eps must be at least 0", c.fn);
  if (c.D < 2 || c.D > 256 || c.D % 2 || c.R < 0 || c.R > c.D || c.R % 2)
    return fail(SSM_ERR_UNSUPPORTED,
                "%s: headdim must be even, 2..256, rotary_dim even, 0..headdim; got %lld, %lld", c.fn,
                (long long)c.D, (long long)c.R);
  if (!rot_sizes_ok(c.batch, c.L, c.Hq, c.Hk, c.D))
    return fail(SSM_ERR_SHAPE, "%s: bad sizes batch %lld, seqlen %lld, heads %lld and %lld", c.fn,
                (long long)c.batch, (long long)c.L, (long long)c.Hq, (long long)c.Hk);
  constexpr int64_t kMaxStride = int64_t{1} << 30;
  if (c.qs < c.Hq * c.D || c.qs > kMaxStride || (c.Hk > 0 && (c.ks < c.Hk * c.D || c.ks > kMaxStride)))
    return fail(SSM_ERR_SHAPE, "%s: a token stride (%lld, %lld) is shorter than its heads or beyond 2^30", c.fn,
                (long long)c.qs, (long long)c.ks);
  const int64_t tokens = c.batch * c.L;
  const bool any = tokens > 0;
  if (c.R > 0 && !c.freq) return fail(SSM_ERR_NULL, "%s: inv_freq is required with rotary_dim > 0", c.fn);
  if (any && (!c.q || !c.qo || (c.bwd && !c.dqo)))
    return fail(SSM_ERR_NULL, "%s: a query tensor is missing", c.fn);
  if (any && c.Hk > 0 && (!c.k || !c.ko || (c.bwd && !c.dko)))
    return fail(SSM_ERR_NULL, "%s: a key tensor is missing", c.fn);
  if (c.Hk == 0 && (c.k || c.ko || c.kw || c.dko || c.dkw))
    return fail(SSM_ERR_NULL, "%s: a key tensor is given with nheads_k = 0", c.fn);
  const size_t es = c.dtype == SSM_DTYPE_F32 ? 4 : 2;
  const char* const oq = c.bwd ? "dq" : "q_out";
  const char* const ok = c.bwd ? "dk" : "k_out";
  const struct { const void* p; size_t k; const char* n; } al[] = {
      {c.q, es, "q"}, {c.k, es, "k"}, {c.qo, es, oq}, {c.ko, es, ok}, {c.dqo, es, "dq_out"},
      {c.dko, es, "dk_out"}, {c.qw, 4, "q_weight"}, {c.kw, 4, "k_weight"}, {c.freq, 4, "inv_freq"},
      {c.pos, 4, "positions"}, {c.dqw, 4, "dq_weight"}, {c.dkw, 4, "dk_weight"}};
  for (const auto& e : al)
    if (e.p && !aligned(e.p, e.k))
      return fail(SSM_ERR_ALIGN, "%s: %s is not %zu-byte aligned", c.fn, e.n, e.k);
  const size_t nq = static_cast<size_t>(tokens) * c.Hq * c.D * es;
  const size_t nk = static_cast<size_t>(tokens) * c.Hk * c.D * es;
  const size_t eq = any ? (static_cast<size_t>(tokens - 1) * c.qs + c.Hq * c.D) * es : 0;
  const size_t ek = any && c.Hk ? (static_cast<size_t>(tokens - 1) * c.ks + c.Hk * c.D) * es : 0;
  const size_t wd = static_cast<size_t>(c.D) * 4;
  const size_t need = c.bwd ? ssm_qk_norm_rotate_bwd_workspace_bytes(c.batch, c.L, c.Hq, c.Hk, c.D) : 0;
  const Span ins[] = {{c.q, eq, "q"}, {c.k, ek, "k"}, {c.dqo, c.dqo ? nq : 0, "dq_out"},
                      {c.dko, c.dko ? nk : 0, "dk_out"}, {c.qw, c.qw ? wd : 0, "q_weight"},
                      {c.kw, c.kw ? wd : 0, "k_weight"},
                      {c.freq, c.freq ? static_cast<size_t>(c.R) * 2 : 0, "inv_freq"},
                      {c.pos, c.pos ? static_cast<size_t>(tokens) * 4 : 0, "positions"}};
  const Span outs[] = {{c.qo, nq, oq}, {c.ko, nk, ok}, {c.dqw, c.dqw ? wd : 0, "dq_weight"},
                       {c.dkw, c.dkw ? wd : 0, "dk_weight"}, {c.ws, c.ws ? need : 0, "workspace"}};
  for (const auto& o : outs)
    for (const auto& n : ins) {
      // a contiguous input may be normalised where it is (forward)
      const bool here = !c.bwd && o.p == n.p &&
                        ((o.p == c.qo && n.p == c.q && c.qs == c.Hq * c.D) ||
                         (o.p == c.ko && n.p == c.k && c.ks == c.Hk * c.D));
      if (overlap(o, n) && !here)
        return fail(SSM_ERR_ALIAS, "%s: output %s overlaps input %s", c.fn, o.name, n.name);
    }
  for (int x = 0; x < 5; ++x)
    for (int y = x + 1; y < 5; ++y)
      if (overlap(outs[x], outs[y]))
        return fail(SSM_ERR_ALIAS, "%s: %s overlaps %s", c.fn, outs[x].name, outs[y].name);
  if (need > 0 && (!c.ws || c.ws_bytes < need))
    return fail(SSM_ERR_WORKSPACE, "%s: workspace of %zu bytes given, %zu needed", c.fn,
                c.ws ? c.ws_bytes : 0, need);
  if (need > 0 && !aligned(c.ws, 256))
    return fail(SSM_ERR_ALIGN, "%s: workspace is not 256-byte aligned", c.fn);
  if (!any && !c.bwd) return SSM_OK;  // (the backward of no tokens leaves zero weight gradients)
  return c.dtype == SSM_DTYPE_F32 ? rot_launch<float>(c) : rot_launch<bf16_t>(c);
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" {

int ssm_qk_norm_rotate_fwd(const void* q, const void* k, const float* q_weight,
                           const float* k_weight, const float* inv_freq, const int32_t* positions,
                           float eps, int interleaved, void* q_out, void* k_out, int64_t batch,
                           int64_t seqlen, int64_t nheads_q, int64_t nheads_k, int64_t headdim,
                           int64_t rotary_dim, int64_t q_token_stride, int64_t k_token_stride,
                           int dtype, hipStream_t stream) {
  return rot_call(RotCall{"ssm_qk_norm_rotate_fwd", q, k, q_weight, k_weight, inv_freq, positions,
                          eps, interleaved, nullptr, nullptr, q_out, k_out, nullptr, nullptr, batch,
                          seqlen, nheads_q, nheads_k, headdim, rotary_dim, q_token_stride,
                          k_token_stride, dtype, nullptr, 0, stream, false});
}

int ssm_qk_norm_rotate_bwd(const void* q, const void* k, const float* q_weight,
                           const float* k_weight, const float* inv_freq, const int32_t* positions,
                           float eps, int interleaved, const void* dq_out, const void* dk_out,
                           void* dq, void* dk, float* dq_weight, float* dk_weight, int64_t batch,
                           int64_t seqlen, int64_t nheads_q, int64_t nheads_k, int64_t headdim,
                           int64_t rotary_dim, int64_t q_token_stride, int64_t k_token_stride,
                           int dtype, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return rot_call(RotCall{"ssm_qk_norm_rotate_bwd", q, k, q_weight, k_weight, inv_freq, positions,
                          eps, interleaved, dq_out, dk_out, dq, dk, dq_weight, dk_weight, batch,
                          seqlen, nheads_q, nheads_k, headdim, rotary_dim, q_token_stride,
                          k_token_stride, dtype, workspace, workspace_bytes, stream, true});
}

size_t ssm_qk_norm_rotate_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads_q,
                                              int64_t nheads_k, int64_t headdim) {
  if (!rot_sizes_ok(batch, seqlen, nheads_q, nheads_k, headdim)) return 0;
  const int64_t rows = batch * seqlen * (nheads_q + nheads_k);
  return static_cast<size_t>(rot_parts(rows)) * 2 * headdim * sizeof(float);
}

}  // extern "C"
