// gated.hpp -- device code shared by the gated linear recurrence's forward,
// backward and decode kernels (gated.hip, gated_bwd.hip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "ssm_recurrent.h"

#include "kernels.hpp"

namespace ssm {

// sigma of v given t = -v log2 e: one hardware exp2 and one reciprocal (an ulp
// each).  v below -88 gives 0 and v = +-inf its limit.
__device__ __forceinline__ float sigmoid2(float t) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(t));
}
__device__ __forceinline__ float sigmoid_f32(float v) { return sigmoid2(v * -kLog2e); }

// The decay a = 2^-v (v = -la log2 e, la the log of the decay) and E = 1 - a.
// Next to a = 1, where a long memory lives, E comes from v q(v) and keeps its
// full precision: a = 1 - E is then rounded to nearest (the hardware exp2
// rounds low on average, which a memory of thousands of tokens adds up), and
// m = sqrt(1 - a^2) = sqrt(E (2 - E)) loses nothing to cancellation.  q(v) =
// (1 - 2^-v) / v as a cubic fitted at Chebyshev points of [0, 3/16], within
// 4.1e-8 of it there and nowhere else (7e-6 at -3/16).  Above, a <= 0.879 and
// E = 1 - a is exact enough; below 0 (growing states) m is 0 and only a counts.
__device__ __forceinline__ float decay_parts(float v, float& a) {
  const float ex = __builtin_amdgcn_exp2f(-v);
  float q = __builtin_fmaf(v, -0.009133012033998966f, 0.055447835475206375f);
  q = __builtin_fmaf(v, q, -0.24022440612316132f);
  q = __builtin_fmaf(v, q, 0.6931471824645996f);
  const bool near = __float_as_uint(v) < __float_as_uint(0.1875f);  // (0 <= v < 3/16: a sign or a NaN compares above)
  // both sides are computed and one is selected: left to itself the compiler
  // branches around each side, and the tokens no longer overlap
  float En = v * q, Ef = 1.0f - ex, an = 1.0f - En;
  asm("" : "+v"(En), "+v"(Ef), "+v"(an));
  a = near ? an : ex;
  return near ? En : Ef;
}
// m^2 = 1 - a^2, 0 for a growing state (the clamp costs nothing: it is a
// modifier of the product).
__device__ __forceinline__ float input_scale2(float E) {
  return __builtin_amdgcn_fmed3f(E * (2.0f - E), 0.0f, 1.0f);
}
template <bool NORM>
__device__ __forceinline__ void decay(float v, float& a, float& m) {
  const float E = decay_parts(v, a);
  m = NORM ? __builtin_amdgcn_sqrtf(input_scale2(E)) : 1.0f;
}

// A channel's parameters as the kernels use them: -A log2 e and the biases
// times -log2 e.
struct Params {
  float A2, rb2, ib2;
};
__device__ __forceinline__ Params params_of(float A, float rb, float ib) {
  float A2 = A * -kLog2e;
  if (A2 > 1e30f) A2 = 1e30f;  // (finite: a token that is masked takes it times 0)
  return Params{A2, rb * -kLog2e, ib * -kLog2e};
}
__device__ __forceinline__ Params load_params(const float* A, const float* rb, const float* ib, int c,
                                              bool have) {
  return params_of(have ? A[c] : 0.0f, have && rb ? rb[c] : 0.0f, have && ib ? ib[c] : 0.0f);
}

// ----------------------------------------------------------------------------
// The walk over time.  A workgroup holds a chunk of tokens of 64 channels: a
// lane has one channel, wave w the tokens [T w, T w + T), everything in
// registers.  A stretch of tokens maps the state before it to the state after
// it, h -> P h + H; the maps of waves and chunks compose.
// ----------------------------------------------------------------------------
constexpr int kGatedC = 64;      // channels of a workgroup
constexpr int kGatedGroup = 16;  // chunks of a group (see gated.hip)

// A lane's value of one token: the raw bits as loaded, widened at use.
template <typename TA>
struct Cell;
template <>
struct Cell<float> {
  using raw_t = uint32_t;
  __device__ static raw_t load(rsrc_t r, uint32_t vo, uint32_t so) {
    return __builtin_amdgcn_raw_buffer_load_b32(r, vo, so, 0);
  }
  __device__ static float get(raw_t v) { return __uint_as_float(v); }
  __device__ static void store(rsrc_t r, float v, uint32_t vo, uint32_t so) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, vo, so, kStoreStream);
  }
};
template <>
struct Cell<bf16_t> {
  using raw_t = uint16_t;
  __device__ static raw_t load(rsrc_t r, uint32_t vo, uint32_t so) {
    return __builtin_amdgcn_raw_buffer_load_b16(r, vo, so, 0);
  }
  __device__ static float get(raw_t v) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
  __device__ static void store(rsrc_t r, float v, uint32_t vo, uint32_t so) {
    const __bf16 b = static_cast<__bf16>(v);  // round to nearest even
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, b), r, vo, so, kStoreStream);
  }
};

// Byte offset that no descriptor here covers (a wave's rows span at most
// 64 * 2^22 * 4 = 2^30 bytes: see gated_sizes_ok): lanes beyond the last
// channel use it, so their loads give 0 and their stores are dropped
// by the range check.
constexpr uint32_t kNoColumn = 0x7fffff00u;

// The map h -> P h + H of a stretch is kept as (y, H).  y >= +0 is P itself;
// y with the sign set is P - 1, for P from 1/2 to 1: a product of decays next
// to 1 loses the same way at every factor when it is rounded (1 - p)(1 - e) ->
// 1 - p - e, which a memory of thousands of tokens shows (1.1e-5 at 6000
// tokens with decays of 1 - 1e-5 to 1 - 1e-3, against 1e-6 in this form).
// y below kCut is -P^(1/4), for P from 2^64 on (a growing state, A > 0; P <= 1
// otherwise): a product beyond float32 acts on a state factor by factor, so
// that only states that are themselves beyond float32 overflow.  Past 2^508,
// where any state but 0 does, it stays at the largest float, and 0 stays 0.
// kCut: a sequence starts inside the stretch, nothing of the incoming state
// passes; it is left out rather than multiplied by zero, so that a NaN or an
// infinity stays in its own sequence.
constexpr float kCut = -2.0f;
__device__ __forceinline__ bool below_one(float y) { return __float_as_int(y) < 0; }

constexpr float kMaxRoot = 0x1.fffffep127f;

// y of a stretch whose v add up to S (the identity for 0).
__device__ __forceinline__ float keep_of(float S) {
  float a;
  const float E = decay_parts(S, a);
  const float y = E < 0.5f && E >= 0.0f ? -__builtin_fabsf(E) : a;
  return S < -64.0f ? -__builtin_fminf(__builtin_amdgcn_exp2f(-0.25f * S), kMaxRoot) : y;
}
// P^(1/4) of a y that is no cut.
__device__ __forceinline__ float root_of(float y) {
  return y < kCut ? -y : __builtin_amdgcn_sqrtf(__builtin_amdgcn_sqrtf(below_one(y) ? 1.0f + y : y));
}
// The state behind a stretch with h before it.  PLAIN: without what follows,
// for a caller that looks at the result.
// An infinite h stays infinite (no decay is 0 in exact arithmetic), also where
// P is the identity or underflows, whose products with it would be NaN.
template <bool VL, bool PLAIN = false>
__device__ __forceinline__ float pass(float y, float H, float h) {
  float r = __builtin_fmaf(y, h, below_one(y) ? h : 0.0f) + H;
  if (!PLAIN) {
    if (y < kCut)
      r = h * -y * -y * -y * -y + H;
    else if (!__builtin_isfinite(r) && __builtin_isinf(h))
      r = h + H;
  }
  if constexpr (VL) return y == kCut ? H : r;
  return r;
}
// (y1, H1) followed by (y2, H2).
template <bool VL, bool PLAIN = false>
__device__ __forceinline__ void compose(float& y1, float& H1, float y2, float H2) {
  H1 = pass<VL, PLAIN>(y2, H2, H1);
  const bool n1 = below_one(y1), n2 = below_one(y2);
  const float both = __builtin_fmaf(y1, y2, y1) + y2;  // (1 + y1)(1 + y2) - 1
  float y = n1 ? (n2 ? (both >= -0.5f ? -__builtin_fabsf(both) : 1.0f + both) : __builtin_fmaf(y1, y2, y2))
               : __builtin_fmaf(y1, y2, n2 ? y1 : 0.0f);
  if (!PLAIN && (y > 0x1p64f || y1 < kCut || y2 < kCut))
    y = -__builtin_fminf(root_of(y1) * root_of(y2), kMaxRoot);
  if constexpr (VL) {
    if (y1 == kCut || y2 == kCut) y = kCut;
  }
  y1 = y;
}

// n maps of the lane's channel, in LDS, composed or applied to a state one
// after the other (BACK: from the last to the first).  The plain forms go
// wrong only where a root is among the maps, or in a way that stays visible in
// the result: an infinity or NaN ends at a cut at most, and P never falls from
// above 2^64 (an overflowed one with the identity behind it is NaN).  Then the fold is done once more with care (with a look at every
// step packed 8192 x 1001 float32 takes 46 us, so 43).
template <bool VL, bool BACK>
__device__ __forceinline__ void fold_maps(const float2 (*maps)[kGatedC], int n, int lane, float& y, float& H) {
  y = -0.0f;
  H = 0.0f;
  float least = 0.0f;
  for (int k = 0; k < n; ++k) {
    const float2 f = maps[BACK ? n - 1 - k : k][lane];
    least = __builtin_fminf(least, f.x);
    compose<VL, true>(y, H, f.x, f.y);
  }
  if (least < kCut || !(y <= 0x1p64f) || !__builtin_isfinite(H)) {
    y = -0.0f;
    H = 0.0f;
    for (int k = 0; k < n; ++k) {
      const float2 f = maps[BACK ? n - 1 - k : k][lane];
      compose<VL>(y, H, f.x, f.y);
    }
  }
}
template <bool VL, bool BACK>
__device__ __forceinline__ float fold_state(const float2 (*maps)[kGatedC], int n, int lane, float h0) {
  float h = h0, least = 0.0f;
  for (int k = 0; k < n; ++k) {
    const float2 f = maps[BACK ? n - 1 - k : k][lane];
    least = __builtin_fminf(least, f.x);
    h = pass<VL, true>(f.x, f.y, h);
  }
  if (least < kCut || !__builtin_isfinite(h)) {
    h = h0;
    for (int k = 0; k < n; ++k) {
      const float2 f = maps[BACK ? n - 1 - k : k][lane];
      h = pass<VL>(f.x, f.y, h);
    }
  }
  return h;
}

// Which of a wave's tokens (64 at most) start and end their sequence, a bit
// each, and each token's sequence (held by lane j for token j).
struct Marks {
  uint64_t starts, ends;
  int seq;
};
// The offsets, read through the scalar cache: nothing writes them meanwhile,
// and a scalar load waits for no row that is on its way.
typedef const int32_t __attribute__((address_space(4)))* scalar_i32;
__device__ __forceinline__ scalar_i32 scalar_of(const int32_t* p) {
  return (scalar_i32)(reinterpret_cast<uintptr_t>(p));
}
__device__ __forceinline__ Marks find_marks(const int32_t* cu, int nseq, int64_t from, int n) {
  const scalar_i32 cs = scalar_of(cu);
  const int t0 = static_cast<int>(from);  // (n > 0: the tokens are below cu[nseq])
  // one search for the whole stretch, until an offset falls inside of it: the
  // sequence of each of its tokens is in [lo, hi), the last s with cu[s] <= t
  // (empty sequences are passed over)
  int lo = 0, hi = nseq;
  while (hi - lo > 1) {
    const int mid = lo + ((hi - lo) >> 1), v = cs[mid];
    if (v <= t0) lo = mid;
    else if (v >= t0 + n) hi = mid;
    else break;
  }
  if (hi - lo == 1)
    return Marks{cs[lo] == t0 ? uint64_t{1} : 0, cs[lo + 1] == t0 + n ? uint64_t{1} << (n - 1) : 0, lo};
  // a lane searches for its token
  const int lane = threadIdx.x & 63;
  Marks m{0, 0, 0};
  bool st = false, en = false;
  if (lane < n) {
    const int t = t0 + lane;
    while (hi - lo > 1) {
      const int mid = lo + ((hi - lo) >> 1);
      if (cu[mid] <= t) lo = mid; else hi = mid;
    }
    m.seq = lo;
    st = cu[lo] == t;
    en = cu[lo + 1] == t + 1;
  }
  m.starts = __ballot(st);
  m.ends = __ballot(en);
  return m;
}

// Publishing between workgroups.  A word is written once, as a whole, and
// says by itself that it is there: the launch before fills the words with
// ones, which no published word equals.  Relaxed 64-bit atomics at device
// scope, so nothing has to be flushed or invalidated around them.
__device__ __forceinline__ void publish(uint64_t* at, float lo, float hi) {
  uint32_t a = __float_as_uint(lo);
  if (a == 0xffffffffu) a = 0x7fc00000u;  // a NaN of another payload
  __hip_atomic_store(at, (static_cast<uint64_t>(__float_as_uint(hi)) << 32) | a, __ATOMIC_RELAXED,
                     __HIP_MEMORY_SCOPE_AGENT);
}
// The lane's V words, once they are all there.  Every wait is for a
// workgroup that took its turn earlier and publishes without waiting for a
// later one, so it ends.  Should the words be overwritten meanwhile (a
// workspace given to two calls at once), the wait still ends, after a quarter
// of a second, and gives NaN.
constexpr int kWaitLimit = 1 << 18;
// K words a lane at once: at + k * stride for k < n (n <= K, uniform).  While
// some are missing the wave polls one of them alone.
template <int K>
__device__ __forceinline__ void await(uint64_t* at, int64_t stride, int n, float (&lo)[K], float (&hi)[K]) {
  uint64_t w[K];
  for (int tries = 0;;) {
    uint64_t* missing = nullptr;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (k < n) w[k] = __hip_atomic_load(at + k * stride, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int k = K - 1; k >= 0; --k)
      if (k < n && w[k] == ~uint64_t{0}) missing = at + k * stride;
    const uint64_t lanes = __ballot(missing != nullptr);
    if (lanes == 0 || tries >= kWaitLimit) break;
    const int l = __builtin_ctzll(lanes);
    const uint64_t p = reinterpret_cast<uint64_t>(missing);
    uint64_t* const one = reinterpret_cast<uint64_t*>(
        static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(p), l))) |
        static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(p >> 32), l))) << 32);
    for (; tries < kWaitLimit; ++tries) {
      if (__hip_atomic_load(one, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != ~uint64_t{0}) break;
      __builtin_amdgcn_s_sleep(1);
    }
    ++tries;
  }
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (k < n) {
      lo[k] = __uint_as_float(static_cast<uint32_t>(w[k]));
      hi[k] = __uint_as_float(static_cast<uint32_t>(w[k] >> 32));
    }
  }
}

// The workspace of a time-split launch.  `cells` channel slots (rows * tiles
// * 64), chunk-major, so that a chunk's words lie together:
//   agg   (chunks, cells): a chunk's map (y, H)
//   carry (groups, cells): the state that enters a group, {0, h}
//   turn  the counter that hands out the units
struct GatedPlan {
  uint32_t chunks, groups, tiles, lines, units;  // lines = rows * tiles, units = lines * chunks
  int64_t cells;
  size_t bytes;  // 0: one chunk per row, no workspace
};
// A grid of `units` workgroups: rows of kGatedGridX, so that neither extent
// times the workgroup's threads passes 32 bits; the last row's surplus returns.
constexpr uint32_t kGatedGridX = 1u << 22;
inline dim3 gated_grid(uint32_t units) {
  return dim3(units < kGatedGridX ? units : kGatedGridX, (units + kGatedGridX - 1) / kGatedGridX);
}
inline GatedPlan gated_plan(int64_t rows, int64_t L, int64_t dim, int chunk) {
  const int64_t chunks = L > 0 ? (L + chunk - 1) / chunk : 1;
  const int64_t groups = (chunks + kGatedGroup - 1) / kGatedGroup;
  const int64_t tiles = (dim + kGatedC - 1) / kGatedC;
  const int64_t cells = rows * tiles * kGatedC;
  return GatedPlan{static_cast<uint32_t>(chunks), static_cast<uint32_t>(groups),
                   static_cast<uint32_t>(tiles), static_cast<uint32_t>(rows * tiles),
                   static_cast<uint32_t>(rows * tiles * chunks), cells,
                   chunks > 1 ? static_cast<size_t>(chunks + groups) * cells * 8 + 256 : 0};
}

// Fills the words with ones and the counter with zero, and moves the state
// of empty sequences (`empty_to`, packed only) through unchanged.
int launch_gated_init(void* ws, size_t bytes, const int32_t* cu, int64_t nseq, int64_t L, int dim,
                      const float* empty_from, float* empty_to, const char* fn, hipStream_t s);

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
  float* part;  // partial sums
};

// Whether these sizes can be launched; bytes of the forward's words; the
// states at the chunks' starts alone (gated.hip).
bool gated_sizes_ok(int64_t rows, int64_t L, int64_t nseq, int64_t dim, bool packed);
size_t gated_fwd_bytes(int64_t rows, int64_t L, int64_t dim);
int gated_states(const char* fn, const void* x, const void* r, const void* i, const float* A,
                 const float* rb, const float* ib, int normalize, const float* h0, float* states,
                 const int32_t* cu, int64_t nseq, int64_t rows, int64_t L, int dim, int dtype,
                 void* ws, hipStream_t stream);

}  // namespace ssm
