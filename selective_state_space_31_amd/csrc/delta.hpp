// delta.hpp -- what the gated delta rule's translation units share: sizes and
// their checks, the launch arguments, and the device helpers of the matrix
// products in float32's precision.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "ssm_layer.h"

#include "host_util.hpp"
#include "kernels.hpp"

namespace ssm {

constexpr int kDeltaC = SSM_DELTA_CHUNK;  // tokens of a chunk
constexpr int64_t kDeltaMaxWidth = 256;   // headdim_k, headdim_v

// Sizes of a call.  Whole sequences: nseq = batch, L tokens each.  Packed:
// nseq sequences in L tokens, cu their offsets.
struct DeltaDims {
  int64_t nseq, L;
  int hk, hv, K, V;
  int64_t qs, ks, vs;  // token strides in values
  bool packed;
  int64_t tokens() const { return packed ? L : nseq * L; }
  // places of chunks: whole sequences have ceil(L / C) each; packed ones have
  // at most L / C + nseq in all, sequence s from place cu[s] / C + s on
  int64_t chunks() const {
    return packed ? L / kDeltaC + nseq : nseq * ((L + kDeltaC - 1) / kDeltaC);
  }
  size_t state_values() const { return static_cast<size_t>(hv) * K * V; }
  // of chunk_states: the state and the chunk's e per place and head
  size_t mid_values() const { return static_cast<size_t>(chunks()) * hv * (K + kDeltaC) * V; }
};

inline bool delta_sizes_ok(int64_t nseq, int64_t L, int64_t hk, int64_t hv, int64_t K, int64_t V, bool packed) {
  if (nseq < 1 || nseq >= (packed ? int64_t{1} << 20 : int64_t{65536}) || L < 0 || L >= (int64_t{1} << 31)) return false;
  if (hk < 1 || hv < hk || hv > 65535 || hv % hk != 0) return false;
  if (K < 1 || K > kDeltaMaxWidth || V < 1 || V > kDeltaMaxWidth) return false;
  if (!packed && nseq * L >= (int64_t{1} << 31)) return false;
  const int64_t chunks = packed ? L / kDeltaC + nseq : nseq * ((L + kDeltaC - 1) / kDeltaC);
  // (a launch has less than 2^32 threads, up to 512 of them for a chunk or a column block)
  return chunks * hv < (int64_t{1} << 22) && nseq * hv * ((V + 15) / 16) < (int64_t{1} << 22);
}

inline bool delta_strides_ok(const DeltaDims& d) {
  const int64_t most = int64_t{1} << 22;  // (64 rows stay within 32-bit byte offsets)
  return d.qs >= int64_t{d.hk} * d.K && d.qs <= most && d.ks >= int64_t{d.hk} * d.K && d.ks <= most &&
         d.vs >= int64_t{d.hv} * d.V && d.vs <= most;
}

// Sequence b's tokens [lo, hi) and its first place among the chunks.  Offsets
// are not checked on the host: here they are bounded by the number of tokens,
// and the places stay below DeltaDims::chunks().
struct DeltaSeq {
  int64_t lo, hi, slot;
};
__device__ __forceinline__ DeltaSeq delta_seq(const int32_t* cu, int64_t b, int64_t L) {
  if (!cu) return DeltaSeq{b * L, (b + 1) * L, b * ((L + kDeltaC - 1) / kDeltaC)};
  int64_t lo = cu[b], hi = cu[b + 1];
  lo = lo < 0 ? 0 : lo > L ? L : lo;
  hi = hi < lo ? lo : hi > L ? L : hi;
  return DeltaSeq{lo, hi, lo / kDeltaC + b};
}

// The rule token by token (delta_step.hip): first may be NULL (zeros), last and
// mids (the states before every kDeltaC-th token) too.
int delta_walk(const char* fn, int dtype, const void* q, const void* k, const void* v, const float* beta,
               const float* g, float scale, void* out, float* last, const float* first, float* mids,
               const int32_t* cu, const DeltaDims& d, hipStream_t stream);

// bytes from the first to the last value of `rows` rows of `width` values
inline size_t strided_bytes(int64_t rows, int64_t width, int64_t stride, size_t es) {
  return rows > 0 ? (static_cast<size_t>(rows - 1) * stride + width) * es : 0;
}

// ---------------------------------------------------------------------------
// matrix products in float32's precision on the bf16 matrix cores
// ---------------------------------------------------------------------------
// A float32 value is the sum of three bf16 ones (8 significant bits each, the
// later parts round what the earlier ones left).  A product of two such values
// keeps the partial products whose parts' indices add up to less than three:
// six of nine, the dropped ones below 2^-26 of it.  A bf16 input is its own first
// part, exactly; what is computed has three parts, also where it reaches bf16
// outputs alone: those are often what is left of a key's much larger old value
// (with two parts outputs of size 1 behind a state of size 1000 are off by 1.7e-2,
// with three by 1.5e-3).  (The float32 matrix instruction has the precision too, at 1/16
// of the bf16 rate: six products are 2.7 times as fast, three 5.3.)
typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8;
typedef __attribute__((ext_vector_type(2))) __bf16 bf16x2;
typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(2))) uint32_t u32x2;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4;

template <typename TA>
constexpr int kInParts = sizeof(TA) == 4 ? 3 : 1;

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
                                                 0);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const bf16x2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xffff0000u); }

// The largest value that has parts: its first one would be infinite beyond, the
// others NaN.
constexpr float kPartsMost = 0x1.fep127f;
__device__ __forceinline__ bool has_parts(float x) { return __builtin_fabsf(x) <= kPartsMost; }

// Two values into N parts each, packed
template <int N>
__device__ __forceinline__ void split2(float a, float b, uint32_t (&p)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    p[i] = pack_bf16(a, b);
    asm("" : "+v"(p[i]));  // (or the compiler converts a second time for each half)
    a -= bf_lo(p[i]);
    b -= bf_hi(p[i]);
  }
}

// c += a b over the parts
template <int NA, int NB>
__device__ __forceinline__ f32x4 mul_parts(const u32x4 (&a)[NA], const u32x4 (&b)[NB], f32x4 c) {
#pragma unroll
  for (int s = 2; s >= 0; --s)
#pragma unroll
    for (int i = 0; i <= s; ++i)
      if (i < NA && s - i < NB) c = mfma16(a[i], b[s - i], c);
  return c;
}

// The same with c rounded twice, whatever the number of products: what the lower
// parts give is summed apart.
template <int NA, int NB>
__device__ __forceinline__ f32x4 mul_parts_apart(const u32x4 (&a)[NA], const u32x4 (&b)[NB], f32x4 c) {
  f32x4 t = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int s = 2; s > 0; --s)
#pragma unroll
    for (int i = 0; i <= s; ++i)
      if (i < NA && s - i < NB) t = mfma16(a[i], b[s - i], t);
  return mfma16(a[0], b[0], c + t);
}

// Matrix fragments.  A product's left operand: lane l holds row l % 16 and eight
// of 32 columns; the right one likewise with rows and columns exchanged; the
// result has column l % 16, rows 4 (l / 16) + 0..3.  Which eight is free as long
// as both operands agree.  Sums over headdim_k take 8 (l / 16) .. + 7, which lie
// together in a row of K or Q.  Sums over tokens take 4 q .. + 3 and 16 + 4 q
// .. + 3 with q = l / 16: then two results below each other are, value by value,
// the right operand of a product over their rows, and two results of the
// transposed product side by side a left one.  In memory a fragment is 64 times
// 16 bytes, lane after lane.
__device__ __forceinline__ int frag_tok(int q, int e) { return (e < 4 ? 4 * q : 12 + 4 * q) + e; }

template <int N>
__device__ __forceinline__ void split4(f32x4 x, u32x2 (&p)[N]) {
  uint32_t lo[N], hi[N];
  split2(x[0], x[1], lo);
  split2(x[2], x[3], hi);
#pragma unroll
  for (int i = 0; i < N; ++i) p[i] = u32x2{lo[i], hi[i]};
}
// A result over row block t goes into the parts' right operands in LDS, base:
// [N][blocks][NC][64], column block nb: for sums over tokens, over headdim_k.
template <int N, int NC>
__device__ __forceinline__ void put_tok(u32x4* base, int blocks, int t, int nb, int lane, f32x4 x) {
  u32x2 p[N];
  split4(x, p);
#pragma unroll
  for (int i = 0; i < N; ++i)
    reinterpret_cast<u32x2*>(base + ((i * blocks + (t >> 1)) * NC + nb) * 64 + lane)[t & 1] = p[i];
}
template <int N, int NC>
__device__ __forceinline__ void put_key(u32x4* base, int blocks, int t, int nb, int lane, f32x4 x) {
  u32x2 p[N];
  split4(x, p);
  const int q = lane >> 4, at = ((t & 1) * 2 + (q >> 1)) * 16 + (lane & 15);
#pragma unroll
  for (int i = 0; i < N; ++i)
    reinterpret_cast<u32x2*>(base + ((i * blocks + (t >> 1)) * NC + nb) * 64 + at)[q & 1] = p[i];
}

// The float32 values that put_key left in three parts (their sum is exact), rows
// of `row` bytes, columns c0 .. of V: a wave of four stores every fourth block of
// 32 rows.
template <int KT, int NC>
__device__ __forceinline__ void store_parts(float* dst, uint32_t bytes, uint32_t row, const u32x4* base, int w, int lane,
                                            int c0, int V) {
  const rsrc_t rs = make_rsrc(dst, bytes);
  const int n = lane & 15, g = lane >> 4;
  for (int kb = w; kb < KT; kb += 4)
#pragma unroll
    for (int nb = 0; nb < NC; ++nb) {
      const int col = c0 + 16 * nb + n;
      const uint32_t at = col < V ? (32u * kb + 8u * g) * row + col * 4u : 0x80000000u;
      const u32x4 a = base[(kb * NC + nb) * 64 + lane], m = base[((KT + kb) * NC + nb) * 64 + lane],
                  z = base[((2 * KT + kb) * NC + nb) * 64 + lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(bf_lo(a[e]) + (bf_lo(m[e]) + bf_lo(z[e]))), rs,
                                              at + (2 * e) * row, 0, 0);
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(bf_hi(a[e]) + (bf_hi(m[e]) + bf_hi(z[e]))), rs,
                                              at + (2 * e + 1) * row, 0, 0);
      }
    }
}

// Triangles of 64 x 64 in 16 x 32 blocks.  Lower: row blocks 0 and 1 have one,
// 2 and 3 have two.  Upper (a lower one transposed): 0 and 1 have two, 2 and 3
// the second alone.
constexpr int kTri = 6;
__device__ __forceinline__ int tri_at(int rowblock, int kb) { return rowblock < 2 ? rowblock : 2 * rowblock - 2 + kb; }
__device__ __forceinline__ int tri_up(int rowblock, int kb) { return rowblock < 2 ? 2 * rowblock + kb : 2 + rowblock; }

// The sequence that chunk place `slot` of a packed call lies in: the largest s
// in [0, nseq) with cu[s] / C + s <= slot, found by a 64-way search.  Probes stay
// inside cu[0, nseq), so unsorted offsets still give an index in range.  slot is
// wave-uniform and all 64 lanes must be active.
__device__ __forceinline__ int delta_owner(const int32_t* cu, int nseq, int64_t slot) {
  const int lane = static_cast<int>(threadIdx.x & 63);
  int lo = 0, cnt = nseq;
  for (;;) {
    const int stride = (cnt + 63) >> 6;
    const int i = lane * stride;
    const bool p = i < cnt && int64_t{cu[lo + i]} / kDeltaC + lo + i <= slot;
    const unsigned long long m = __ballot(p);
    const int k = m ? 63 - __builtin_clzll(m) : 0;
    lo = __builtin_amdgcn_readfirstlane(lo + k * stride);
    if (stride == 1) return lo;
    cnt = (cnt - k * stride < stride) ? cnt - k * stride : stride;
  }
}

// (Several workgroups write a line of an output: it stays in L2 for them.)
template <typename TA>
__device__ __forceinline__ void buffer_store_act(float v, rsrc_t r, uint32_t off) {
  TA t;
  store_act(&t, v);
  if constexpr (sizeof(TA) == 4) __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, off, 0, 0);
  else __builtin_amdgcn_raw_buffer_store_b16(t.bits, r, off, 0, 0);
}

// ---------------------------------------------------------------------------
// chunks
// ---------------------------------------------------------------------------
// With S0 the state before a chunk, G the running sum of g, gamma_i = e^{G_i},
// D_ij = e^{G_i - G_j} and e_i = v_i - S^T k_i what a token finds missing (so u =
// beta e):
//   (I + A) e = V - gamma (K S0),  A_ij = beta_j D_ij k_i.k_j below the diagonal
//   out = scale (gamma (Q S0) + P e),  P_ij = beta_j D_ij q_i.k_j on and below it
//   S1 = gamma_63 S0 + K^T (d e),  d_j = beta_j e^{G_63 - G_j}
// e rather than u, so that beta = 0 needs no division for beta's gradient, which is
// y.e.  The backward solves with beta_i in A_ij and keeps beta out of P and d: that
// is the transposed system of u.
// What does not depend on the state is prepared per chunk (delta_prep.hip), T =
// (I + A)^-1 among it.
struct ChunkSpace {
  // per place and key head, parts in turn: fragments of K and Q (4 row blocks x
  // KT of 32 columns) and of K^T and Q^T (2 KT row blocks x 2 of 32 tokens)
  u32x4 *kf, *qf, *ktf, *qtf;
  // per place and value head, in three parts: fragments of T and P (forward), of
  // T^T and P^T (backward)
  u32x4 *tf, *pf;
  float* vec;  // gamma (64), d (64); for the backward -beta gamma (64) too
};

template <typename TA>
struct PrepArgs {
  const TA *q, *k;
  const float *beta, *g;
  const int32_t* cu;
  int64_t nseq, L, qs, ks;
  int hk, hv, K;
  ChunkSpace c;
};

inline int delta_kt(int K) { return K <= 32 ? 1 : K <= 64 ? 2 : K <= 128 ? 4 : 8; }  // columns in blocks of 32

// Carves the forward's or the backward's space from `base` (NULL: counts only);
// returns the bytes.
inline size_t chunk_space(const DeltaDims& d, int dtype, bool back, char* base, ChunkSpace* c) {
  const size_t in = dtype == SSM_DTYPE_F32 ? 3 : 1, kt = delta_kt(d.K);
  const size_t n = static_cast<size_t>(d.chunks()), frag = 64 * sizeof(u32x4);
  const size_t rows = n * d.hk * in * 4 * kt * frag, tri = n * d.hv * kTri * frag;
  size_t at = 0;
  const auto take = [&](size_t bytes) {
    char* const r = base ? base + at : nullptr;
    at += bytes;
    return r;
  };
  ChunkSpace s;
  s.kf = reinterpret_cast<u32x4*>(take(rows));
  s.qf = reinterpret_cast<u32x4*>(take(back ? 0 : rows));
  s.ktf = reinterpret_cast<u32x4*>(take(rows));
  s.qtf = reinterpret_cast<u32x4*>(take(back ? rows : 0));
  s.tf = reinterpret_cast<u32x4*>(take(3 * tri));
  s.pf = reinterpret_cast<u32x4*>(take(3 * tri));
  s.vec = reinterpret_cast<float*>(take(n * d.hv * (back ? 3 : 2) * kDeltaC * 4));
  if (c) *c = s;
  return at;
}

// Whether a workgroup of the passes over chunks takes two column blocks of 16
// rather than one: the same left operands then serve twice the columns, and rows of
// the states are written in whole lines, but a chunk takes longer.  So where one
// block each would be more workgroups than compute units.  Calls of 1024 tokens a
// sequence, heads of 128, one block and two (workgroups of one block; bf16 and
// float32):
//   96 (1 x 12 heads)   forward 45 / 57 us, 61 / 74; gradients 84 / 99, 100 / 122
//   192                 46 / 58, 66 / 78; 100 / 113, 132 / 155
//   256 (heads of 64)   45 / 56, 61 / 73; 98 / 110, 152 / 166
//   288                 62 / 60, 116 / 93; with the states 77 / 64, 124 / 104
//   480                 66 / 66, 146 / 120; states 81 / 69, 185 / 154
//   576                 92 / 107, 227 / 196; states 141 / 134, 280 / 242
//   768                 114 / 121, 282 / 233; states 168 / 157, 324 / 278
//   1536                266 / 224, 533 / 395; states 388 / 293, 619 / 457
// Not for packed sequences: a few long ones may be all that is there to do, and a
// chunk of theirs takes 2.8 us instead of 1.65 (11 of 0 to 3000 tokens: 715
// workgroups 108 / 137 and 160 / 181, 1056 139 / 155 and 345 / 301, 3520 464 / 393
// and 914 / 690; of equal lengths two would be better: 16 of 512, 1536: 118 / 113
// and 298 / 216), and the lengths are not known here; nor is how many are empty.
inline bool two_blocks(const DeltaDims& d) {
  return !d.packed && d.K <= 128 && d.V > 16 && d.nseq * d.hv * ((d.V + 15) / 16) > device_cus();
}

// Launches the preparation of every chunk, the forward's or the backward's.
void delta_prep(int dtype, bool back, const void* q, const void* k, const float* beta, const float* g,
                const int32_t* cu, const DeltaDims& d, const ChunkSpace& c, hipStream_t stream);

// The forward over chunks; out, last and mids may be NULL (delta_fwd.hip).
void delta_chunks(int dtype, const void* v, float scale, void* out, float* last, const float* first, float* mids,
                  const int32_t* cu, const DeltaDims& d, const ChunkSpace& c, hipStream_t stream);

}  // namespace ssm
