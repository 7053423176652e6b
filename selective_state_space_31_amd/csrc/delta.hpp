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
};

inline bool delta_sizes_ok(int64_t nseq, int64_t L, int64_t hk, int64_t hv, int64_t K, int64_t V, bool packed) {
  if (nseq < 1 || nseq >= (packed ? int64_t{1} << 20 : int64_t{65536}) || L < 0 || L >= (int64_t{1} << 31)) return false;
  if (hk < 1 || hv < hk || hv > 65535 || hv % hk != 0) return false;
  if (K < 1 || K > kDeltaMaxWidth || V < 1 || V > kDeltaMaxWidth) return false;
  if (!packed && nseq * L >= (int64_t{1} << 31)) return false;
  const int64_t chunks = packed ? L / kDeltaC + nseq : nseq * ((L + kDeltaC - 1) / kDeltaC);
  return (chunks > nseq ? chunks : nseq) * hv < (int64_t{1} << 26);
}

inline bool delta_strides_ok(const DeltaDims& d) {
  const int64_t most = int64_t{1} << 30;
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

}  // namespace ssm
