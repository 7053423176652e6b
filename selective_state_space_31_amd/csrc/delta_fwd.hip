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
//   X = V - gamma (K S0);  E = T X;  S1 = gamma_63 S0 + K^T (d E)
//   out = scale (gamma (Q S0) + P E)
// A workgroup takes one column block of a head (columns do not meet).  Its first
// four waves carry the chain X, E, S1: wave w has the tokens 16 w .. + 15 and
// every fourth row block of S, in registers.  The other four form the outputs, 16
// tokens each, in the time that the chain leaves.  S, X, d E and E pass through LDS
// as right operands in bf16 parts, each split by one wave (16 heads over 131072
// tokens: 4.12 ms for the call, with the outputs' waves each splitting all of E
// 4.20); the left operands come from memory as fragments, each needed by one wave
// alone, the next chunk's while this one is worked on.  What bounds it is the chain through a chunk: three products, three
// splits and three barriers, one after another (heads of 128, bf16: 1.65 us a chunk
// with one column block, 131072 tokens of 16 heads 3.4 ms at 1.2 TB/s, matrix cores
// busy a fifth of the time on the compute units in use; 2.8 us with two, 4 x 2048
// x 12 heads 91 us; float32 8192 x 13 heads of 64 x 77 116 us).
template <typename TA, int KT, int NC, bool MIDS>
__global__ void __launch_bounds__(512, KT <= 4 ? 2 : 1) delta_rec_kernel(const RecArgs<TA> p) {
  constexpr int IN = kInParts<TA>, TW = (KT + 1) / 2;
  __shared__ u32x4 sS[3][KT][NC][64], sX[3][2][NC][64], sD[3][2][NC][64], sU[3][2][NC][64];  // (sU: the parts of E)
  __shared__ f32x4 sE[4][NC][64];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave & 3;
  // The workgroups of a head read the same fragments: they go to the same XCD
  // (workgroups are dealt to the eight XCDs in turn).
  const unsigned wide = 8u * static_cast<unsigned>(p.slices);
  const int64_t pair = int64_t{blockIdx.x / wide} * 8 + (blockIdx.x % wide & 7);
  if (pair >= p.nseq * p.hv) return;
  const int c0 = static_cast<int>(blockIdx.x % wide >> 3) * 16 * NC;
  const int64_t b = pair / p.hv;
  const int h = static_cast<int>(pair - b * p.hv), j = h / (p.hv / p.hk);
  const DeltaSeq q = delta_seq(p.cu, b, p.L);
  const int nc = static_cast<int>((q.hi - q.lo + kDeltaC - 1) / kDeltaC);
  const size_t sv = static_cast<size_t>(p.K) * p.V, mv = sv + static_cast<size_t>(kDeltaC) * p.V;
  // Buffer accesses outside the range read zeros and write nothing: rows behind
  // the sequence or the state, and by this offset columns behind the last one.
  constexpr uint32_t es = sizeof(TA), kNone = 0x80000000u;
  const uint32_t sbytes = static_cast<uint32_t>(sv * 4), srow = static_cast<uint32_t>(p.V) * 4;
  const auto rows_of = [&](int64_t t0) {
    return static_cast<uint32_t>(q.hi - t0 < kDeltaC ? q.hi - t0 : kDeltaC);
  };
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  const bool two = w >= 2;  // the triangles' rows w have two blocks

  // the wave's rows of K or Q as fragments
  u32x4 fr[KT][IN];
  const auto load_rows = [&](int64_t slot) {
    const u32x4* const src = (wave < 4 ? p.c.kf : p.c.qf) + ((slot * p.hk + j) * (IN * 4 * KT) + w * KT) * 64;
#pragma unroll
    for (int kb = 0; kb < KT; ++kb)
#pragma unroll
      for (int i = 0; i < IN; ++i) fr[kb][i] = (src + (i * 4 * KT + kb) * 64)[lane];
  };

  if (wave >= 4) {
    // ---- outputs ----
    const uint32_t orow = static_cast<uint32_t>(p.hv * p.V) * es;
    uint32_t oat[NC][4];
#pragma unroll
    for (int nb = 0; nb < NC; ++nb)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        oat[nb][r] = c0 + 16 * nb + n < p.V ? (16u * w + 4u * g + r) * orow + (16 * nb + n) * es : kNone;
    u32x4 fp[2][3];
    f32x4 nga;
    const auto load_p = [&](int64_t slot) {
      nga = reinterpret_cast<const f32x4*>(p.c.vec + (slot * p.hv + h) * 2 * kDeltaC)[4 * w + g];
      const u32x4* const src = p.c.pf + ((slot * p.hv + h) * (3 * kTri) + tri_at(w, 0)) * 64;
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        fp[0][i] = (src + i * kTri * 64)[lane];
        fp[1][i] = (src + (i * kTri + (two ? 1 : 0)) * 64)[lane];  // (short rows' own again: see below)
      }
    };
    if (nc > 0) {
      load_p(q.slot);
      load_rows(q.slot);
    }
    // A token whose x is not finite meets the zeros of T's rows before it in its
    // column: their e is formed again without it, and that of the rows from it on is
    // NaN, as the column's state is by the chain.  (What finds it is e itself: it
    // reaches every row behind it.)
    const auto e_without = [&](int64_t slot, int nb) {
      const u32x4* const src = p.c.tf + ((slot * p.hv + h) * (3 * kTri) + tri_at(w, 0)) * 64;
      f32x4 e = zero;
      int first = kDeltaC;
      for (int kb = 0; kb <= w >> 1; ++kb) {
        u32x4 t[3], x[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          t[i] = (src + (i * kTri + kb) * 64)[lane];
          x[i] = sX[i][kb][nb][lane];
        }
#pragma unroll
        for (int k = 7; k >= 0; --k) {
          const uint32_t half = k & 1 ? 0xffff0000u : 0xffffu, top = half & 0x7f807f80u;
          if ((x[0][k >> 1] & top) != top) continue;
          first = min(first, 32 * kb + frag_tok(g, k));
#pragma unroll
          for (int i = 0; i < 3; ++i) x[i][k >> 1] &= ~half;
        }
        e = mul_parts(t, x, e);
      }
      first = min(first, __shfl_xor(first, 16));
      first = min(first, __shfl_xor(first, 32));
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (16 * w + 4 * g + r >= first) e[r] = __builtin_nanf("");
      return e;
    };
    f32x4 y[NC];
#pragma unroll
    for (int nb = 0; nb < NC; ++nb) y[nb] = zero;
    __syncthreads();
    if (nc == 0) return;  // (the chain waits at no further barrier either)
    // (The first trip finishes no chunk: it stores nothing.  Loads and stores are the
    // same in every trip, so that a wait for the oldest waits for no others: the
    // call with 131072 tokens 3.94 ms, with branches around them 4.22.)
    for (int c = 0;; ++c) {
      const int64_t slot = q.slot + c;
      const int more = c + 1 < nc ? 1 : 0;  // (the last chunk's loads ahead are its own again)
      // the chunk before: its e came behind the last barrier but one
#pragma unroll
      for (int nb = 0; nb < NC; ++nb) {
        u32x4 e[2][3];
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int i = 0; i < 3; ++i) e[kb][i] = sU[i][kb][nb][lane];
        y[nb] = mul_parts(fp[0], e[0], y[nb]);
        if (two) y[nb] = mul_parts(fp[1], e[1], y[nb]);
      }
      if (p.out) {
        const int64_t t0 = q.lo + int64_t{c - 1} * kDeltaC;
        const rsrc_t rs = make_rsrc(p.out + (t0 * p.hv + h) * p.V + c0,
                                    c > 0 ? (rows_of(t0) - 1) * orow + static_cast<uint32_t>(p.V - c0) * es : 0);
#pragma unroll
        for (int nb = 0; nb < NC; ++nb)
#pragma unroll
          for (int r = 0; r < 4; ++r) buffer_store_act<TA>(p.scale * y[nb][r], rs, oat[nb][r]);
      }
      if (c == nc) break;
      load_p(slot);
      __syncthreads();
#pragma unroll
      for (int nb = 0; nb < NC; ++nb) {
        y[nb] = zero;
#pragma unroll
        for (int kb = 0; kb < KT; ++kb) {
          u32x4 s[3];
#pragma unroll
          for (int i = 0; i < 3; ++i) s[i] = sS[i][kb][nb][lane];
          y[nb] = mul_parts(fr[kb], s, y[nb]);
        }
        y[nb] *= nga;
      }
      load_rows(slot + more);
      if constexpr (MIDS) store_parts<KT, NC>(p.mids + (slot * p.hv + h) * mv, sbytes, srow, &sS[0][0][0][0], w, lane, c0, p.V);
      __syncthreads();
      f32x4 e[NC];
      float size = 0.0f;
#pragma unroll
      for (int nb = 0; nb < NC; ++nb) {
        e[nb] = sE[w][nb][lane];
        put_tok<3, NC>(&sU[0][0][0][0], 2, w, nb, lane, e[nb]);
#pragma unroll
        for (int r = 0; r < 4; ++r) size += __builtin_fabsf(e[nb][r]);
      }
      if (__any(!has_parts(size)))  // (or a sum of large ones: no harm)
#pragma unroll
        for (int nb = 0; nb < NC; ++nb) {
          f32x4 kept = e[nb] = e_without(slot, nb);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (!has_parts(kept[r])) {
              kept[r] = 0.0f;
              y[nb][r] = __builtin_nanf("");
            }
          put_tok<3, NC>(&sU[0][0][0][0], 2, w, nb, lane, kept);
        }
      if constexpr (MIDS) {
        const rsrc_t rs = make_rsrc(p.mids + (slot * p.hv + h) * mv + sv, kDeltaC * srow);
#pragma unroll
        for (int nb = 0; nb < NC; ++nb) {
          const uint32_t at = c0 + 16 * nb + n < p.V ? (16u * w + 4u * g) * srow + (c0 + 16 * nb + n) * 4u : kNone;
#pragma unroll
          for (int r = 0; r < 4; ++r)
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(e[nb][r]), rs, at + r * srow, 0, 0);
        }
      }
      __syncthreads();
    }
    return;
  }

  // ---- chain ----
  const bool tiles = TW > 1 || w < 2 * KT;  // (with 32 rows two waves hold none)
  const uint32_t vrow = static_cast<uint32_t>(p.vs) * es;
  uint32_t sat[NC], vat[NC][4];
#pragma unroll
  for (int nb = 0; nb < NC; ++nb) {
    const bool mine = c0 + 16 * nb + n < p.V;
    sat[nb] = mine ? (16u * w + 4u * g) * srow + (c0 + 16 * nb + n) * 4u : kNone;
#pragma unroll
    for (int r = 0; r < 4; ++r) vat[nb][r] = mine ? (16u * w + 4u * g + r) * vrow + (16 * nb + n) * es : kNone;
  }
  f32x4 S[TW][NC];
#pragma unroll
  for (int i = 0; i < TW; ++i)
#pragma unroll
    for (int nb = 0; nb < NC; ++nb) S[i][nb] = zero;
  if (p.first && tiles) {
    const rsrc_t rs = make_rsrc(p.first + pair * sv, sbytes);
#pragma unroll
    for (int i = 0; i < TW; ++i)
#pragma unroll
      for (int nb = 0; nb < NC; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          S[i][nb][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, sat[nb] + (64 * i + r) * srow, 0, 0));
  }
  const auto state_store = [&](float* dst) {
    const rsrc_t rs = make_rsrc(dst, sbytes);
#pragma unroll
    for (int i = 0; i < TW; ++i)
#pragma unroll
      for (int nb = 0; nb < NC; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[i][nb][r]), rs, sat[nb] + (64 * i + r) * srow, 0, 0);
  };
  const auto put_state = [&]() {
    if (tiles)
#pragma unroll
      for (int i = 0; i < TW; ++i)
#pragma unroll
        for (int nb = 0; nb < NC; ++nb) put_key<3, NC>(&sS[0][0][0][0], KT, w + 4 * i, nb, lane, S[i][nb]);
  };
  // K's and K^T's fragments are fetched a chunk ahead, or where both do not fit
  // the registers each behind the other's use (float32 keys beyond 128, 2 x 1024 x
  // 4 heads of 256: 78 us, with both ahead and 100 registers spilled 127; the pass
  // back 79 and 100).
  constexpr bool kTight = KT * IN > 12;
  u32x4 ft[2][3], fkt[TW][2][IN];
  f32x4 nga, nde;
  float ngC;
  typename Io<TA>::raw_t rv[NC][4];
  const auto load_v = [&](int64_t slot, int64_t t0) {
    const float* const vec = p.c.vec + (slot * p.hv + h) * 2 * kDeltaC;
    nga = reinterpret_cast<const f32x4*>(vec)[4 * w + g];
    nde = reinterpret_cast<const f32x4*>(vec + kDeltaC)[4 * w + g];
    ngC = vec[kDeltaC - 1 + (tid >> 9)];  // (by a vector load: a scalar one would be waited for at the barrier)
    const rsrc_t rs = make_rsrc(p.v + t0 * p.vs + h * p.V + c0,
                                (rows_of(t0) - 1) * vrow + static_cast<uint32_t>(p.V - c0) * es);
#pragma unroll
    for (int nb = 0; nb < NC; ++nb)
#pragma unroll
      for (int r = 0; r < 4; ++r) rv[nb][r] = Io<TA>::load(rs, vat[nb][r], 0);
  };
  const auto load_t = [&](int64_t slot) {
    const u32x4* const src = p.c.tf + ((slot * p.hv + h) * (3 * kTri) + tri_at(w, 0)) * 64;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      ft[0][i] = (src + i * kTri * 64)[lane];
      if (two) ft[1][i] = (src + (i * kTri + 1) * 64)[lane];
    }
  };
  const auto load_kt = [&](int64_t slot) {
    const u32x4* const kt = p.c.ktf + ((slot * p.hk + j) * (IN * 4 * KT) + 2 * w) * 64;
    if (tiles)
#pragma unroll
      for (int x = 0; x < TW; ++x)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int i = 0; i < IN; ++i) fkt[x][kb][i] = (kt + (i * 4 * KT + 8 * x + kb) * 64)[lane];
  };
  if (nc > 0) {
    load_rows(q.slot);
    load_v(q.slot, q.lo);
    load_t(q.slot);
    if constexpr (!kTight) load_kt(q.slot);
    put_state();
  }
  __syncthreads();
  for (int c = 0; c < nc; ++c) {
    const int64_t slot = q.slot + c, t0 = q.lo + int64_t{c} * kDeltaC;
    const int more = c + 1 < nc ? 1 : 0;
    // ---- X ----
    const f32x4 de = nde;
    f32x4 x[NC];
#pragma unroll
    for (int nb = 0; nb < NC; ++nb) {
      x[nb] = zero;
#pragma unroll
      for (int kb = 0; kb < KT; ++kb) {
        u32x4 s[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) s[i] = sS[i][kb][nb][lane];
        x[nb] = mul_parts(fr[kb], s, x[nb]);
      }
    }
#pragma unroll
    for (int i = 0; i < TW; ++i)
#pragma unroll
      for (int nb = 0; nb < NC; ++nb) S[i][nb] *= ngC;
#pragma unroll
    for (int nb = 0; nb < NC; ++nb) {
#pragma unroll
      for (int r = 0; r < 4; ++r) x[nb][r] = Io<TA>::f32(rv[nb][r]) - nga[r] * x[nb][r];
      put_tok<3, NC>(&sX[0][0][0][0], 2, w, nb, lane, x[nb]);
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (kTight) load_kt(slot);
    else load_rows(slot + more);
    __syncthreads();
    // ---- E ----
    u32x4 xp[2][NC][3];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int nb = 0; nb < NC; ++nb)
#pragma unroll
        for (int i = 0; i < 3; ++i) xp[kb][nb][i] = sX[i][kb][nb][lane];
    load_v(slot + more, t0 + more * kDeltaC);
    f32x4 u[NC];
#pragma unroll
    for (int nb = 0; nb < NC; ++nb) u[nb] = mul_parts(ft[0], xp[0][nb], zero);
    if (two)
#pragma unroll
      for (int nb = 0; nb < NC; ++nb) u[nb] = mul_parts(ft[1], xp[1][nb], u[nb]);
#pragma unroll
    for (int nb = 0; nb < NC; ++nb) {
      sE[w][nb][lane] = u[nb];
      put_tok<3, NC>(&sD[0][0][0][0], 2, w, nb, lane, u[nb] * de);
    }
    __builtin_amdgcn_sched_barrier(0);
    __syncthreads();
    // ---- S1 ----
    if (tiles) {
      u32x4 d[2][NC][3];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int nb = 0; nb < NC; ++nb)
#pragma unroll
          for (int i = 0; i < 3; ++i) d[kb][nb][i] = sD[i][kb][nb][lane];
      load_t(slot + more);
#pragma unroll
      for (int i = 0; i < TW; ++i) {
        f32x4 add[NC];  // (summed apart: the state itself is rounded once)
#pragma unroll
        for (int nb = 0; nb < NC; ++nb) add[nb] = zero;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int nb = 0; nb < NC; ++nb) add[nb] = mul_parts(fkt[i][kb], d[kb][nb], add[nb]);
#pragma unroll
        for (int nb = 0; nb < NC; ++nb) S[i][nb] += add[nb];
      }
      put_state();
    } else {
      load_t(slot + more);
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (kTight) load_rows(slot + more);
    else load_kt(slot + more);
    __syncthreads();
  }
  if (p.last && tiles) state_store(p.last + pair * sv);
}

template <typename TA, int KT, int NC>
void launch_rec(RecArgs<TA> a, hipStream_t stream) {
  const int64_t pairs = a.nseq * a.hv;
  a.slices = (a.V + 16 * NC - 1) / (16 * NC);
  const dim3 grid(static_cast<unsigned>((pairs + 7) / 8 * 8 * a.slices)), block(512);
  if (a.mids) hipLaunchKernelGGL((delta_rec_kernel<TA, KT, NC, true>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((delta_rec_kernel<TA, KT, NC, false>), grid, block, 0, stream, a);
}

template <typename TA>
void run_chunks(const void* v, float scale, void* out, float* last, const float* first, float* mids,
                const int32_t* cu, const DeltaDims& d, const ChunkSpace& c, hipStream_t stream) {
  const RecArgs<TA> a{static_cast<const TA*>(v), static_cast<TA*>(out), first, last, mids, cu, c, scale, d.nseq, d.L,
                      d.vs, d.hk, d.hv, d.K, d.V, 1};
  const bool pairs = two_blocks(d);
  switch (delta_kt(d.K)) {
    case 1: pairs ? launch_rec<TA, 1, 2>(a, stream) : launch_rec<TA, 1, 1>(a, stream); break;
    case 2: pairs ? launch_rec<TA, 2, 2>(a, stream) : launch_rec<TA, 2, 1>(a, stream); break;
    case 4: pairs ? launch_rec<TA, 4, 2>(a, stream) : launch_rec<TA, 4, 1>(a, stream); break;
    default: launch_rec<TA, 8, 1>(a, stream); break;
  }
}

// Sequences of few tokens go token by token: one launch, the state read and
// written once.  Up to 8 tokens that is quicker everywhere (16 heads of 128, bf16:
// 1 token 4.4 against 15.5 us, 8 tokens 14.1 and 15.5, 16 tokens 25 and 14), up to
// 16 where the heads fill the device (32 sequences: 46 against 52 us, 32 tokens 80
// and 53).  Of packed sequences only the sum of the lengths is known here, and one
// may have them all, at 1.9 us a token: so by the same 8, although many short ones
// would gain (16 heads of 128, bf16 and float32: 256 sequences of 1 token 109
// against 490 us in chunks and 109 against 988, of 8 tokens 327 and 506, 289 and
// 1009; but 255 of 1 and one of 500 1065 and 507).
bool few_tokens(const DeltaDims& d) {
  return d.L <= 8 || (!d.packed && d.L <= 16 && d.nseq * d.hv > device_cus());
}

size_t fwd_bytes(const DeltaDims& d, int dtype) {
  return few_tokens(d) ? 0 : chunk_space(d, dtype, false, nullptr, nullptr);
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
  if (few_tokens(d))
    return delta_walk(fn, dtype, q, k, v, beta, g, scale, out, last, first, mids, cu, d, stream);
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
