// delta_bwd.hip -- gradients of the gated delta rule, behind
// ssm_delta_rule_bwd and _bwd_varlen of include/ssm_layer.h.
#include "delta.hpp"

namespace ssm {
namespace {

// ---------------------------------------------------------------------------
// the states' gradients, chunk after chunk from the last one
// ---------------------------------------------------------------------------
template <typename TA>
struct BackArgs {
  const TA* dout;
  TA* dv;
  const float *dlast, *beta;
  float *dfirst, *dmid, *y;  // dmid: the gradient of the state behind every chunk; y: T^T dU of its tokens
  const int32_t* cu;
  ChunkSpace c;
  float scale;
  int64_t nseq, L;
  int hk, hv, K, V, slices;
};

// With dS1 the gradient of the state behind a chunk, per block of 16 NC columns:
//   dU = d (K dS1) + scale P^T dO;  Y = T^T dU;  dV = beta Y
//   dS0 = gamma_63 dS1 + scale Q^T (gamma dO) - K^T (gamma beta Y)
// The forward's layout: four waves carry the chain dU, Y, dS0 (wave w the tokens
// 16 w .. + 15 and every fourth row block of dS), the other four what it does not
// wait for: a chunk ahead dO's parts, scale P^T dO and scale Q^T (gamma dO), which
// the chain adds, and the stores.
//   window A (up to barrier 1)  chain: dU     others: the next dO's parts in, Q^T (gamma dO) out
//   window B (up to barrier 2)  chain: Y      others: the next P^T dO, the states' gradients
//   window C (up to barrier 3)  chain: dS0    others: the next Q^T (gamma dO), Y and dV
// The chain bounds it as in the forward (4 x 2048 x 12 heads of 128, bf16: 122 us,
// 340 MB at 2.8 TB/s; packed float32 3001 x 5 heads of 80 x 103 63 us).
template <typename TA, int KT, int NC>
__global__ void __launch_bounds__(512, 2) delta_back_kernel(const BackArgs<TA> p) {
  constexpr int IN = kInParts<TA>, TW = (KT + 1) / 2;
  __shared__ u32x4 sS[3][KT][NC][64], sU[3][2][NC][64], sZ[3][2][NC][64], sG[3][2][NC][64], sO[IN][2][NC][64];
  __shared__ f32x4 sP[4][NC][64], sY[4][NC][64], sW[2 * KT][NC][64];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave & 3;
  // (a head's workgroups on one XCD, as in the forward)
  const unsigned wide = 8u * static_cast<unsigned>(p.slices);
  const int64_t pair = int64_t{blockIdx.x / wide} * 8 + (blockIdx.x % wide & 7);
  if (pair >= p.nseq * p.hv) return;
  const int c0 = static_cast<int>(blockIdx.x % wide >> 3) * 16 * NC;
  const int64_t b = pair / p.hv;
  const int h = static_cast<int>(pair - b * p.hv), j = h / (p.hv / p.hk);
  const DeltaSeq q = delta_seq(p.cu, b, p.L);
  const int nc = static_cast<int>((q.hi - q.lo + kDeltaC - 1) / kDeltaC);
  const size_t sv = static_cast<size_t>(p.K) * p.V;
  constexpr uint32_t es = sizeof(TA), kNone = 0x80000000u;
  const uint32_t sbytes = static_cast<uint32_t>(sv * 4), srow = static_cast<uint32_t>(p.V) * 4;
  const uint32_t orow = static_cast<uint32_t>(p.hv * p.V) * es;
  const auto rows_of = [&](int64_t t0) {
    return static_cast<uint32_t>(q.hi - t0 < kDeltaC ? q.hi - t0 : kDeltaC);
  };
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  const bool tiles = TW > 1 || w < 2 * KT;  // (with 32 rows two waves hold none)
  uint32_t sat[NC];
#pragma unroll
  for (int nb = 0; nb < NC; ++nb)
    sat[nb] = c0 + 16 * nb + n < p.V ? (16u * w + 4u * g) * srow + (c0 + 16 * nb + n) * 4u : kNone;
  const int kb0 = w >> 1;  // the transposed triangles' rows w have the blocks kb0 .. 1
  const auto vec_of = [&](int64_t slot, int i) {
    return reinterpret_cast<const f32x4*>(p.c.vec + (slot * p.hv + h) * 3 * kDeltaC + i * kDeltaC)[4 * w + g];
  };
  const auto load_tri = [&](const u32x4* base, int64_t slot, u32x4 (&f)[2][3]) {
    const u32x4* const src = base + (slot * p.hv + h) * (3 * kTri) * 64;
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (kb >= kb0) f[kb][i] = (src + (i * kTri + tri_up(w, kb)) * 64)[lane];
  };
  const auto load_cols = [&](const u32x4* base, int64_t slot, u32x4 (&f)[TW][2][IN]) {
    const u32x4* const src = base + ((slot * p.hk + j) * (IN * 4 * KT) + 2 * w) * 64;
    if (tiles)
#pragma unroll
      for (int x = 0; x < TW; ++x)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int i = 0; i < IN; ++i) f[x][kb][i] = (src + (i * 4 * KT + 8 * x + kb) * 64)[lane];
  };

  if (wave >= 4) {
    u32x4 fp[2][3], fqt[TW][2][IN];
    uint32_t oat[NC][4];
#pragma unroll
    for (int nb = 0; nb < NC; ++nb)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        oat[nb][r] = c0 + 16 * nb + n < p.V ? (16u * w + 4u * g + r) * orow + (16 * nb + n) * es : kNone;
    typename Io<TA>::raw_t ro[NC][4];
    f32x4 rga, W[TW][NC];
    float be[4];
    const auto load_o = [&](int64_t slot, int64_t t0) {
      const rsrc_t rs = make_rsrc(p.dout + (t0 * p.hv + h) * p.V + c0,
                                  (rows_of(t0) - 1) * orow + static_cast<uint32_t>(p.V - c0) * es);
#pragma unroll
      for (int nb = 0; nb < NC; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r) ro[nb][r] = Io<TA>::load(rs, oat[nb][r], 0);
      rga = vec_of(slot, 0);
    };
    const auto put_o = [&]() {
#pragma unroll
      for (int nb = 0; nb < NC; ++nb) {
        f32x4 o, z;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          o[r] = Io<TA>::f32(ro[nb][r]);
          z[r] = p.scale * rga[r] * o[r];
        }
        put_tok<IN, NC>(&sO[0][0][0][0], 2, w, nb, lane, o);
        put_tok<3, NC>(&sG[0][0][0][0], 2, w, nb, lane, z);
      }
    };
    const auto form_p = [&]() {
#pragma unroll
      for (int nb = 0; nb < NC; ++nb) {
        f32x4 y = zero;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          if (kb < kb0) continue;
          u32x4 o[IN];
#pragma unroll
          for (int i = 0; i < IN; ++i) o[i] = sO[i][kb][nb][lane];
          y = mul_parts(fp[kb], o, y);
        }
        sP[w][nb][lane] = y * p.scale;
      }
    };
    const auto form_w = [&]() {
      if (!tiles) return;
#pragma unroll
      for (int nb = 0; nb < NC; ++nb) {
#pragma unroll
        for (int x = 0; x < TW; ++x) W[x][nb] = zero;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          u32x4 z[3];
#pragma unroll
          for (int i = 0; i < 3; ++i) z[i] = sG[i][kb][nb][lane];
#pragma unroll
          for (int x = 0; x < TW; ++x) W[x][nb] = mul_parts(fqt[x][kb], z, W[x][nb]);
        }
      }
    };
    const auto put_w = [&]() {
      if (tiles)
#pragma unroll
        for (int x = 0; x < TW; ++x)
#pragma unroll
          for (int nb = 0; nb < NC; ++nb) sW[w + 4 * x][nb][lane] = W[x][nb];
    };
    const auto load_b = [&](int64_t t0) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t t = t0 + 16 * w + 4 * g + r;
        be[r] = t < q.hi ? p.beta[t * p.hv + h] : 0.0f;
      }
    };
    if (nc > 0) {
      const int64_t slot = q.slot + nc - 1, t0 = q.lo + int64_t{nc - 1} * kDeltaC;
      const int less = nc > 1 ? 1 : 0;
      load_o(slot, t0);
      load_tri(p.c.pf, slot, fp);
      load_cols(p.c.qtf, slot, fqt);
      load_b(t0);
      put_o();
      load_o(slot - less, t0 - less * kDeltaC);
    }
    __syncthreads();
    if (nc > 0) {
      const int64_t slot = q.slot + nc - 1 - (nc > 1 ? 1 : 0);
      form_p();
      form_w();
      load_tri(p.c.pf, slot, fp);
      load_cols(p.c.qtf, slot, fqt);
    }
    __syncthreads();
    for (int c = nc - 1; c >= 0; --c) {
      const int64_t slot = q.slot + c, t0 = q.lo + int64_t{c} * kDeltaC;
      const int less2 = c > 1 ? 2 : c > 0 ? 1 : 0;  // (the first chunks' loads ahead are theirs again)
      // ---- window A: what the chain adds this time is in W; the next chunk's dO ----
      put_w();
      put_o();
      load_o(slot - less2, t0 - less2 * kDeltaC);
      __syncthreads();
      // ---- window B ----
      form_p();
      load_tri(p.c.pf, slot - less2, fp);
      store_parts<KT, NC>(p.dmid + (slot * p.hv + h) * sv, sbytes, srow, &sS[0][0][0][0], w, lane, c0, p.V);
      __syncthreads();
      // ---- window C ----
      {
        const rsrc_t ry = make_rsrc(p.y + (slot * p.hv + h) * kDeltaC * p.V, kDeltaC * srow);
        const rsrc_t rv = make_rsrc(p.dv + (t0 * p.hv + h) * p.V + c0,
                                    (rows_of(t0) - 1) * orow + static_cast<uint32_t>(p.V - c0) * es);
#pragma unroll
        for (int nb = 0; nb < NC; ++nb) {
          const f32x4 y = sY[w][nb][lane];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(y[r]), ry, sat[nb] + r * srow, 0, 0);
            buffer_store_act<TA>(be[r] * y[r], rv, oat[nb][r]);
          }
        }
      }
      load_b(t0 - (c > 0 ? kDeltaC : 0));
      form_w();
      load_cols(p.c.qtf, slot - less2, fqt);
      __syncthreads();
    }
    return;
  }

  // ---- chain ----
  f32x4 S[TW][NC];
#pragma unroll
  for (int i = 0; i < TW; ++i)
#pragma unroll
    for (int nb = 0; nb < NC; ++nb) S[i][nb] = zero;
  if (p.dlast && tiles) {
    const rsrc_t rs = make_rsrc(p.dlast + pair * sv, sbytes);
#pragma unroll
    for (int i = 0; i < TW; ++i)
#pragma unroll
      for (int nb = 0; nb < NC; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          S[i][nb][r] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rs, sat[nb] + (64 * i + r) * srow, 0, 0));
  }
  const auto put_state = [&]() {
    if (tiles)
#pragma unroll
      for (int i = 0; i < TW; ++i)
#pragma unroll
        for (int nb = 0; nb < NC; ++nb) put_key<3, NC>(&sS[0][0][0][0], KT, w + 4 * i, nb, lane, S[i][nb]);
  };
  constexpr bool kTight = KT * IN > 12;  // (K's and K^T's fragments: as in the forward)
  u32x4 fk[KT][IN], ft[2][3], fkt[TW][2][IN];
  f32x4 nde, nz;
  float ngC;
  const auto load_k = [&](int64_t slot) {
    const u32x4* const src = p.c.kf + ((slot * p.hk + j) * (IN * 4 * KT) + w * KT) * 64;
#pragma unroll
    for (int kb = 0; kb < KT; ++kb)
#pragma unroll
      for (int i = 0; i < IN; ++i) fk[kb][i] = (src + (i * 4 * KT + kb) * 64)[lane];
  };
  const auto load_vec = [&](int64_t slot) {
    nde = vec_of(slot, 1);
    nz = vec_of(slot, 2);
    ngC = p.c.vec[(slot * p.hv + h) * 3 * kDeltaC + kDeltaC - 1 + (tid >> 9)];  // (a vector load)
  };
  if (nc > 0) {
    const int64_t slot = q.slot + nc - 1;
    load_k(slot);
    load_vec(slot);
    load_tri(p.c.tf, slot, ft);
    if constexpr (!kTight) load_cols(p.c.ktf, slot, fkt);
    put_state();
  }
  __syncthreads();
  __syncthreads();
  for (int c = nc - 1; c >= 0; --c) {
    const int64_t slot = q.slot + c;
    const int less = c > 0 ? 1 : 0;
    // ---- dU ----
    f32x4 x[NC];
#pragma unroll
    for (int nb = 0; nb < NC; ++nb) {
      x[nb] = zero;
#pragma unroll
      for (int kb = 0; kb < KT; ++kb) {
        u32x4 s[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) s[i] = sS[i][kb][nb][lane];
        x[nb] = mul_parts(fk[kb], s, x[nb]);
      }
    }
#pragma unroll
    for (int i = 0; i < TW; ++i)
#pragma unroll
      for (int nb = 0; nb < NC; ++nb) S[i][nb] *= ngC;
#pragma unroll
    for (int nb = 0; nb < NC; ++nb)
      put_tok<3, NC>(&sU[0][0][0][0], 2, w, nb, lane, x[nb] * nde + sP[w][nb][lane]);
    const f32x4 z = nz;
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (kTight) load_cols(p.c.ktf, slot, fkt);
    else load_k(slot - less);
    __syncthreads();
    // ---- Y ----
    u32x4 u[2][NC][3];
#pragma unroll
    for (int kb = 0; kb < 2; ++kb)
#pragma unroll
      for (int nb = 0; nb < NC; ++nb)
#pragma unroll
        for (int i = 0; i < 3; ++i) u[kb][nb][i] = sU[i][kb][nb][lane];
    load_vec(slot - less);
    f32x4 y[NC];
#pragma unroll
    for (int nb = 0; nb < NC; ++nb) y[nb] = mul_parts(ft[1], u[1][nb], zero);
    if (kb0 == 0)
#pragma unroll
      for (int nb = 0; nb < NC; ++nb) y[nb] = mul_parts(ft[0], u[0][nb], y[nb]);
#pragma unroll
    for (int nb = 0; nb < NC; ++nb) {
      sY[w][nb][lane] = y[nb];
      put_tok<3, NC>(&sZ[0][0][0][0], 2, w, nb, lane, y[nb] * z);
    }
    __syncthreads();
    // ---- dS0 ----
    if (tiles) {
      u32x4 d[2][NC][3];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
#pragma unroll
        for (int nb = 0; nb < NC; ++nb)
#pragma unroll
          for (int i = 0; i < 3; ++i) d[kb][nb][i] = sZ[i][kb][nb][lane];
      load_tri(p.c.tf, slot - less, ft);
#pragma unroll
      for (int i = 0; i < TW; ++i)
#pragma unroll
        for (int nb = 0; nb < NC; ++nb) {
          f32x4 add = sW[w + 4 * i][nb][lane];  // (summed apart: the state itself is rounded once)
#pragma unroll
          for (int kb = 0; kb < 2; ++kb) add = mul_parts(fkt[i][kb], d[kb][nb], add);
          S[i][nb] += add;
        }
      put_state();
    } else {
      load_tri(p.c.tf, slot - less, ft);
    }
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (kTight) load_k(slot - less);
    else load_cols(p.c.ktf, slot - less, fkt);
    __syncthreads();
  }
  if (p.dfirst && tiles) {
    const rsrc_t rs = make_rsrc(p.dfirst + pair * sv, sbytes);
#pragma unroll
    for (int i = 0; i < TW; ++i)
#pragma unroll
      for (int nb = 0; nb < NC; ++nb)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[i][nb][r]), rs, sat[nb] + (64 * i + r) * srow, 0, 0);
  }
}

// ---------------------------------------------------------------------------
// the inputs' gradients, every chunk by itself
// ---------------------------------------------------------------------------
template <typename TA>
struct GradArgs {
  const TA* dout;
  const float *beta, *g, *mids, *dmid, *y;
  TA *dq, *dk;
  float *dbeta, *dg, *dqh, *dkh;  // dqh, dkh: of every value head, or NULL
  const int32_t* cu;
  ChunkSpace c;
  float scale;
  int64_t nseq, L;
  int hk, hv, K, V;
};

constexpr int kGradRow = kDeltaC + 4;

// A lane's x and that of the lane ROR places back in its row of 16
template <int ROR>
__device__ __forceinline__ float row_add(float x) {
  return x + __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x120 + ROR, 0xf, 0xf, false));
}

// The sum over the 16 lanes of a row, in each of them
__device__ __forceinline__ float row_sum16(float x) {
  return row_add<1>(row_add<2>(row_add<4>(row_add<8>(x))));
}

template <int N>
__device__ __forceinline__ void split8(const float (&x)[8], u32x4 (&f)[N]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t part[N];
    split2(x[2 * e], x[2 * e + 1], part);
#pragma unroll
    for (int i = 0; i < N; ++i) f[i][e] = part[i];
  }
}
// Per value head, with S0 and E from the forward, dS1 and Y from the pass back
// (G1 = dO E^T on and below the diagonal, G2 = Y E^T below it):
//   F_ij = scale beta_j D_ij G1_ij;  H_ij = -beta_i beta_j D_ij G2_ij
//   dQ = scale gamma (dO S0^T) + F K
//   dK = [H K - gamma beta (Y S0^T)] + [d beta (E dS1^T) + H^T K + F^T Q] = read + write
//   dbeta_i = y_i.e_i
//   dG_i = q_i.dq_i + k_i.(read - write)_i  (e^{G_i} goes with what reads, e^{-G_i}
//   with what writes), and <S1, dS1> for the last one; dg is their sum from behind
// One workgroup of eight waves a chunk and key head, over its value heads in turn
// (SHARED), or a chunk and value head; where several of those share a key head
// their dQ and dK go out in float32 and delta_join_kernel sums them.
// dQ and dK are cut into RT row by CT column blocks a wave; waves 0-3 have G1's and
// F's rows, waves 4-7 G2's and H's.  The row operands (dO, Y, E, then H and F) pass
// through LDS in parts; S0 and dS1 come as rows straight from memory, where each is
// the right operand as it lies.
template <int KT>
struct GradCut {
  static constexpr int RT = KT < 4 ? KT : 4, RG = 4 / RT, CG = 8 / RG, CT = 2 * KT / CG;
};

// What bounds it (4 sequences of 2048 tokens, 12 heads of 128, bf16: 182 us for 440
// MB and 280 MB of spilled registers, 3.9 TB/s): no unit by itself (vector ALU 32%,
// matrix cores 17%, LDS about 30% of the time), but the phases between barriers,
// each on another one.  Two workgroups a CU (128 registers, 59 spilled) are 4%
// faster than one without spills; float32 has too many values for two.
template <typename TA, int KT, bool SHARED>
__global__ void __launch_bounds__(512, SHARED || kInParts<TA> > 1 || KT > 4 ? 2 : 4) delta_grad_kernel(const GradArgs<TA> p) {
  constexpr int IN = kInParts<TA>, RT = GradCut<KT>::RT, CG = GradCut<KT>::CG, CT = GradCut<KT>::CT;
  typedef float Mat[kDeltaC][kGradRow];
  __shared__ u32x4 sF[12][3][64];  // dO, Y, E: 4 row blocks of 32 columns; then two triangles' 6 blocks
  __shared__ Mat sH, sP;
  __shared__ double sG[kDeltaC];
  __shared__ float sga[kDeltaC], sde[kDeltaC], sbe[kDeltaC], sdb[kDeltaC], sdot[CG][kDeltaC];
  __shared__ double sone[2][8];
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave & 3;
  const int cg = wave % CG, rg = wave / CG;
  const unsigned heads = static_cast<unsigned>(SHARED ? p.hk : p.hv);
  const int64_t slot = blockIdx.x / heads;
  const int rep = p.hv / p.hk, of = static_cast<int>(blockIdx.x % heads), j = SHARED ? of : of / rep;
  const int64_t per = (p.L + kDeltaC - 1) / kDeltaC;
  const int64_t b = p.cu ? delta_owner(p.cu, static_cast<int>(p.nseq), slot) : slot / per;
  const DeltaSeq q = delta_seq(p.cu, b, p.L);
  const int64_t t0 = q.lo + (slot - q.slot) * kDeltaC;
  if (slot < q.slot || t0 >= q.hi) return;  // (a place that no chunk has)
  const int valid = static_cast<int>(q.hi - t0 < kDeltaC ? q.hi - t0 : kDeltaC);
  const size_t sv = static_cast<size_t>(p.K) * p.V, mv = sv + static_cast<size_t>(kDeltaC) * p.V;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  const int row = 16 * w + n;

  const auto value = [&](const u32x4 (&f)[2][IN], int rt, int r) {
    float x = 0.0f;
    const int e = 4 * (rt & 1) + r;
#pragma unroll
    for (int i = IN - 1; i >= 0; --i) {
      const u32x4 v = RT == 4 ? f[rt >> 1][i] : rg * RT >= 2 ? f[1][i] : f[0][i];
      x += e & 1 ? bf_hi(v[e >> 1]) : bf_lo(v[e >> 1]);
    }
    return x;
  };

  f32x4 dq[RT][CT], dk[RT][CT];  // with several value heads: the sums over them
#pragma unroll
  for (int x = 0; x < RT; ++x)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) dq[x][ct] = dk[x][ct] = zero;

  const int h0 = SHARED ? j * rep : of;
  for (int h = h0; h < h0 + (SHARED ? rep : 1); ++h) {
    const int64_t at = slot * p.hv + h;
    bool gone = false;  // (wave 0) this token's decay is 0: no slope, where dg's sums leave the rest of what cancels
    if (wave == 0) {  // as in the preparation
      const bool in = lane < valid;
      const float x = in && p.g ? p.g[(t0 + lane) * p.hv + h] : 0.0f;
      gone = expf(x) == 0.0f;
      double G = x < -1e4f ? -1e4 : static_cast<double>(x);
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) {
        const double up = __shfl_up(G, m);
        if (lane >= m) G += up;
      }
      sG[lane] = G;
      sga[lane] = expf(static_cast<float>(G));
      sde[lane] = expf(static_cast<float>(__shfl(G, 63) - G));
      sbe[lane] = in ? p.beta[(t0 + lane) * p.hv + h] : 0.0f;
    }
    f32x4 r1[RT][CT], r2[RT][CT], r3[RT][CT], gg[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) gg[x] = zero;
#pragma unroll
    for (int x = 0; x < RT; ++x)
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) r1[x][ct] = r2[x][ct] = r3[x][ct] = zero;
    float ye = 0.0f;
    double ss = 0.0;  // (dg is what is left of larger sums: those over many terms are in float64)
    // Rows of 32 columns at a time: waves 0-3 E (and Y for y.e), waves 4-7 Y and dO.
    // Where the last block is not full, columns behind V are made zeros in the left
    // operands and in S0 (what is multiplied with them is finite: the next row's).
    const uint32_t vw = static_cast<uint32_t>(p.V) * 4;
    const rsrc_t rS = make_rsrc(p.mids + at * mv, static_cast<uint32_t>(sv * 4));
    const rsrc_t rD = make_rsrc(p.dmid + at * sv, static_cast<uint32_t>(sv * 4));
    const rsrc_t rE = make_rsrc(p.mids + at * mv + sv, kDeltaC * vw);
    const rsrc_t rY = make_rsrc(p.y + at * kDeltaC * p.V, kDeltaC * vw);
    const TA* const orow = p.dout + ((t0 + row) * p.hv + h) * p.V + 8 * g;
    const auto rows8 = [&](float (&x)[8], rsrc_t r, uint32_t off) {
      const u32x4 lo = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
      const u32x4 hi = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off + 16, 0, 0));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[e] = __uint_as_float(lo[e]);
        x[4 + e] = __uint_as_float(hi[e]);
      }
    };
    for (int vb = 0; vb < p.V; vb += 32) {
      const uint32_t c = static_cast<uint32_t>(vb + 8 * g) * 4;
      const bool full = vb + 32 <= p.V;
      float xs[CT][8], xd[CT][8];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const uint32_t d = static_cast<uint32_t>(16 * (cg + CG * ct) + n) * vw + c;
        rows8(xs[ct], rS, d);
        rows8(xd[ct], rD, d);
      }
      u32x4 fa[3], fo[IN];
      {
        float xa[8], xb[8];
        rows8(xa, wave < 4 ? rE : rY, static_cast<uint32_t>(row) * vw + c);
        if (wave < 4) {
          rows8(xb, rY, static_cast<uint32_t>(row) * vw + c);
        } else {
          TA xo[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) xo[e] = TA{};
          if (row < valid) {
            if (full) {
              __builtin_memcpy(xo, orow + vb, sizeof(xo));
            } else {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (vb + 8 * g + e < p.V) xo[e] = orow[vb + e];
            }
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) xb[e] = to_f32(xo[e]);
        }
        if (!full)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (vb + 8 * g + e >= p.V) {
              xa[e] = 0.0f;
#pragma unroll
              for (int ct = 0; ct < CT; ++ct) xs[ct][e] = 0.0f;
            }
        split8(xa, fa);
        if (wave < 4) {
#pragma unroll
          for (int e = 0; e < 8; ++e) ye = __builtin_fmaf(xa[e], xb[e], ye);
        } else {
          split8(xb, fo);
        }
      }
      __syncthreads();  // (what was in LDS has been used)
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        sF[(wave < 4 ? 8 : 4) + w][i][lane] = fa[i];
        if (i < IN && wave >= 4) sF[w][i][lane] = fo[i < IN ? i : 0];
      }
      u32x4 fs[CT][3];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        float sd = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) sd = __builtin_fmaf(xs[ct][e], xd[ct][e], sd);
        ss += sd;
        split8(xs[ct], fs[ct]);
      }
      __syncthreads();
#pragma unroll
      for (int x = 0; x < RT; ++x) {
        const int rt = rg * RT + x;
        u32x4 a[IN], y[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          if (i < IN) a[i < IN ? i : 0] = sF[rt][i][lane];
          y[i] = sF[4 + rt][i][lane];
        }
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          r1[x][ct] = mul_parts_apart(a, fs[ct], r1[x][ct]);
          r2[x][ct] = mul_parts_apart(y, fs[ct], r2[x][ct]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      u32x4 fd[CT][3];
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) split8(xd[ct], fd[ct]);
#pragma unroll
      for (int x = 0; x < RT; ++x) {
        u32x4 u[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) u[i] = sF[8 + rg * RT + x][i][lane];
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) r3[x][ct] = mul_parts_apart(u, fd[ct], r3[x][ct]);
        __builtin_amdgcn_sched_barrier(0);
      }
      u32x4 left[3];
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < IN || wave >= 4) left[i] = sF[(wave < 4 ? 0 : 4) + w][i][lane];
#pragma unroll
      for (int jt = 0; jt < 4; ++jt) {
        if (jt > w) continue;
        u32x4 u[3];
#pragma unroll
        for (int i = 0; i < 3; ++i) u[i] = sF[8 + jt][i][lane];
        if (wave < 4) {
          u32x4 fo[IN];
#pragma unroll
          for (int i = 0; i < IN; ++i) fo[i] = left[i];
          gg[jt] = mul_parts(fo, u, gg[jt]);
        } else {
          gg[jt] = mul_parts(left, u, gg[jt]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    // ---- F (waves 0-3) and H (waves 4-7) ----
    Mat& mine = wave < 4 ? sP : sH;
#pragma unroll
    for (int jt = 0; jt < 4; ++jt) {
      if (jt > w) continue;
      const int col = 16 * jt + n;
      const double Gc = sG[col];
      const float bc = sbe[col];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 16 * w + 4 * g + e;
        const float D = (wave < 4 ? i >= col : i > col) ? bc * expf(static_cast<float>(sG[i] - Gc)) : 0.0f;
        mine[i][col] = D * gg[jt][e] * (wave < 4 ? p.scale : -sbe[i]);
        if (i < col) mine[i][col] = 0.0f;
      }
    }
    if (w % 2 == 0)  // the block right of the diagonal completes a fragment's 32 columns
#pragma unroll
      for (int e = 0; e < 4; ++e) mine[16 * w + 4 * g + e][16 * w + 16 + n] = 0.0f;
    if (wave < 4) {
      ye += __shfl_xor(ye, 16);
      ye += __shfl_xor(ye, 32);
      if (g == 0) sdb[row] = ye;
    }
    __builtin_amdgcn_sched_barrier(0);
    // K^T and Q^T of the wave's columns: right operands of the triangles' products,
    // and value by value what a result's place is multiplied with in the sums
    u32x4 kt[CT][2][IN], qt[CT][2][IN];
    {
      const size_t cat = static_cast<size_t>(slot * p.hk + j) * IN * 2 * KT * 2 * 64 + lane;
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb)
#pragma unroll
          for (int i = 0; i < IN; ++i) {
            kt[ct][kb][i] = p.c.ktf[cat + ((i * 2 * KT + cg + CG * ct) * 2 + kb) * 64];
            qt[ct][kb][i] = p.c.qtf[cat + ((i * 2 * KT + cg + CG * ct) * 2 + kb) * 64];
          }
    }
    // ---- the rows' scales, and K^T d E's part of <S1, dS1> ----
    float cross = 0.0f;
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      const int rt = rg * RT + x;
      const f32x4 ga = *reinterpret_cast<const f32x4*>(&sga[16 * rt + 4 * g]);
      const f32x4 de = *reinterpret_cast<const f32x4*>(&sde[16 * rt + 4 * g]);
      const f32x4 be = *reinterpret_cast<const f32x4*>(&sbe[16 * rt + 4 * g]);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          const float kx = value(kt[ct], RT == 1 ? rt : x, r);
          r1[x][ct][r] *= p.scale * ga[r];
          r2[x][ct][r] *= -ga[r] * be[r];
          r3[x][ct][r] *= de[r] * be[r];
          cross = __builtin_fmaf(kx, r3[x][ct][r], cross);
        }
      }
    }
    // ---- the triangles as left operands: H and F, then H^T and F^T ----
#pragma unroll
    for (int turn = 0; turn < 2; ++turn) {
      __syncthreads();
      const Mat& m = wave < 4 ? sH : sP;
      for (int kb = turn ? w >> 1 : 0; kb <= (turn ? 1 : w >> 1); ++kb) {
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int c = 32 * kb + frag_tok(g, e);
          x[e] = turn ? m[c][row] : m[row][c];
        }
        u32x4 f[3];
        split8(x, f);
#pragma unroll
        for (int i = 0; i < 3; ++i) sF[(wave < 4 ? 0 : 6) + (turn ? tri_up(w, kb) : tri_at(w, kb))][i][lane] = f[i];
      }
      __syncthreads();
#pragma unroll
      for (int x = 0; x < RT; ++x) {
        const int rt = rg * RT + x;
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          if (turn ? kb < rt >> 1 : kb > rt >> 1) continue;
          const int f = turn ? tri_up(rt, kb) : tri_at(rt, kb);
          u32x4 e[3], y[3];
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            e[i] = sF[f][i][lane];
            y[i] = sF[6 + f][i][lane];
          }
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) {
            if (turn) {
              r3[x][ct] = mul_parts_apart(e, kt[ct][kb], r3[x][ct]);
              r3[x][ct] = mul_parts_apart(y, qt[ct][kb], r3[x][ct]);
            } else {
              r2[x][ct] = mul_parts_apart(e, kt[ct][kb], r2[x][ct]);
              r1[x][ct] = mul_parts_apart(y, kt[ct][kb], r1[x][ct]);
            }
          }
        }
      }
    }
    // ---- dG: sums over the rows ----
#pragma unroll
    for (int x = 0; x < RT; ++x) {
      const int rt = rg * RT + x;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float dot = 0.0f;
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          const float kx = value(kt[ct], RT == 1 ? rt : x, r), qx = value(qt[ct], RT == 1 ? rt : x, r);
          dot = __builtin_fmaf(qx, r1[x][ct][r], dot);
          dot = __builtin_fmaf(kx, r2[x][ct][r] - r3[x][ct][r], dot);
          if constexpr (SHARED) {
            dq[x][ct][r] += r1[x][ct][r];
            dk[x][ct][r] += r2[x][ct][r] + r3[x][ct][r];
          } else {
            dq[x][ct][r] = r1[x][ct][r];
            dk[x][ct][r] = r2[x][ct][r] + r3[x][ct][r];
          }
        }
        dot = row_sum16(dot);
        if (n == 0) sdot[cg][16 * rt + 4 * g + r] = dot;
      }
    }
    if (rg != 0) ss = 0.0;  // (the row groups read the same states)
    double crosses = cross;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      ss += __shfl_xor(ss, m);
      crosses += __shfl_xor(crosses, m);
    }
    if (lane == 0) {
      sone[0][wave] = ss;
      sone[1][wave] = crosses;
    }
    __syncthreads();
    if (wave == 0) {
      double last = 0.0, top = 0.0, d = 0.0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        last += sone[1][i];
        top += sone[0][i];
      }
#pragma unroll
      for (int i = 0; i < CG; ++i) d += sdot[i][lane];
      last += sga[kDeltaC - 1] * top;
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) {  // the sum from behind
        const double up = __shfl_down(d, m);
        if (lane + m < 64) d += up;
      }
      if (lane < valid) {
        p.dbeta[(t0 + lane) * p.hv + h] = sdb[lane];
        if (p.dg) p.dg[(t0 + lane) * p.hv + h] = gone ? 0.0f : static_cast<float>(d + last);
      }
    }
    __syncthreads();
  }
#pragma unroll
  for (int x = 0; x < RT; ++x)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = 16 * (rg * RT + x) + 4 * g + r;
#pragma unroll
      for (int ct = 0; ct < CT; ++ct) {
        const int d = 16 * (cg + CG * ct) + n;
        if (i < valid && d < p.K) {
          const size_t to = ((t0 + i) * heads + of) * p.K + d;
          if (!SHARED && p.dqh) {
            p.dqh[to] = dq[x][ct][r];
            p.dkh[to] = dk[x][ct][r];
          } else {
            store_act(p.dq + to, dq[x][ct][r]);
            store_act(p.dk + to, dk[x][ct][r]);
          }
        }
      }
    }
}

// dq and dk of a key head from those of its `rep` value heads, in their order; a
// wave a row (token and key head).
template <typename TA>
__global__ void __launch_bounds__(256) delta_join_kernel(const float* __restrict__ dqh, const float* __restrict__ dkh,
                                                         TA* __restrict__ dq, TA* __restrict__ dk, const int32_t* cu,
                                                         int64_t nseq, int64_t tokens, int hk, int rep, int K) {
  int64_t end = tokens;
  if (cu) {  // (rows behind the last sequence stay as they are)
    const int64_t last = cu[nseq];
    end = last < 0 ? 0 : last < tokens ? last : tokens;
  }
  const int64_t rows = end * hk;
  for (int64_t i = int64_t{blockIdx.x} * 4 + (threadIdx.x >> 6); i < rows; i += int64_t{gridDim.x} * 4)
    for (int d = static_cast<int>(threadIdx.x & 63); d < K; d += 64) {
      const size_t from = static_cast<size_t>(i) * rep * K + d;
      float a = dqh[from], b = dkh[from];
      for (int r = 1; r < rep; ++r) {
        a += dqh[from + static_cast<size_t>(r) * K];
        b += dkh[from + static_cast<size_t>(r) * K];
      }
      store_act(dq + i * K + d, a);
      store_act(dk + i * K + d, b);
    }
}

// Value heads that share a key head: a workgroup each, or one for all of them?
// Apart they need fewer rounds of the device where a round of key heads is not
// full, and a fifth more a round to write and join (calls of the backward, apart
// against together; heads of 128, bf16: 512 tokens of 8 + 16 heads 72 and 85 us,
// 1536: 115 and 115, 2560: 190 and 187, 4096: 274 and 242, of 4 + 16: 263 and 234;
// 2 x 4096 of 1 + 8 heads of 64 167 and 227; 3001 of 1 + 5 of 80 x 103, float32, 173
// and 261, 4 x 3001 287 and 303, 6 x 3001 403 and 477).
bool heads_apart(const DeltaDims& d) {
  if (d.hv == d.hk) return false;
  const int64_t cus = device_cus(), apart = (d.chunks() * d.hv + cus - 1) / cus;
  const int64_t together = (d.chunks() * d.hk + cus - 1) / cus * (d.hv / d.hk);
  return 5 * apart <= 4 * together;
}

// The gradients' own space: the backward's chunk parts, the state gradients, Y,
// and without chunk_states those and the forward's chunk parts.
struct BackSpace {
  ChunkSpace back, fwd;
  float *dmid, *y, *mids, *dqh, *dkh;
};

size_t back_space(const DeltaDims& d, int dtype, bool have, char* base, BackSpace* s) {
  BackSpace x{};
  size_t at = chunk_space(d, dtype, true, base, &x.back);
  const auto take = [&](size_t bytes) {
    char* const r = base ? base + at : nullptr;
    at += (bytes + 255) / 256 * 256;
    return reinterpret_cast<float*>(r);
  };
  x.dmid = take(static_cast<size_t>(d.chunks()) * d.state_values() * 4);
  x.y = take(static_cast<size_t>(d.chunks()) * d.hv * kDeltaC * d.V * 4);
  x.dqh = x.dkh = x.mids = nullptr;
  if (heads_apart(d)) {
    x.dqh = take(static_cast<size_t>(d.tokens()) * d.hv * d.K * 4);
    x.dkh = take(static_cast<size_t>(d.tokens()) * d.hv * d.K * 4);
  }
  if (!have) {
    x.mids = take(d.mid_values() * 4);
    at += chunk_space(d, dtype, false, base ? base + at : nullptr, &x.fwd);
  }
  if (s) *s = x;
  return at;
}

size_t bwd_bytes(const DeltaDims& d, int dtype, bool have) { return back_space(d, dtype, have, nullptr, nullptr); }

template <typename TA, int KT, int NC>
void launch_back(BackArgs<TA> a, hipStream_t stream) {
  a.slices = (a.V + 16 * NC - 1) / (16 * NC);
  const dim3 grid(static_cast<unsigned>((a.nseq * a.hv + 7) / 8 * 8 * a.slices)), block(512);
  hipLaunchKernelGGL((delta_back_kernel<TA, KT, NC>), grid, block, 0, stream, a);
}

template <typename TA, int KT>
void launch_bwd(const BackArgs<TA>& a, const GradArgs<TA>& e, const DeltaDims& d, hipStream_t stream) {
  if constexpr (KT <= 4) {
    if (two_blocks(d)) launch_back<TA, KT, 2>(a, stream);
    else launch_back<TA, KT, 1>(a, stream);
  } else {
    launch_back<TA, KT, 1>(a, stream);
  }
  if (a.L == 0) return;
  const bool together = a.hv > a.hk && !e.dqh;
  const dim3 grid(static_cast<unsigned>(d.chunks() * (together ? a.hk : a.hv))), block(512);
  if (together) hipLaunchKernelGGL((delta_grad_kernel<TA, KT, true>), grid, block, 0, stream, e);
  else hipLaunchKernelGGL((delta_grad_kernel<TA, KT, false>), grid, block, 0, stream, e);
  if (!e.dqh) return;
  const int64_t rows = d.tokens() * d.hk, most = int64_t{device_cus()} * 8;
  hipLaunchKernelGGL((delta_join_kernel<TA>), dim3(static_cast<unsigned>(rows / 4 + 1 < most ? rows / 4 + 1 : most)),
                     dim3(256), 0, stream, e.dqh, e.dkh, e.dq, e.dk, e.cu, d.nseq, d.tokens(), d.hk, d.hv / d.hk, d.K);
}

template <typename TA>
int run_bwd(const char* fn, const float* beta, const float* g, float scale, const float* mids, const void* dout, const float* dlast, void* dq, void* dk, void* dv,
            float* dbeta, float* dg, float* dfirst, const int32_t* cu, const DeltaDims& d, const BackSpace& s,
            hipStream_t stream) {
  const BackArgs<TA> a{static_cast<const TA*>(dout), static_cast<TA*>(dv), dlast, beta, dfirst, s.dmid, s.y, cu,
                       s.back, scale, d.nseq, d.L, d.hk, d.hv, d.K, d.V, 1};
  const GradArgs<TA> e{static_cast<const TA*>(dout), beta, g, mids, s.dmid, s.y, static_cast<TA*>(dq),
                       static_cast<TA*>(dk), dbeta, dg, s.dqh, s.dkh, cu, s.back, scale, d.nseq, d.L, d.hk, d.hv, d.K, d.V};
  switch (delta_kt(d.K)) {
    case 1: launch_bwd<TA, 1>(a, e, d, stream); break;
    case 2: launch_bwd<TA, 2>(a, e, d, stream); break;
    case 4: launch_bwd<TA, 4>(a, e, d, stream); break;
    default: launch_bwd<TA, 8>(a, e, d, stream); break;
  }
  return launch_status(fn);
}

int delta_bwd(const char* fn, const void* q, const void* k, const void* v, const float* beta, const float* g,
              float scale, const float* first, const float* mids, const void* dout, const float* dlast, void* dq,
              void* dk, void* dv, float* dbeta, float* dg, float* dfirst, const int32_t* cu, bool packed,
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
  if (L > 0 && (!q || !k || !v || !beta || !dout || !dq || !dk || !dv || !dbeta))
    return fail(SSM_ERR_NULL, "%s: q, k, v, beta, dout, dq, dk, dv and dbeta are required", fn);
  if (dg && !g) return fail(SSM_ERR_NULL, "%s: dg needs g", fn);
  const size_t es = dtype == SSM_DTYPE_F32 ? 4 : 2;
  const struct { const void* p; size_t k; const char* n; } al[] = {
      {q, es, "q"}, {k, es, "k"}, {v, es, "v"}, {dout, es, "dout"}, {dq, es, "dq"}, {dk, es, "dk"}, {dv, es, "dv"},
      {beta, 4, "beta"}, {g, 4, "g"}, {first, 4, "initial_state"}, {mids, 4, "chunk_states"},
      {dlast, 4, "dlast_state"}, {dbeta, 4, "dbeta"}, {dg, 4, "dg"}, {dfirst, 4, "dinitial_state"},
      {cu, 4, "cu_seqlens"}};
  for (const auto& e : al)
    if (e.p && !aligned(e.p, e.k)) return fail(SSM_ERR_ALIGN, "%s: %s is not %zu-byte aligned", fn, e.n, e.k);
  const size_t gate = static_cast<size_t>(d.tokens()) * hv * 4, st = nseq * d.state_values() * 4;
  const size_t key = static_cast<size_t>(d.tokens()) * hk * K * es, val = static_cast<size_t>(d.tokens()) * hv * V * es;
  const size_t need = bwd_bytes(d, dtype, mids != nullptr);
  const Span ins[] = {{q, strided_bytes(d.tokens(), hk * K, qs, es), "q"},
                      {k, strided_bytes(d.tokens(), hk * K, ks, es), "k"},
                      {v, strided_bytes(d.tokens(), hv * V, vs, es), "v"},
                      {beta, gate, "beta"},
                      {g, g ? gate : 0, "g"},
                      {first, first ? st : 0, "initial_state"},
                      {mids, mids ? d.mid_values() * 4 : 0, "chunk_states"},
                      {dout, val, "dout"},
                      {dlast, dlast ? st : 0, "dlast_state"},
                      {cu, packed ? static_cast<size_t>(nseq + 1) * 4 : 0, "cu_seqlens"}};
  const Span outs[] = {{dq, key, "dq"}, {dk, key, "dk"}, {dv, val, "dv"}, {dbeta, gate, "dbeta"},
                       {dg, dg ? gate : 0, "dg"}, {dfirst, dfirst ? st : 0, "dinitial_state"},
                       {ws, ws ? need : 0, "workspace"}};
  constexpr int no = sizeof(outs) / sizeof(outs[0]);
  for (const auto& o : outs)
    for (const auto& n : ins)
      if (overlap(o, n)) return fail(SSM_ERR_ALIAS, "%s: output %s overlaps input %s", fn, o.name, n.name);
  for (int a = 0; a < no; ++a)
    for (int b = a + 1; b < no; ++b)
      if (overlap(outs[a], outs[b]))
        return fail(SSM_ERR_ALIAS, "%s: %s overlaps %s", fn, outs[a].name, outs[b].name);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(SSM_ERR_WORKSPACE, "%s: workspace of %zu bytes given, %zu needed", fn, ws ? ws_bytes : 0, need);
  if (need > 0 && !aligned(ws, 256))
    return fail(SSM_ERR_ALIGN, "%s: workspace is not 256-byte aligned", fn);
  if (L == 0 && !dfirst) return SSM_OK;
  if (!packed) cu = nullptr;
  BackSpace x;
  back_space(d, dtype, mids != nullptr, static_cast<char*>(ws), &x);
  if (L > 0) {
    if (!mids) {
      delta_prep(dtype, false, q, k, beta, g, cu, d, x.fwd, stream);
      delta_chunks(dtype, v, scale, nullptr, nullptr, first, x.mids, cu, d, x.fwd, stream);
    }
    delta_prep(dtype, true, q, k, beta, g, cu, d, x.back, stream);
  }
  return (dtype == SSM_DTYPE_F32 ? run_bwd<float> : run_bwd<bf16_t>)(
      fn, beta, g, scale, mids ? mids : x.mids, dout, dlast, dq, dk, dv, dbeta, dg, dfirst, cu, d, x, stream);
}

size_t query(int64_t nseq, int64_t L, int64_t hk, int64_t hv, int64_t K, int64_t V, bool packed, int dtype, int have) {
  if ((dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16) || !delta_sizes_ok(nseq, L, hk, hv, K, V, packed)) return 0;
  return bwd_bytes(DeltaDims{nseq, L, static_cast<int>(hk), static_cast<int>(hv), static_cast<int>(K),
                             static_cast<int>(V), hk * K, hk * K, hv * V, packed},
                   dtype, have != 0);
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" {

int ssm_delta_rule_bwd(const void* q, const void* k, const void* v, const float* beta, const float* g, float scale,
                       const float* initial_state, const float* chunk_states, const void* dout,
                       const float* dlast_state, void* dq, void* dk, void* dv, float* dbeta, float* dg,
                       float* dinitial_state, int64_t batch, int64_t seqlen, int64_t nheads_k, int64_t nheads_v,
                       int64_t headdim_k, int64_t headdim_v, int64_t q_token_stride, int64_t k_token_stride,
                       int64_t v_token_stride, int dtype, void* workspace, size_t workspace_bytes,
                       hipStream_t stream) {
  return delta_bwd("ssm_delta_rule_bwd", q, k, v, beta, g, scale, initial_state, chunk_states, dout, dlast_state, dq,
                   dk, dv, dbeta, dg, dinitial_state, nullptr, false, batch, seqlen, nheads_k, nheads_v, headdim_k,
                   headdim_v, q_token_stride, k_token_stride, v_token_stride, dtype, workspace, workspace_bytes,
                   stream);
}

size_t ssm_delta_rule_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t nheads_k, int64_t nheads_v,
                                          int64_t headdim_k, int64_t headdim_v, int dtype, int with_chunk_states) {
  return query(batch, seqlen, nheads_k, nheads_v, headdim_k, headdim_v, false, dtype, with_chunk_states);
}

int ssm_delta_rule_bwd_varlen(const void* q, const void* k, const void* v, const float* beta, const float* g,
                              float scale, const float* initial_state, const float* chunk_states, const void* dout,
                              const float* dlast_state, void* dq, void* dk, void* dv, float* dbeta, float* dg,
                              float* dinitial_state, const int32_t* cu_seqlens, int64_t nseq, int64_t total_len,
                              int64_t nheads_k, int64_t nheads_v, int64_t headdim_k, int64_t headdim_v,
                              int64_t q_token_stride, int64_t k_token_stride, int64_t v_token_stride, int dtype,
                              void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return delta_bwd("ssm_delta_rule_bwd_varlen", q, k, v, beta, g, scale, initial_state, chunk_states, dout,
                   dlast_state, dq, dk, dv, dbeta, dg, dinitial_state, cu_seqlens, true, nseq, total_len, nheads_k,
                   nheads_v, headdim_k, headdim_v, q_token_stride, k_token_stride, v_token_stride, dtype, workspace,
                   workspace_bytes, stream);
}

size_t ssm_delta_rule_bwd_varlen_workspace_bytes(int64_t nseq, int64_t total_len, int64_t nheads_k, int64_t nheads_v,
                                                 int64_t headdim_k, int64_t headdim_v, int dtype,
                                                 int with_chunk_states) {
  return query(nseq, total_len, nheads_k, nheads_v, headdim_k, headdim_v, true, dtype, with_chunk_states);
}

}  // extern "C"
