// delta_prep.hip -- the part of the gated delta rule's chunks that does not
// depend on the state (delta.hpp says what).
#include "delta.hpp"

namespace ssm {
namespace {

constexpr int kRow = kDeltaC + 4;  // floats from row to row of a 64 x 64 matrix in LDS

typedef float Mat[kDeltaC][kRow];

// 16 x 16 block (i, j) of x as the left operand of the float32 instruction
// (row l % 16, column l / 16 of every fourth), j-th of the right one likewise
__device__ __forceinline__ f32x4 mul16(const Mat& a, int ai, int aj, const Mat& b, int bi, int bj, f32x4 c) {
  const int n = static_cast<int>(threadIdx.x & 15), g = static_cast<int>(threadIdx.x & 63) >> 4;
#pragma unroll
  for (int s = 0; s < 4; ++s)
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[16 * ai + n][16 * aj + 4 * s + g], b[16 * bi + 4 * s + g][16 * bj + n], c,
                                             0, 0, 0);
  return c;
}

__device__ __forceinline__ void put16(Mat& m, int i, int j, f32x4 c, float sign) {
  const int n = static_cast<int>(threadIdx.x & 15), g = static_cast<int>(threadIdx.x & 63) >> 4;
#pragma unroll
  for (int r = 0; r < 4; ++r) m[16 * i + 4 * g + r][16 * j + n] = sign * c[r];
}

// One workgroup a chunk and value head; wave w has the tokens 16 w .. + 15.
// Products are formed transposed (K K^T and K Q^T with the wave's tokens as
// columns): a lane then holds four neighbours of a row of A, and two results
// side by side are a fragment of P.  K^T comes out of products with the columns
// of the unit matrix, which are exact.
// Memory bounds it where chunks are many (16 heads of 128 over 131072 tokens, bf16:
// 519 us for 3.2 GB read and written, 6.2 TB/s); a round of few takes 17 us (4 x
// 2048 x 12 heads 43 us, 4.4 TB/s), the chain of the inverse's barriers.
template <typename TA, int KT, bool BACK>
__global__ void __launch_bounds__(256) delta_prep_kernel(const PrepArgs<TA> p) {
  constexpr int IN = kInParts<TA>;
  typedef u32x4 Frags[IN][4][KT][64];
  __shared__ union { Frags k; Mat t; } both;  // T takes K's place (and Q, in the backward, T's)
  __shared__ Mat sA;
  Frags& sk = both.k;
  Mat& sT = both.t;
  __shared__ double sG[kDeltaC];
  __shared__ float sbeta[kDeltaC];
  __shared__ int sbad;  // T holds a value that is not finite
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t slot = blockIdx.x / static_cast<unsigned>(p.hv);
  const int h = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.hv)), r = p.hv / p.hk, j = h / r;
  const int64_t per = (p.L + kDeltaC - 1) / kDeltaC;
  const int64_t b = p.cu ? delta_owner(p.cu, static_cast<int>(p.nseq), slot) : slot / per;
  const DeltaSeq q = delta_seq(p.cu, b, p.L);
  const int64_t t0 = q.lo + (slot - q.slot) * kDeltaC;
  if (slot < q.slot || t0 >= q.hi) return;  // (a place that no chunk has)
  const int valid = static_cast<int>(q.hi - t0 < kDeltaC ? q.hi - t0 : kDeltaC);
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  const bool first = h % r == 0;  // the key head's own fragments are written once
  const int row = 16 * w + n;

  // ---- rows of K and Q: into fragments ----
  u32x4 fk[KT][IN], fq[KT][IN];
  const auto load_rows = [&](const TA* src, u32x4 (&f)[KT][IN]) {
#pragma unroll
    for (int kb = 0; kb < KT; ++kb) {
      TA raw[8];
      const int c = 32 * kb + 8 * g;
      if (row < valid && c + 8 <= p.K) {
        __builtin_memcpy(raw, src + c, sizeof(raw));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          raw[e] = TA{};
          if (row < valid && c + e < p.K) raw[e] = src[c + e];
        }
      }
      if constexpr (IN == 1) {
        __builtin_memcpy(&f[kb][0], raw, sizeof(f[kb][0]));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t part[IN];
          split2(to_f32(raw[2 * e]), to_f32(raw[2 * e + 1]), part);
#pragma unroll
          for (int i = 0; i < IN; ++i) f[kb][i][e] = part[i];
        }
      }
    }
  };
  load_rows(p.k + (t0 + row) * p.ks + j * p.K, fk);
  load_rows(p.q + (t0 + row) * p.qs + j * p.K, fq);
  if (tid == 0) sbad = 0;
  if (w == 0) {
    const bool in = lane < valid;
    sbeta[lane] = in ? p.beta[(t0 + lane) * p.hv + h] : 0.0f;
    // The running sum in float64: its differences stand in exponents.  A decay
    // below e^-10000 is none, and minus infinity is taken so.
    const float x = in && p.g ? p.g[(t0 + lane) * p.hv + h] : 0.0f;
    double G = x < -1e4f ? -1e4 : static_cast<double>(x);
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const double up = __shfl_up(G, m);
      if (lane >= m) G += up;
    }
    sG[lane] = G;
    float* const vec = p.c.vec + (slot * p.hv + h) * (BACK ? 3 : 2) * kDeltaC;
    const float gamma = expf(static_cast<float>(G));
    vec[lane] = gamma;
    if constexpr (BACK) vec[2 * kDeltaC + lane] = -gamma * sbeta[lane];
    vec[kDeltaC + lane] = expf(static_cast<float>(__shfl(G, 63) - G)) * (BACK ? 1.0f : sbeta[lane]);
  }
#pragma unroll
  for (int kb = 0; kb < KT; ++kb)
#pragma unroll
    for (int i = 0; i < IN; ++i) {
      sk[i][w][kb][lane] = fk[kb][i];
      if (first) {
        const int64_t at = ((((slot * p.hk + j) * IN + i) * 4 + w) * KT + kb) * 64 + lane;
        p.c.kf[at] = fk[kb][i];
        if constexpr (!BACK) p.c.qf[at] = fq[kb][i];
      }
    }
  __syncthreads();

  // ---- A (into LDS) and P: beta_j D_ij k_i.k_j and beta_j D_ij q_i.k_j, lane's
  // i = row; for the backward A alone, with beta_i ----
  const double Gr = sG[row];
  const float br = sbeta[row];
  const int64_t at = slot * p.hv + h;
#pragma unroll
  for (int pair = 0; pair < 2; ++pair) {
    u32x4 fp[3];
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int jt = 2 * pair + half;
      const bool below = jt <= w;
      f32x4 kk = zero, qk = zero;
      if (below) {
#pragma unroll
        for (int kb = 0; kb < KT; ++kb) {
          u32x4 a[IN];
#pragma unroll
          for (int i = 0; i < IN; ++i) a[i] = sk[i][jt][kb][lane];
          kk = mul_parts(a, fk[kb], kk);
          if constexpr (!BACK) qk = mul_parts(a, fq[kb], qk);
        }
      }
      float4 a4 = {0.0f, 0.0f, 0.0f, 0.0f};
      if (below) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int o = 16 * jt + 4 * g + e;
          const float D = row >= o ? expf(static_cast<float>(Gr - sG[o])) : 0.0f;
          const float bo = BACK ? br : sbeta[o];
          qk[e] = row >= o ? qk[e] * (D * bo) : 0.0f;  // (a later token that is not finite stays out)
          reinterpret_cast<float*>(&a4)[e] = row > o ? bo * D * kk[e] : 0.0f;
        }
        *reinterpret_cast<float4*>(&sA[row][16 * jt + 4 * g]) = a4;
      }
      if constexpr (!BACK) {
        uint32_t lo[3], hi[3];
        split2(qk[0], qk[1], lo);
        split2(qk[2], qk[3], hi);
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          fp[i][2 * half] = lo[i];
          fp[i][2 * half + 1] = hi[i];
        }
      }
    }
    if constexpr (!BACK)
      if (pair <= w >> 1)
#pragma unroll
        for (int i = 0; i < 3; ++i) p.c.pf[((at * 3 + i) * kTri + tri_at(w, pair)) * 64 + lane] = fp[i];
  }
  // ---- fragments of K^T (later Q^T): products with the unit matrix's columns ----
  u32x4 unit;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int c = 8 * g + 2 * e - 16 * (w & 1);
    unit[e] = (c == n ? 0x3f80u : 0u) | (c + 1 == n ? 0x3f800000u : 0u);
  }
  const auto transposed = [&](u32x4* dst) {
    for (int t = w; t < 2 * KT; t += 4)
#pragma unroll
      for (int i = 0; i < IN; ++i)
#pragma unroll
        for (int kb = 0; kb < 2; ++kb) {
          u32x4 v;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const f32x4 x = mfma16(sk[i][2 * kb + half][t >> 1][lane], unit, zero);
            v[2 * half] = pack_bf16(x[0], x[1]);
            v[2 * half + 1] = pack_bf16(x[2], x[3]);
          }
          dst[((((slot * p.hk + j) * IN + i) * 2 * KT + t) * 2 + kb) * 64 + lane] = v;
        }
  };
  if (first) transposed(p.c.ktf);
  __syncthreads();
  if (w % 2 == 0)  // the block right of the diagonal completes a fragment's 32 columns
    *reinterpret_cast<float4*>(&sT[row][16 * w + 16 + 4 * g]) = float4{0.0f, 0.0f, 0.0f, 0.0f};
  __syncthreads();

  // ---- T = (I + A)^-1: the diagonal blocks of 16 by substitution, a column a
  // lane; then [[T1, 0], [-T2 A21 T1, T2]] joins two blocks to one.  The inner
  // product goes through blocks above the diagonal, which nothing reads. ----
  float size = 0.0f;
  {
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float x = i == n ? 1.0f : 0.0f;
#pragma unroll
      for (int c = 0; c < i; ++c) x = __builtin_fmaf(-sA[16 * w + i][16 * w + c], t[c], x);
      t[i] = x;
      size += __builtin_fabsf(x);
    }
    if (g == 0)
#pragma unroll
      for (int i = 0; i < 16; ++i) sT[16 * w + i][16 * w + n] = t[i];
  }
  __syncthreads();
  // blocks (1, 0) and (3, 2)
  if (w < 2) put16(sT, w, w + 2, mul16(sA, 2 * w + 1, 2 * w, sT, 2 * w, 2 * w, zero), 1.0f);
  __syncthreads();
  if (w < 2) {
    const f32x4 m = mul16(sT, 2 * w + 1, 2 * w + 1, sT, w, w + 2, zero);
    put16(sT, 2 * w + 1, 2 * w, m, -1.0f);
    size += (__builtin_fabsf(m[0]) + __builtin_fabsf(m[1])) + (__builtin_fabsf(m[2]) + __builtin_fabsf(m[3]));
  }
  __syncthreads();
  {  // blocks (2..3, 0..1), one a wave
    const int bi = 2 + (w >> 1), bj = w & 1;
    f32x4 m = mul16(sA, bi, 1, sT, 1, bj, zero);
    if (bj == 0) m = mul16(sA, bi, 0, sT, 0, 0, m);
    put16(sT, bi - 2, bj + 2, m, 1.0f);
    __syncthreads();
    m = mul16(sT, bi, 2, sT, 0, bj + 2, zero);
    if (bi == 3) m = mul16(sT, 3, 3, sT, 1, bj + 2, m);
    put16(sT, bi, bj, m, -1.0f);
    size += (__builtin_fabsf(m[0]) + __builtin_fabsf(m[1])) + (__builtin_fabsf(m[2]) + __builtin_fabsf(m[3]));
  }
  if constexpr (!BACK)
    if (!has_parts(size)) sbad = 1;
  __syncthreads();
  // A token that is not finite, or an overflow, may not reach the rows before it by
  // way of the products' zeros: then T by substitution, each column by itself from
  // its diagonal on.  (The backward's tokens depend on those behind them anyway.)
  if constexpr (!BACK)
    if (sbad) {
      if (w == 0)
        for (int i = 0; i < kDeltaC; ++i) {
          float x = i == lane ? 1.0f : 0.0f;
          for (int c = 0; c < i; ++c)
            if (c >= lane) x = __builtin_fmaf(-sA[i][c], sT[c][lane], x);
          sT[i][lane] = x;
        }
      __syncthreads();
    }

  // ---- fragments of T, or of T^T; wave w its row block ----
  for (int kb = BACK ? w >> 1 : 0; kb <= (BACK ? 1 : w >> 1); ++kb) {
    u32x4 ft[3];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t part[3];
      const int x = 32 * kb + frag_tok(g, 2 * e);
      if constexpr (BACK) split2(sT[x][row], sT[x + 1][row], part);
      else split2(sT[row][x], sT[row][x + 1], part);
#pragma unroll
      for (int i = 0; i < 3; ++i) ft[i][e] = part[i];
    }
    const int f = BACK ? tri_up(w, kb) : tri_at(w, kb);
#pragma unroll
    for (int i = 0; i < 3; ++i) p.c.tf[((at * 3 + i) * kTri + f) * 64 + lane] = ft[i];
  }
  // ---- P^T: D_ij q_i.k_j with the lane's j = row.  Q goes where K was, whose
  // fragments the wave still has ----
  if constexpr (BACK) {
    __syncthreads();
#pragma unroll
    for (int kb = 0; kb < KT; ++kb)
#pragma unroll
      for (int i = 0; i < IN; ++i) sk[i][w][kb][lane] = fq[kb][i];
    __syncthreads();
    if (first) transposed(p.c.qtf);
#pragma unroll
    for (int pair = 0; pair < 2; ++pair) {
      if (pair < w >> 1) continue;
      u32x4 fp[3];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int it = 2 * pair + half;
        f32x4 qk = zero;
        if (it >= w) {
#pragma unroll
          for (int kb = 0; kb < KT; ++kb) {
            u32x4 a[IN];
#pragma unroll
            for (int i = 0; i < IN; ++i) a[i] = sk[i][it][kb][lane];
            qk = mul_parts(a, fk[kb], qk);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int o = 16 * it + 4 * g + e;
            qk[e] *= o >= row ? expf(static_cast<float>(sG[o] - Gr)) : 0.0f;
            if (o < row) qk[e] = 0.0f;
          }
        }
        uint32_t lo[3], hi[3];
        split2(qk[0], qk[1], lo);
        split2(qk[2], qk[3], hi);
#pragma unroll
        for (int i = 0; i < 3; ++i) {
          fp[i][2 * half] = lo[i];
          fp[i][2 * half + 1] = hi[i];
        }
      }
#pragma unroll
      for (int i = 0; i < 3; ++i) p.c.pf[((at * 3 + i) * kTri + tri_up(w, pair)) * 64 + lane] = fp[i];
    }
  }
}

template <typename TA, bool BACK>
void launch(const void* q, const void* k, const float* beta, const float* g, const int32_t* cu, const DeltaDims& d,
            const ChunkSpace& c, hipStream_t stream) {
  const PrepArgs<TA> a{static_cast<const TA*>(q), static_cast<const TA*>(k), beta, g, cu, d.nseq, d.L, d.qs, d.ks,
                       d.hk, d.hv, d.K, c};
  const dim3 grid(static_cast<unsigned>(d.chunks() * d.hv)), block(256);
  switch (delta_kt(d.K)) {
    case 1: hipLaunchKernelGGL((delta_prep_kernel<TA, 1, BACK>), grid, block, 0, stream, a); break;
    case 2: hipLaunchKernelGGL((delta_prep_kernel<TA, 2, BACK>), grid, block, 0, stream, a); break;
    case 4: hipLaunchKernelGGL((delta_prep_kernel<TA, 4, BACK>), grid, block, 0, stream, a); break;
    default: hipLaunchKernelGGL((delta_prep_kernel<TA, 8, BACK>), grid, block, 0, stream, a); break;
  }
}

}  // namespace

void delta_prep(int dtype, bool back, const void* q, const void* k, const float* beta, const float* g,
                const int32_t* cu, const DeltaDims& d, const ChunkSpace& c, hipStream_t stream) {
  if (dtype == SSM_DTYPE_F32) (back ? launch<float, true> : launch<float, false>)(q, k, beta, g, cu, d, c, stream);
  else (back ? launch<bf16_t, true> : launch<bf16_t, false>)(q, k, beta, g, cu, d, c, stream);
}

}  // namespace ssm
