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

// One workgroup a chunk and value head; wave w has rows 16 w .. + 15.
template <typename TA, int KT, bool BACK>
__global__ void __launch_bounds__(256) delta_prep_kernel(const PrepArgs<TA> p) {
  constexpr int IN = ActParts<TA>::in, OUT = BACK ? 3 : ActParts<TA>::out;
  __shared__ u32x4 sk[IN][4][KT][64];
  __shared__ Mat sA, sP, sT;
  __shared__ double sG[kDeltaC];
  __shared__ float sbeta[kDeltaC];
  const int tid = static_cast<int>(threadIdx.x), w = tid >> 6, lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int64_t slot = blockIdx.x / static_cast<unsigned>(p.hv);
  const int h = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.hv)), r = p.hv / p.hk, j = h / r;
  const int64_t per = (p.L + kDeltaC - 1) / kDeltaC;
  const int64_t b = p.cu ? delta_owner(p.cu, static_cast<int>(p.nseq), slot) : slot / per;
  const DeltaSeq q = delta_seq(p.cu, b, p.L);
  const int64_t t0 = q.lo + (slot - q.slot) * kDeltaC;
  if (slot < q.slot || t0 >= q.hi) return;  // (a place that no chunk has)
  const int valid = static_cast<int>(q.hi - t0 < kDeltaC ? q.hi - t0 : kDeltaC);

  // ---- rows of K and Q: into fragments ----
  u32x4 qa[KT][IN];
  const int row = 16 * w + n;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    const TA* const src = which ? p.q + (t0 + row) * p.qs + j * p.K : p.k + (t0 + row) * p.ks + j * p.K;
#pragma unroll
    for (int kb = 0; kb < KT; ++kb) {
      const int c = 32 * kb + 8 * g;
      TA raw[8];
      if (row < valid && c + 8 <= p.K) {
        __builtin_memcpy(raw, src + c, sizeof(raw));
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          raw[e] = TA{};
          if (row < valid && c + e < p.K) raw[e] = src[c + e];
        }
      }
      u32x4 f[IN];
      if constexpr (IN == 1) {
        __builtin_memcpy(&f[0], raw, sizeof(f[0]));
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t part[IN];
          split2(to_f32(raw[2 * e]), to_f32(raw[2 * e + 1]), part);
#pragma unroll
          for (int i = 0; i < IN; ++i) f[i][e] = part[i];
        }
      }
#pragma unroll
      for (int i = 0; i < IN; ++i) {
        if (which) qa[kb][i] = f[i];
        else sk[i][w][kb][lane] = f[i];
        if (h % r == 0 && !(BACK && which))
          (which ? p.c.qf : p.c.kf)[((((slot * p.hk + j) * IN + i) * 4 + w) * KT + kb) * 64 + lane] = f[i];
      }
    }
  }
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
    float* const vec = p.c.vec + (slot * p.hv + h) * 2 * kDeltaC;
    vec[lane] = expf(static_cast<float>(G));
    vec[kDeltaC + lane] = expf(static_cast<float>(__shfl(G, 63) - G));
  }
  __syncthreads();

  // ---- K K^T and Q K^T, decayed: A and P ----
  for (int jt = 0; jt <= w; ++jt) {
    f32x4 kk = {0.0f, 0.0f, 0.0f, 0.0f}, qk = kk;
#pragma unroll
    for (int kb = 0; kb < KT; ++kb) {
      u32x4 a[IN], c[IN];
#pragma unroll
      for (int i = 0; i < IN; ++i) {
        a[i] = sk[i][w][kb][lane];
        c[i] = sk[i][jt][kb][lane];
      }
      kk = mul_parts<3>(a, c, kk);
      qk = mul_parts<3>(qa[kb], c, qk);
    }
    const int col = 16 * jt + n;
    const double Gc = sG[col];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 16 * w + 4 * g + e;
      const float D = i >= col ? expf(static_cast<float>(sG[i] - Gc)) : 0.0f;
      sA[i][col] = i > col ? sbeta[i] * D * kk[e] : 0.0f;
      sP[i][col] = i >= col ? D * qk[e] : 0.0f;
    }
  }
  if (w % 2 == 0) {  // the block right of the diagonal completes a fragment's 32 columns
#pragma unroll
    for (int e = 0; e < 4; ++e) sP[16 * w + 4 * g + e][16 * w + 16 + n] = sT[16 * w + 4 * g + e][16 * w + 16 + n] = 0.0f;
  }
  __syncthreads();

  // ---- T = (I + A)^-1: the diagonal blocks of 16 by substitution, a column a
  // lane; then [[T1, 0], [-T2 A21 T1, T2]] joins two blocks to one ----
  {
    float t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float x = i == n ? 1.0f : 0.0f;
#pragma unroll
      for (int c = 0; c < i; ++c) x = __builtin_fmaf(-sA[16 * w + i][16 * w + c], t[c], x);
      t[i] = x;
    }
    if (g == 0)
#pragma unroll
      for (int i = 0; i < 16; ++i) sT[16 * w + i][16 * w + n] = t[i];
  }
  __syncthreads();
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  // blocks (1, 0) and (3, 2); the inner product goes through A's own block
  if (w < 2) put16(sA, 2 * w + 1, 2 * w, mul16(sA, 2 * w + 1, 2 * w, sT, 2 * w, 2 * w, zero), 1.0f);
  __syncthreads();
  if (w < 2) put16(sT, 2 * w + 1, 2 * w, mul16(sT, 2 * w + 1, 2 * w + 1, sA, 2 * w + 1, 2 * w, zero), -1.0f);
  __syncthreads();
  {  // blocks (2..3, 0..1), one a wave
    const int bi = 2 + (w >> 1), bj = w & 1;
    f32x4 m = mul16(sA, bi, 1, sT, 1, bj, zero);
    if (bj == 0) m = mul16(sA, bi, 0, sT, 0, 0, m);
    __syncthreads();
    put16(sA, bi, bj, m, 1.0f);
    __syncthreads();
    m = mul16(sT, bi, 2, sA, 2, bj, zero);
    if (bi == 3) m = mul16(sT, 3, 3, sA, 3, bj, m);
    put16(sT, bi, bj, m, -1.0f);
  }
  __syncthreads();

  // ---- fragments of T diag(beta) and P, or of T^T and P^T; wave w its row block ----
  for (int kb = BACK ? w >> 1 : 0; kb <= (BACK ? 1 : w >> 1); ++kb) {
    const int c = 32 * kb + 8 * g;
    u32x4 ft[3], fp[OUT];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t part[3], op[OUT];
      const int x = c + 2 * e;
      if constexpr (BACK) {
        split2(sT[x][row], sT[x + 1][row], part);
        split2(sP[x][row], sP[x + 1][row], op);
      } else {
        split2(sT[row][x] * sbeta[x], sT[row][x + 1] * sbeta[x + 1], part);
        split2(sP[row][x], sP[row][x + 1], op);
      }
#pragma unroll
      for (int i = 0; i < 3; ++i) ft[i][e] = part[i];
#pragma unroll
      for (int i = 0; i < OUT; ++i) fp[i][e] = op[i];
    }
    const int64_t at = slot * p.hv + h;
    const int f = BACK ? tri_up(w, kb) : tri_at(w, kb);
#pragma unroll
    for (int i = 0; i < 3; ++i) p.c.tf[((at * 3 + i) * kTri + f) * 64 + lane] = ft[i];
#pragma unroll
    for (int i = 0; i < OUT; ++i) p.c.pf[((at * OUT + i) * kTri + f) * 64 + lane] = fp[i];
  }
  // ---- fragments of K^T (and Q^T) ----
  if (h % r != 0) return;
  const auto transposed = [&](u32x4* dst) {
    const uint16_t* const flat = reinterpret_cast<const uint16_t*>(&sk[0][0][0][0]);
    for (int f = w; f < IN * 2 * KT * 2; f += 4) {
      const int i = f / (4 * KT), t = f / 2 % (2 * KT), kb = f & 1;
      const int d = 16 * t + n;  // the row of the transposed matrix
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t two = 0;
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const int tok = 32 * kb + 8 * g + 2 * e + o;
          const int unit = ((i * 4 + tok / 16) * KT + d / 32) * 64 + (d % 32 / 8) * 16 + tok % 16;
          two |= static_cast<uint32_t>(flat[unit * 8 + d % 8]) << (16 * o);
        }
        v[e] = two;
      }
      dst[((((slot * p.hk + j) * IN + i) * 2 * KT + t) * 2 + kb) * 64 + lane] = v;
    }
  };
  transposed(p.c.ktf);
  if constexpr (BACK) {
    __syncthreads();
#pragma unroll
    for (int kb = 0; kb < KT; ++kb)
#pragma unroll
      for (int i = 0; i < IN; ++i) sk[i][w][kb][lane] = qa[kb][i];
    __syncthreads();
    transposed(p.c.qtf);
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
