// conv1d_bwd.hip -- the gradients of the causal depthwise convolution (+ SiLU)
// of conv1d.hip, behind the C ABI in include/ssm_recurrent.h.
//
// With xx the input extended to the left by the conv state,
//   pre_t = bias + sum_k w_k xx_{t-(W-1)+k},  d_t = dout_t silu'(pre_t)
//   dxx_s = sum_k w_k d_{s+(W-1)-k}   (d = 0 outside the sequence)
//           (+ dfinal for the last W-1 inputs)
//   dw_k = sum_t d_t xx_{t-(W-1)+k};  dbias = sum_t d_t
#include <hip/hip_runtime.h>

#include <cstdint>

#include "ssm_recurrent.h"

#include "host_util.hpp"
#include "kernels.hpp"

namespace ssm {

template <typename TA>
struct ConvBwdArgs {
  const TA* x;
  const float *w, *bias;
  const TA *state0, *dout, *dstate1;  // state0, dstate1: (batch, dim, W-1) or NULL
  TA* dx;
  TA* dstate0;
  float* part;  // (batch * chunks, W + 1, dim)
  int64_t batch, L;
  int dim;
  uint32_t tiles, chunks, units;  // of 64 V channels, of kConvBwdChunk tokens; workgroups
};

// Workgroups of a grid's row: neither extent times the threads passes 32 bits.
constexpr uint32_t kConvGridX = 1u << 22;

// Tokens of a wave and waves of a workgroup, one stretch after the other.  The
// layer of 4 x 2048 x 1536 bf16 and 3 x 1001 x 515 float32 (3 taps): 16 x 8 20.3
// and 8.3 us, 32 x 4 21.4 and 10.1, 8 x 16 23.7 and 7.9, 16 x 16 26.8 and 9.2.
constexpr int kConvBwdT = 16;
constexpr int kConvBwdWaves = 8;
constexpr int kConvBwdChunk = kConvBwdT * kConvBwdWaves;

// V channels of one token: raw bits as loaded, widened at use (as in the
// forward: for bf16 two channels a lane, 4-byte accesses).
template <typename TA, int V>
struct ConvCell;
template <>
struct ConvCell<float, 1> {
  using raw_t = uint32_t;
  __device__ static raw_t load(rsrc_t r, uint32_t vo, uint32_t so) {
    return __builtin_amdgcn_raw_buffer_load_b32(r, vo, so, 0);
  }
  __device__ static float get(raw_t v, int) { return __uint_as_float(v); }
  __device__ static void store(rsrc_t r, const float (&v)[1], uint32_t vo, uint32_t so) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[0]), r, vo, so, kStoreStream);
  }
};
template <>
struct ConvCell<bf16_t, 1> {
  using raw_t = uint16_t;
  __device__ static raw_t load(rsrc_t r, uint32_t vo, uint32_t so) {
    return __builtin_amdgcn_raw_buffer_load_b16(r, vo, so, 0);
  }
  __device__ static float get(raw_t v, int) { return __uint_as_float(static_cast<uint32_t>(v) << 16); }
  __device__ static void store(rsrc_t r, const float (&v)[1], uint32_t vo, uint32_t so) {
    const __bf16 b = static_cast<__bf16>(v[0]);  // round to nearest even
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, b), r, vo, so, kStoreStream);
  }
};
template <>
struct ConvCell<bf16_t, 2> {
  using raw_t = uint32_t;
  __device__ static raw_t load(rsrc_t r, uint32_t vo, uint32_t so) {
    return __builtin_amdgcn_raw_buffer_load_b32(r, vo, so, 0);
  }
  __device__ static float get(raw_t v, int k) { return __uint_as_float(k ? (v & 0xffff0000u) : (v << 16)); }
  __device__ static void store(rsrc_t r, const float (&v)[2], uint32_t vo, uint32_t so) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 b = __builtin_convertvector((f32x2{v[0], v[1]}), bf16x2);
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, b), r, vo, so, kStoreStream);
  }
};
// Byte offset that no descriptor here covers (a stretch spans less than 2^30
// bytes): loads give 0, stores are dropped.
constexpr uint32_t kConvNoColumn = 0x7fffff00u;

// One pass: a wave takes kConvBwdT tokens of 64 V channels.  Going through
// them it keeps the last W inputs and the last W gradients before the SiLU in
// registers; the W - 1 tokens behind its stretch are computed once more for
// the inputs at its end, and the rows around the stretch are the neighbouring
// waves' (found in cache).  All loads are issued before the first use.  The
// sums over tokens stay in registers, are added over the workgroup's waves in
// LDS and leave one row of partials per workgroup.
// Two reads and one write of the activations bound it, with 69 vector
// instructions per token and two channels (70% of the time) next to them:
// 4 x 2048 x 1536 bf16, 4 taps, 20.3 us, 3.7 TB/s; 3 x 1001 x 515 float32 8.3 us.
template <typename TA, int V, int W, bool SILU>
__global__ void __launch_bounds__(64 * kConvBwdWaves) conv_bwd_kernel(ConvBwdArgs<TA> a) {
  constexpr int T = kConvBwdT, C = 64 * V, K = W - 1;
  using IO = ConvCell<TA, V>;
  __shared__ float s_sum[kConvBwdWaves][W + 1][C];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t unit = blockIdx.y * kConvGridX + blockIdx.x;
  if (unit >= a.units) return;
  const uint32_t tile = unit % a.tiles, rest = unit / a.tiles;
  const uint32_t chunk = rest % a.chunks, b = rest / a.chunks;
  const int dim = a.dim, col0 = static_cast<int>(tile) * C, col = col0 + lane * V;
  const bool have = col < dim;
  const int64_t L = a.L, t0 = static_cast<int64_t>(chunk) * kConvBwdChunk + w * T;
  const int n = t0 >= L ? 0 : (L - t0 < T ? static_cast<int>(L - t0) : T);  // the wave's tokens
  float dw[V][W], db[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int k = 0; k < W; ++k) dw[v][k] = 0.0f;
    db[v] = 0.0f;
  }
  // (an empty sequence's first wave moves the state's gradient through)
  if (n > 0 || (L == 0 && t0 == 0)) {
    const uint32_t rowb = static_cast<uint32_t>(dim) * sizeof(TA);
    const uint32_t voff = have ? static_cast<uint32_t>(lane * V * sizeof(TA)) : kConvNoColumn;
    // rows [t0, min(t0 + T + K, L)) of this sequence, from the wave's column on
    const int rows = L - t0 < T + K ? static_cast<int>(L - t0) : T + K;
    const int64_t base = (static_cast<int64_t>(b) * L + t0) * dim + col0;
    const uint32_t span = rows > 0 ? static_cast<uint32_t>(rows) * rowb - col0 * static_cast<uint32_t>(sizeof(TA)) : 0;
    const rsrc_t rx = make_rsrc(a.x + base, span), rd = make_rsrc(a.dout + base, span);
    const uint32_t lastrow = rows > 0 ? static_cast<uint32_t>(rows - 1) * rowb : 0;
    const auto at = [&](int j) {  // rows behind the last are that one again
      const uint32_t o = static_cast<uint32_t>(j) * rowb;
      return o < lastrow ? o : lastrow;
    };
    typename IO::raw_t xr[T + K], dr[T + K], xb[K];
    if (rows > 0) {
#pragma unroll
      for (int j = 0; j < T + K; ++j) {
        xr[j] = IO::load(rx, voff, at(j));
        dr[j] = IO::load(rd, voff, at(j));
      }
    }
    float wt[V][W], bias[V], xw[V][W], dd[V][W];  // the last W inputs and gradients, the newest last
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int k = 0; k < W; ++k) {
        wt[v][k] = have ? a.w[static_cast<size_t>(col + v) * W + k] : 0.0f;
        dd[v][k] = 0.0f;
        xw[v][k] = 0.0f;
      }
      bias[v] = have && a.bias ? a.bias[col + v] : 0.0f;
    }
    if (t0 > 0) {  // the K rows before
      const rsrc_t rb = make_rsrc(a.x + base - static_cast<int64_t>(K) * dim, K * rowb);
#pragma unroll
      for (int j = 0; j < K; ++j) xb[j] = IO::load(rb, voff, static_cast<uint32_t>(j) * rowb);
#pragma unroll
      for (int j = 0; j < K; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) xw[v][j + 1] = IO::get(xb[j], v);
    } else if (a.state0 && have) {
#pragma unroll
      for (int j = 0; j < K; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v)
          xw[v][j + 1] = to_f32(a.state0[(static_cast<int64_t>(b) * dim + col + v) * K + j]);
    }
    const rsrc_t ro = make_rsrc(a.dx + base, n > 0 ? static_cast<uint32_t>(n) * rowb - col0 * static_cast<uint32_t>(sizeof(TA)) : 0);
#pragma unroll
    for (int j = 0; j < T + K; ++j) {
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
          xw[v][k] = xw[v][k + 1];
          dd[v][k] = dd[v][k + 1];
        }
        xw[v][K] = rows > 0 ? IO::get(xr[j], v) : 0.0f;
        float d = rows > 0 ? IO::get(dr[j], v) : 0.0f;
        if (SILU) {
          float pre = bias[v];
#pragma unroll
          for (int k = 0; k < W; ++k) pre = __builtin_fmaf(wt[v][k], xw[v][k], pre);
          const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-pre * kLog2e));
          d *= s * __builtin_fmaf(pre, 1.0f - s, 1.0f);
        }
        d = j < rows ? d : 0.0f;  // tokens behind the sequence
        dd[v][K] = d;
        if (j < T && j < n) {  // (not d = 0 times what a window behind the end holds)
#pragma unroll
          for (int k = 0; k < W; ++k) dw[v][k] = __builtin_fmaf(d, xw[v][k], dw[v][k]);
          db[v] += d;
        }
        // the input K tokens back has all its gradients now
        o[v] = 0.0f;
#pragma unroll
        for (int k = 0; k < W; ++k) o[v] = __builtin_fmaf(wt[v][K - k], dd[v][k], o[v]);
      }
      const int64_t s = t0 + j - K;
      if (j < K) {  // before the stretch: the wave in front has it, or the state
        if (t0 == 0 && a.dstate0 && have) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            const int64_t st = (static_cast<int64_t>(b) * dim + col + v) * K;
            const int64_t f = s - (L - K);  // its place in the final state
            if (a.dstate1 && f >= 0) o[v] += to_f32(a.dstate1[st + f]);
            store_act(a.dstate0 + st + j, o[v]);
          }
        }
      } else if (j - K < n) {
        if (a.dstate1 && s >= L - K && have) {
#pragma unroll
          for (int v = 0; v < V; ++v)
            o[v] += to_f32(a.dstate1[(static_cast<int64_t>(b) * dim + col + v) * K + (s - (L - K))]);
        }
        IO::store(ro, o, voff, static_cast<uint32_t>(j - K) * rowb);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
#pragma unroll
    for (int k = 0; k < W; ++k) s_sum[w][k][lane * V + v] = dw[v][k];
    s_sum[w][W][lane * V + v] = db[v];
  }
  __syncthreads();
  for (int q = threadIdx.x; q < (W + 1) * C; q += 64 * kConvBwdWaves) {
    const int k = q / C, cc = q % C;
    float v = s_sum[0][k][cc];
#pragma unroll
    for (int u = 1; u < kConvBwdWaves; ++u) v += s_sum[u][k][cc];
    if (col0 + cc < dim)
      a.part[((static_cast<int64_t>(b) * a.chunks + chunk) * (W + 1) + k) * dim + col0 + cc] = v;
  }
}

// Sums of the workgroups' partials: a workgroup takes 64 channels of one tap
// (the last one the bias), wave w every kConvSumWaves-th row, and the waves'
// sums are added in order.
// 2 MB for 4 x 2048 x 1536: its launch and one round trip, 3.9 us.
constexpr int kConvSumWaves = 8;
__global__ void __launch_bounds__(64 * kConvSumWaves) conv_bwd_sum_kernel(const float* part, int64_t n, int dim,
                                                                          int W, float* dweight, float* dbias) {
  __shared__ float s_part[kConvSumWaves][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane, k = blockIdx.y;
  if (k == W && !dbias) return;
  float v = 0.0f;
  if (c < dim) {
    const float* from = part + static_cast<int64_t>(k) * dim + c;
#pragma unroll 8
    for (int64_t j = w; j < n; j += kConvSumWaves) v += from[j * (W + 1) * dim];
  }
  s_part[w][lane] = v;
  __syncthreads();
  if (w == 0 && c < dim) {
#pragma unroll
    for (int u = 1; u < kConvSumWaves; ++u) v += s_part[u][lane];
    if (k == W)
      dbias[c] = v;
    else
      dweight[static_cast<size_t>(c) * W + k] = v;
  }
}

namespace {

constexpr int64_t kConvBwdMaxDim = int64_t{1} << 22;

bool conv_bwd_sizes_ok(int64_t batch, int64_t L, int64_t dim) {
  return batch >= 1 && dim >= 1 && L >= 0 && dim <= kConvBwdMaxDim && batch <= 65535 &&
         L <= (int64_t{1} << 40) / dim &&
         batch * ((L + 15) / 16) * ((dim + 63) / 64) < (int64_t{1} << 25);
}

int64_t conv_bwd_chunks(int64_t L) { return L > 0 ? (L + kConvBwdChunk - 1) / kConvBwdChunk : 1; }

template <typename TA, int V>
int conv_bwd_launch(ConvBwdArgs<TA> a, int W, bool silu, float* dweight, float* dbias, hipStream_t s) {
  a.tiles = static_cast<uint32_t>((a.dim + 64 * V - 1) / (64 * V));
  a.chunks = static_cast<uint32_t>(conv_bwd_chunks(a.L));
  const int64_t n = a.batch * a.chunks;
  a.units = static_cast<uint32_t>(n * a.tiles);  // (65535 * 65536 at most, of empty sequences)
  const dim3 grid(a.units < kConvGridX ? a.units : kConvGridX, (a.units + (kConvGridX - 1ull)) / kConvGridX), block(64 * kConvBwdWaves);
#define SSM_CONV_BWD_CASE(WW)                                                            \
  case WW:                                                                               \
    if (silu)                                                                            \
      hipLaunchKernelGGL((conv_bwd_kernel<TA, V, WW, true>), grid, block, 0, s, a);      \
    else                                                                                 \
      hipLaunchKernelGGL((conv_bwd_kernel<TA, V, WW, false>), grid, block, 0, s, a);     \
    break;
  switch (W) {
    SSM_CONV_BWD_CASE(2)
    SSM_CONV_BWD_CASE(3)
    SSM_CONV_BWD_CASE(4)
    default: break;
  }
#undef SSM_CONV_BWD_CASE
  hipLaunchKernelGGL(conv_bwd_sum_kernel, dim3((a.dim + 63) / 64, W + 1), dim3(64 * kConvSumWaves), 0, s, a.part,
                     n, a.dim, W, dweight, dbias);
  return launch_status("ssm_causal_conv1d_bwd");
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" {

size_t ssm_causal_conv1d_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim,
                                             int64_t width) {
  if (!conv_bwd_sizes_ok(batch, seqlen, dim) || width < 2 || width > 4) return 0;
  return static_cast<size_t>(width + 1) * batch * conv_bwd_chunks(seqlen) * dim * sizeof(float);
}

int ssm_causal_conv1d_bwd(const void* x, const float* weight, const float* bias,
                          const void* initial_conv_state, const void* dout,
                          const void* dfinal_conv_state, void* dx, float* dweight, float* dbias,
                          void* dinitial_conv_state, int64_t batch, int64_t seqlen, int64_t dim,
                          int64_t width, int silu, int dtype, void* workspace,
                          size_t workspace_bytes, hipStream_t stream) {
  clear_error();
  const char* fn = "ssm_causal_conv1d_bwd";
  if (dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16)
    return fail(SSM_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, dtype);
  if (silu != 0 && silu != 1)
    return fail(SSM_ERR_UNSUPPORTED, "%s: silu must be 0 or 1, got %d", fn, silu);
  if (width < 2 || width > 4)
    return fail(SSM_ERR_UNSUPPORTED, "%s: width must be 2, 3 or 4, got %lld", fn, (long long)width);
  if (!conv_bwd_sizes_ok(batch, seqlen, dim))
    return fail(SSM_ERR_SHAPE, "%s: bad sizes batch %lld, seqlen %lld, dim %lld", fn,
                (long long)batch, (long long)seqlen, (long long)dim);
  if (!weight || !dweight || (seqlen > 0 && (!x || !dout || !dx)))
    return fail(SSM_ERR_NULL, "%s: weight, dweight, x, dout and dx are required", fn);
  const size_t es = dtype == SSM_DTYPE_F32 ? 4 : 2;
  const struct { const void* p; size_t k; const char* n; } al[] = {
      {x, es, "x"}, {dout, es, "dout"}, {dx, es, "dx"}, {weight, 4, "weight"}, {bias, 4, "bias"},
      {initial_conv_state, es, "initial_conv_state"}, {dfinal_conv_state, es, "dfinal_conv_state"},
      {dinitial_conv_state, es, "dinitial_conv_state"}, {dweight, 4, "dweight"}, {dbias, 4, "dbias"}};
  for (const auto& e : al)
    if (e.p && !aligned(e.p, e.k))
      return fail(SSM_ERR_ALIGN, "%s: %s is not %zu-byte aligned", fn, e.n, e.k);
  const size_t tok = static_cast<size_t>(batch) * seqlen * dim * es;
  const size_t st = static_cast<size_t>(batch) * dim * (width - 1) * es;
  const size_t wt = static_cast<size_t>(dim) * width * 4, pd = static_cast<size_t>(dim) * 4;
  const size_t need = ssm_causal_conv1d_bwd_workspace_bytes(batch, seqlen, dim, width);
  const Span ins[] = {{x, tok, "x"}, {dout, tok, "dout"}, {weight, wt, "weight"},
                      {bias, bias ? pd : 0, "bias"},
                      {initial_conv_state, initial_conv_state ? st : 0, "initial_conv_state"},
                      {dfinal_conv_state, dfinal_conv_state ? st : 0, "dfinal_conv_state"}};
  const Span outs[] = {{dx, tok, "dx"}, {dweight, wt, "dweight"}, {dbias, dbias ? pd : 0, "dbias"},
                       {dinitial_conv_state, dinitial_conv_state ? st : 0, "dinitial_conv_state"},
                       {workspace, workspace ? need : 0, "workspace"}};
  for (const auto& o : outs)
    for (const auto& i : ins)
      if (overlap(o, i))
        return fail(SSM_ERR_ALIAS, "%s: output %s overlaps input %s", fn, o.name, i.name);
  for (int p = 0; p < 5; ++p)
    for (int q = p + 1; q < 5; ++q)
      if (overlap(outs[p], outs[q]))
        return fail(SSM_ERR_ALIAS, "%s: %s overlaps %s", fn, outs[p].name, outs[q].name);
  if (!workspace || workspace_bytes < need)
    return fail(SSM_ERR_WORKSPACE, "%s: workspace of %zu bytes given, %zu needed", fn,
                workspace ? workspace_bytes : 0, need);
  if (!aligned(workspace, 256))
    return fail(SSM_ERR_ALIGN, "%s: workspace is not 256-byte aligned", fn);
  const auto go = [&](auto tag) {
    using TA = decltype(tag);
    ConvBwdArgs<TA> a{static_cast<const TA*>(x), weight, bias,
                      static_cast<const TA*>(initial_conv_state), static_cast<const TA*>(dout),
                      static_cast<const TA*>(dfinal_conv_state), static_cast<TA*>(dx),
                      static_cast<TA*>(dinitial_conv_state), static_cast<float*>(workspace), batch,
                      seqlen, static_cast<int>(dim), 0, 0, 0};
    if constexpr (sizeof(TA) == 2) {
      // two channels a lane where every row starts on four bytes (8 x 4096 x
      // 5120: 197 us, one channel 212; 4 x 2048 x 1536: 20.3 and 19.6)
      if (dim % 2 == 0 && aligned(x, 4) && aligned(dout, 4) && aligned(dx, 4))
        return conv_bwd_launch<TA, 2>(a, static_cast<int>(width), silu != 0, dweight, dbias, stream);
    }
    return conv_bwd_launch<TA, 1>(a, static_cast<int>(width), silu != 0, dweight, dbias, stream);
  };
  return dtype == SSM_DTYPE_F32 ? go(float{}) : go(bf16_t{});
}

}  // extern "C"
