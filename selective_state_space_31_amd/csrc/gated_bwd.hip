// gated_bwd.hip -- the gradients of the gated linear recurrence, behind the C
// ABI in include/ssm_recurrent.h.
//
// With g_t = dout_t silu(z_t), h_t as in the forward:
//   G_t = g_t + a_{t+1} G_{t+1}  (+ dlast at a sequence's last token)
//   dz = dout h silu'(z);  dx = G m u;  di = G m x u (1 - u)
//   dla = G (a h_{t-1} - u x a^2 / m);  dr = dla A s (1 - s)
//   dA = sum dla s;  drb = sum dr;  dib = sum di;  dh0 = a_0 G_0
// (s = sigma(r + rb), u = sigma(i + ib); the a^2 / m term only with normalize.)
#include "gated.hpp"
#include "host_util.hpp"

namespace ssm {

// Partial sums of dA, drb, dib: (rows * chunks, 3, dim), one row per chunk.

constexpr int kBwdWaves = SSM_GATED_CHUNK / kGatedT;

// The forward's layout with the adjoint running back: a workgroup takes one
// chunk of 64 tokens and reads its data once.  The states inside the chunk
// come from the one the forward left at its start, without waiting; the
// adjoint k_t = a_t G_t that enters from the chunk behind is handed over as
// the forward hands over states (maps within a group of chunks, one value per
// group), with the units given out last chunk first.
// Per token and channel six values stay in registers between the two walks
// (a, g, s and the factors of G in dx, di and dla), so a lane has one channel:
// two would need 200 registers, and one workgroup per CU.
template <typename TA, int V, bool NORM, bool GATE, bool VL>
__global__ void __launch_bounds__(64 * kBwdWaves, 3) gated_bwd_kernel(GatedBwdArgs<TA> p, GatedPlan pl) {
  constexpr int T = kGatedT, W = kBwdWaves, C = 64 * V, kPolls = kGatedGroup / W;
  using IO = Cell<TA, V>;
  __shared__ float2 s_fwd[W][C], s_rev[W][C];
  __shared__ float2 s_in[kGatedGroup][C];
  __shared__ float s_carry[C];
  __shared__ uint32_t s_turn;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int dim = p.dim;
  uint64_t* const maps = static_cast<uint64_t*>(p.ws);
  uint64_t* const carries = maps + pl.chunks * pl.cells;
  uint32_t unit = blockIdx.x;
  if (pl.chunks > 1) {
    if (threadIdx.x == 0)
      s_turn = atomicAdd(reinterpret_cast<uint32_t*>(carries + pl.groups * pl.cells), 1u);
    __syncthreads();
    unit = __builtin_amdgcn_readfirstlane(s_turn);
    if (unit >= pl.units) return;  // (a workspace that another call uses at the same time)
  }
  const uint32_t chunks = pl.chunks;
  const uint32_t c = chunks - 1 - unit / pl.lines, line = unit % pl.lines;
  const uint32_t row = line / pl.tiles, tile = line % pl.tiles;
  const int col0 = static_cast<int>(tile) * C, col = col0 + lane * V;
  const bool have = col < dim;
  const int64_t t0 = static_cast<int64_t>(c) * SSM_GATED_CHUNK + w * T;
  int64_t end = p.L;
  if (VL) {
    const int64_t e = p.cu[p.nseq];
    end = e < 0 ? 0 : (e < end ? e : end);
  }
  const int n = end <= t0 ? 0 : (end - t0 < T ? static_cast<int>(end - t0) : T);  // the wave's tokens

  // a; b, then g; the subtrahend of dla / G, then dla / G; dx / G; di / G; s
  float a[V][T], g[V][T], cl[V][T], cx[V][T], ci[V][T], sr[V][T], y[V], H[V], A[V];
  Marks mk{0, 0, 0};
  const uint32_t voff = have ? static_cast<uint32_t>(lane * V * sizeof(TA)) : kNoColumn;
  const uint32_t rowb = static_cast<uint32_t>(dim) * sizeof(TA);
  const int64_t base = (static_cast<int64_t>(row) * p.L + t0) * dim + col0;
  const uint32_t span = n > 0 ? (static_cast<uint32_t>(n) * rowb - col0 * static_cast<uint32_t>(sizeof(TA))) : 0;
  const int64_t mid = (static_cast<int64_t>(row) * chunks + c) * dim + col;
  float h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    y[v] = H[v] = 0.0f;
    A[v] = have ? p.A[col + v] : 0.0f;
    h[v] = have ? p.chunk_states[mid + v] : 0.0f;
  }
  typename IO::raw_t zr[GATE ? T : 1], dr[T];
  if (n > 0) {
    typename IO::raw_t xr[T], rr[T], ir[T];
    const rsrc_t rx = make_rsrc(p.x + base, span), rg = make_rsrc(p.r + base, span),
                 ri = make_rsrc(p.i + base, span), rd = make_rsrc(p.dout + base, span);
#pragma unroll
    for (int j = 0; j < T; ++j) {  // rows behind the last are that one again
      const uint32_t so = static_cast<uint32_t>(j < n ? j : n - 1) * rowb;
      rr[j] = IO::load(rg, voff, so);
      ir[j] = IO::load(ri, voff, so);
      xr[j] = IO::load(rx, voff, so);
    }
    if (VL) mk = find_marks(p.cu, static_cast<int>(p.nseq), t0, n);
    Params pr[V];
#pragma unroll
    for (int v = 0; v < V; ++v) pr[v] = load_params(p.A, p.rb, p.ib, col + v, have);
    // every token as if it were there (rows behind the last repeat it), y
    // over the n that are
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const float there = j < n ? 1.0f : 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float s = sigmoid2(__builtin_fmaf(IO::get(rr[j], v), -kLog2e, pr[v].rb2));
        const float u = sigmoid2(__builtin_fmaf(IO::get(ir[j], v), -kLog2e, pr[v].ib2));
        const float x = IO::get(xr[j], v), d = pr[v].A2 * s;
        const float E = decay_parts(d, a[v][j]);
        float m = 1.0f;
        cl[v][j] = 0.0f;
        if (NORM) {
          const float M = input_scale2(E);
          const float inv = M > 0.0f ? __builtin_amdgcn_rsqf(M) : 0.0f;
          m = M * inv;
          cl[v][j] = u * x * (a[v][j] * a[v][j] * inv);
        }
        sr[v][j] = s;
        cx[v][j] = m * u;
        g[v][j] = cx[v][j] * x;
        ci[v][j] = g[v][j] * (1.0f - u);
        y[v] = __builtin_fmaf(d, there, y[v]);
        H[v] = __builtin_fmaf(a[v][j], H[v], g[v][j]);
        // (the six values are formed here: moved to where they are used, their
        // sources would have to stay as well)
        asm volatile("" : "+v"(a[v][j]), "+v"(g[v][j]), "+v"(cl[v][j]), "+v"(cx[v][j]), "+v"(ci[v][j]),
                     "+v"(sr[v][j]));
      }
      if (j & 1) __builtin_amdgcn_sched_barrier(0);
    }
    if (n < T || (VL && mk.starts)) {
#pragma unroll
      for (int v = 0; v < V; ++v) H[v] = 0.0f;
#pragma unroll
      for (int j = 0; j < T; ++j) {
        const bool start = VL && (mk.starts >> j & 1);
        const int64_t s = start ? __builtin_amdgcn_readlane(mk.seq, j) : 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          if (j >= n) {
            a[v][j] = 1.0f;
            g[v][j] = 0.0f;
          }
          const float before = start ? (p.h0 && have ? p.h0[s * dim + col + v] : 0.0f) : H[v];
          H[v] = __builtin_fmaf(a[v][j], before, g[v][j]);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < T; ++j) dr[j] = IO::load(rd, voff, static_cast<uint32_t>(j < n ? j : n - 1) * rowb);
    if (GATE) {
      const rsrc_t rz = make_rsrc(p.z + base, span);
#pragma unroll
      for (int j = 0; j < T; ++j) zr[j] = IO::load(rz, voff, static_cast<uint32_t>(j < n ? j : n - 1) * rowb);
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    y[v] = keep_of(y[v]);
    s_fwd[w][lane * V + v] = make_float2(VL && mk.starts ? kCut : y[v], H[v]);
  }
  __syncthreads();
  for (int k = 0; k < w; ++k) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float2 f = s_fwd[k][lane * V + v];
      h[v] = pass<VL>(f.x, f.y, h[v]);
    }
  }
  // the states inside the wave's tokens: dz, and what multiplies G in dla
  float Q[V];
#pragma unroll
  for (int v = 0; v < V; ++v) Q[v] = 0.0f;
  if (n > 0) {
    const rsrc_t rdz = make_rsrc(p.dz + (GATE ? base : 0), GATE ? span : 0);
#pragma unroll
    for (int j = 0; j < T; ++j) {
      float dz[V];
      if (VL && (mk.starts >> j & 1)) {
        const int64_t s = __builtin_amdgcn_readlane(mk.seq, j);
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = p.h0 && have ? p.h0[s * dim + col + v] : 0.0f;
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float ah = a[v][j] * h[v];
        h[v] = __builtin_fmaf(a[v][j], h[v], g[v][j]);
        cl[v][j] = ah - cl[v][j];
        const float dout = IO::get(dr[j], v);
        if (GATE) {
          const float z = IO::get(zr[j], v), sz = sigmoid_f32(z);
          dz[v] = dout * h[v] * sz * __builtin_fmaf(z, 1.0f - sz, 1.0f);
          g[v][j] = dout * (z * sz);
        } else {
          g[v][j] = dout;
        }
      }
      if (GATE && j < n) IO::store(rdz, dz, voff, static_cast<uint32_t>(j) * rowb);
      if (j & 1) __builtin_amdgcn_sched_barrier(0);
    }
    if (n < T) {
#pragma unroll
      for (int j = 0; j < T; ++j) {
#pragma unroll
        for (int v = 0; v < V; ++v) g[v][j] = j < n ? g[v][j] : 0.0f;
      }
    }
    // the map of the wave's tokens on the adjoint that enters from behind
#pragma unroll
    for (int j = T - 1; j >= 0; --j) {
      if (VL && (mk.ends >> j & 1)) {
        const int64_t s = __builtin_amdgcn_readlane(mk.seq, j);
#pragma unroll
        for (int v = 0; v < V; ++v) Q[v] = p.dlast && have ? p.dlast[s * dim + col + v] : 0.0f;
      }
      if (VL && (mk.starts >> j & 1)) {
#pragma unroll
        for (int v = 0; v < V; ++v) Q[v] = 0.0f;
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v) Q[v] = a[v][j] * (g[v][j] + Q[v]);
      }
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (VL && (mk.starts | mk.ends)) y[v] = kCut;
    s_rev[w][lane * V + v] = make_float2(y[v], Q[v]);
  }
  __syncthreads();
  float yw[V], Qw[V], yt[V], Qt[V], k[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    yw[v] = -0.0f;
    Qw[v] = 0.0f;
  }
  for (int q = W - 1; q > w; --q) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float2 f = s_rev[q][lane * V + v];
      compose<VL>(yw[v], Qw[v], f.x, f.y);
    }
  }
  const int64_t cell = static_cast<int64_t>(line) * C + lane * V;
  if (w == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      yt[v] = yw[v];
      Qt[v] = Qw[v];
      compose<VL>(yt[v], Qt[v], y[v], Q[v]);
      if (c > 0) publish(maps + c * pl.cells + cell + v, yt[v], Qt[v]);
    }
  }
  // the adjoint that enters the chunk from behind
  const uint32_t first = c / kGatedGroup * kGatedGroup;
  const uint32_t lastc = first + kGatedGroup < chunks ? first + kGatedGroup - 1 : chunks - 1;
  const int there = static_cast<int>(lastc - c);  // chunks of the group behind this one
  {
    float lo[kPolls][V], hi[kPolls][V];
    const int polls = there > w ? (there - w + W - 1) / W : 0;  // chunks c + 1 + w, c + 1 + w + W, ...
    if (polls > 0)
      await<V>(maps + (c + 1 + w) * pl.cells + cell, W * pl.cells, polls, lo, hi);
#pragma unroll
    for (int k2 = 0; k2 < kPolls; ++k2) {
      if (k2 < polls) {
#pragma unroll
        for (int v = 0; v < V; ++v) s_in[w + k2 * W][lane * V + v] = make_float2(lo[k2][v], hi[k2][v]);
      }
    }
  }
  if (w == W - 1) {
    float lo[1][V], hi[1][V];
    if (lastc + 1 < chunks) {
      await<V>(carries + (c / kGatedGroup + 1) * pl.cells + cell, 0, 1, lo, hi);
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v)
        hi[0][v] = !VL && p.dlast && have ? p.dlast[static_cast<int64_t>(row) * dim + col + v] : 0.0f;
    }
#pragma unroll
    for (int v = 0; v < V; ++v) s_carry[lane * V + v] = hi[0][v];
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) k[v] = s_carry[lane * V + v];
  for (int j = there - 1; j >= 0; --j) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float2 f = s_in[j][lane * V + v];
      k[v] = pass<VL>(f.x, f.y, k[v]);
    }
  }
  if (w == 0 && c == first && c > 0) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      publish(carries + c / kGatedGroup * pl.cells + cell + v, 0.0f, pass<VL>(yt[v], Qt[v], k[v]));
  }
#pragma unroll
  for (int v = 0; v < V; ++v) k[v] = pass<VL>(yw[v], Qw[v], k[v]);
  float dA[V], drb[V], dib[V];
#pragma unroll
  for (int v = 0; v < V; ++v) dA[v] = drb[v] = dib[v] = 0.0f;
  if (n > 0) {
    const rsrc_t rdx = make_rsrc(p.dx + base, span), rdr = make_rsrc(p.dr + base, span),
                 rdi = make_rsrc(p.di + base, span);
#pragma unroll
    for (int j = T - 1; j >= 0; --j) {
      if (j < n) {
        if (VL && (mk.ends >> j & 1)) {
          const int64_t s = __builtin_amdgcn_readlane(mk.seq, j);
#pragma unroll
          for (int v = 0; v < V; ++v) k[v] = p.dlast && have ? p.dlast[s * dim + col + v] : 0.0f;
        }
        float ox[V], orr[V], oi[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float G = g[v][j] + k[v], dla = G * cl[v][j], s = sr[v][j];
          ox[v] = G * cx[v][j];
          oi[v] = G * ci[v][j];
          orr[v] = dla * (A[v] * s * (1.0f - s));
          dA[v] = __builtin_fmaf(dla, s, dA[v]);
          drb[v] += orr[v];
          dib[v] += oi[v];
          k[v] = a[v][j] * G;
        }
        const uint32_t so = static_cast<uint32_t>(j) * rowb;
        IO::store(rdx, ox, voff, so);
        IO::store(rdr, orr, voff, so);
        IO::store(rdi, oi, voff, so);
        if (VL && (mk.starts >> j & 1)) {
          const int64_t s = __builtin_amdgcn_readlane(mk.seq, j);
#pragma unroll
          for (int v = 0; v < V; ++v) {
            if (p.dh0 && have) p.dh0[s * dim + col + v] = k[v];
            k[v] = 0.0f;
          }
        }
      }
    }
  }
  if (!VL && p.dh0 && c == 0 && w == 0 && have) {
#pragma unroll
    for (int v = 0; v < V; ++v) p.dh0[static_cast<int64_t>(row) * dim + col + v] = k[v];
  }
  // the chunk's sums: over the waves, last tokens first
  __syncthreads();
  float* const s_sum = reinterpret_cast<float*>(&s_in[0][0]);  // (W, 3, C)
  static_assert(sizeof(s_in) >= sizeof(float) * W * 3 * C, "the sums fit where the maps were");
#pragma unroll
  for (int v = 0; v < V; ++v) {
    s_sum[(w * 3 + 0) * C + lane * V + v] = dA[v];
    s_sum[(w * 3 + 1) * C + lane * V + v] = drb[v];
    s_sum[(w * 3 + 2) * C + lane * V + v] = dib[v];
  }
  __syncthreads();
  for (int q = threadIdx.x; q < 3 * C; q += 64 * W) {
    float v = 0.0f;
#pragma unroll
    for (int k2 = W - 1; k2 >= 0; --k2) v += s_sum[k2 * 3 * C + q];
    const int what = q / C, cc = col0 + q % C;
    if (cc < dim)
      p.part[((static_cast<int64_t>(row) * chunks + c) * 3 + what) * dim + cc] = v;
  }
}

// Sums of the chunks' partials: a workgroup takes 64 channels of one of the
// three, wave w every kSumWaves-th chunk, and the waves' sums are added in
// order.
constexpr int kSumWaves = 8;
__global__ void __launch_bounds__(64 * kSumWaves) gated_sum_kernel(const float* part, int64_t n, int dim,
                                                                   float* dA, float* drb, float* dib) {
  __shared__ float s_part[kSumWaves][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + lane, what = blockIdx.y;
  float* to = what == 0 ? dA : what == 1 ? drb : dib;
  if (!to) return;
  float v = 0.0f;
  if (c < dim) {
    const float* from = part + static_cast<int64_t>(what) * dim + c;
#pragma unroll 8
    for (int64_t k = w; k < n; k += kSumWaves) v += from[k * 3 * dim];
  }
  s_part[w][lane] = v;
  __syncthreads();
  if (w == 0 && c < dim) {
#pragma unroll
    for (int k = 1; k < kSumWaves; ++k) v += s_part[k][lane];
    to[c] = v;
  }
}

template <typename TA, int V>
int launch_gated_bwd(const GatedBwdArgs<TA>& a, const GatedPlan& pl, bool norm, const char* fn,
                     hipStream_t s) {
  int rc = launch_gated_init(a.ws, pl.bytes, a.cu, a.cu ? a.nseq : a.rows, a.L, a.dim, a.dlast, a.dh0, fn, s);
  if (rc != SSM_OK) return rc;
  if (a.L > 0) {
    const dim3 grid(static_cast<unsigned>(pl.units)), block(64 * kBwdWaves);
#define SSM_GATED_CASE(N, G, VLN)                                                              \
  if (norm == N && (a.z != nullptr) == G && (a.cu != nullptr) == VLN)                          \
    hipLaunchKernelGGL((gated_bwd_kernel<TA, V, N, G, VLN>), grid, block, 0, s, a, pl);
    SSM_GATED_CASE(true, true, false)
    SSM_GATED_CASE(true, false, false)
    SSM_GATED_CASE(false, true, false)
    SSM_GATED_CASE(false, false, false)
    SSM_GATED_CASE(true, true, true)
    SSM_GATED_CASE(true, false, true)
    SSM_GATED_CASE(false, true, true)
    SSM_GATED_CASE(false, false, true)
#undef SSM_GATED_CASE
  }
  const int64_t n = a.L > 0 ? a.rows * pl.chunks : 0;
  hipLaunchKernelGGL(gated_sum_kernel, dim3((a.dim + 63) / 64, 3), dim3(64 * kSumWaves), 0, s, a.part, n,
                     a.dim, a.dA, a.drb, a.dib);
  return launch_status(fn);
}

namespace {

// The walk's words, the chunk states if the caller has none, the partial
// sums; each part starts on 256 bytes.
struct BwdSpace {
  size_t states, part, bytes;  // offsets, total
};
BwdSpace bwd_space(int64_t rows, int64_t L, int64_t dim, bool have_states) {
  const auto up = [](size_t v) { return (v + 255) & ~size_t{255}; };
  const size_t chunks = static_cast<size_t>(rows) * ((L + SSM_GATED_CHUNK - 1) / SSM_GATED_CHUNK);
  BwdSpace b;
  b.states = up(gated_walk_bytes(rows, L, dim));
  b.part = b.states + (have_states ? 0 : up(chunks * dim * 4));
  b.bytes = b.part + up(chunks * 3 * dim * 4);
  return b;
}

size_t bwd_ws_bytes(int64_t rows, int64_t L, int64_t nseq, int64_t dim, int dtype, bool packed,
                    bool have_states) {
  if ((dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16) ||
      !gated_sizes_ok(rows, L, nseq, dim, packed))
    return 0;
  return bwd_space(rows, L, dim, have_states).bytes;
}

int gated_bwd(const char* fn, const void* x, const void* r, const void* i, const float* A,
              const float* rb, const float* ib, int normalize, const void* z, const float* h0,
              const float* chunk_states, const void* dout, const float* dlast, void* dx, void* dr,
              void* di, void* dz, float* dA, float* drb, float* dib, float* dh0, const int32_t* cu,
              int64_t nseq, int64_t rows, int64_t L, int64_t dim, int dtype, bool packed, void* ws,
              size_t ws_bytes, hipStream_t stream) {
  clear_error();
  if (dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16)
    return fail(SSM_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, dtype);
  if (normalize != 0 && normalize != 1)
    return fail(SSM_ERR_UNSUPPORTED, "%s: normalize must be 0 or 1, got %d", fn, normalize);
  if (!gated_sizes_ok(rows, L, nseq, dim, packed))
    return fail(SSM_ERR_SHAPE, "%s: bad sizes: %lld sequence(s), %lld tokens, dim %lld", fn,
                (long long)(packed ? nseq : rows), (long long)L, (long long)dim);
  if (!A || !dA || (packed && !cu))
    return fail(SSM_ERR_NULL, "%s: A, dA%s are required", fn, packed ? " and cu_seqlens" : "");
  if (L > 0 && (!x || !r || !i || !dout || !dx || !dr || !di))
    return fail(SSM_ERR_NULL, "%s: x, rgate, igate, dout, dx, drgate and digate are required", fn);
  if (L > 0 && z && !dz) return fail(SSM_ERR_NULL, "%s: dz is required with z", fn);
  if (!z && dz) return fail(SSM_ERR_NULL, "%s: dz given without z", fn);
  const size_t es = dtype == SSM_DTYPE_F32 ? 4 : 2;
  const struct { const void* p; size_t k; const char* n; } al[] = {
      {x, es, "x"}, {r, es, "rgate"}, {i, es, "igate"}, {z, es, "z"}, {dout, es, "dout"},
      {dx, es, "dx"}, {dr, es, "drgate"}, {di, es, "digate"}, {dz, es, "dz"}, {A, 4, "A"},
      {rb, 4, "rgate_bias"}, {ib, 4, "igate_bias"}, {h0, 4, "initial_state"},
      {chunk_states, 4, "chunk_states"}, {dlast, 4, "dlast_state"}, {dA, 4, "dA"},
      {drb, 4, "drgate_bias"}, {dib, 4, "digate_bias"}, {dh0, 4, "dinitial_state"},
      {cu, 4, "cu_seqlens"}};
  for (const auto& e : al)
    if (e.p && !aligned(e.p, e.k))
      return fail(SSM_ERR_ALIGN, "%s: %s is not %zu-byte aligned", fn, e.n, e.k);
  const size_t tok = static_cast<size_t>(rows) * L * dim * es;
  const size_t st = static_cast<size_t>(packed ? nseq : rows) * dim * 4;
  const size_t cst =
      static_cast<size_t>(rows) * ((L + SSM_GATED_CHUNK - 1) / SSM_GATED_CHUNK) * dim * 4;
  const size_t pd = static_cast<size_t>(dim) * 4;
  const BwdSpace sp = bwd_space(rows, L, dim, chunk_states != nullptr);
  const size_t need = sp.bytes;
  const Span ins[] = {{x, tok, "x"}, {r, tok, "rgate"}, {i, tok, "igate"}, {z, z ? tok : 0, "z"},
                      {dout, tok, "dout"}, {A, pd, "A"}, {rb, rb ? pd : 0, "rgate_bias"},
                      {ib, ib ? pd : 0, "igate_bias"}, {h0, h0 ? st : 0, "initial_state"},
                      {chunk_states, chunk_states ? cst : 0, "chunk_states"},
                      {dlast, dlast ? st : 0, "dlast_state"},
                      {cu, packed ? static_cast<size_t>(nseq + 1) * 4 : 0, "cu_seqlens"}};
  const Span outs[] = {{dx, tok, "dx"}, {dr, tok, "drgate"}, {di, tok, "digate"},
                       {dz, dz ? tok : 0, "dz"}, {dA, pd, "dA"}, {drb, drb ? pd : 0, "drgate_bias"},
                       {dib, dib ? pd : 0, "digate_bias"}, {dh0, dh0 ? st : 0, "dinitial_state"},
                       {ws, ws ? need : 0, "workspace"}};
  constexpr int kOuts = sizeof(outs) / sizeof(outs[0]);
  for (const auto& o : outs)
    for (const auto& n : ins)
      if (overlap(o, n))
        return fail(SSM_ERR_ALIAS, "%s: output %s overlaps input %s", fn, o.name, n.name);
  for (int a = 0; a < kOuts; ++a)
    for (int b = a + 1; b < kOuts; ++b)
      if (overlap(outs[a], outs[b]))
        return fail(SSM_ERR_ALIAS, "%s: %s overlaps %s", fn, outs[a].name, outs[b].name);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(SSM_ERR_WORKSPACE, "%s: workspace of %zu bytes given, %zu needed", fn,
                ws ? ws_bytes : 0, need);
  if (need > 0 && !aligned(ws, 256))
    return fail(SSM_ERR_ALIGN, "%s: workspace is not 256-byte aligned", fn);
  char* const at = static_cast<char*>(ws);
  if (!chunk_states && L > 0) {
    float* const mid = reinterpret_cast<float*>(at + sp.states);
    const int rc = gated_states(fn, x, r, i, A, rb, ib, normalize, h0, mid, packed ? cu : nullptr, nseq,
                                rows, L, static_cast<int>(dim), dtype, ws, stream);
    if (rc != SSM_OK) return rc;
    chunk_states = mid;
  }
  const auto go = [&](auto tag) {
    using TA = decltype(tag);
    GatedBwdArgs<TA> a{static_cast<const TA*>(x), static_cast<const TA*>(r),
                       static_cast<const TA*>(i), static_cast<const TA*>(z),
                       static_cast<const TA*>(dout), A, rb, ib, h0, chunk_states, dlast,
                       static_cast<TA*>(dx), static_cast<TA*>(dr), static_cast<TA*>(di),
                       static_cast<TA*>(dz), dA, drb, dib, dh0, packed ? cu : nullptr, rows, L, nseq,
                       static_cast<int>(dim), ws, reinterpret_cast<float*>(at + sp.part)};
    return launch_gated_bwd<TA, 1>(a, gated_plan(rows, L, dim, 1, SSM_GATED_CHUNK), normalize != 0, fn, stream);
  };
  return dtype == SSM_DTYPE_F32 ? go(float{}) : go(bf16_t{});
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" {

int ssm_gated_scan_bwd(const void* x, const void* rgate, const void* igate, const float* A,
                       const float* rgate_bias, const float* igate_bias, int normalize,
                       const void* z, const float* initial_state, const float* chunk_states,
                       const void* dout, const float* dlast_state, void* dx, void* drgate,
                       void* digate, void* dz, float* dA, float* drgate_bias, float* digate_bias,
                       float* dinitial_state, int64_t batch, int64_t seqlen, int64_t dim, int dtype,
                       void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return gated_bwd("ssm_gated_scan_bwd", x, rgate, igate, A, rgate_bias, igate_bias, normalize, z,
                   initial_state, chunk_states, dout, dlast_state, dx, drgate, digate, dz, dA,
                   drgate_bias, digate_bias, dinitial_state, nullptr, batch, batch, seqlen, dim,
                   dtype, false, workspace, workspace_bytes, stream);
}

size_t ssm_gated_scan_bwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int dtype,
                                          int with_chunk_states) {
  return bwd_ws_bytes(batch, seqlen, batch, dim, dtype, false, with_chunk_states != 0);
}

int ssm_gated_scan_bwd_varlen(const void* x, const void* rgate, const void* igate, const float* A,
                              const float* rgate_bias, const float* igate_bias, int normalize,
                              const void* z, const float* initial_state,
                              const float* chunk_states, const void* dout,
                              const float* dlast_state, void* dx, void* drgate, void* digate,
                              void* dz, float* dA, float* drgate_bias, float* digate_bias,
                              float* dinitial_state, const int32_t* cu_seqlens, int64_t nseq,
                              int64_t total_len, int64_t dim, int dtype, void* workspace,
                              size_t workspace_bytes, hipStream_t stream) {
  return gated_bwd("ssm_gated_scan_bwd_varlen", x, rgate, igate, A, rgate_bias, igate_bias,
                   normalize, z, initial_state, chunk_states, dout, dlast_state, dx, drgate, digate,
                   dz, dA, drgate_bias, digate_bias, dinitial_state, cu_seqlens, nseq, 1, total_len,
                   dim, dtype, true, workspace, workspace_bytes, stream);
}

size_t ssm_gated_scan_bwd_varlen_workspace_bytes(int64_t nseq, int64_t total_len, int64_t dim,
                                                 int dtype, int with_chunk_states) {
  return bwd_ws_bytes(1, total_len, nseq, dim, dtype, true, with_chunk_states != 0);
}

}  // extern "C"
