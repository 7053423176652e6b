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

// Tokens of a lane, rows in flight (a ring of registers), waves.
constexpr int kBwdT = 16, kBwdBatch = 2, kBwdRing = 2;
constexpr int kBwdWaves = 8;
constexpr int kBwdChunk = kBwdT * kBwdWaves;
static_assert(SSM_GATED_CHUNK == kBwdT, "a wave starts where the forward kept the state");

// The forward's layout with the adjoint running back: one pass over the data,
// a wave starts from the state that the forward left at its first token, and
// the adjoint k_t = a_t G_t that enters from the chunk behind is handed over
// as the forward hands over states (maps within a group of chunks, one value
// per group), the units given out last chunk first.
// Per token six values stay in registers between the walk that rebuilds the
// states and the walk back: a, g, s and the factors of G in dx, di and dla.  T =
// 16 of them are 96 of the 128 registers that let four waves share a SIMD; the
// ring holds four tokens on the way (all sixteen at two waves a SIMD: 70 us
// against 58 for the layer, 22.5 against 23 for few workgroups; no variant is
// kept for that).  88 vector instructions a token keep the vector ALU busy for
// 57% of the time; the rest waits on memory.
// Measured (kernel alone): 4 x 2048 x 1536 with z, 9 activation tensors, bf16 59
// us, 3.8 TB/s, float32 97 us, 4.7 TB/s; packed 8192 x 1001 float32 96 us, bf16
// 65 us; packed 3001 x 515 float32 23 us, bf16 21 us.
template <typename TA, bool NORM, bool GATE, bool VL>
__global__ void __launch_bounds__(64 * kBwdWaves, 4) gated_bwd_kernel(GatedBwdArgs<TA> p, GatedPlan pl) {
  constexpr int T = kBwdT, W = kBwdWaves, C = kGatedC, NB = kBwdBatch, kPolls = (kGatedGroup + W - 1) / W;
  using IO = Cell<TA>;
  __shared__ float2 s_rev[W][C];
  __shared__ float2 s_in[kGatedGroup][C];
  __shared__ float s_carry[C];
  __shared__ uint32_t s_turn;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int dim = p.dim;
  uint64_t* const maps = static_cast<uint64_t*>(p.ws);
  uint64_t* const carries = maps + pl.chunks * pl.cells;
  uint32_t unit = blockIdx.y * kGatedGridX + blockIdx.x;
  if (pl.chunks > 1) {
    if (threadIdx.x == 0) s_turn = atomicAdd(reinterpret_cast<uint32_t*>(carries + pl.groups * pl.cells), 1u);
    __syncthreads();
    unit = __builtin_amdgcn_readfirstlane(s_turn);
  }
  if (unit >= pl.units) return;  // (the grid's surplus, or a workspace that another call uses at the same time)
  const uint32_t chunks = pl.chunks;
  const uint32_t c = chunks - 1 - unit / pl.lines, line = unit % pl.lines;
  const uint32_t row = line / pl.tiles, tile = line % pl.tiles;
  const int col0 = static_cast<int>(tile) * C, col = col0 + lane;
  const bool have = col < dim;
  const int64_t t0 = static_cast<int64_t>(c) * kBwdChunk + w * T;
  int64_t end = p.L;
  if (VL) {
    const int64_t e = scalar_of(p.cu)[p.nseq];
    end = e < 0 ? 0 : (e < end ? e : end);
  }
  const int n = end <= t0 ? 0 : (end - t0 < T ? static_cast<int>(end - t0) : T);  // the wave's tokens

  const uint32_t voff = have ? static_cast<uint32_t>(lane * sizeof(TA)) : kNoColumn;
  const uint32_t rowb = static_cast<uint32_t>(dim) * sizeof(TA);
  const int64_t base = (static_cast<int64_t>(row) * p.L + t0) * dim + col0;
  const uint32_t span = n > 0 ? (static_cast<uint32_t>(n) * rowb - col0 * static_cast<uint32_t>(sizeof(TA))) : 0;
  const uint32_t lastrow = n > 0 ? static_cast<uint32_t>(n - 1) * rowb : 0;
  const auto at = [&](int j) {  // rows behind the last are that one again
    const uint32_t o = static_cast<uint32_t>(j) * rowb;
    return o < lastrow ? o : lastrow;
  };
  const auto only = [&](int j) { return j < n ? voff : kNoColumn; };  // stores of tokens that are not there are dropped
  const Params pr = load_params(p.A, p.rb, p.ib, col, have);

  // a; g; dla / G; dx / G; di / G; s
  float a[T], g[T], cl[T], cx[T], ci[T], sr[T], y = 0.0f, Q = 0.0f;
  Marks mk{0, 0, 0};
  if (n > 0) {
    constexpr int R = kBwdRing;
    typename IO::raw_t xr[R][NB], rr[R][NB], ir[R][NB], dr[R][NB], zr[GATE ? R : 1][NB];
    const rsrc_t rx = make_rsrc(p.x + base, span), rg = make_rsrc(p.r + base, span),
                 ri = make_rsrc(p.i + base, span), rd = make_rsrc(p.dout + base, span),
                 rz = make_rsrc(GATE ? p.z + base : p.z, GATE ? span : 0),
                 rdz = make_rsrc(GATE ? p.dz + base : p.dz, GATE ? span : 0);
#pragma unroll
    for (int j = 0; j < R * NB; ++j) {
      rr[j / NB][j % NB] = IO::load(rg, voff, at(j));
      ir[j / NB][j % NB] = IO::load(ri, voff, at(j));
      xr[j / NB][j % NB] = IO::load(rx, voff, at(j));
      dr[j / NB][j % NB] = IO::load(rd, voff, at(j));
      if (GATE) zr[j / NB][j % NB] = IO::load(rz, voff, at(j));
    }
    float h = have ? p.chunk_states[(row * ((p.L + T - 1) / T) + t0 / T) * dim + col] : 0.0f;
    if (VL) mk = find_marks(p.cu, static_cast<int>(p.nseq), t0, n);
    // every token as if it were there (rows behind the last repeat it), y
    // over the n that are
#pragma unroll
    for (int k = 0; k < T / NB; ++k) {
#pragma unroll
      for (int jj = 0; jj < NB; ++jj) {
        const int j = k * NB + jj;
        const float there = j < n ? 1.0f : 0.0f;
        const float s = sigmoid2(__builtin_fmaf(IO::get(rr[k % R][jj]), -kLog2e, pr.rb2));
        const float u = sigmoid2(__builtin_fmaf(IO::get(ir[k % R][jj]), -kLog2e, pr.ib2));
        const float x = IO::get(xr[k % R][jj]), dout = IO::get(dr[k % R][jj]), d = pr.A2 * s;
        const float E = decay_parts(d, a[j]);
        float m = 1.0f, sub = 0.0f;
        if (NORM) {
          const float M = input_scale2(E);
          const float inv = M >= 0x1p-126f ? __builtin_amdgcn_rsqf(M) : 0.0f;  // (subnormals have no rsq)
          m = M * inv;
          sub = u * x * (a[j] * inv * a[j]);  // (a^2 alone may overflow where A > 0)
        }
        if (VL && (mk.starts >> j & 1))
          h = p.h0 && have ? p.h0[static_cast<int64_t>(__builtin_amdgcn_readlane(mk.seq, j)) * dim + col] : 0.0f;
        sr[j] = s;
        cx[j] = m * u;
        const float b = cx[j] * x, ah = a[j] * h;
        ci[j] = b * (1.0f - u);
        cl[j] = ah - sub;
        h = __builtin_fmaf(a[j], h, b);
        y = __builtin_fmaf(d, there, y);
        if (GATE) {
          const float z = IO::get(zr[k % R][jj]), sz = sigmoid_f32(z);
          IO::store(rdz, dout * h * sz * __builtin_fmaf(z, 1.0f - sz, 1.0f), only(j), at(j));
          g[j] = dout * (z * sz);
        } else {
          g[j] = dout;
        }
        // (the six values are formed here: moved to where they are used, their
        // sources would have to stay as well)
        asm volatile("" : "+v"(a[j]), "+v"(g[j]), "+v"(cl[j]), "+v"(cx[j]), "+v"(ci[j]), "+v"(sr[j]));
      }
      __builtin_amdgcn_sched_barrier(0);
      if (k + R < T / NB) {
#pragma unroll
        for (int jj = 0; jj < NB; ++jj) {
          const uint32_t o = at((k + R) * NB + jj);
          rr[k % R][jj] = IO::load(rg, voff, o);
          ir[k % R][jj] = IO::load(ri, voff, o);
          xr[k % R][jj] = IO::load(rx, voff, o);
          dr[k % R][jj] = IO::load(rd, voff, o);
          if (GATE) zr[k % R][jj] = IO::load(rz, voff, o);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (n < T) {
#pragma unroll
      for (int j = 0; j < T; ++j) {
        if (j >= n) {
          a[j] = 1.0f;
          g[j] = cl[j] = cx[j] = ci[j] = 0.0f;
        }
      }
    }
    // the map of the wave's tokens on the adjoint that enters from behind
#pragma unroll
    for (int j = T - 1; j >= 0; --j) {
      if (VL && (mk.ends >> j & 1))
        Q = p.dlast && have ? p.dlast[static_cast<int64_t>(__builtin_amdgcn_readlane(mk.seq, j)) * dim + col] : 0.0f;
      Q = VL && (mk.starts >> j & 1) ? 0.0f : a[j] * (g[j] + Q);
    }
  }
  y = VL && (mk.starts | mk.ends) ? kCut : keep_of(y);
  s_rev[w][lane] = make_float2(y, Q);
  __syncthreads();
  float yw, Qw, yt = 0.0f, Qt = 0.0f;
  fold_maps<VL, true>(s_rev + w + 1, W - 1 - w, lane, yw, Qw);
  const int64_t cell = static_cast<int64_t>(line) * C + lane;
  if (w == 0) {
    yt = yw;
    Qt = Qw;
    compose<VL>(yt, Qt, y, Q);
    if (c > 0) publish(maps + c * pl.cells + cell, yt, Qt);
  }
  // the adjoint that enters the chunk from behind
  const uint32_t first = c / kGatedGroup * kGatedGroup;
  const uint32_t lastc = first + kGatedGroup < chunks ? first + kGatedGroup - 1 : chunks - 1;
  const int there = static_cast<int>(lastc - c);  // chunks of the group behind this one
  {
    float lo[kPolls], hi[kPolls];
    const int polls = there > w ? (there - w + W - 1) / W : 0;  // chunks c + 1 + w, c + 1 + w + W, ...
    if (polls > 0) await(maps + (c + 1 + w) * pl.cells + cell, W * pl.cells, polls, lo, hi);
#pragma unroll
    for (int q = 0; q < kPolls; ++q)
      if (q < polls) s_in[w + q * W][lane] = make_float2(lo[q], hi[q]);
  }
  if (w == W - 1) {
    float zero[1], from[1] = {!VL && p.dlast && have ? p.dlast[static_cast<int64_t>(row) * dim + col] : 0.0f};
    if (lastc + 1 < chunks) await(carries + (c / kGatedGroup + 1) * pl.cells + cell, 0, 1, zero, from);
    s_carry[lane] = from[0];
  }
  __syncthreads();
  float k = fold_state<VL, true>(s_in, there, lane, s_carry[lane]);
  if (w == 0 && c == first && c > 0)
    publish(carries + c / kGatedGroup * pl.cells + cell, 0.0f, pass<VL>(yt, Qt, k));
  k = pass<VL>(yw, Qw, k);
  float dA = 0.0f, drb = 0.0f, dib = 0.0f;
  if (n > 0) {
    const rsrc_t rdx = make_rsrc(p.dx + base, span), rdr = make_rsrc(p.dr + base, span),
                 rdi = make_rsrc(p.di + base, span);
    float A = have ? p.A[col] : 0.0f;
    if (A < -1e30f) A = -1e30f;  // (finite, as in A2: a decay of 0 has no slope)
#pragma unroll
    for (int j = T - 1; j >= 0; --j) {
      if (VL && (mk.ends >> j & 1))
        k = p.dlast && have ? p.dlast[static_cast<int64_t>(__builtin_amdgcn_readlane(mk.seq, j)) * dim + col] : 0.0f;
      const float G = g[j] + k, dla = G * cl[j], s = sr[j];
      const float di = G * ci[j], drr = dla * (A * s * (1.0f - s));
      dA = __builtin_fmaf(dla, s, dA);
      drb += drr;
      dib += di;
      k = a[j] * G;
      IO::store(rdx, G * cx[j], only(j), at(j));
      IO::store(rdr, drr, only(j), at(j));
      IO::store(rdi, di, only(j), at(j));
      if (VL && (mk.starts >> j & 1)) {
        if (p.dh0 && have) p.dh0[static_cast<int64_t>(__builtin_amdgcn_readlane(mk.seq, j)) * dim + col] = k;
        k = 0.0f;
      }
    }
  }
  if (!VL && p.dh0 && c == 0 && w == 0 && have) p.dh0[static_cast<int64_t>(row) * dim + col] = k;
  // the chunk's sums: over the waves, last tokens first
  __syncthreads();
  float* const s_sum = reinterpret_cast<float*>(&s_in[0][0]);  // (W, 3, C)
  static_assert(sizeof(s_in) >= sizeof(float) * W * 3 * C, "the sums fit where the maps were");
  s_sum[(w * 3 + 0) * C + lane] = dA;
  s_sum[(w * 3 + 1) * C + lane] = drb;
  s_sum[(w * 3 + 2) * C + lane] = dib;
  __syncthreads();
  for (int q = threadIdx.x; q < 3 * C; q += 64 * W) {
    float v = 0.0f;
#pragma unroll
    for (int k2 = W - 1; k2 >= 0; --k2) v += s_sum[k2 * 3 * C + q];
    const int what = q / C, cc = col0 + q % C;
    if (cc < dim) p.part[((static_cast<int64_t>(row) * chunks + c) * 3 + what) * dim + cc] = v;
  }
}

// Sums of the chunks' partials: a workgroup takes 64 channels of one of the
// three, wave w every kSumWaves-th chunk, and the waves' sums are added in
// order.  1.2 MB for 4 x 2048 x 1536: its launch and one round trip, 4.7 us.
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

template <typename TA>
int launch_gated_bwd(const GatedBwdArgs<TA>& a, const GatedPlan& pl, bool norm, const char* fn,
                     hipStream_t s) {
  int rc = launch_gated_init(a.ws, pl.bytes, a.cu, a.cu ? a.nseq : a.rows, a.L, a.dim, a.dlast, a.dh0, fn, s);
  if (rc != SSM_OK) return rc;
  if (a.L > 0) {
    const dim3 grid = gated_grid(pl.units), block(64 * kBwdWaves);
#define SSM_GATED_CASE(N, G, VLN)                                                              \
  if (norm == N && (a.z != nullptr) == G && (a.cu != nullptr) == VLN)                          \
    hipLaunchKernelGGL((gated_bwd_kernel<TA, N, G, VLN>), grid, block, 0, s, a, pl);
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
  const size_t own = gated_plan(rows, L, dim, kBwdChunk).bytes, fwd = have_states ? 0 : gated_fwd_bytes(rows, L, dim);
  const size_t states = static_cast<size_t>(rows) * ((L + SSM_GATED_CHUNK - 1) / SSM_GATED_CHUNK);
  const size_t chunks = static_cast<size_t>(rows) * ((L + kBwdChunk - 1) / kBwdChunk);
  BwdSpace b;
  b.states = up(own > fwd ? own : fwd);
  b.part = b.states + (have_states ? 0 : up(states * dim * 4));
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
    return launch_gated_bwd<TA>(a, gated_plan(rows, L, dim, kBwdChunk), normalize != 0, fn, stream);
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
