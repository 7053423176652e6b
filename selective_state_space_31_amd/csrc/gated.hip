// gated.hip -- the gated linear recurrence, forward and decode step, behind
// the C ABI in include/ssm_recurrent.h.
//
//   a_t = e^(A sigma(r_t + rb)),  h_t = a_t h_{t-1} + m_t sigma(i_t + ib) x_t
//   out_t = h_t silu(z_t)
//
// 37 vector instructions per token and channel, 44 with z, stand against 8 to 20
// bytes, so memory bounds a long run (vector ALU busy 70% of the time at 131072
// tokens) and latency a short one.
//
#include "gated.hpp"
#include "host_util.hpp"

namespace ssm {

// Ones into the published words, zero into the counter; empty sequences'
// states.  A grid-stride loop over each; a launch (2 to 5 us) more than work
// (0.4 MB for 4 x 2048 x 1536).
__global__ void __launch_bounds__(256) gated_init_kernel(uint64_t* words, int64_t nwords,
                                                         uint32_t* turn, const int32_t* cu,
                                                         int64_t nstates, int dim,
                                                         const float* from, float* to) {
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 256;
  for (int64_t i = i0; i < nwords; i += step) words[i] = ~uint64_t{0};
  if (i0 == 0 && turn) *turn = 0;
  for (int64_t i = i0; i < nstates; i += step) {
    const int64_t s = i / dim;
    if (!cu || cu[s + 1] <= cu[s]) to[i] = from ? from[i] : 0.0f;
  }
}

int launch_gated_init(void* ws, size_t bytes, const int32_t* cu, int64_t nseq, int64_t L, int dim,
                      const float* from, float* to, const char* fn, hipStream_t s) {
  const int64_t nwords = bytes ? static_cast<int64_t>(bytes - 256) / 8 : 0;
  const int64_t nstates = to && (cu || L == 0) ? nseq * dim : 0;
  const int64_t n = nwords > nstates ? nwords : nstates;
  if (n == 0) return SSM_OK;
  uint32_t* turn = bytes ? reinterpret_cast<uint32_t*>(static_cast<uint64_t*>(ws) + nwords) : nullptr;
  const int64_t blocks = (n + 255) / 256;
  hipLaunchKernelGGL(gated_init_kernel, dim3(static_cast<unsigned>(blocks < 2048 ? blocks : 2048)),
                     dim3(256), 0, s, static_cast<uint64_t*>(ws), nwords, turn, cu, nstates, dim, from,
                     to);
  return launch_status(fn);
}

// Tokens of a lane, waves of a workgroup, rows of the inputs a wave has in
// flight (batch * ring: a ring of registers, filled again as it is used up),
// waves a SIMD holds.
struct FwdLong {  // few folds per token, 3 workgroups to a CU: throughput
  // (4 x 2048 x 1536 bf16: 37 us; T 32 with z fetched before the wait 45)
  static constexpr int T = 64, W = 4, batch = 4, ring = 2, occupancy = 3;
};
struct FwdShort {  // every load issued at once: the latency of few workgroups
  // (8192 x 1001 float32: 43 us; half as many waves and T 8 each 5 more)
  static constexpr int T = 16, W = 16, batch = 4, ring = 4, occupancy = 4;
};

// One pass over the data: a workgroup loads its tokens once, turns them into
// (a, b) in registers and composes its chunk's map; publishes that; waits for
// the state that enters the chunk; and walks its tokens from there.  Chunks
// come in groups of kGatedGroup.  A chunk reads the maps of the chunks before
// it in its group, which exist as soon as those workgroups have read their
// data, and one state per group, which the last chunk of the group before
// hands on: the chain over the sequence is one step per 4096 tokens.  The
// folds have a fixed order, so results repeat bit for bit.
// Units are handed out by a counter, earlier chunks first: a workgroup waits
// only for ones that are running or done.
// Reading the data once is what the split is for: chunk maps in a launch of
// their own would read x and both gates twice (7 units of traffic for 5).
// Measured (kernel alone): 1 x 131072 x 2048 bf16 450 us, 4.8 TB/s of the
// algorithm's bytes (copies of the same size reach 4.9 to 6.1); 4 x 2048 x 1536
// with z bf16 37 us, 3.4 TB/s, float32 54 us, 4.6 TB/s; packed 8192 x 1001 with
// z float32 43 us, 3.8 TB/s, bf16 35 us; packed 3001 x 515 of either type 16 us, the chain ticket -> loads -> publish ->
// wait -> stores of one round of workgroups.
template <typename TA, typename CF, bool NORM, bool GATE, bool VL>
__global__ void __launch_bounds__(64 * CF::W, CF::occupancy) gated_fwd_kernel(GatedFwdArgs<TA> p, GatedPlan pl) {
  constexpr int T = CF::T, W = CF::W, C = kGatedC, NB = CF::batch, R = CF::ring, kPolls = kGatedGroup / W;
  // rows of z in flight; before the wait for the entering state where the
  // registers have room for them
  constexpr int kZ = 16;
  constexpr bool kZEarly = T == kZ;
  using IO = Cell<TA>;
  __shared__ float2 s_agg[W][C];
  __shared__ float2 s_in[kGatedGroup][C];
  __shared__ float s_carry[C];
  __shared__ uint32_t s_turn;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int dim = p.dim;
  uint64_t* const agg = static_cast<uint64_t*>(p.ws);
  uint64_t* const carries = agg + pl.chunks * pl.cells;
  uint32_t unit = blockIdx.y * kGatedGridX + blockIdx.x;
  if (pl.chunks > 1) {
    if (threadIdx.x == 0) s_turn = atomicAdd(reinterpret_cast<uint32_t*>(carries + pl.groups * pl.cells), 1u);
    __syncthreads();
    unit = __builtin_amdgcn_readfirstlane(s_turn);
  }
  if (unit >= pl.units) return;  // (the grid's surplus, or a workspace that another call uses at the same time)
  const uint32_t c = unit / pl.lines, line = unit % pl.lines;
  const uint32_t row = line / pl.tiles, tile = line % pl.tiles;
  const int col0 = static_cast<int>(tile) * C, col = col0 + lane;
  const bool have = col < dim;
  const int64_t t0 = static_cast<int64_t>(c) * (T * W) + w * T;
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
  float a[T], b[T], y = 0.0f, H = 0.0f;  // y: first the sum of the tokens' v
  Marks mk{0, 0, 0};
  if (n > 0) {
    typename IO::raw_t xr[R][NB], rr[R][NB], ir[R][NB];
    const rsrc_t rx = make_rsrc(p.x + base, span), rg = make_rsrc(p.r + base, span),
                 ri = make_rsrc(p.i + base, span);
#pragma unroll
    for (int j = 0; j < R * NB; ++j) {
      rr[j / NB][j % NB] = IO::load(rg, voff, at(j));
      ir[j / NB][j % NB] = IO::load(ri, voff, at(j));
      xr[j / NB][j % NB] = IO::load(rx, voff, at(j));
    }
    if (VL) mk = find_marks(p.cu, static_cast<int>(p.nseq), t0, n);
    const Params pr = load_params(p.A, p.rb, p.ib, col, have);
    // every token as if it were there (rows behind the last repeat it), y
    // over the n that are
#pragma unroll
    for (int k = 0; k < T / NB; ++k) {
#pragma unroll
      for (int jj = 0; jj < NB; ++jj) {
        const int j = k * NB + jj;
        const float there = j < n ? 1.0f : 0.0f;
        const float d = pr.A2 * sigmoid2(__builtin_fmaf(IO::get(rr[k % R][jj]), -kLog2e, pr.rb2));
        float m;
        decay<NORM>(d, a[j], m);
        b[j] = m * sigmoid2(__builtin_fmaf(IO::get(ir[k % R][jj]), -kLog2e, pr.ib2)) * IO::get(xr[k % R][jj]);
        y = __builtin_fmaf(d, there, y);
        H = __builtin_fmaf(a[j], H, b[j]);
      }
      // (a batch of tokens overlaps; more would not fit the registers)
      __builtin_amdgcn_sched_barrier(0);
      if (k + R < T / NB) {
#pragma unroll
        for (int jj = 0; jj < NB; ++jj) {
          rr[k % R][jj] = IO::load(rg, voff, at((k + R) * NB + jj));
          ir[k % R][jj] = IO::load(ri, voff, at((k + R) * NB + jj));
          xr[k % R][jj] = IO::load(rx, voff, at((k + R) * NB + jj));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (n < T || (VL && mk.starts)) {
      H = 0.0f;
#pragma unroll
      for (int j = 0; j < T; ++j) {
        const bool start = VL && (mk.starts >> j & 1);
        const int64_t s = start ? __builtin_amdgcn_readlane(mk.seq, j) : 0;
        if (j >= n) {
          a[j] = 1.0f;
          b[j] = 0.0f;
        }
        // (without an initial state a * 0, so that a NaN gate counts as it does in a whole sequence)
        if (start) b[j] = __builtin_fmaf(a[j], p.h0 && have ? p.h0[s * dim + col] : 0.0f, b[j]);
        H = start ? b[j] : __builtin_fmaf(a[j], H, b[j]);
      }
    }
  }
  const rsrc_t rz = make_rsrc(GATE && n > 0 ? p.z + base : p.z, GATE ? span : 0);
  typename IO::raw_t zr[GATE ? kZ : 1];
  if (GATE && kZEarly && n > 0) {
#pragma unroll
    for (int j = 0; j < kZ; ++j) zr[j] = IO::load(rz, voff, at(j));
  }
  // The state that the first group folds from.  last_state may be its buffer,
  // written by the row's last chunk behind the words of every chunk before it:
  // with h0 here (the pin waits for the load) ahead of this chunk's word, nobody
  // still reads it by then.
  float h0 = 0.0f;
  if (!VL && p.h0 && c < kGatedGroup) {
    if (have) h0 = p.h0[static_cast<int64_t>(row) * dim + col];
    asm volatile("" : "+v"(h0));
  }
  y = VL && mk.starts ? kCut : keep_of(y);
  s_agg[w][lane] = make_float2(y, H);
  __syncthreads();
  // the map of the waves before this one; the last wave also the chunk's
  float yw, Hw, yt = 0.0f, Ht = 0.0f, h;
  fold_maps<VL, false>(s_agg, w, lane, yw, Hw);
  const int64_t cell = static_cast<int64_t>(line) * C + lane;
  if (w == W - 1) {
    yt = yw;
    Ht = Hw;
    compose<VL>(yt, Ht, y, H);
    if (c + 1 < pl.chunks) publish(agg + c * pl.cells + cell, yt, Ht);
  }
  // the state that enters the chunk
  if (c == 0) {
    h = h0;
  } else {
    const uint32_t first = c / kGatedGroup * kGatedGroup;
    const int there = static_cast<int>(c - first);  // chunks of the group before this one
    const int polls = there > w ? (there - w + W - 1) / W : 0;  // chunks w, w + W, ...
    float lo[kPolls], hi[kPolls];
    if (polls > 0) await(agg + (first + w) * pl.cells + cell, W * pl.cells, polls, lo, hi);
#pragma unroll
    for (int k = 0; k < kPolls; ++k)
      if (k < polls) s_in[w + k * W][lane] = make_float2(lo[k], hi[k]);
    if (w == W - 1) {
      float zero[1], state[1] = {h0};
      if (first > 0) await(carries + c / kGatedGroup * pl.cells + cell, 0, 1, zero, state);
      s_carry[lane] = state[0];
    }
    __syncthreads();
    h = fold_state<VL, false>(s_in, there, lane, s_carry[lane]);
  }
  if (w == W - 1 && (c + 1) % kGatedGroup == 0 && c + 1 < pl.chunks)
    publish(carries + (c + 1) / kGatedGroup * pl.cells + cell, 0.0f, pass<VL>(yt, Ht, h));
  h = pass<VL>(yw, Hw, h);
  if (n > 0) {
    // without out (the chunks' states alone) every store is out of range
    const rsrc_t ro = make_rsrc(p.out + base, p.out ? span : 0);
    const uint32_t outb = p.out ? rowb : 0;
    if (GATE && !kZEarly) {
#pragma unroll
      for (int j = 0; j < kZ; ++j) zr[j] = IO::load(rz, voff, at(j));
    }
    float* const states =
        p.chunk_states && have
            ? p.chunk_states + (row * ((p.L + SSM_GATED_CHUNK - 1) / SSM_GATED_CHUNK) + t0 / SSM_GATED_CHUNK) * dim + col
            : nullptr;
    const auto before = [&](int j) {
      if (j % SSM_GATED_CHUNK == 0 && states) states[static_cast<int64_t>(j / SSM_GATED_CHUNK) * dim] = h;
    };
    const auto emit = [&](int j) {
      const float o = GATE ? h * silu_f32(IO::get(zr[GATE ? j % kZ : 0])) : h;
      if (GATE && j + kZ < T) zr[j % kZ] = IO::load(rz, voff, at(j + kZ));
      IO::store(ro, o, voff, static_cast<uint32_t>(j) * outb);
      if ((j & 3) == 3) __builtin_amdgcn_sched_barrier(0);
    };
    if (n == T && (!VL || !(mk.starts | mk.ends))) {
#pragma unroll
      for (int j = 0; j < T; ++j) {
        before(j);
        h = __builtin_fmaf(a[j], h, b[j]);
        emit(j);
      }
    } else {
#pragma unroll
      for (int j = 0; j < T; ++j) {
        if (j < n) {
          before(j);
          h = VL && (mk.starts >> j & 1) ? b[j] : __builtin_fmaf(a[j], h, b[j]);
          emit(j);
          if (VL && p.last && (mk.ends >> j & 1) && have)
            p.last[static_cast<int64_t>(__builtin_amdgcn_readlane(mk.seq, j)) * dim + col] = h;
        }
      }
    }
  }
  // (waves behind the row's end hold the identity)
  if (!VL && p.last && c + 1 == pl.chunks && w == W - 1 && have) p.last[static_cast<int64_t>(row) * dim + col] = h;
}

template <typename CF>
GatedPlan fwd_plan(int64_t rows, int64_t L, int64_t dim) {
  return gated_plan(rows, L, dim, CF::T * CF::W);
}

template <typename TA, typename CF>
int launch_gated_fwd(const GatedFwdArgs<TA>& a, bool norm, const char* fn, hipStream_t s) {
  const GatedPlan pl = fwd_plan<CF>(a.rows, a.L, a.dim);
  const int rc = launch_gated_init(a.ws, pl.bytes, a.cu, a.cu ? a.nseq : a.rows, a.L, a.dim, a.h0, a.last,
                                   fn, s);
  if (rc != SSM_OK || a.L == 0) return rc;
  const dim3 grid = gated_grid(pl.units), block(64 * CF::W);
#define SSM_GATED_CASE(N, G, VLN)                                                              \
  if (norm == N && (a.z != nullptr) == G && (a.cu != nullptr) == VLN)                          \
    hipLaunchKernelGGL((gated_fwd_kernel<TA, CF, N, G, VLN>), grid, block, 0, s, a, pl);
  SSM_GATED_CASE(true, true, false)
  SSM_GATED_CASE(true, false, false)
  SSM_GATED_CASE(false, true, false)
  SSM_GATED_CASE(false, false, false)
  SSM_GATED_CASE(true, true, true)
  SSM_GATED_CASE(true, false, true)
  SSM_GATED_CASE(false, true, true)
  SSM_GATED_CASE(false, false, true)
#undef SSM_GATED_CASE
  return launch_status(fn);
}

template <typename TA>
struct GatedStepArgs {
  float* state;
  const TA *x, *r, *i, *z;
  const float *A, *rb, *ib;
  TA* out;
  int64_t n;
  int dim;
};

// One step: h <- a h + m u x, out = h silu(z).  V neighbouring channels of one
// sequence per lane, each array moved as one access.  Bound by memory where
// there is enough of it (256 x 5120 float32: 36.7 MB in 8.0 us, 4.6 TB/s),
// otherwise by its launch (1 x 2048 bf16: 2.5 us).
template <typename T, int V>
struct alignas(V * sizeof(T)) Pack {
  T v[V];
};
template <typename TA, int V, bool NORM>
__global__ void __launch_bounds__(256) gated_step_kernel(GatedStepArgs<TA> p) {
  const uint32_t o = (blockIdx.x * 256 + threadIdx.x) * V;
  if (o >= p.n) return;
  const uint32_t c = o % static_cast<uint32_t>(p.dim);
  using Act = Pack<TA, V>;
  using F32 = Pack<float, V>;
  const auto f32 = [](const float* q, uint32_t k) { return *reinterpret_cast<const F32*>(q + k); };
  const auto act = [&](const TA* q) { return *reinterpret_cast<const Act*>(q + o); };
  const F32 none{};
  const Act r = act(p.r), i = act(p.i), x = act(p.x), z = p.z ? act(p.z) : Act{};
  F32 h = f32(p.state, o);
  const F32 A = f32(p.A, c), rb = p.rb ? f32(p.rb, c) : none, ib = p.ib ? f32(p.ib, c) : none;
  Act out;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float a, m;
    const Params pr = params_of(A.v[v], rb.v[v], ib.v[v]);
    decay<NORM>(pr.A2 * sigmoid2(__builtin_fmaf(to_f32(r.v[v]), -kLog2e, pr.rb2)), a, m);
    const float u = sigmoid2(__builtin_fmaf(to_f32(i.v[v]), -kLog2e, pr.ib2));
    h.v[v] = __builtin_fmaf(a, h.v[v], m * u * to_f32(x.v[v]));
    store_act(&out.v[v], p.z ? h.v[v] * silu_f32(to_f32(z.v[v])) : h.v[v]);
  }
  *reinterpret_cast<F32*>(p.state + o) = h;
  *reinterpret_cast<Act*>(p.out + o) = out;
}

template <int V>
struct Lane {
  static constexpr int value = V;
};

constexpr int64_t kGatedMaxDim = int64_t{1} << 22;
constexpr int64_t kGatedMaxSeqs = int64_t{1} << 24;

// Whether batch, seqlen (or nseq, total_len) and dim can be launched: the
// byte offsets inside a wave's 64 rows fit 31 bits, and a workgroup per 64
// channels and (in the backward) 128 tokens fits a grid.
bool gated_sizes_ok(int64_t rows, int64_t L, int64_t nseq, int64_t dim, bool packed) {
  if (dim < 1 || dim > kGatedMaxDim || L < 0 || L > (int64_t{1} << 40) / dim) return false;
  if (packed ? (nseq < 1 || nseq >= kGatedMaxSeqs) : (rows < 1 || rows > 65535)) return false;
  return rows * ((L + 127) / 128) * ((dim + 63) / 64) < (int64_t{1} << 31);
}

size_t gated_fwd_bytes(int64_t rows, int64_t L, int64_t dim) {
  const size_t a = fwd_plan<FwdLong>(rows, L, dim).bytes, b = fwd_plan<FwdShort>(rows, L, dim).bytes;
  return a > b ? a : b;
}

template <typename TA>
int run_gated_fwd(const char* fn, const void* x, const void* r, const void* i, const float* A,
                  const float* rb, const float* ib, bool norm, const void* z, void* out, float* last,
                  const float* h0, float* states, const int32_t* cu, int64_t nseq, int64_t rows,
                  int64_t L, int dim, void* ws, hipStream_t stream) {
  const GatedFwdArgs<TA> a{static_cast<const TA*>(x), static_cast<const TA*>(r), static_cast<const TA*>(i),
                           static_cast<const TA*>(z), A, rb, ib, static_cast<TA*>(out), last, h0, states, cu,
                           rows, L, nseq, dim, ws};
  // Long stretches where they give every CU more than two workgroups (768 of
  // them, 4 x 2048 x 1536 bf16: 37 against 42 us); below, a lane that goes
  // through its tokens in rounds of loads takes longer than the device is kept
  // busy by them (512, 8192 x 1001 float32: 54 against 41 us; 108, 3001 x 515
  // float32: 25 against 16 us).  The length needs no rule of its own: rows that
  // fill neither stretch cost what their workgroups' starts and whole stretches
  // cost, and the long ones still less (512 x 4 x 2048 bf16 189 against 241 us,
  // 256 x 16 x 2048 104 against 123, 16 x 64 x 5120 21 against 28; float32 the
  // same within 8%, in the same order).
  return fwd_plan<FwdLong>(rows, L, dim).units > 2u * static_cast<unsigned>(device_cus())
             ? launch_gated_fwd<TA, FwdLong>(a, norm, fn, stream)
             : launch_gated_fwd<TA, FwdShort>(a, norm, fn, stream);
}

int gated_states(const char* fn, const void* x, const void* r, const void* i, const float* A,
                 const float* rb, const float* ib, int normalize, const float* h0, float* states,
                 const int32_t* cu, int64_t nseq, int64_t rows, int64_t L, int dim, int dtype,
                 void* ws, hipStream_t stream) {
  return dtype == SSM_DTYPE_F32
             ? run_gated_fwd<float>(fn, x, r, i, A, rb, ib, normalize != 0, nullptr, nullptr, nullptr, h0,
                                    states, cu, nseq, rows, L, dim, ws, stream)
             : run_gated_fwd<bf16_t>(fn, x, r, i, A, rb, ib, normalize != 0, nullptr, nullptr, nullptr, h0,
                                     states, cu, nseq, rows, L, dim, ws, stream);
}

namespace {

int gated_fwd(const char* fn, const void* x, const void* r, const void* i, const float* A,
              const float* rb, const float* ib, int normalize, const void* z, void* out,
              float* last, const float* h0, float* chunk_states, const int32_t* cu, int64_t nseq,
              int64_t rows, int64_t L, int64_t dim, int dtype, bool packed, void* ws,
              size_t ws_bytes, hipStream_t stream) {
  clear_error();
  if (dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16)
    return fail(SSM_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, dtype);
  if (normalize != 0 && normalize != 1)
    return fail(SSM_ERR_UNSUPPORTED, "%s: normalize must be 0 or 1, got %d", fn, normalize);
  if (!gated_sizes_ok(rows, L, nseq, dim, packed))
    return fail(SSM_ERR_SHAPE, "%s: bad sizes: %lld sequence(s), %lld tokens, dim %lld", fn,
                (long long)(packed ? nseq : rows), (long long)L, (long long)dim);
  if (!A || (packed && !cu)) return fail(SSM_ERR_NULL, "%s: A%s required", fn, packed ? " and cu_seqlens are" : " is");
  if (L > 0 && (!x || !r || !i || !out))
    return fail(SSM_ERR_NULL, "%s: x, rgate, igate and out are required", fn);
  const size_t es = dtype == SSM_DTYPE_F32 ? 4 : 2;
  const struct { const void* p; size_t k; const char* n; } al[] = {
      {x, es, "x"}, {r, es, "rgate"}, {i, es, "igate"}, {z, es, "z"}, {out, es, "out"}, {A, 4, "A"},
      {rb, 4, "rgate_bias"}, {ib, 4, "igate_bias"}, {h0, 4, "initial_state"},
      {last, 4, "last_state"}, {chunk_states, 4, "chunk_states"}, {cu, 4, "cu_seqlens"}};
  for (const auto& e : al)
    if (e.p && !aligned(e.p, e.k))
      return fail(SSM_ERR_ALIGN, "%s: %s is not %zu-byte aligned", fn, e.n, e.k);
  const size_t tok = static_cast<size_t>(rows) * L * dim * es;
  const size_t st = static_cast<size_t>(packed ? nseq : rows) * dim * 4;
  const size_t cst = static_cast<size_t>(rows) * ((L + SSM_GATED_CHUNK - 1) / SSM_GATED_CHUNK) * dim * 4;
  const size_t pd = static_cast<size_t>(dim) * 4;
  const size_t need = gated_fwd_bytes(rows, L, dim);
  const Span ins[] = {{x, tok, "x"}, {r, tok, "rgate"}, {i, tok, "igate"}, {z, z ? tok : 0, "z"},
                      {A, pd, "A"}, {rb, rb ? pd : 0, "rgate_bias"}, {ib, ib ? pd : 0, "igate_bias"},
                      {cu, packed ? static_cast<size_t>(nseq + 1) * 4 : 0, "cu_seqlens"},
                      {h0, h0 ? st : 0, "initial_state"}};
  const Span outs[] = {{out, tok, "out"}, {last, last ? st : 0, "last_state"},
                       {chunk_states, chunk_states ? cst : 0, "chunk_states"},
                       {ws, ws ? need : 0, "workspace"}};
  for (const auto& o : outs)
    for (const auto& n : ins)
      if (overlap(o, n) && !(o.p == last && n.p == h0 && last == h0 && !packed))
        return fail(SSM_ERR_ALIAS, "%s: output %s overlaps input %s", fn, o.name, n.name);
  for (int a = 0; a < 4; ++a)
    for (int b = a + 1; b < 4; ++b)
      if (overlap(outs[a], outs[b]))
        return fail(SSM_ERR_ALIAS, "%s: %s overlaps %s", fn, outs[a].name, outs[b].name);
  if (need > 0 && (!ws || ws_bytes < need))
    return fail(SSM_ERR_WORKSPACE, "%s: workspace of %zu bytes given, %zu needed", fn,
                ws ? ws_bytes : 0, need);
  if (need > 0 && !aligned(ws, 256))
    return fail(SSM_ERR_ALIGN, "%s: workspace is not 256-byte aligned", fn);
  const int32_t* const offsets = packed ? cu : nullptr;
  return dtype == SSM_DTYPE_F32
             ? run_gated_fwd<float>(fn, x, r, i, A, rb, ib, normalize != 0, z, out, last, h0, chunk_states,
                                    offsets, nseq, rows, L, static_cast<int>(dim), ws, stream)
             : run_gated_fwd<bf16_t>(fn, x, r, i, A, rb, ib, normalize != 0, z, out, last, h0,
                                     chunk_states, offsets, nseq, rows, L, static_cast<int>(dim), ws,
                                     stream);
}

}  // namespace
}  // namespace ssm

using namespace ssm;

extern "C" {

int ssm_gated_scan_fwd(const void* x, const void* rgate, const void* igate, const float* A,
                       const float* rgate_bias, const float* igate_bias, int normalize,
                       const void* z, void* out, float* last_state, const float* initial_state,
                       float* chunk_states, int64_t batch, int64_t seqlen, int64_t dim, int dtype,
                       void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return gated_fwd("ssm_gated_scan_fwd", x, rgate, igate, A, rgate_bias, igate_bias, normalize, z,
                   out, last_state, initial_state, chunk_states, nullptr, batch, batch, seqlen, dim,
                   dtype, false, workspace, workspace_bytes, stream);
}

size_t ssm_gated_scan_fwd_workspace_bytes(int64_t batch, int64_t seqlen, int64_t dim, int dtype) {
  if ((dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16) ||
      !gated_sizes_ok(batch, seqlen, batch, dim, false))
    return 0;
  return gated_fwd_bytes(batch, seqlen, dim);
}

int ssm_gated_scan_fwd_varlen(const void* x, const void* rgate, const void* igate, const float* A,
                              const float* rgate_bias, const float* igate_bias, int normalize,
                              const void* z, void* out, float* last_state,
                              const float* initial_state, float* chunk_states,
                              const int32_t* cu_seqlens, int64_t nseq, int64_t total_len,
                              int64_t dim, int dtype, void* workspace, size_t workspace_bytes,
                              hipStream_t stream) {
  return gated_fwd("ssm_gated_scan_fwd_varlen", x, rgate, igate, A, rgate_bias, igate_bias,
                   normalize, z, out, last_state, initial_state, chunk_states, cu_seqlens, nseq, 1,
                   total_len, dim, dtype, true, workspace, workspace_bytes, stream);
}

size_t ssm_gated_scan_fwd_varlen_workspace_bytes(int64_t nseq, int64_t total_len, int64_t dim,
                                                 int dtype) {
  if ((dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16) ||
      !gated_sizes_ok(1, total_len, nseq, dim, true))
    return 0;
  return gated_fwd_bytes(1, total_len, dim);
}

int ssm_gated_state_update(float* state, const void* x, const void* rgate, const void* igate,
                           const float* A, const float* rgate_bias, const float* igate_bias,
                           int normalize, const void* z, void* out, int64_t batch, int64_t dim,
                           int dtype, hipStream_t stream) {
  clear_error();
  const char* fn = "ssm_gated_state_update";
  if (dtype != SSM_DTYPE_F32 && dtype != SSM_DTYPE_BF16)
    return fail(SSM_ERR_UNSUPPORTED, "%s: unknown dtype %d", fn, dtype);
  if (normalize != 0 && normalize != 1)
    return fail(SSM_ERR_UNSUPPORTED, "%s: normalize must be 0 or 1, got %d", fn, normalize);
  if (batch < 1 || dim < 1 || dim > kGatedMaxDim || batch > (int64_t{1} << 31) ||
      batch * dim > (int64_t{1} << 31) - 2048)  // (batch bounded first: no overflow)
    return fail(SSM_ERR_SHAPE, "%s: bad sizes batch %lld, dim %lld", fn, (long long)batch,
                (long long)dim);
  if (!state || !x || !rgate || !igate || !A || !out)
    return fail(SSM_ERR_NULL, "%s: state, x, rgate, igate, A and out are required", fn);
  const size_t es = dtype == SSM_DTYPE_F32 ? 4 : 2;
  const struct { const void* p; size_t k; const char* n; } al[] = {
      {state, 4, "state"}, {x, es, "x"}, {rgate, es, "rgate"}, {igate, es, "igate"}, {z, es, "z"},
      {out, es, "out"}, {A, 4, "A"}, {rgate_bias, 4, "rgate_bias"}, {igate_bias, 4, "igate_bias"}};
  for (const auto& e : al)
    if (e.p && !aligned(e.p, e.k))
      return fail(SSM_ERR_ALIGN, "%s: %s is not %zu-byte aligned", fn, e.n, e.k);
  const size_t tok = static_cast<size_t>(batch) * dim * es, pd = static_cast<size_t>(dim) * 4;
  const Span ins[] = {{x, tok, "x"}, {rgate, tok, "rgate"}, {igate, tok, "igate"},
                      {z, z ? tok : 0, "z"}, {A, pd, "A"},
                      {rgate_bias, rgate_bias ? pd : 0, "rgate_bias"},
                      {igate_bias, igate_bias ? pd : 0, "igate_bias"}};
  const Span outs[] = {{out, tok, "out"}, {state, static_cast<size_t>(batch) * dim * 4, "state"}};
  for (const auto& o : outs)
    for (const auto& n : ins)
      if (overlap(o, n))
        return fail(SSM_ERR_ALIAS, "%s: %s overlaps input %s", fn, o.name, n.name);
  if (overlap(outs[0], outs[1])) return fail(SSM_ERR_ALIAS, "%s: out overlaps state", fn);
  const int64_t n = batch * dim;
  const auto go = [&](auto tag, auto lane) {
    using TA = decltype(tag);
    constexpr int V = decltype(lane)::value;
    const dim3 grid(static_cast<unsigned>((n / V + 255) / 256)), block(256);
    GatedStepArgs<TA> a{state, static_cast<const TA*>(x), static_cast<const TA*>(rgate),
                        static_cast<const TA*>(igate), static_cast<const TA*>(z), A, rgate_bias,
                        igate_bias, static_cast<TA*>(out), n, static_cast<int>(dim)};
    if (normalize)
      hipLaunchKernelGGL((gated_step_kernel<TA, V, true>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((gated_step_kernel<TA, V, false>), grid, block, 0, stream, a);
  };
  // two channels a lane where every row allows it (256 x 5120 float32: 8.0 us,
  // one 8.8, four 8.4; 1 x 2048 bf16: 2.5, 2.6, 2.5)
  constexpr int V = 2;
  bool wide = dim % V == 0;
  for (const auto& e : al) wide = wide && aligned(e.p, V * e.k);  // (a NULL is)
  if (dtype == SSM_DTYPE_F32)
    wide ? go(float{}, Lane<V>{}) : go(float{}, Lane<1>{});
  else
    wide ? go(bf16_t{}, Lane<V>{}) : go(bf16_t{}, Lane<1>{});
  return launch_status(fn);
}

}  // extern "C"
