// gated.hip -- the gated linear recurrence, forward and decode step, behind
// the C ABI in include/ssm_recurrent.h.
//
//   a_t = e^(A sigma(r_t + rb)),  h_t = a_t h_{t-1} + m_t sigma(i_t + ib) x_t
//   out_t = h_t silu(z_t)
//
#include "gated.hpp"
#include "host_util.hpp"

namespace ssm {

// Whether a call goes through the sequence without a time split.
bool gated_streams(int64_t rows, int64_t L, int64_t dim) {
  return dim <= (int64_t{1} << 20) && L > SSM_GATED_CHUNK && rows * ((dim + 31) / 32) >= 160;
}

// Ones into the published words, zero into the counter; empty sequences'
// states.  A grid-stride loop over each.
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

constexpr int kFwdT = 32, kFwdBatch = 8;
constexpr int kFwdWaves = 4;  // a chunk is 128 tokens

// One pass over the data: a workgroup loads its tokens once, turns them into
// (a, b) in registers and composes its chunk's map; publishes that; waits for
// the state that enters the chunk; and walks its tokens from there.  Chunks
// come in groups of kGatedGroup.  A chunk reads the maps of the chunks before
// it in its group, which exist as soon as those workgroups have read their
// data, and one state per group, which the last chunk of the group before
// hands on: the chain over the sequence is one step per 2048 tokens.  The
// folds have a fixed order, so results repeat bit for bit.
// Units are handed out by a counter, earlier chunks first: a workgroup waits
// only for ones that are running or done.
template <typename TA, int V, bool NORM, bool GATE, bool VL>
__global__ void __launch_bounds__(64 * kFwdWaves, 4) gated_fwd_kernel(GatedFwdArgs<TA> p, GatedPlan pl) {
  constexpr int T = kFwdT, W = kFwdWaves, C = 64 * V, kPolls = kGatedGroup / W;
  constexpr int kPerState = SSM_GATED_CHUNK / T;  // waves from one chunk state to the next
  using IO = Cell<TA, V>;
  __shared__ float2 s_agg[W][C];
  __shared__ float2 s_in[kGatedGroup][C];
  __shared__ float s_carry[C];
  __shared__ uint32_t s_turn;
  const int lane = threadIdx.x & 63;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int dim = p.dim;
  uint64_t* const agg = static_cast<uint64_t*>(p.ws);
  uint64_t* const carries = agg + pl.chunks * pl.cells;
  uint32_t unit = blockIdx.x;
  if (pl.chunks > 1) {
    if (threadIdx.x == 0)
      s_turn = atomicAdd(reinterpret_cast<uint32_t*>(carries + pl.groups * pl.cells), 1u);
    __syncthreads();
    unit = __builtin_amdgcn_readfirstlane(s_turn);
    if (unit >= pl.units) return;  // (a workspace that another call uses at the same time)
  }
  const uint32_t c = unit / pl.lines, line = unit % pl.lines;
  const uint32_t row = line / pl.tiles, tile = line % pl.tiles;
  const int col0 = static_cast<int>(tile) * C, col = col0 + lane * V;
  const bool have = col < dim;
  const int64_t t0 = static_cast<int64_t>(c) * (T * W) + w * T;
  int64_t end = p.L;
  if (VL) {
    const int64_t e = p.cu[p.nseq];
    end = e < 0 ? 0 : (e < end ? e : end);
  }
  const int n = end <= t0 ? 0 : (end - t0 < T ? static_cast<int>(end - t0) : T);  // the wave's tokens

  float a[V][T], b[V][T], y[V], H[V];  // y: first the sum of the tokens' v
  Marks mk{0, 0, 0};
  const uint32_t voff = have ? static_cast<uint32_t>(lane * V * sizeof(TA)) : kNoColumn;
  const uint32_t rowb = static_cast<uint32_t>(dim) * sizeof(TA);
  const int64_t base = (static_cast<int64_t>(row) * p.L + t0) * dim + col0;
  const uint32_t span = n > 0 ? (static_cast<uint32_t>(n) * rowb - col0 * static_cast<uint32_t>(sizeof(TA))) : 0;
  const uint32_t lastrow = n > 0 ? static_cast<uint32_t>(n - 1) * rowb : 0;
  const auto at = [&](int j) {  // rows behind the last are that one again
    const uint32_t o = static_cast<uint32_t>(j) * rowb;
    return o < lastrow ? o : lastrow;
  };
  constexpr int ZB = 16;  // rows of z in flight
  typename IO::raw_t zr[GATE ? ZB : 1];
  const rsrc_t rz = make_rsrc(GATE && n > 0 ? p.z + base : p.z, GATE ? span : 0);
#pragma unroll
  for (int v = 0; v < V; ++v) {
    y[v] = 0.0f;
    H[v] = 0.0f;
  }
  if (n > 0) {
    constexpr int NB = kFwdBatch;
    typename IO::raw_t xr[2][NB], rr[2][NB], ir[2][NB];
    const rsrc_t rx = make_rsrc(p.x + base, span), rg = make_rsrc(p.r + base, span),
                 ri = make_rsrc(p.i + base, span);
    const auto fetch = [&](int k) {
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        rr[k & 1][j] = IO::load(rg, voff, at(k * NB + j));
        ir[k & 1][j] = IO::load(ri, voff, at(k * NB + j));
        xr[k & 1][j] = IO::load(rx, voff, at(k * NB + j));
      }
    };
    fetch(0);
    fetch(1);
    if (VL) mk = find_marks(p.cu, static_cast<int>(p.nseq), t0, n);
    Params pr[V];
#pragma unroll
    for (int v = 0; v < V; ++v) pr[v] = load_params(p.A, p.rb, p.ib, col + v, have);
    // every token as if it were there (rows behind the last repeat it), y
    // over the n that are
#pragma unroll
    for (int k = 0; k < T / NB; ++k) {
#pragma unroll
      for (int jj = 0; jj < NB; ++jj) {
        const int j = k * NB + jj;
        const float there = j < n ? 1.0f : 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float d = pr[v].A2 * sigmoid2(__builtin_fmaf(IO::get(rr[k & 1][jj], v), -kLog2e, pr[v].rb2));
          float m;
          decay<NORM>(d, a[v][j], m);
          b[v][j] = m * sigmoid2(__builtin_fmaf(IO::get(ir[k & 1][jj], v), -kLog2e, pr[v].ib2)) *
                    IO::get(xr[k & 1][jj], v);
          y[v] = __builtin_fmaf(d, there, y[v]);
          H[v] = __builtin_fmaf(a[v][j], H[v], b[v][j]);
        }
        // a few tokens overlap; more would not fit the registers
        if ((j & 3) == 3) __builtin_amdgcn_sched_barrier(0);
      }
      if (k + 2 < T / NB) {
#pragma unroll
        for (int j = 0; j < NB; ++j) {
          rr[k & 1][j] = IO::load(rg, voff, at((k + 2) * NB + j));
          ir[k & 1][j] = IO::load(ri, voff, at((k + 2) * NB + j));
          xr[k & 1][j] = IO::load(rx, voff, at((k + 2) * NB + j));
        }
        __builtin_amdgcn_sched_barrier(0);
      }
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
            b[v][j] = 0.0f;
          }
          if (start && p.h0 && have) b[v][j] = __builtin_fmaf(a[v][j], p.h0[s * dim + col + v], b[v][j]);
          H[v] = start ? b[v][j] : __builtin_fmaf(a[v][j], H[v], b[v][j]);
        }
      }
    }
    if (GATE) {
#pragma unroll
      for (int j = 0; j < ZB; ++j) zr[j] = IO::load(rz, voff, at(j));
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) {
    y[v] = VL && mk.starts ? kCut : keep_of(y[v]);
    s_agg[w][lane * V + v] = make_float2(y[v], H[v]);
  }
  __syncthreads();
  // the map of the waves before this one; the last wave also the chunk's
  float yw[V], Hw[V], yt[V], Ht[V], h[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    yw[v] = -0.0f;
    Hw[v] = 0.0f;
  }
  for (int k = 0; k < w; ++k) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float2 f = s_agg[k][lane * V + v];
      compose<VL>(yw[v], Hw[v], f.x, f.y);
    }
  }
  const int64_t cell = static_cast<int64_t>(line) * C + lane * V;
  if (w == W - 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      yt[v] = yw[v];
      Ht[v] = Hw[v];
      compose<VL>(yt[v], Ht[v], y[v], H[v]);
      if (c + 1 < pl.chunks) publish(agg + c * pl.cells + cell + v, yt[v], Ht[v]);
    }
  }
  // the state that enters the chunk
  if (c == 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = !VL && p.h0 && have ? p.h0[static_cast<int64_t>(row) * dim + col + v] : 0.0f;
  } else {
    const uint32_t first = c / kGatedGroup * kGatedGroup;
    const int there = static_cast<int>(c - first);  // chunks of the group before this one
    {
      float lo[kPolls][V], hi[kPolls][V];
      const int polls = there > w ? (there - w + W - 1) / W : 0;  // chunks w, w + W, ...
      if (polls > 0)
        await<V>(agg + (first + w) * pl.cells + cell, W * pl.cells, polls, lo, hi);
#pragma unroll
      for (int k = 0; k < kPolls; ++k) {
        if (k < polls) {
#pragma unroll
          for (int v = 0; v < V; ++v) s_in[w + k * W][lane * V + v] = make_float2(lo[k][v], hi[k][v]);
        }
      }
    }
    if (w == W - 1) {
      float lo[1][V], hi[1][V];
      if (first > 0) {
        await<V>(carries + c / kGatedGroup * pl.cells + cell, 0, 1, lo, hi);
      } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
          hi[0][v] = !VL && p.h0 && have ? p.h0[static_cast<int64_t>(row) * dim + col + v] : 0.0f;
      }
#pragma unroll
      for (int v = 0; v < V; ++v) s_carry[lane * V + v] = hi[0][v];
    }
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v) h[v] = s_carry[lane * V + v];
    for (int j = 0; j < there; ++j) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float2 f = s_in[j][lane * V + v];
        h[v] = pass<VL>(f.x, f.y, h[v]);
      }
    }
  }
  if (w == W - 1 && (c + 1) % kGatedGroup == 0 && c + 1 < pl.chunks) {
#pragma unroll
    for (int v = 0; v < V; ++v)
      publish(carries + (c + 1) / kGatedGroup * pl.cells + cell + v, 0.0f, pass<VL>(yt[v], Ht[v], h[v]));
  }
#pragma unroll
  for (int v = 0; v < V; ++v) h[v] = pass<VL>(yw[v], Hw[v], h[v]);
  if (w % kPerState == 0 && p.chunk_states && have && t0 < p.L) {
    const int64_t states = (p.L + SSM_GATED_CHUNK - 1) / SSM_GATED_CHUNK;
#pragma unroll
    for (int v = 0; v < V; ++v)
      p.chunk_states[(row * states + t0 / SSM_GATED_CHUNK) * dim + col + v] = h[v];
  }
  if (n > 0 && p.out) {  // (without out: the chunks' states alone)
    const rsrc_t ro = make_rsrc(p.out + base, span);
    const auto emit = [&](int j) {
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) o[v] = GATE ? h[v] * silu_f32(IO::get(zr[GATE ? j % ZB : 0], v)) : h[v];
      if (GATE && j + ZB < T) zr[j % ZB] = IO::load(rz, voff, at(j + ZB));
      IO::store(ro, o, voff, static_cast<uint32_t>(j) * rowb);
    };
    if (n == T && (!VL || !(mk.starts | mk.ends))) {
#pragma unroll
      for (int j = 0; j < T; ++j) {
#pragma unroll
        for (int v = 0; v < V; ++v) h[v] = __builtin_fmaf(a[v][j], h[v], b[v][j]);
        emit(j);
      }
    } else {
#pragma unroll
      for (int j = 0; j < T; ++j) {
        if (j < n) {
#pragma unroll
          for (int v = 0; v < V; ++v)
            h[v] = VL && (mk.starts >> j & 1) ? b[v][j] : __builtin_fmaf(a[v][j], h[v], b[v][j]);
          emit(j);
          if (VL && p.last && (mk.ends >> j & 1) && have) {
            const int64_t s = __builtin_amdgcn_readlane(mk.seq, j);
#pragma unroll
            for (int v = 0; v < V; ++v) p.last[s * dim + col + v] = h[v];
          }
        }
      }
    }
  }
  if (!VL && p.last && c + 1 == pl.chunks && w == W - 1 && have && p.L > 0) {
#pragma unroll
    for (int v = 0; v < V; ++v) p.last[static_cast<int64_t>(row) * dim + col + v] = h[v];
  }
}

// The walk without a time split, for calls whose channels fill the device: a
// workgroup takes 32 channels of one row through the whole sequence, 512
// tokens a turn.  A wave's lanes are 32 channels and two stretches of 32
// tokens, so a row access is 64 bytes (bf16) and the other half of the line
// belongs to the next workgroup, which runs on the same XCD.  The state goes
// from turn to turn through LDS, one barrier a turn; nothing is handed between
// workgroups, and there is no workspace and no second launch.  The next turn's
// inputs are loaded into registers as this turn's are used up (a wave has all
// 256 registers: one workgroup fits a CU).
constexpr int kStreamT = 32, kStreamC = 32, kStreamWaves = 8;
constexpr int kStreamTurn = kStreamWaves * 64 / kStreamC * kStreamT;  // tokens
constexpr int kXcds = 8;  // workgroups are dealt to the XCDs in turn

template <typename TA, bool NORM, bool GATE>
__global__ void __launch_bounds__(64 * kStreamWaves, 2)
    gated_stream_kernel(GatedFwdArgs<TA> p, uint32_t tiles, uint32_t units) {
  constexpr int T = kStreamT, C = kStreamC, W = kStreamWaves, NB = 8;
  using IO = Cell<TA, 1>;
  __shared__ float2 s_map[2][2 * W][C];
  __shared__ float s_carry[2][C];
  static_assert(SSM_GATED_CHUNK == 2 * T, "a wave starts where a chunk state is kept");
  const uint32_t unit = blockIdx.x % kXcds * (gridDim.x / kXcds) + blockIdx.x / kXcds;
  if (unit >= units) return;
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane % C, seg = lane / C;
  const uint32_t row = unit / tiles, tile = unit % tiles;
  const int dim = p.dim, col0 = static_cast<int>(tile) * C, col = col0 + c;
  const bool have = col < dim;
  const uint32_t rowb = static_cast<uint32_t>(dim) * sizeof(TA);
  const uint32_t voff = have ? seg * T * rowb + c * static_cast<uint32_t>(sizeof(TA)) : kNoColumn;
  const Params pr = load_params(p.A, p.rb, p.ib, col, have);
  const int turns = static_cast<int>((p.L + kStreamTurn - 1) / kStreamTurn);
  const int64_t states = (p.L + SSM_GATED_CHUNK - 1) / SSM_GATED_CHUNK;

  // a wave's rows of one turn: [t0, t0 + n), n <= 64, from its column on
  struct Rows {
    int64_t t0, base;
    int n;
    uint32_t span;
  };
  const auto rows_of = [&](int turn) {
    Rows r;
    r.t0 = static_cast<int64_t>(turn) * kStreamTurn + w * (2 * T);
    const int64_t left = p.L - r.t0;
    r.n = left <= 0 ? 0 : (left < 2 * T ? static_cast<int>(left) : 2 * T);
    r.base = r.n > 0 ? (static_cast<int64_t>(row) * p.L + r.t0) * dim + col0 : 0;
    r.span = r.n > 0 ? r.n * rowb - col0 * static_cast<uint32_t>(sizeof(TA)) : 0;
    return r;
  };
  // (the scalar offset stays inside the span; what is behind it reads as 0)
  const auto at = [&](const Rows& r, int j) { return static_cast<uint32_t>(j < r.n ? j : (r.n > 0 ? r.n - 1 : 0)) * rowb; };

  typename IO::raw_t xr[T], rr[T], ir[T], zr[GATE ? T : 1];
  Rows now = rows_of(0);
  {
    const rsrc_t rx = make_rsrc(p.x + now.base, now.span), rg = make_rsrc(p.r + now.base, now.span),
                 ri = make_rsrc(p.i + now.base, now.span);
#pragma unroll
    for (int j = 0; j < T; ++j) {
      rr[j] = IO::load(rg, voff, at(now, j));
      ir[j] = IO::load(ri, voff, at(now, j));
      xr[j] = IO::load(rx, voff, at(now, j));
    }
  }
  if (threadIdx.x < C) s_carry[0][c] = p.h0 && have ? p.h0[static_cast<int64_t>(row) * dim + col] : 0.0f;
  for (int turn = 0; turn < turns; ++turn) {
    const Rows next = rows_of(turn + 1);
    if (GATE) {
      const rsrc_t rz = make_rsrc(p.z + now.base, now.span);
#pragma unroll
      for (int j = 0; j < T; ++j) zr[j] = IO::load(rz, voff, at(now, j));
    }
    const rsrc_t rx = make_rsrc(p.x + next.base, next.span), rg = make_rsrc(p.r + next.base, next.span),
                 ri = make_rsrc(p.i + next.base, next.span);
    // Tokens behind the row's end take part with what they read: only
    // stretches behind them would see it, and those have no token.
    float a[T], b[T], y = 0.0f, H = 0.0f;
#pragma unroll
    for (int k = 0; k < T / NB; ++k) {
#pragma unroll
      for (int jj = 0; jj < NB; ++jj) {
        const int j = k * NB + jj;
        const float d = pr.A2 * sigmoid2(__builtin_fmaf(IO::get(rr[j], 0), -kLog2e, pr.rb2));
        float m;
        decay<NORM>(d, a[j], m);
        b[j] = m * sigmoid2(__builtin_fmaf(IO::get(ir[j], 0), -kLog2e, pr.ib2)) * IO::get(xr[j], 0);
        y += d;
        H = __builtin_fmaf(a[j], H, b[j]);
      }
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int jj = 0; jj < NB; ++jj) {
        const int j = k * NB + jj;
        rr[j] = IO::load(rg, voff, at(next, j));
        ir[j] = IO::load(ri, voff, at(next, j));
        xr[j] = IO::load(rx, voff, at(next, j));
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    s_map[turn & 1][2 * w + seg][c] = make_float2(keep_of(y), H);
    __syncthreads();
    float h = s_carry[turn & 1][c];
#pragma unroll 4
    for (int k = 0; k < 2 * w; ++k) {
      const float2 f = s_map[turn & 1][k][c];
      h = pass<false>(f.x, f.y, h);
    }
    if (seg) {
      const float2 f = s_map[turn & 1][2 * w][c];
      h = pass<false>(f.x, f.y, h);
    }
    if (p.chunk_states && seg == 0 && have && now.n > 0)
      p.chunk_states[(row * states + now.t0 / SSM_GATED_CHUNK) * dim + col] = h;
    // (without out, for the states alone, every store is out of range)
    const rsrc_t ro = make_rsrc(p.out + now.base, p.out ? now.span : 0);
    const uint32_t outb = p.out ? rowb : 0;
    if (now.n == 2 * T) {
#pragma unroll
      for (int j = 0; j < T; ++j) {
        h = __builtin_fmaf(a[j], h, b[j]);
        const float o[1] = {GATE ? h * silu_f32(IO::get(zr[GATE ? j : 0], 0)) : h};
        IO::store(ro, o, voff, static_cast<uint32_t>(j) * outb);
      }
    } else {
      const int mine = now.n - seg * T;  // tokens of this lane's stretch
#pragma unroll
      for (int j = 0; j < T; ++j) {
        if (j < now.n) {
          const float g = __builtin_fmaf(a[j], h, b[j]);
          h = j < mine ? g : h;
          const float o[1] = {GATE ? g * silu_f32(IO::get(zr[GATE ? j : 0], 0)) : g};
          IO::store(ro, o, voff, static_cast<uint32_t>(j) * outb);  // (dropped behind the last row)
        }
      }
    }
    // the row's last token is this lane's last one
    if (p.last && have && now.t0 + seg * T < p.L && now.t0 + seg * T + T >= p.L)
      p.last[static_cast<int64_t>(row) * dim + col] = h;
    if (w == W - 1 && seg == 1) s_carry[(turn + 1) & 1][c] = h;
    now = next;
  }
}

template <typename TA, int V>
int launch_gated_fwd(const GatedFwdArgs<TA>& a, bool norm, const char* fn, hipStream_t s) {
  if (!a.cu && a.L > 0 && gated_streams(a.rows, a.L, a.dim)) {
    const uint32_t tiles = (a.dim + kStreamC - 1) / kStreamC;
    const uint32_t units = static_cast<uint32_t>(a.rows * tiles);
    const dim3 grid((units + kXcds - 1) / kXcds * kXcds), block(64 * kStreamWaves);
#define SSM_GATED_CASE(N, G)                                                                  \
  if (norm == N && (a.z != nullptr) == G)                                                      \
    hipLaunchKernelGGL((gated_stream_kernel<TA, N, G>), grid, block, 0, s, a, tiles, units);
    SSM_GATED_CASE(true, true)
    SSM_GATED_CASE(true, false)
    SSM_GATED_CASE(false, true)
    SSM_GATED_CASE(false, false)
#undef SSM_GATED_CASE
    return launch_status(fn);
  }
  const GatedPlan pl = gated_plan(a.rows, a.L, a.dim, V, kFwdWaves * kFwdT);
  const int rc = launch_gated_init(a.ws, pl.bytes, a.cu, a.cu ? a.nseq : a.rows, a.L, a.dim, a.h0, a.last,
                                   fn, s);
  if (rc != SSM_OK || a.L == 0) return rc;
  const dim3 grid(static_cast<unsigned>(pl.units)), block(64 * kFwdWaves);
#define SSM_GATED_CASE(N, G, VLN)                                                              \
  if (norm == N && (a.z != nullptr) == G && (a.cu != nullptr) == VLN)                          \
    hipLaunchKernelGGL((gated_fwd_kernel<TA, V, N, G, VLN>), grid, block, 0, s, a, pl);
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

// One lane per (sequence, channel).
template <typename TA, bool NORM>
__global__ void __launch_bounds__(256) gated_step_kernel(GatedStepArgs<TA> p) {
  const int64_t o = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (o >= p.n) return;
  const int c = static_cast<int>(o % p.dim);
  float a, m;
  const Params pr = load_params(p.A, p.rb, p.ib, c, true);
  decay<NORM>(pr.A2 * sigmoid2(__builtin_fmaf(to_f32(p.r[o]), -kLog2e, pr.rb2)), a, m);
  const float u = sigmoid2(__builtin_fmaf(to_f32(p.i[o]), -kLog2e, pr.ib2));
  const float h = __builtin_fmaf(a, p.state[o], m * u * to_f32(p.x[o]));
  p.state[o] = h;
  store_act(p.out + o, p.z ? h * silu_f32(to_f32(p.z[o])) : h);
}

constexpr int64_t kGatedMaxDim = int64_t{1} << 24;
constexpr int64_t kGatedMaxSeqs = int64_t{1} << 24;

// Whether batch, seqlen (or nseq, total_len) and dim can be launched.
bool gated_sizes_ok(int64_t rows, int64_t L, int64_t nseq, int64_t dim, bool packed) {
  if (dim < 1 || dim > kGatedMaxDim || L < 0 || L > (int64_t{1} << 40) / dim) return false;
  if (packed ? (nseq < 1 || nseq >= kGatedMaxSeqs) : (rows < 1 || rows > 65535)) return false;
  // one launch: a workgroup per chunk and tile of at least 64 channels
  return rows * ((L + SSM_GATED_CHUNK - 1) / SSM_GATED_CHUNK) * ((dim + 63) / 64) < (int64_t{1} << 31);
}

// Workspace of a time-split walk: for the narrowest tiles and the shortest
// chunks a call may take.
size_t gated_walk_bytes(int64_t rows, int64_t L, int64_t dim) {
  size_t most = 0;
  for (int V = 1; V <= 2; ++V) {
    const size_t b = gated_plan(rows, L, dim, V, SSM_GATED_CHUNK).bytes;
    most = b > most ? b : most;
  }
  return most;
}

// The forward's launch for either type; bf16 with two channels a lane where
// every row starts on four bytes.
template <typename TA>
int run_gated_fwd(const char* fn, const void* x, const void* r, const void* i, const float* A,
                  const float* rb, const float* ib, bool norm, const void* z, void* out, float* last,
                  const float* h0, float* states, const int32_t* cu, int64_t nseq, int64_t rows,
                  int64_t L, int dim, void* ws, hipStream_t stream) {
  const GatedFwdArgs<TA> a{static_cast<const TA*>(x), static_cast<const TA*>(r),
                           static_cast<const TA*>(i), static_cast<const TA*>(z), A, rb, ib,
                           static_cast<TA*>(out), last, h0, states, cu, rows, L, nseq, dim, ws};
  if constexpr (sizeof(TA) == 2) {
    if (dim % 2 == 0 && aligned(x, 4) && aligned(r, 4) && aligned(i, 4) && aligned(z, 4) && aligned(out, 4))
      return launch_gated_fwd<TA, 1>(a, norm, fn, stream);
  }
  return launch_gated_fwd<TA, 1>(a, norm, fn, stream);
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
  const size_t need = gated_walk_bytes(rows, L, dim);
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
  return gated_walk_bytes(batch, seqlen, dim);
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
  return gated_walk_bytes(1, total_len, dim);
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
  const dim3 grid(static_cast<unsigned>((n + 255) / 256)), block(256);
  const auto go = [&](auto tag) {
    using TA = decltype(tag);
    GatedStepArgs<TA> a{state, static_cast<const TA*>(x), static_cast<const TA*>(rgate),
                        static_cast<const TA*>(igate), static_cast<const TA*>(z), A, rgate_bias,
                        igate_bias, static_cast<TA*>(out), n, static_cast<int>(dim)};
    if (normalize)
      hipLaunchKernelGGL((gated_step_kernel<TA, true>), grid, block, 0, stream, a);
    else
      hipLaunchKernelGGL((gated_step_kernel<TA, false>), grid, block, 0, stream, a);
  };
  if (dtype == SSM_DTYPE_F32)
    go(float{});
  else
    go(bf16_t{});
  return launch_status(fn);
}

}  // extern "C"
