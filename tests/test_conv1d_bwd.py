"""The causal convolution's gradients on the GPU against float64."""
import numpy as np
import pytest
import torch

import selective_state_space_31_amd as pkg
from oracle import conv_bwd as oc
from tests._recurrent import DT, act, f32, np64, within

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E = 2.0 ** -24
BF16 = 2.0 ** -8


class Case:
    def __init__(self, b, L, d, W, dtype, seed, silu=True, bias=True, state=True, dfinal=True):
        rng = np.random.default_rng(seed)
        self.dtype, self.silu = dtype, silu
        self.x, self.dout = act(rng, (b, L, d), dtype, DEV), act(rng, (b, L, d), dtype, DEV)
        self.w = f32(rng, (d, W), DEV, W ** -0.5)
        self.bias = f32(rng, (d,), DEV, 0.5) if bias else None
        self.state = act(rng, (b, d, W - 1), dtype, DEV) if state else None
        self.dfinal = act(rng, (b, d, W - 1), dtype, DEV) if dfinal else None

    def args(self):
        return (self.x, self.w, self.dout)

    def kw(self):
        return dict(bias=self.bias, initial_conv_state=self.state, dfinal_conv_state=self.dfinal, silu=self.silu)


def check(c, g):
    """pre: W products and additions, (W + 1) e of the absolute terms P; silu'
    has slope at most 1/2, and its own roundings are (4|pre| + 16) e of its
    absolute terms; d = dout silu'.  dxx: W products of d, (W + 2) e more;
    sums over tokens add (chunk of 128 + chunks + a few) e of the terms."""
    x, w, dout = np64(c.x), np64(c.w), np64(c.dout)
    b, L, d = x.shape
    W = w.shape[1]
    ref = oc.conv1d_bwd(x, w, np64(c.bias), dout, c.silu, np64(c.state), np64(c.dfinal))
    before = np.zeros((b, W - 1, d)) if c.state is None else np64(c.state).transpose(0, 2, 1)
    xx = np.concatenate([before, x], 1)
    bias = 0.0 if c.bias is None else np64(c.bias)
    pre = np.zeros((b, L, d)) + bias
    P = np.zeros((b, L, d)) + np.abs(bias)
    for k in range(W):
        pre += w[:, k] * xx[:, k:k + L]
        P += np.abs(w[:, k] * xx[:, k:k + L])
    mag, err = np.abs(dout), np.abs(dout) * 0
    if c.silu:
        s = 1 / (1 + np.exp(-pre))
        sl = s * (1 + np.abs(pre) * (1 - s))
        err = np.abs(dout) * (0.5 * (W + 1) * E * P + sl * (4 * np.abs(pre) + 16) * E)
        mag = np.abs(dout) * sl
    dm, de = np.zeros_like(xx), np.zeros_like(xx)
    dw, db = {}, (mag.sum((0, 1)), err.sum((0, 1)))
    for k in range(W):
        dm[:, k:k + L] += np.abs(w[:, k]) * mag
        de[:, k:k + L] += np.abs(w[:, k]) * err
        dw[k] = ((mag * np.abs(xx[:, k:k + L])).sum((0, 1)), (err * np.abs(xx[:, k:k + L])).sum((0, 1)))
    if c.dfinal is not None:
        dm[:, L:] += np.abs(np64(c.dfinal)).transpose(0, 2, 1)
    bound = 2 * (de + dm * (W + 2) * E) + 1e-30
    steps = (128 + 8 + b * (L // 128 + 2)) * E

    def cast(bd, rf):
        return bd + BF16 * (np.abs(rf) + bd) if c.dtype == "bf16" else bd
    within(g["dx"], ref["dx"], cast(bound[:, W - 1:], ref["dx"]), "dx")
    if c.state is not None:
        within(g["dinitial_conv_state"], ref["dinitial_conv_state"],
               cast(bound[:, :W - 1].transpose(0, 2, 1), ref["dinitial_conv_state"]), "dstate")
    for k in range(W):
        within(g["dweight"][:, k], ref["dweight"][:, k], 2 * dw[k][1] + steps * dw[k][0] + 1e-30, "dw%d" % k)
    if c.bias is not None:
        within(g["dbias"], ref["dbias"], 2 * db[1] + steps * db[0] + 1e-30, "dbias")


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("b,L,d", [(1, 1, 1), (2, 2, 5), (1, 3, 64), (3, 16, 66), (2, 33, 130), (1, 257, 64),
                                   (2, 1030, 70)])
def test_gradients(b, L, d, W, dtype):
    c = Case(b, L, d, W, dtype, b + L + d + W)
    check(c, pkg.ssm_causal_conv1d_bwd(*c.args(), **c.kw()))


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("silu,bias,state,dfinal", [(False, True, True, True), (True, False, False, False),
                                                    (True, True, False, True), (False, False, True, False)])
def test_optional_parts(silu, bias, state, dfinal, dtype):
    c = Case(2, 150, 64, 4, dtype, 3, silu, bias, state, dfinal)
    check(c, pkg.ssm_causal_conv1d_bwd(*c.args(), **c.kw()))


def test_empty_sequence():
    c = Case(2, 0, 66, 4, "fp32", 4)
    g = pkg.ssm_causal_conv1d_bwd(*c.args(), **c.kw())
    assert torch.equal(g["dinitial_conv_state"], c.dfinal)  # the state passes through unchanged
    assert not g["dweight"].any() and not g["dbias"].any()


def test_infinite_input_at_the_end():
    """Without SiLU an infinite last input gives infinite weight gradients,
    not NaN from the tokens behind the sequence."""
    for L in (7, 32, 40):
        c = Case(1, L, 64, 4, "fp32", 8, silu=False, state=False, dfinal=False)
        c.x[0, L - 1, 5] = float("inf")
        c.dout[:] = 1.0
        g = pkg.ssm_causal_conv1d_bwd(*c.args(), **c.kw())
        assert torch.isinf(g["dweight"][5, 3]) and torch.isfinite(g["dweight"][5, :3]).all()
        assert torch.isfinite(g["dx"]).all()


def test_large_inputs_and_nan():
    """Pre-activations past where the logistic function saturates, and a NaN
    that reaches only its own neighbourhood and channel."""
    c = Case(1, 100, 64, 4, "fp32", 5)
    c.x *= 200.0
    check(c, pkg.ssm_causal_conv1d_bwd(*c.args(), **c.kw()))
    base = pkg.ssm_causal_conv1d_bwd(*c.args(), **c.kw())
    c.x[0, 50, 7] = float("nan")
    g = pkg.ssm_causal_conv1d_bwd(*c.args(), **c.kw())
    bad = torch.isnan(g["dx"])
    assert bad[0, 47:54, 7].all() and int(bad.sum()) == 7
    assert torch.equal(g["dx"][~bad], base["dx"][~bad])
    assert torch.isnan(g["dweight"][7]).all() and int(torch.isnan(g["dweight"]).sum()) == 4


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("off", [0, 1])
def test_writes_stay_in_their_buffers(dtype, off):
    c = Case(2, 77, 66, 4, dtype, 6)
    bufs = []

    def shift(t):
        flat = torch.full((t.numel() + 128,), 5.0, dtype=t.dtype, device=DEV)
        v = flat[64 + off:64 + off + t.numel()].view(t.shape)
        v.copy_(t)
        bufs.append((flat, v))
        return v
    c.x, c.dout, c.state, c.dfinal = (shift(t) for t in (c.x, c.dout, c.state, c.dfinal))
    g = dict(dx=shift(c.x), dweight=shift(c.w), dbias=shift(c.bias), dinitial_conv_state=shift(c.state))
    pkg.ssm_causal_conv1d_bwd(*c.args(), grads=g, **c.kw())
    check(c, g)
    for flat, v in bufs:
        keep = torch.ones(flat.numel(), dtype=torch.bool, device=DEV)
        keep[64 + off:64 + off + v.numel()] = False
        assert (flat[keep] == 5.0).all()


def test_repeats_bit_for_bit_and_captured():
    c = Case(2, 3000, 200, 4, "bf16", 7)
    run = lambda: [v for _, v in sorted(pkg.ssm_causal_conv1d_bwd(*c.args(), **c.kw()).items())]
    want = run()
    assert all(torch.equal(a, b) for a, b in zip(run(), want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        run()
        torch.cuda.synchronize()
    assert got[-1].dtype == DT["bf16"] or got[-1].dtype == torch.float32


def test_more_workgroups_than_a_grid_row():
    """65535 one-token sequences of so many channels that the threads of one
    grid row would pass 32 bits; every sequence has the same inputs."""
    d = 16447
    c = Case(1, 1, d, 2, "bf16", 31)
    want = pkg.ssm_causal_conv1d_bwd(*c.args(), **c.kw())
    many = lambda t: t.expand((65535,) + t.shape[1:]).contiguous()
    g = pkg.ssm_causal_conv1d_bwd(many(c.x), c.w, many(c.dout), bias=c.bias, initial_conv_state=many(c.state),
                                  dfinal_conv_state=many(c.dfinal), silu=c.silu)
    assert bool((g["dx"] == want["dx"]).all())
    assert bool((g["dinitial_conv_state"] == want["dinitial_conv_state"]).all())
    for k in ("dweight", "dbias"):  # sums of equal values: a relative 65535 2^-24 at most
        torch.testing.assert_close(g[k], want[k] * 65535.0, rtol=65535 * 2.0 ** -24, atol=0)
