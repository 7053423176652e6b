"""Infinite states, inputs and gradients through the gated recurrence's maps:
an infinity stays one across the borders of waves, chunks, groups of chunks
and padding, as it does token by token (GPU)."""
import numpy as np
import pytest
import torch

import selective_state_space_31_amd as pkg
from oracle import gated as og
from tests import _gated_bound as gb
from tests._recurrent import Gated, np64, within

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
INF = float("inf")
# few workgroups and many (short and long stretches); rows that end inside a wave; more than one group of chunks
SHAPES = [(1, 1, 3), (2, 40, 5), (2, 700, 5), (1, 9001, 4), (300, 301, 66)]


def same_class(got, ref, what):
    """Finite, NaN, +inf and -inf in the same places."""
    got = np64(got)
    for name, f in (("NaN", np.isnan), ("+inf", np.isposinf), ("-inf", np.isneginf)):
        assert np.array_equal(f(got), f(ref)), "%s: %s in %d places, expected %d" % (
            what, name, f(got).sum(), f(ref).sum())


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("b,L,d", SHAPES)
def test_infinite_states_and_inputs(b, L, d, gate, dtype):
    p = Gated((b, L), b, d, dtype, DEV, 31, gate=gate)
    p.h0[0, 0], p.h0[-1, 1] = INF, -INF
    p.x[0, L // 3, 2] = INF
    if d > 3:
        p.h0[0, 3], p.x[0, L - 1, 3] = INF, -INF  # inf - inf at the last token
    out, last, mid = pkg.ssm_gated_scan_fwd(*p.args(), return_last_state=True, return_chunk_states=True, **p.kw())
    h, _, _ = p.host()
    with np.errstate(invalid="ignore"):
        ref, rl, H = og.gated_scan(**h)
        bo, bl, bs, _ = gb.forward(**h, dtype=dtype)
    rm = H[:, 0:L:pkg.SSM_GATED_CHUNK]
    for got, want, bound, what in ((out, ref, bo, "out"), (last, rl, bl, "last"),
                                   (mid, rm, bs[:, 0:L:pkg.SSM_GATED_CHUNK], "chunk_states")):
        same_class(got, want, what)
        within(got, want, bound, what)


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("d", [5, 2500])
def test_packed(d, dtype):
    lengths = [200, 0, 1500, 33, 1, 700]
    cu = np.concatenate([[0], np.cumsum(lengths)])
    T = int(cu[-1])
    p = Gated((T,), len(lengths), d, dtype, DEV, 32)
    p.h0[0, 0], p.h0[2, 1], p.h0[3, 1], p.h0[1, 2] = INF, -INF, INF, INF
    p.x[cu[2] + 700, 2] = -INF
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    out, last = pkg.ssm_gated_scan_fwd_varlen(*p.args(), cut, return_last_state=True, **p.kw())
    out, last = out[:, :5].contiguous(), last[:, :5].contiguous()
    for k in ("x", "r", "i", "z", "dout", "A", "rb", "ib", "h0", "dlast"):
        setattr(p, k, getattr(p, k)[..., :5].contiguous())
    for s in range(len(lengths)):
        h, _, _ = p.host(s, cu[s], cu[s + 1])
        with np.errstate(invalid="ignore"):
            ref, rl, _ = og.gated_scan(**h)
        same_class(out[None, cu[s]:cu[s + 1]], ref, "out %d" % s)
        same_class(last[s:s + 1], rl, "last %d" % s)


@pytest.mark.parametrize("b,L,d", SHAPES)
def test_infinite_gradients(b, L, d):
    """An infinite gradient reaches every token before it, as an infinity."""
    p = Gated((b, L), b, d, "fp32", DEV, 33)
    p.dlast[0, 0] = INF
    p.dout[0, L - 1 - L // 3, 1] = -INF
    g = pkg.ssm_gated_scan_bwd(*p.args(), p.dout, dlast_state=p.dlast, **p.kw())
    h, dout, dl = p.host()
    with np.errstate(invalid="ignore"):
        ref = og.gated_scan_bwd(dout=dout, dlast=dl, **h)
        bound = gb.backward(dout=dout, dlast=dl, **h)
    for k in ("dx", "digate", "dz", "dinitial_state"):
        same_class(g[k], ref[k], k)
    for k in ref:
        within(g[k], ref[k], bound[k], k)


@pytest.mark.parametrize("b,L,d", SHAPES)
def test_gradients_at_infinite_states(b, L, d):
    """dx, digate and the state's gradient do not depend on the state; the
    decay's gradient and dz do, and are not finite there."""
    p = Gated((b, L), b, d, "fp32", DEV, 34)
    want = pkg.ssm_gated_scan_bwd(*p.args(), p.dout, dlast_state=p.dlast, **p.kw())
    p.h0[0, 0], p.h0[-1, 1] = INF, -INF
    g = pkg.ssm_gated_scan_bwd(*p.args(), p.dout, dlast_state=p.dlast, **p.kw())
    for k in ("dx", "digate", "digate_bias", "dinitial_state"):
        assert torch.equal(g[k], want[k]), k
    for k in ("drgate", "dz"):
        bad = ~torch.isfinite(g[k])
        assert bad[0, :, 0].all() and bad[-1, :, 1].all() and int(bad.sum()) == 2 * L, k
        assert torch.equal(g[k][~bad], want[k][~bad]), k
    for k in ("dA", "drgate_bias"):
        assert not torch.isfinite(g[k][:2]).any() and torch.equal(g[k][2:], want[k][2:]), k


def test_step_is_the_scan_of_one_token():
    p = Gated((3,), 3, 5, "fp32", DEV, 35)
    p.h0[0, 0], p.h0[1, 1], p.x[2, 2] = INF, -INF, INF
    state = p.h0.clone()
    kw = {k: v for k, v in p.kw().items() if k != "initial_state"}
    one = pkg.ssm_gated_state_update(state, *p.args(), **kw)
    kw["z"] = p.z[:, None]
    out, last = pkg.ssm_gated_scan_fwd(p.x[:, None], p.r[:, None], p.i[:, None], p.A, initial_state=p.h0,
                                       return_last_state=True, **kw)
    same_class(out[:, 0], np64(one), "out")
    same_class(last, np64(state), "state")
    assert int(torch.isinf(state).sum()) == 3
