"""The gated recurrence with A > 0, where decays are factors above 1 (GPU)."""
import numpy as np
import pytest
import torch

import selective_state_space_31_amd as pkg
from oracle import gated as og
from tests import _gated_bound as gb
from tests._recurrent import Gated, np64, within

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
GRADS = ("dx", "drgate", "digate", "dz", "dA", "drgate_bias", "digate_bias", "dinitial_state")


def growing(lead, n, d, A, dtype="fp32", seed=41, **kw):
    p = Gated(lead, n, d, dtype, DEV, seed, bias=False, **kw)
    p.r.mul_(0.1)
    p.A.fill_(A)
    return p


@pytest.mark.parametrize("b,L,d", [(2, 700, 5), (1, 9001, 3), (300, 301, 66)])
def test_zero_states_stay_zero(b, L, d):
    """With normalize nothing enters (m = 0): all zeros, however large the
    product of the factors gets."""
    p = growing((b, L), b, d, 1.0, state=False)
    out, last, mid = pkg.ssm_gated_scan_fwd(*p.args(), return_last_state=True, return_chunk_states=True, **p.kw())
    assert not out.any() and not last.any() and not mid.any()


@pytest.mark.parametrize("b,L,d", [(2, 700, 5), (1, 3001, 3)])
def test_zero_gradients_stay_zero(b, L, d):
    """Nothing comes from behind the first tokens: the adjoint is 0 there,
    however large the product of the factors is, and grows in front."""
    p = growing((b, L), b, d, 3.0, state=False, dlast=False)
    p.dout[:, 40:] = 0.0
    g = pkg.ssm_gated_scan_bwd(*p.args(), p.dout, **p.kw())
    h, dout, dl = p.host()
    ref, bound = og.gated_scan_bwd(dout=dout, dlast=dl, **h), gb.backward(dout=dout, dlast=dl, **h)
    for k in GRADS:
        within(g[k], ref[k], bound[k], k)
    assert not g["dinitial_state"].eq(0).any()


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("b,L,d,A", [(2, 290, 70, 1.0), (300, 290, 66, 1.0), (2, 90, 70, 3.0), (300, 90, 66, 3.0)])
def test_states_in_range_behind_products_that_are_not(b, L, d, A, normalize):
    """A small state times a product beyond float32: e^(A L / 2) 10^-30."""
    p = growing((b, L), b, d, A, normalize=normalize, gate=False)
    p.h0.mul_(1e-30)
    p.x.mul_(1e-30)
    out, last = pkg.ssm_gated_scan_fwd(*p.args(), return_last_state=True, **p.kw())
    h, _, _ = p.host()
    ref, rl, _ = og.gated_scan(**h)
    bo, bl, _, _ = gb.forward(**h)
    assert np.abs(ref).max() < 1e37
    within(out, ref, bo, "out")
    within(last, rl, bl, "last")


@pytest.mark.parametrize("b", [2, 40])
def test_gradients_in_range_behind_products_that_are_not(b):
    """The same with the adjoint: e^130 10^-30 over a chunk of 128 tokens and
    two more."""
    p = growing((b, 130), b, 70, 2.0, normalize=False, gate=False)
    for t in (p.h0, p.x, p.dlast, p.dout):
        t.mul_(1e-30)
    g = pkg.ssm_gated_scan_bwd(*p.args(), p.dout, dlast_state=p.dlast, **p.kw())
    h, dout, dl = p.host()
    ref, bound = og.gated_scan_bwd(dout=dout, dlast=dl, **h), gb.backward(dout=dout, dlast=dl, **h)
    for k in GRADS:
        if k != "dz":
            assert np.abs(ref[k]).max() < 1e37
            within(g[k], ref[k], bound[k], k)


def test_packed():
    lengths = [290, 0, 100, 290, 7]
    cu = np.concatenate([[0], np.cumsum(lengths)])
    p = growing((int(cu[-1]),), len(lengths), 70, 1.0, gate=False)
    p.h0.mul_(1e-30)
    cut = torch.tensor(cu, dtype=torch.int32, device=DEV)
    out, last = pkg.ssm_gated_scan_fwd_varlen(*p.args(), cut, return_last_state=True, **p.kw())
    for s in range(len(lengths)):
        h, _, _ = p.host(s, cu[s], cu[s + 1])
        ref, rl, _ = og.gated_scan(**h)
        bo, bl, _, _ = gb.forward(**h)
        within(out[None, cu[s]:cu[s + 1]], ref, bo, "out %d" % s)
        within(last[s:s + 1], rl, bl, "last %d" % s)


def test_states_beyond_range_are_not_finite():
    """Past float32's range a state is infinite or NaN, and stays so."""
    p = growing((2, 700), 2, 70, 1.0, normalize=False, gate=False)
    out = np64(pkg.ssm_gated_scan_fwd(*p.args(), **p.kw()))
    ref, _, _ = og.gated_scan(**p.host()[0])
    assert not np.isfinite(out[np.abs(ref) > 1e39]).any()
    bo, _, _, _ = gb.forward(**p.host()[0])
    low = np.abs(ref) < 1e37  # (until the state passes the range for good)
    low &= np.cumprod(np.abs(ref) < 1e37, axis=1).astype(bool)
    assert (np.abs(out - ref)[low] <= bo[low]).all()


@pytest.mark.parametrize("L", [1, 2])
def test_steep_factors(L):
    """Factors near the largest allowed A, whose square passes float32."""
    p = growing((2, L), 2, 70, 60.0, gate=False)
    p.r.fill_(4.0)
    p.h0.mul_(1e-30)
    out, last = pkg.ssm_gated_scan_fwd(*p.args(), return_last_state=True, **p.kw())
    g = pkg.ssm_gated_scan_bwd(*p.args(), p.dout, dlast_state=p.dlast, **p.kw())
    h, dout, dl = p.host()
    ref, rl, _ = og.gated_scan(**h)
    bo, bl, _, _ = gb.forward(**h)
    within(out, ref, bo, "out")
    within(last, rl, bl, "last")
    ref, bound = og.gated_scan_bwd(dout=dout, dlast=dl, **h), gb.backward(dout=dout, dlast=dl, **h)
    # (e^118 = 1.8 10^51, the gradient of the state before two such tokens, is no float32: infinite)
    big = lambda v: np.where(np.abs(v) > np.finfo(np.float32).max, np.copysign(np.inf, v), v)
    for k in GRADS:
        if k != "dz":
            within(g[k], big(ref[k]), bound[k], k)
