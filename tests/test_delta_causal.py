"""A value that is not finite acts on its own token and those behind it, in its
sequence and head, and on nothing before it: wherever it stands in a chunk of
64 tokens, and for every input (GPU)."""
import numpy as np
import pytest
import torch

import selective_state_space_31_amd as pkg
from oracle import delta
from tests._layer import HALF, Delta, bound, check_close, largest
from tests._recurrent import np64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def before(p, out, s, t, t0=None, t1=None):
    """Outputs of the first t tokens of sequence s against float64 (with the
    bound of tests/_layer.py)."""
    h, _, _ = p.host(s, t0, t1)
    cut = {n: a if n == "h0" or a is None else a[:t] for n, a in h.items()}
    ref, _, _ = delta.delta_rule(**cut)
    if t:
        check_close(out[:t], ref, bound(ref, p.dtype, 64, (0, 2)), "out before")


def behind(p, out, last, s, t0=None, t1=None):
    """What is not finite by the formulas is not finite in the results."""
    h, _, _ = p.host(s, t0, t1)
    with np.errstate(all="ignore"):
        ref, ref_last, _ = delta.delta_rule(**h)
    assert not np.isfinite(ref).all()
    assert not np.isfinite(np64(out)[~np.isfinite(ref)]).any()
    assert not np.isfinite(np64(last)[~np.isfinite(ref_last)]).any()


def spoil(p, what, at, value):
    """`value` in one place of input `what`, at token index `at`."""
    x = getattr(p, what)[at]
    x.view(-1)[x.numel() // 2] = value


KINDS = [("q", "nan"), ("k", "nan"), ("k", "inf"), ("v", "nan"), ("v", "-inf"), ("beta", "nan"), ("beta", "inf"), ("g", "nan"),
         ("g", "inf")]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("what,value", KINDS)
@pytest.mark.parametrize("t", [0, 1, 15, 16, 17, 31, 32, 40, 50, 63, 64, 100, 129])
def test_whole(t, what, value, dtype):
    p = Delta((2, 130), 2, 1, 2, 64, 40, dtype, DEV, seed=t)
    spoil(p, what, (1, t), float(value))
    out, last, mids = pkg.ssm_delta_rule_fwd(*p.args(), return_last_state=True, return_chunk_states=True, **p.kw())
    torch.cuda.synchronize()
    before(p, out[0], 0, 130)
    before(p, out[1], 1, t)
    behind(p, out[1], last[1], 1)
    # the states in front of the token's chunk, and what the tokens before it found missing
    h, _, _ = p.host(1)
    cut = {n: a if n == "h0" or a is None else a[:t] for n, a in h.items()}
    _, end, states = delta.delta_rule(**cut)
    top = np.concatenate([states, end[None]])
    size = 64 * HALF * largest(top, (0, 2, 3))
    starts = np.arange(0, t + 1, 64)
    check_close(mids[1, :len(starts), :, :64], top[starts], size + 1e-30, "chunk_states")
    miss = delta.missing(**cut)
    got = np64(mids[1])
    for i in range(t):
        check_close(got[i // 64, :, 64 + i % 64], miss[i], 64 * HALF * (largest(top, (0, 2, 3))[0, :, 0] + largest(miss, (0, 2))[0])
                    + 1e-30, "e of token %d" % i)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("what,value", KINDS)
@pytest.mark.parametrize("shape", [(4, 70, 32, 64, 128, 77), (1, 100, 1, 1, 256, 200), (1, 40, 1, 3, 16, 16), (2, 90, 2, 2, 100, 128)],
                         ids=str)
def test_other_sizes(shape, what, value, dtype):
    """Two column blocks a workgroup, shared key heads, wide and narrow keys."""
    b, L, hk, hv, K, V = shape
    p = Delta((b, L), b, hk, hv, K, V, dtype, DEV, seed=L)
    t = L - 9
    spoil(p, what, (b - 1, t), float(value))
    out, last = pkg.ssm_delta_rule_fwd(*p.args(), return_last_state=True, **p.kw())
    torch.cuda.synchronize()
    before(p, out[b - 1], b - 1, t)
    behind(p, out[b - 1], last[b - 1], b - 1)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_several_in_a_chunk(dtype):
    """Two columns of the values and a key, in that order; a packed sequence
    between others."""
    cu = [0, 70, 170, 260]
    p = Delta((260,), 3, 1, 2, 64, 48, dtype, DEV, seed=5)
    clean = Delta((260,), 3, 1, 2, 64, 48, dtype, DEV, seed=5)
    off = torch.tensor(cu, dtype=torch.int32, device=DEV)
    p.v[100, 0, 3], p.v[90, 0, 40], p.k[120, 0, 7] = float("nan"), float("inf"), float("nan")
    f = lambda q: pkg.ssm_delta_rule_fwd_varlen(*q.args(), off, return_last_state=True, **q.kw())
    out, last = f(p)
    want, wlast = f(clean)
    torch.cuda.synchronize()
    for s in (0, 2):
        assert torch.equal(out[cu[s]:cu[s + 1]], want[cu[s]:cu[s + 1]]) and torch.equal(last[s], wlast[s])
    before(p, out[70:170], 1, 20, 70, 170)
    behind(p, out[70:170], last[1], 1, 70, 170)
    # columns do not meet before the key: head 0's column 40 is gone from its token on, column 3 from its own, the rest not
    assert torch.isfinite(out[70:120, 1]).all()
    for c, t in ((40, 90), (3, 100)):
        assert torch.isfinite(out[70:t, 0, c]).all() and not torch.isfinite(out[t:170, 0, c]).any()
    keep = [c for c in range(48) if c not in (3, 40)]
    assert torch.isfinite(out[70:120, 0][:, keep]).all() and not torch.isfinite(out[120:170]).any()


def test_a_state_that_overflows():
    """Keys of length 6: states grow past float32's range inside a chunk.  What
    lies before is finite, and is what a call of those tokens alone gives."""
    p = Delta((1, 64), 1, 1, 1, 64, 64, "fp32", DEV, seed=6, decay=False)
    p.k *= 6.0
    p.k[:] = p.k[:, :1]  # (one key: the state grows by 1 - 36 with every token)
    p.beta.fill_(1.0)
    out = pkg.ssm_delta_rule_fwd(*p.args(), **p.kw())
    h, _, _ = p.host(0)
    ref, _, _ = delta.delta_rule(**h)
    small = int(np.argmax(np.abs(ref).max((1, 2)) > 1e34))
    assert 18 <= small < 30
    torch.cuda.synchronize()
    got = np64(out[0])
    assert np.isfinite(got[:small]).all()
    # (a token multiplies what is there, its errors among it: 64 half steps a token of the size at hand)
    size = np.maximum.accumulate(np.abs(ref).max((1, 2)))[:, None, None]
    err = np.abs(got[:small] - ref[:small])
    assert (err <= 64 * 64 * HALF * size[:small]).all()
