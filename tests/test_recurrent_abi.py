"""The C ABI of the recurrent operators and their Python binding: declared,
exported, and refusing bad arguments on the host before anything is enqueued
(CPU)."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import selective_state_space_31_amd as pkg
from selective_state_space_31_amd import recurrent

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = ctypes.c_void_p
NULL, SHAPE, UNSUPPORTED, ALIGN, ALIAS, WORKSPACE = -1, -2, -3, -4, -5, -6


def fake(k, off=0):
    """Distinct device addresses, far apart, never dereferenced."""
    return P(0x10000000000 * k + off)


@pytest.fixture(scope="module")
def lib():
    return recurrent._load()


def declared_functions():
    src = open(os.path.join(ROOT, "include", "ssm_recurrent.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    return sorted(set(re.findall(r"\b(ssm_[a-z0-9_]+)\s*\(", src)))


def test_header_binding_and_library_agree():
    assert declared_functions() == sorted(recurrent.EXPORTS)
    out = subprocess.run(["nm", "-D", "--defined-only", pkg.LIB_PATH], stdout=subprocess.PIPE, text=True,
                         check=True).stdout
    exported = set(l.split()[-1] for l in out.splitlines() if l.strip())
    for name in declared_functions():
        assert name in exported, name
        assert callable(getattr(pkg, name))


def gfwd(lib, packed=False, **kw):
    a = dict(x=fake(1), r=fake(2), i=fake(3), A=fake(4), rb=None, ib=None, norm=1, z=None, out=fake(5), last=None,
             h0=None, mid=None, cu=fake(20), n=2, L=300, d=64, dt=0, ws=fake(30), wsb=1 << 40)
    a.update(kw)
    head = (a["x"], a["r"], a["i"], a["A"], a["rb"], a["ib"], a["norm"], a["z"], a["out"], a["last"], a["h0"], a["mid"])
    tail = (a["n"], a["L"], a["d"], a["dt"], a["ws"], a["wsb"], None)
    return lib.ssm_gated_scan_fwd_varlen(*head, a["cu"], *tail) if packed else lib.ssm_gated_scan_fwd(*head, *tail)


BAD_SIZES = [dict(n=0), dict(n=-3), dict(L=-1), dict(d=0), dict(d=-1), dict(d=(1 << 22) + 1), dict(L=1 << 50),
             dict(L=(1 << 63) - 1), dict(n=(1 << 63) - 1)]


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), UNSUPPORTED), (dict(dt=-1), UNSUPPORTED), (dict(norm=2), UNSUPPORTED), (dict(A=None), NULL),
    (dict(x=None), NULL), (dict(r=None), NULL), (dict(i=None), NULL), (dict(out=None), NULL),
    (dict(x=fake(1, 2)), ALIGN), (dict(A=fake(4, 2)), ALIGN), (dict(rb=fake(6, 1)), ALIGN), (dict(h0=fake(7, 2)), ALIGN),
    (dict(mid=fake(8, 1)), ALIGN), (dict(out=fake(1)), ALIAS), (dict(out=fake(2, 64)), ALIAS),
    (dict(last=fake(5, 128)), ALIAS), (dict(mid=fake(5, 128)), ALIAS), (dict(z=fake(5)), ALIAS),
    (dict(last=fake(7, 4), h0=fake(7)), ALIAS), (dict(last=fake(4)), ALIAS),
] + [(k, SHAPE) for k in BAD_SIZES])
def test_gated_fwd_refuses(lib, packed, kw, code):
    assert gfwd(lib, packed, **kw) == code
    assert lib.ssm_last_error()


def test_gated_fwd_refuses_more(lib):
    assert gfwd(lib, n=65536) == SHAPE
    assert gfwd(lib, True, n=1 << 24) == SHAPE
    assert gfwd(lib, True, cu=None) == NULL
    assert gfwd(lib, True, cu=fake(20, 2)) == ALIGN
    assert gfwd(lib, True, last=fake(20)) == ALIAS
    assert gfwd(lib, True, last=fake(7), h0=fake(7)) == ALIAS  # (resuming in place is for whole sequences)
    need = lib.ssm_gated_scan_fwd_workspace_bytes(2, 3000, 64, 0)
    if need:
        assert gfwd(lib, L=3000, wsb=need - 1) == WORKSPACE
        assert gfwd(lib, L=3000, ws=None) == WORKSPACE
        assert gfwd(lib, L=3000, ws=fake(30, 128)) == ALIGN
        assert gfwd(lib, L=3000, ws=fake(1)) == ALIAS


def gbwd(lib, packed=False, **kw):
    a = dict(x=fake(1), r=fake(2), i=fake(3), A=fake(4), rb=None, ib=None, norm=1, z=None, h0=None, mid=None,
             dout=fake(5), dlast=None, dx=fake(6), dr=fake(7), di=fake(8), dz=None, dA=fake(9), drb=None, dib=None,
             dh0=None, cu=fake(20), n=2, L=300, d=64, dt=0, ws=fake(30), wsb=1 << 40)
    a.update(kw)
    head = tuple(a[k] for k in ("x", "r", "i", "A", "rb", "ib", "norm", "z", "h0", "mid", "dout", "dlast", "dx", "dr",
                                "di", "dz", "dA", "drb", "dib", "dh0"))
    tail = (a["n"], a["L"], a["d"], a["dt"], a["ws"], a["wsb"], None)
    return lib.ssm_gated_scan_bwd_varlen(*head, a["cu"], *tail) if packed else lib.ssm_gated_scan_bwd(*head, *tail)


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(dt=7), UNSUPPORTED), (dict(norm=-1), UNSUPPORTED), (dict(A=None), NULL), (dict(dA=None), NULL),
    (dict(dout=None), NULL), (dict(dx=None), NULL), (dict(dr=None), NULL), (dict(di=None), NULL),
    (dict(z=fake(10)), NULL), (dict(dz=fake(10)), NULL), (dict(dout=fake(5, 2)), ALIGN), (dict(dA=fake(9, 2)), ALIGN),
    (dict(dx=fake(1)), ALIAS), (dict(dx=fake(7, 32)), ALIAS), (dict(dr=fake(5)), ALIAS), (dict(dA=fake(4)), ALIAS),
    (dict(mid=fake(6)), ALIAS), (dict(dh0=fake(9)), ALIAS), (dict(ws=fake(6)), ALIAS), (dict(ws=None), WORKSPACE),
    (dict(wsb=16), WORKSPACE), (dict(ws=fake(30, 64)), ALIGN),
] + [(k, SHAPE) for k in BAD_SIZES])
def test_gated_bwd_refuses(lib, packed, kw, code):
    assert gbwd(lib, packed, **kw) == code
    assert lib.ssm_last_error()


def gstep(lib, **kw):
    a = dict(h=fake(1), x=fake(2), r=fake(3), i=fake(4), A=fake(5), rb=None, ib=None, norm=1, z=None, out=fake(6), n=4,
             d=64, dt=1)
    a.update(kw)
    return lib.ssm_gated_state_update(*(a[k] for k in ("h", "x", "r", "i", "A", "rb", "ib", "norm", "z", "out", "n", "d",
                                                       "dt")), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=3), UNSUPPORTED), (dict(norm=5), UNSUPPORTED), (dict(h=None), NULL), (dict(x=None), NULL),
    (dict(A=None), NULL), (dict(out=None), NULL), (dict(n=0), SHAPE), (dict(d=0), SHAPE), (dict(n=1 << 40), SHAPE),
    (dict(n=1 << 20, d=1 << 12), SHAPE), (dict(d=1 << 40), SHAPE), (dict(x=fake(2, 1)), ALIGN), (dict(h=fake(1, 2)), ALIGN),
    (dict(out=fake(2)), ALIAS), (dict(out=fake(1, 16)), ALIAS), (dict(h=fake(5)), ALIAS)])
def test_gated_step_refuses(lib, kw, code):
    assert gstep(lib, **kw) == code
    assert lib.ssm_last_error()


def rot(lib, bwd=False, **kw):
    a = dict(q=fake(1), k=fake(2), qw=None, kw=None, f=fake(3), pos=None, eps=1e-6, inter=0, dqo=fake(4), dko=fake(5),
             qo=fake(6), ko=fake(7), dqw=fake(8), dkw=fake(9), b=2, L=10, hq=4, hk=2, D=64, R=64, qs=256, ks=128, dt=1,
             ws=fake(30), wsb=1 << 40)
    a.update(kw)
    head = tuple(a[k] for k in ("q", "k", "qw", "kw", "f", "pos", "eps", "inter"))
    size = tuple(a[k] for k in ("b", "L", "hq", "hk", "D", "R", "qs", "ks", "dt"))
    if bwd:
        return lib.ssm_qk_norm_rotate_bwd(*head, a["dqo"], a["dko"], a["qo"], a["ko"], a["dqw"], a["dkw"], *size, a["ws"],
                                          a["wsb"], None)
    return lib.ssm_qk_norm_rotate_fwd(*head, a["qo"], a["ko"], *size, None)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(dt=2), UNSUPPORTED), (dict(inter=2), UNSUPPORTED), (dict(eps=-1.0), UNSUPPORTED),
    (dict(eps=float("nan")), UNSUPPORTED), (dict(D=63), UNSUPPORTED), (dict(D=0), UNSUPPORTED),
    (dict(D=258, qs=4096, ks=4096), UNSUPPORTED), (dict(R=66), UNSUPPORTED), (dict(R=3), UNSUPPORTED),
    (dict(R=-2), UNSUPPORTED), (dict(b=0), SHAPE), (dict(L=-1), SHAPE), (dict(hq=0), SHAPE), (dict(hk=-1), SHAPE),
    (dict(b=1 << 20, L=1 << 20), SHAPE), (dict(L=1 << 62), SHAPE), (dict(qs=255), SHAPE), (dict(ks=0), SHAPE),
    (dict(qs=1 << 60), SHAPE), (dict(f=None), NULL), (dict(q=None), NULL), (dict(k=None), NULL), (dict(qo=None), NULL),
    (dict(ko=None), NULL), (dict(hk=0, ks=0), NULL), (dict(q=fake(1, 1)), ALIGN), (dict(f=fake(3, 2)), ALIGN),
    (dict(pos=fake(10, 2)), ALIGN), (dict(qo=fake(6, 1)), ALIGN), (dict(qo=fake(2)), ALIAS), (dict(ko=fake(6)), ALIAS),
    (dict(qo=fake(1, 2)), ALIAS), (dict(qo=fake(1), qs=300), ALIAS), (dict(qo=fake(3)), ALIAS)])
def test_rotate_refuses(lib, bwd, kw, code):
    assert rot(lib, bwd, **kw) == code
    assert lib.ssm_last_error()


@pytest.mark.parametrize("kw,code", [
    (dict(dqo=None), NULL), (dict(dko=None), NULL), (dict(qo=fake(1)), ALIAS), (dict(qo=fake(4)), ALIAS),
    (dict(dqw=fake(6)), ALIAS), (dict(dkw=fake(8)), ALIAS), (dict(ws=None), WORKSPACE), (dict(wsb=8), WORKSPACE),
    (dict(ws=fake(30, 8)), ALIGN), (dict(ws=fake(6)), ALIAS)])
def test_rotate_bwd_refuses(lib, kw, code):
    assert rot(lib, True, **kw) == code


def conv(lib, **kw):
    a = dict(x=fake(1), w=fake(2), b=None, s0=None, dout=fake(3), ds1=None, dx=fake(4), dw=fake(5), db=None, ds0=None, n=2,
             L=40, d=64, W=4, silu=1, dt=1, ws=fake(30), wsb=1 << 40)
    a.update(kw)
    return lib.ssm_causal_conv1d_bwd(*(a[k] for k in ("x", "w", "b", "s0", "dout", "ds1", "dx", "dw", "db", "ds0", "n", "L",
                                                      "d", "W", "silu", "dt", "ws", "wsb")), None)


@pytest.mark.parametrize("kw,code", [
    (dict(dt=4), UNSUPPORTED), (dict(silu=2), UNSUPPORTED), (dict(W=1), UNSUPPORTED), (dict(W=5), UNSUPPORTED),
    (dict(n=0), SHAPE), (dict(L=-1), SHAPE), (dict(d=0), SHAPE), (dict(L=1 << 50), SHAPE), (dict(n=65536), SHAPE),
    (dict(n=65535, L=1 << 20), SHAPE), (dict(w=None), NULL), (dict(dw=None), NULL), (dict(x=None), NULL),
    (dict(dout=None), NULL), (dict(dx=None), NULL), (dict(x=fake(1, 1)), ALIGN), (dict(dw=fake(5, 2)), ALIGN),
    (dict(ds1=fake(6, 1)), ALIGN), (dict(dx=fake(1)), ALIAS), (dict(dx=fake(3, 8)), ALIAS), (dict(dw=fake(2)), ALIAS),
    (dict(ds0=fake(4)), ALIAS), (dict(s0=fake(6), ds0=fake(6)), ALIAS), (dict(ws=None), WORKSPACE), (dict(wsb=4), WORKSPACE),
    (dict(ws=fake(30, 16)), ALIGN), (dict(ws=fake(4)), ALIAS)])
def test_conv_bwd_refuses(lib, kw, code):
    assert conv(lib, **kw) == code
    assert lib.ssm_last_error()


def test_workspace_queries(lib):
    big = (1 << 63) - 1
    for f, k in ((lib.ssm_gated_scan_fwd_workspace_bytes, (1,)), (lib.ssm_gated_scan_fwd_varlen_workspace_bytes, (1,)),
                 (lib.ssm_gated_scan_bwd_workspace_bytes, (1, 0)),
                 (lib.ssm_gated_scan_bwd_varlen_workspace_bytes, (1, 1))):
        for bad in ((0, 8, 8), (1, -1, 8), (1, 8, 0), (big, 8, 8), (1, big, 8), (1, 8, big)):
            assert f(*bad, *k) == 0
        assert f(1, 100, 8, 5, *k[1:]) == 0
    assert lib.ssm_gated_scan_bwd_workspace_bytes(2, 300, 64, 1, 1) > 0
    assert lib.ssm_qk_norm_rotate_bwd_workspace_bytes(2, 10, 4, 2, 64) > 0
    assert lib.ssm_qk_norm_rotate_bwd_workspace_bytes(2, big, 4, 2, 64) == 0
    assert lib.ssm_causal_conv1d_bwd_workspace_bytes(2, 10, 64, 4) > 0
    assert lib.ssm_causal_conv1d_bwd_workspace_bytes(2, 10, 64, 5) == 0


# ---- the Python binding (tensors on the CPU: nothing can be launched) ----
def gated_tensors(b=2, L=5, d=6, dtype=torch.float32):
    t = lambda *s: torch.zeros(*s, dtype=dtype)
    return dict(x=t(b, L, d), rgate=t(b, L, d), igate=t(b, L, d), A=torch.zeros(d))


@pytest.mark.parametrize("kw,exc", [
    (dict(x=torch.zeros(5, 6)), ValueError), (dict(x=torch.zeros(2, 5, 6, dtype=torch.float16)), TypeError),
    (dict(rgate=torch.zeros(2, 5, 7)), ValueError), (dict(igate=torch.zeros(2, 5, 6, dtype=torch.bfloat16)), TypeError),
    (dict(A=torch.zeros(7)), ValueError), (dict(A=torch.zeros(6, dtype=torch.float64)), TypeError), (dict(A=None), ValueError),
    (dict(z=torch.zeros(2, 6, 5).transpose(1, 2)), ValueError), (dict(rgate_bias=torch.zeros(5)), ValueError),
    (dict(initial_state=torch.zeros(3, 6)), ValueError), (dict(out=torch.zeros(2, 5, 5)), ValueError),
    (dict(last_state=torch.zeros(2, 7)), ValueError), (dict(chunk_states=torch.zeros(2, 3, 6)), ValueError),
    (dict(x="no"), TypeError), (dict(), ValueError)])  # (the last: right, but not on a HIP device)
def test_gated_binding_refuses(kw, exc):
    with pytest.raises(exc):
        pkg.ssm_gated_scan_fwd(**dict(gated_tensors(), **kw))


def test_more_binding_refusals():
    g = gated_tensors()
    with pytest.raises(ValueError):
        pkg.ssm_gated_scan_fwd_varlen(g["x"][0], g["rgate"][0], g["igate"][0], g["A"], None)
    with pytest.raises(TypeError):
        pkg.ssm_gated_scan_fwd_varlen(g["x"][0], g["rgate"][0], g["igate"][0], g["A"], torch.tensor([0, 5]))
    with pytest.raises(ValueError):
        pkg.ssm_gated_scan_fwd_varlen(g["x"][0], g["rgate"][0], g["igate"][0], g["A"],
                                      torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        pkg.ssm_gated_scan_bwd(**g, dout=torch.zeros(2, 5, 5))
    with pytest.raises(ValueError):
        pkg.ssm_gated_state_update(torch.zeros(2, 5), torch.zeros(2, 6), torch.zeros(2, 6), torch.zeros(2, 6), g["A"])
    q, k, f = torch.zeros(2, 3, 4, 8), torch.zeros(2, 3, 2, 8), torch.zeros(4)
    for bad in (dict(q=q[0]), dict(k=k[:, :2]), dict(k=torch.zeros(2, 3, 2, 6)), dict(q=q.transpose(1, 2)),
                dict(q=torch.zeros(2, 3, 4, 16)[..., ::2]), dict(k=k.bfloat16()), dict(inv_freq=torch.zeros(2, 2)),
                dict(q_weight=torch.zeros(4)), dict(positions=torch.zeros(2, 3)), dict(k=None, k_weight=torch.zeros(8)),
                dict(q=torch.zeros(1, 3, 4, 8).expand(2, 3, 4, 8)), dict(q=torch.zeros(2, 1, 4, 8).expand(2, 3, 4, 8)),
                dict(k=torch.zeros(2, 3, 0, 8)), dict(q=q.half())):
        with pytest.raises((ValueError, TypeError)):
            pkg.ssm_qk_norm_rotate_fwd(**dict(dict(q=q, k=k, inv_freq=f), **bad))
    with pytest.raises(ValueError):
        pkg.ssm_qk_norm_rotate_bwd(q, k, f, torch.zeros(2, 3, 4, 7), k)
    x = torch.zeros(2, 5, 6)
    for bad in (dict(weight=torch.zeros(6)), dict(weight=torch.zeros(5, 4)), dict(dout=torch.zeros(2, 4, 6)),
                dict(bias=torch.zeros(5)), dict(initial_conv_state=torch.zeros(2, 6, 2)), dict(x=x[0]), dict(x=x.double())):
        with pytest.raises((ValueError, TypeError)):
            pkg.ssm_causal_conv1d_bwd(**dict(dict(x=x, weight=torch.zeros(6, 4), dout=x), **bad))


def test_head_strides_are_read_right():
    """What the C call gets for slices of wider rows."""
    rows = torch.zeros(2, 3, 100)
    q = rows[..., 4:36].unflatten(-1, (4, 8))
    assert recurrent._heads(q, "q", 2, 3, 8, q) == (4, 100)
    one = torch.zeros(5, 1, 100)[..., 4:36].unflatten(-1, (4, 8))
    assert recurrent._heads(one, "q", 5, 1, 8, q) == (4, 100)
    assert recurrent._heads(one[:1], "q", 1, 1, 8, q) == (4, 32)
