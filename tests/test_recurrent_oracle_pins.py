"""Pins of the float64 references of the recurrent operators: closed forms,
independent forms and differences (CPU)."""
import numpy as np
import pytest

from oracle import conv_bwd as oc
from oracle import gated as og
from oracle import norm_rotate as on
from tests import _gated_bound as gb


def problem(seed, b=2, L=9, d=3, gate=True, normalize=True):
    r = np.random.default_rng(seed)
    n = lambda *s: r.standard_normal(s)
    return dict(x=n(b, L, d), r=n(b, L, d), i=n(b, L, d), A=-np.exp(n(d)), z=n(b, L, d) if gate else None,
                rb=n(d), ib=n(d), normalize=normalize, h0=n(b, d))


@pytest.mark.parametrize("normalize", [True, False])
def test_scan_is_the_unrolled_sum(normalize):
    p = problem(1, gate=False, normalize=normalize)
    out, last, H = og.gated_scan(**p)
    s = 1 / (1 + np.exp(-(p["r"] + p["rb"])))
    a = np.exp(p["A"] * s)
    b = p["x"] / (1 + np.exp(-(p["i"] + p["ib"]))) * (np.sqrt(1 - a * a) if normalize else 1.0)
    for t in range(9):
        want = a[:, :t + 1].prod(1) * p["h0"]
        for k in range(t + 1):
            want = want + a[:, k + 1:t + 1].prod(1) * b[:, k]
        np.testing.assert_allclose(out[:, t], want, rtol=1e-12, atol=1e-13)
    np.testing.assert_array_equal(H[:, 1:], out)
    np.testing.assert_array_equal(last, out[:, -1])


def test_constant_gates_are_a_filter():
    """a and m constant: a first-order recursive filter."""
    from scipy.signal import lfilter
    x = np.random.default_rng(2).standard_normal((1, 50, 1))
    o = np.zeros_like(x)
    out, _, _ = og.gated_scan(x, o, o + 1e4, np.array([2 * np.log(0.9)]))  # sigma(0) = 1/2: a = 0.9
    want = lfilter([np.sqrt(1 - 0.81)], [1, -0.9], x[0, :, 0])
    np.testing.assert_allclose(out[0, :, 0], want, rtol=1e-12)


def test_gate_limits():
    x = np.random.default_rng(3).standard_normal((1, 6, 2))
    h0 = np.array([[1.5, -2.0]])
    closed = np.full_like(x, -1e4)
    out, last, _ = og.gated_scan(x, closed, closed, np.array([-1.0, -1.0]), h0=h0)  # holds the state
    np.testing.assert_array_equal(out, np.broadcast_to(h0[:, None], x.shape))
    out, _, _ = og.gated_scan(x, -closed, -closed, np.array([-1e4, -1e4]), h0=h0)  # passes the input through
    np.testing.assert_array_equal(out, x)


def difference(f, v, e=1e-6):
    g = np.zeros_like(v)
    for i in np.ndindex(v.shape):
        w = v.copy()
        w[i] += e
        up = f(w)
        w[i] -= 2 * e
        g[i] = (up - f(w)) / (2 * e)
    return g


@pytest.mark.parametrize("gate,normalize", [(True, True), (False, True), (True, False)])
def test_gated_gradients_are_differences(gate, normalize):
    p = problem(4, b=2, L=4, d=2, gate=gate, normalize=normalize)
    r = np.random.default_rng(5)
    dout, dl = r.standard_normal((2, 4, 2)), r.standard_normal((2, 2))

    def loss(**kw):
        out, last, _ = og.gated_scan(**dict(p, **kw))
        return (out * dout).sum() + (last * dl).sum()
    g = og.gated_scan_bwd(dout=dout, dlast=dl, **p)
    for name, key in (("dx", "x"), ("drgate", "r"), ("digate", "i"), ("dz", "z"), ("dA", "A"), ("drgate_bias", "rb"),
                      ("digate_bias", "ib"), ("dinitial_state", "h0")):
        if p[key] is None:
            assert g[name] is None
            continue
        np.testing.assert_allclose(g[name], difference(lambda v: loss(**{key: v}), p[key]), rtol=2e-6, atol=1e-8,
                                   err_msg=name)


def float32_walk(p):
    """The recurrence with every operation rounded to float32 (numpy)."""
    f = np.float32
    c = {k: (f(v) if isinstance(v, np.ndarray) else v) for k, v in p.items()}
    sg = lambda v: f(1) / (f(1) + np.exp(-v))
    la = c["A"] * sg(c["r"] + c["rb"])
    a = np.exp(la)
    m = np.sqrt(-np.expm1(f(2) * la))
    b = m * sg(c["i"] + c["ib"]) * c["x"]
    h, H = c["h0"], []
    for t in range(c["x"].shape[1]):
        h = a[:, t] * h + b[:, t]
        H.append(h)
    return np.stack(H, 1)


def test_rounding_bound_holds_and_is_tight():
    """Float32 arithmetic stays inside the bound, and not by orders of
    magnitude: the bound can catch a wrong kernel."""
    p = problem(6, b=3, L=400, d=16, gate=False)
    p = {k: (v.astype(np.float32).astype(np.float64) if isinstance(v, np.ndarray) else v) for k, v in p.items()}
    bo, _, _, _ = gb.forward(**p)
    out, _, _ = og.gated_scan(**p)
    ratio = np.abs(float32_walk(p) - out) / bo
    assert ratio.max() < 1.0
    assert np.median(bo / (np.abs(out) + 1e-3)) < 2e-4


@pytest.mark.parametrize("inter", [False, True])
def test_rotation_keeps_norms_and_relative_angles(inter):
    """A turned pair keeps its length, and the product of a query and a key
    depends on the difference of their positions alone."""
    r = np.random.default_rng(7)
    freq = 100.0 ** (-np.arange(4) / 4)
    q, k = r.standard_normal((1, 1, 1, 8)), r.standard_normal((1, 1, 1, 8))
    dots = [float((on.norm_rotate(q, None, [[t]], freq, 0.0, inter) *
                   on.norm_rotate(k, None, [[t + 5]], freq, 0.0, inter)).sum()) for t in (0, 3, 1000)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-10)
    y = on.norm_rotate(q, None, [[77]], freq, 0.0, inter)
    np.testing.assert_allclose((y * y).mean(), 1.0, rtol=1e-12)


def test_quarter_turn():
    v = np.array([1.0, 2.0, 3.0, 4.0]).reshape(1, 1, 1, 4)
    n = v / np.sqrt(7.5)
    quarter = np.array([np.pi / 2, np.pi])
    half = on.norm_rotate(v, None, [[1]], quarter, 0.0, False)[0, 0, 0]
    np.testing.assert_allclose(half, n[0, 0, 0][[2, 1, 0, 3]] * [-1, -1, 1, -1], atol=1e-15)
    inter = on.norm_rotate(v, None, [[1]], quarter, 0.0, True)[0, 0, 0]
    np.testing.assert_allclose(inter, n[0, 0, 0][[1, 0, 2, 3]] * [-1, 1, -1, -1], atol=1e-15)


@pytest.mark.parametrize("inter", [False, True])
def test_norm_rotate_gradients_are_differences(inter):
    r = np.random.default_rng(8)
    v, w, dy = r.standard_normal((2, 3, 2, 6)), r.standard_normal(6), r.standard_normal((2, 3, 2, 6))
    pos, freq = r.integers(0, 50, (2, 3)), np.array([1.0, 0.1])
    f = lambda vv, ww: (on.norm_rotate(vv, ww, pos, freq, 1e-3, inter) * dy).sum()
    dv, dw = on.norm_rotate_bwd(v, w, pos, freq, 1e-3, inter, dy)
    np.testing.assert_allclose(dv, difference(lambda t: f(t, w), v), rtol=1e-6, atol=1e-8)
    np.testing.assert_allclose(dw, difference(lambda t: f(v, t), w), rtol=1e-6, atol=1e-8)


@pytest.mark.parametrize("silu", [True, False])
@pytest.mark.parametrize("L", [1, 2, 6])
def test_conv_gradients_are_differences(L, silu):
    """Against the forward oracle of the convolution, a C program."""
    import oracle
    r = np.random.default_rng(9)
    x, w, b = r.standard_normal((2, L, 3)), r.standard_normal((3, 4)), r.standard_normal(3)
    st, dout, df = r.standard_normal((2, 3, 3)), r.standard_normal((2, L, 3)), r.standard_normal((2, 3, 3))

    def loss(x=x, w=w, b=b, st=st):
        f = lambda v: v.astype(np.float32)
        out, fin = oracle.conv1d_fwd(f(x), f(w), f(b), silu, f(st))
        return float((out * dout).sum() + (fin * df).sum())
    g = oc.conv1d_bwd(x, w, b, dout, silu, st, df)
    # the forward oracle takes float32 inputs: a step of 2^-9 keeps their rounding below 2^-24 / 2^-9 of a slope
    for name, key, v in (("dx", "x", x), ("dweight", "w", w), ("dbias", "b", b), ("dinitial_conv_state", "st", st)):
        np.testing.assert_allclose(g[name], difference(lambda t: loss(**{key: t}), v, 2.0 ** -9), rtol=2e-3, atol=2e-3,
                                   err_msg=name)
