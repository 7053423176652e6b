"""Rounding bounds of the gated recurrence in float32, per element.

With e = 2^-24 (half a float32 step, relative), v = r + rb, w = i + ib:
  * the logistic function: -v log2 e is formed as r (-log2 e) + rb (-log2 e)
    in one fused operation, which rounds by e|v|, on a product that rounds by
    e|rb|, with a constant off by less than e/4: (5/4 |v| + |rb|) e; below v
    and w stand for |v| + |rb| and |w| + |ib|.  The hardware exp2 and
    reciprocal are within 2e each, the sum 1 + e^-v rounds by e: s and u are
    within (2|v| + 6) e of themselves;
  * la = A s: one rounding more, (2|v| + 7) e |la|;
  * a = e^la: that times a, A log2 e (e|la|), the exp2 (2e) or the polynomial
    and the difference 1 - E (2e): a (|la| (2|v| + 8) + 2) e;
  * m: E is within (2|v| + 8 + 4) e where the polynomial (within 4.1e-8 < e)
    is used; elsewhere E >= 0.121, a/E <= 7.3 and |la| a/E <= 1, so within (2|v| + 8 + 16) e; the root
    halves it, the product and the root itself add 3e: (|v| + 15) e;
  * b = m u x: (|v| + 15 + 2|w| + 6 + 2) e = (|v| + 2|w| + 23) e;
  * h = a h' + b adds e|h|.
The error obeys err_t = a err_{t-1} + da |h'| + db + e|h|, walked here with
the absolute states Habs_t = a Habs_{t-1} + |b_t| in h's place.  The kernels
compose chunks of tokens: the carry passes a product of decays instead of one
decay at a time (the same roundings) and a composition rounds once more per
chunk, on values below Habs.  All bounds are doubled for that and for what is
second order.  bf16 outputs round once more: 2^-8 of the value.
"""
import numpy as np

from oracle import gated as og

E = 2.0 ** -24
BF16 = 2.0 ** -8
TINY = 1e-30


def _in(v, b):
    return np.asarray(v, np.float64) + (0.0 if b is None else np.asarray(b, np.float64))


def _coeff(x, r, i, A, rb, ib, normalize):
    s, u, la, a, m = og.gates(x, r, i, A, rb, ib, normalize)
    v, w = np.abs(_in(r, rb)) + np.abs(_in(0.0, rb)), np.abs(_in(i, ib)) + np.abs(_in(0.0, ib))
    ca = (np.abs(la) * (2 * v + 8) + 2) * E
    cb = (v + 2 * w + 23) * E
    return s, u, la, a, m, v, w, ca, cb


def forward(x, r, i, A, z=None, rb=None, ib=None, normalize=True, h0=None, dtype="fp32"):
    """(bound of out, bound of last_state, bounds of the states (batch, L + 1,
    dim), Habs)."""
    x = np.asarray(x, np.float64)
    s, u, la, a, m, v, w, ca, cb = _coeff(x, r, i, A, rb, ib, normalize)
    n, L, d = x.shape
    ab = np.abs(m * u * x)
    Ha, er = np.zeros((n, L + 1, d)), np.zeros((n, L + 1, d))
    if h0 is not None:
        Ha[:, 0] = np.abs(h0)
    for t in range(L):
        Ha[:, t + 1] = a[:, t] * Ha[:, t] + ab[:, t]
        er[:, t + 1] = (a[:, t] * er[:, t] + ca[:, t] * a[:, t] * Ha[:, t] + cb[:, t] * ab[:, t]
                        + E * Ha[:, t + 1])
    er = 2 * er
    eo, mag = er[:, 1:], Ha[:, 1:]
    if z is not None:
        z = np.asarray(z, np.float64)
        sl = np.abs(z * og._sig(z))
        eo = sl * eo + sl * mag * 2 * (2 * np.abs(z) + 8) * E
    if dtype == "bf16":
        out, _, _ = og.gated_scan(x, r, i, A, z, rb, ib, normalize, h0)
        eo = eo + BF16 * (np.abs(out) + eo)
    return eo + TINY, er[:, L] + TINY, er + TINY, Ha


def backward(x, r, i, A, dout, z=None, rb=None, ib=None, normalize=True, h0=None, dlast=None,
             dtype="fp32"):
    """Bounds of gated_scan_bwd's values, by name.  Products take the sum of
    their factors' relative bounds; G obeys the forward's recursion with the
    tokens reversed.  Sums over tokens add e times (chunk length + chunks + a
    few) times the sum of the absolute terms."""
    x, dout, A = (np.asarray(k, np.float64) for k in (x, dout, A))
    s, u, la, a, m, v, w, ca, cb = _coeff(x, r, i, A, rb, ib, normalize)
    _, _, eh, Ha = forward(x, r, i, A, z, rb, ib, normalize, h0)
    n, L, d = x.shape
    ga = np.abs(dout)
    cg = 0.0
    res = {}
    if z is not None:
        z = np.asarray(z, np.float64)
        sz = og._sig(z)
        slope = np.abs(sz * (1 + z * (1 - sz)))
        # silu' cancels near its zero: its absolute error is that of its terms
        slope_abs = sz * (1 + np.abs(z) * (1 - sz))
        res["dz"] = ga * (eh[:, 1:] * slope + Ha[:, 1:] * slope_abs * 2 * (4 * np.abs(z) + 16) * E)
        cg = 2 * (2 * np.abs(z) + 8) * E
        ga = ga * np.abs(z * sz)
    Ga, eg = np.zeros_like(x), np.zeros_like(x)
    k, ek = (np.zeros((n, d)) if dlast is None else np.abs(np.asarray(dlast, np.float64))), np.zeros((n, d))
    for t in range(L - 1, -1, -1):
        Ga[:, t] = ga[:, t] + k
        c = cg[:, t] if z is not None else 0.0
        eg[:, t] = ek + c * ga[:, t] + E * Ga[:, t]
        k = a[:, t] * Ga[:, t]
        ek = a[:, t] * eg[:, t] + ca[:, t] * k + E * k
    eg, ek = 2 * eg, 2 * ek
    mu, cm = m * u, cb + 4 * E
    res["dx"] = eg * mu + Ga * mu * cm
    # u (1 - u): 1 - u is within (2|w| + 7) e absolutely; likewise s
    uu, ss = u * (1 - u), s * (1 - s)
    au, as_ = uu * (2 * w + 8) * E + u * (2 * w + 8) * E * np.minimum(1.0, u + E), None
    as_ = ss * (2 * v + 8) * E + s * (2 * v + 8) * E * np.minimum(1.0, s + E)
    mx = m * np.abs(x)
    res["digate"] = eg * mx * uu + Ga * mx * (au + uu * cm)
    t1, e1 = a * Ha[:, :-1], a * eh[:, :-1] + a * Ha[:, :-1] * (ca + 2 * E)
    if normalize:
        with np.errstate(divide="ignore"):
            inv = np.where(m > 0, 1.0 / m, 0.0)
        t2 = u * np.abs(x) * a * a * inv
        t1, e1 = t1 + t2, e1 + t2 * (2 * ca + cb + 8 * E)
    dla, el = Ga * t1, eg * t1 + Ga * e1 + Ga * t1 * 2 * E
    aA = np.abs(A)
    res["drgate"] = el * aA * ss + dla * aA * (as_ + ss * 4 * E)
    res["dinitial_state"] = ek
    steps = (128 + 16 + n * (L // 128 + 2)) * E
    for name, e, mag in (("dA", el * s + dla * s * (2 * v + 8) * E, dla * s),
                         ("drgate_bias", res["drgate"], dla * aA * ss),
                         ("digate_bias", res["digate"], Ga * mx * uu)):
        res[name] = (e.sum((0, 1)) + steps * mag.sum((0, 1))) + TINY
    if dtype == "bf16":
        ref = og.gated_scan_bwd(x, r, i, A, dout, z, rb, ib, normalize, h0, dlast)
        for name in ("dx", "drgate", "digate", "dz"):
            if name in res:
                res[name] = res[name] + BF16 * (np.abs(ref[name]) + res[name])
    return {k: v + TINY for k, v in res.items()}
