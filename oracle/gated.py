"""float64 reference of the gated linear recurrence and its gradients: the
definition's loop over the tokens, in numpy.  Test infrastructure; shares no
code with the kernels."""
import numpy as np


def _sig(v):
    v = np.asarray(v, np.float64)
    with np.errstate(over="ignore"):
        return np.where(v >= 0, 1.0 / (1.0 + np.exp(-np.abs(v))), np.exp(-np.abs(v)) / (1.0 + np.exp(-np.abs(v))))


def gates(x, r, i, A, rb=None, ib=None, normalize=True):
    """s, u, la, a, m of every token (float64)."""
    f = lambda v: np.asarray(v, np.float64)
    s = _sig(f(r) + (0.0 if rb is None else f(rb)))
    u = _sig(f(i) + (0.0 if ib is None else f(ib)))
    la = f(A) * s
    a = np.exp(la)
    m = np.sqrt(np.maximum(-np.expm1(2.0 * la), 0.0)) if normalize else np.ones_like(la)
    return s, u, la, a, m


def gated_scan(x, r, i, A, z=None, rb=None, ib=None, normalize=True, h0=None):
    """One batch of sequences (batch, L, dim): (out, last_state, states), with
    states (batch, L + 1, dim) the state before every token and the last."""
    x = np.asarray(x, np.float64)
    s, u, la, a, m = gates(x, r, i, A, rb, ib, normalize)
    b, L, d = x.shape
    H = np.zeros((b, L + 1, d))
    if h0 is not None:
        H[:, 0] = h0
    for t in range(L):
        H[:, t + 1] = a[:, t] * H[:, t] + m[:, t] * u[:, t] * x[:, t]
    out = H[:, 1:].copy()
    if z is not None:
        z = np.asarray(z, np.float64)
        out = out * z * _sig(z)
    return out, H[:, L].copy(), H


def gated_scan_bwd(x, r, i, A, dout, z=None, rb=None, ib=None, normalize=True, h0=None, dlast=None):
    """Gradients of sum(dout*out) + sum(dlast*last), as a dict."""
    x, dout, A = (np.asarray(v, np.float64) for v in (x, dout, A))
    s, u, la, a, m = gates(x, r, i, A, rb, ib, normalize)
    _, _, H = gated_scan(x, r, i, A, z, rb, ib, normalize, h0)
    b, L, d = x.shape
    g, dz = dout, None
    if z is not None:
        z = np.asarray(z, np.float64)
        sz = _sig(z)
        g = dout * z * sz
        dz = dout * H[:, 1:] * sz * (1.0 + z * (1.0 - sz))
    k = np.zeros((b, d)) if dlast is None else np.asarray(dlast, np.float64).copy()
    G = np.zeros_like(x)
    for t in range(L - 1, -1, -1):
        G[:, t] = g[:, t] + k
        k = a[:, t] * G[:, t]
    dla = G * a * H[:, :-1]
    if normalize:
        with np.errstate(divide="ignore"):
            inv = np.where(m > 0, 1.0 / m, 0.0)
        dla = dla - G * u * x * a * a * inv
    dr = dla * A * s * (1.0 - s)
    di = G * m * x * u * (1.0 - u)
    return dict(dx=G * m * u, drgate=dr, digate=di, dz=dz, dA=(dla * s).sum((0, 1)),
                drgate_bias=dr.sum((0, 1)), digate_bias=di.sum((0, 1)), dinitial_state=k)
