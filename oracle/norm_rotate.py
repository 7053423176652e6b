"""float64 reference of the per-head RMS norm with the position rotation and
of its gradients, in numpy.  Test infrastructure; shares no code with the
kernels."""
import numpy as np


def _pairs(R, interleaved):
    if interleaved:
        return np.arange(0, R, 2), np.arange(1, R, 2)
    return np.arange(R // 2), np.arange(R // 2, R)


def _turn(v, pos, freq, interleaved, back=False):
    R = 0 if freq is None else 2 * len(freq)
    y = v.copy()
    if R:
        p, q = _pairs(R, interleaved)
        ang = np.asarray(pos, np.float64)[:, :, None, None] * np.asarray(freq, np.float64)
        c, s = np.cos(ang), np.sin(ang) * (-1.0 if back else 1.0)
        y[..., p] = v[..., p] * c - v[..., q] * s
        y[..., q] = v[..., p] * s + v[..., q] * c
    return y


def norm_rotate(v, w, pos, freq, eps, interleaved):
    """v (batch, L, heads, D); w (D) or None; pos (batch, L)."""
    v = np.asarray(v, np.float64)
    w = 1.0 if w is None else np.asarray(w, np.float64)
    n = v / np.sqrt((v * v).mean(-1, keepdims=True) + eps) * w
    return _turn(n, pos, freq, interleaved)


def norm_rotate_bwd(v, w, pos, freq, eps, interleaved, dy):
    """(dv, dw) of sum(dy * norm_rotate(v))."""
    v, dy = np.asarray(v, np.float64), np.asarray(dy, np.float64)
    w = np.ones(v.shape[-1]) if w is None else np.asarray(w, np.float64)
    rstd = 1.0 / np.sqrt((v * v).mean(-1, keepdims=True) + eps)
    vh = v * rstd
    g = _turn(dy, pos, freq, interleaved, back=True)
    gw = g * w
    return rstd * (gw - vh * (gw * vh).mean(-1, keepdims=True)), (g * vh).sum((0, 1, 2))
