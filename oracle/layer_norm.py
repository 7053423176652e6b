"""Plain float64 form of layer norm over rows and its gradients (numpy):
y = (x - mean) / sqrt(var + eps) * w + b."""
import numpy as np


def layer_norm(x, w, b, eps):
    """(y, normalised rows, 1 / sqrt(var + eps))."""
    c = x - x.mean(-1, keepdims=True)
    rstd = 1.0 / np.sqrt((c * c).mean(-1, keepdims=True) + eps)
    h = c * rstd
    return h * (1.0 if w is None else w) + (0.0 if b is None else b), h, rstd


def layer_norm_bwd(x, w, eps, dy, dres=None):
    """(dx, dw, db) of sum(dy * y) + sum(dres * x)."""
    _, h, rstd = layer_norm(x, w, None, eps)
    gw = dy * (1.0 if w is None else w)
    dx = rstd * (gw - gw.mean(-1, keepdims=True) - h * (gw * h).mean(-1, keepdims=True))
    over = tuple(range(x.ndim - 1))
    return dx if dres is None else dx + dres, (dy * h).sum(over), dy.sum(over)
