"""float64 reference of the causal depthwise convolution's gradients, in
numpy.  Test infrastructure; shares no code with the kernels."""
import numpy as np


def conv1d_bwd(x, w, bias, dout, silu=True, state=None, dfinal=None):
    """x, dout (batch, L, dim); w (dim, W); states (batch, dim, W-1), oldest
    first.  Returns dict(dx, dweight, dbias, dinitial_conv_state)."""
    x, w, dout = (np.asarray(v, np.float64) for v in (x, w, dout))
    b, L, d = x.shape
    W = w.shape[1]
    before = np.zeros((b, W - 1, d)) if state is None else np.asarray(state, np.float64).transpose(0, 2, 1)
    xx = np.concatenate([before, x], 1)
    pre = np.zeros((b, L, d)) + (0.0 if bias is None else np.asarray(bias, np.float64))
    for k in range(W):
        pre += w[:, k] * xx[:, k:k + L]
    g = dout
    if silu:
        s = 1.0 / (1.0 + np.exp(-pre))
        g = dout * s * (1.0 + pre * (1.0 - s))
    dxx = np.zeros_like(xx)
    dw = np.zeros_like(w)
    for k in range(W):
        dxx[:, k:k + L] += w[:, k] * g
        dw[:, k] = (g * xx[:, k:k + L]).sum((0, 1))
    if dfinal is not None:
        dxx[:, L:] += np.asarray(dfinal, np.float64).transpose(0, 2, 1)
    return dict(dx=dxx[:, W - 1:], dweight=dw, dbias=g.sum((0, 1)),
                dinitial_conv_state=dxx[:, :W - 1].transpose(0, 2, 1))
