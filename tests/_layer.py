"""Shared helpers of the delta rule's and layer norm's tests: seeded inputs,
the float64 results of a call, and the bounds of its errors.

Bounds.  The kernels hold every product and sum that a state, an output or a
gradient goes through to float32's precision.  A chunk's results pass through
at most four products one after another (state by key, the chunk's triangular
solve, the outer product, the decay), each a sum of at most 256 terms; rounding
such a sum is off by 2^-24 relative to its terms' 2-norm times at most
sqrt(256) = 16 when the roundings are independent.  What reaches a result is so
at most 4 * 16 = 64 half steps of its largest size in the head, and the
recurrence (|I - beta k k^T| <= 1, decays <= 1) does not magnify what earlier
chunks left.  Gradients come out of a second such chain over the results of the
first, with up to three more products: 2 * (4 + 4) * 16 = 256 half steps.  A
bf16 result adds half a step of its own type, 2^-8 of the value; what reaches
only bf16 results is carried in two bf16 parts (2^-17 relative), which adds at
most 2^-15 of the largest size over the products of a chain.

dbeta and dg are inner products (du . e, <dS, S>); their errors scale with the
product of the factors' norms, not with what is left of it.
"""
import numpy as np
import torch

from oracle import delta
from tests._recurrent import DT, act, f32, np64

HALF = 2.0 ** -24


def unit(rng, shape, dtype, device):
    """Rows of unit norm with a positive share in common."""
    r = rng.standard_normal(shape) + 0.3
    r = r / (1.0 + np.exp(-r)) + 1e-3 * rng.standard_normal(shape)
    r = r / np.sqrt((r * r).sum(-1, keepdims=True))
    return torch.from_numpy(r.astype(np.float32)).to(DT[dtype]).to(device)


class Delta:
    """Inputs of a delta rule call over rows ``lead`` (batch, L) or (T,)."""

    def __init__(self, lead, n, hk, hv, K, V, dtype, device, seed, decay=True, state=True, dlast=True, rate=(1e-3, 1.0),
                 fused=False):
        rng = np.random.default_rng(seed)
        lead = tuple(lead)
        self.dtype, self.n = dtype, n
        self.q, self.k = unit(rng, lead + (hk, K), dtype, device), unit(rng, lead + (hk, K), dtype, device)
        self.v = act(rng, lead + (hv, V), dtype, device)
        if fused:  # slices of wider rows
            wide = [act(rng, lead + (7 + w + 9,), dtype, device) for w in (hk * K, hk * K, hv * V)]
            for name, rows, h in (("q", wide[0], hk), ("k", wide[1], hk), ("v", wide[2], hv)):
                t = rows[..., 7:-9].unflatten(-1, (h, -1))
                t.copy_(getattr(self, name))
                setattr(self, name, t)
        self.beta = torch.sigmoid(f32(rng, lead + (hv,), device))
        r = np.exp(rng.uniform(np.log(rate[0]), np.log(rate[1]), hv))
        g = -r * np.log1p(np.exp(rng.standard_normal(lead + (hv,))))
        self.g = torch.from_numpy(g.astype(np.float32)).to(device) if decay else None
        self.h0 = f32(rng, (n, hv, K, V), device) if state else None
        self.dout = act(rng, lead + (hv, V), dtype, device)
        self.dlast = f32(rng, (n, hv, K, V), device) if dlast else None

    def args(self):
        return (self.q, self.k, self.v, self.beta)

    def kw(self):
        return dict(g=self.g, initial_state=self.h0)

    def host(self, s, t0=None, t1=None):
        """float64 copies of sequence s (packed: tokens t0..t1)."""
        tok = lambda t: None if t is None else (np64(t[s]) if t0 is None else np64(t[t0:t1]))
        st = lambda t: None if t is None else np64(t[s])
        return dict(q=tok(self.q), k=tok(self.k), v=tok(self.v), beta=tok(self.beta), g=tok(self.g), h0=st(self.h0)), \
            tok(self.dout), st(self.dlast)


def largest(ref, axes):
    return np.abs(ref).max(axis=axes, keepdims=True) if ref.size else np.zeros((1,) * ref.ndim)


def bound(ref, dtype, halves, axes):
    """Per element: ``halves`` half steps of the largest size over ``axes``,
    and the result's own rounding."""
    b = halves * HALF * largest(ref, axes) + 1e-30
    return b + 2.0 ** -24 * np.abs(ref) if dtype == "fp32" else b + 2.0 ** -8 * np.abs(ref) + 2.0 ** -15 * largest(ref, axes)


def check_close(got, ref, b, what):
    got = np64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    assert np.isfinite(got).all(), "%s: not finite" % what
    err = np.abs(got - ref)
    b = np.broadcast_to(b, ref.shape)
    if (err > b).any():
        i = np.unravel_index(np.argmax(err / b), err.shape)
        raise AssertionError("%s: %d of %d outside the bound; worst at %s: got %r ref %r bound %r"
                             % (what, int((err > b).sum()), err.size, i, got[i], ref[i], b[i]))


def check_forward(p, out, last, s, t0=None, t1=None, what="", mids=None):
    """out (L, Hv, V), last (Hv, K, V), mids (chunks, Hv, K, V) of sequence s."""
    h, _, _ = p.host(s, t0, t1)
    ref, ref_last, before = delta.delta_rule(**h)
    if ref.shape[0]:
        check_close(out, ref, bound(ref, p.dtype, 64, (0, 2)), what + " out")
    # (a state's columns gather what all earlier ones were worth)
    top = np.concatenate([before, ref_last[None]])
    size = 64 * HALF * largest(top, (0, 2, 3))
    check_close(last, ref_last, size[0] + 1e-30, what + " last_state")
    if mids is not None:
        K = ref_last.shape[1]
        mids = np64(mids)
        check_close(mids[:, :, :K], before[::64], size + 1e-30, what + " chunk_states")
        u = delta.missing(**h)
        for c in range(mids.shape[0]):
            part = u[64 * c:64 * c + 64].transpose(1, 0, 2)
            check_close(mids[c, :, K:K + part.shape[1]], part, 64 * HALF * largest(top, (0, 2, 3))[0] + 64 * HALF *
                        largest(u, (0, 2))[0][:, :, None] + 1e-30, what + " e")
            assert (mids[c, :, K + part.shape[1]:] == 0).all(), what


def check_grads(p, got, s, t0=None, t1=None, what=""):
    h, dout, dlast = p.host(s, t0, t1)
    ref = delta.delta_rule_bwd(dout=dout, dlast=dlast, **h)
    sizes = delta.grad_sizes(dout=dout, dlast=dlast, **h)
    for name in ("dq", "dk", "dv"):
        if ref[name].size:
            # (what a token's gradient is formed from is as large as the sizes say, also where little of it is left)
            b = bound(ref[name], p.dtype, 0, (0, 2)) + 256 * HALF * sizes[name] + \
                (2.0 ** -15 * sizes[name] if p.dtype == "bf16" else 0.0)
            check_close(got[name], ref[name], b, what + " " + name)
    for name in ("dbeta", "dg"):
        if got.get(name) is not None and ref[name].size:
            check_close(got[name], ref[name], 256 * HALF * sizes[name] + 1e-30, what + " " + name)
    check_close(got["dinitial_state"], ref["dinitial_state"], 256 * HALF * sizes["dstate"] + 1e-30,
                what + " dinitial_state")
