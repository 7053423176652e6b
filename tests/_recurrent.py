"""Shared helpers of the recurrent operators' tests: seeded inputs, float64
copies and comparison against a bound per element."""
import numpy as np
import torch

DT = {"fp32": torch.float32, "bf16": torch.bfloat16}


def act(rng, shape, dtype, device, scale=1.0):
    v = (scale * rng.standard_normal(shape)).astype(np.float32)
    return torch.from_numpy(v).to(DT[dtype]).to(device)


def f32(rng, shape, device, scale=1.0):
    return torch.from_numpy((scale * rng.standard_normal(shape)).astype(np.float32)).to(device)


def np64(t):
    return None if t is None else t.detach().to(torch.float64).cpu().numpy()


def within(got, ref, bound, what):
    """|got - ref| <= bound everywhere, and the same non-finite values."""
    got, ref = np64(got) if isinstance(got, torch.Tensor) else np.asarray(got, np.float64), np.asarray(ref)
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    fine = np.isfinite(ref)
    assert np.array_equal(fine, np.isfinite(got)), "%s: non-finite values differ" % what
    err = np.where(fine, np.abs(np.where(fine, got, 0.0) - np.where(fine, ref, 0.0)), 0.0)
    bound = np.broadcast_to(bound, ref.shape)
    bad = (err > bound) & fine
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(fine, err / bound, 0.0)), err.shape)
        raise AssertionError("%s: %d of %d outside the bound; worst at %s: got %r ref %r bound %r"
                             % (what, int(bad.sum()), bad.size, i, got[i], ref[i], bound[i]))


class Gated:
    """Inputs of a gated recurrence over rows ``lead`` (batch, L) or (T,)."""

    def __init__(self, lead, nstates, dim, dtype, device, seed, gate=True, normalize=True, bias=True,
                 state=True, dlast=True, A_range=(1e-3, 1.0)):
        rng = np.random.default_rng(seed)
        lo, hi = np.log(A_range[0]), np.log(A_range[1])
        self.dtype, self.normalize = dtype, normalize
        a = lambda: act(rng, tuple(lead) + (dim,), dtype, device)
        self.x, self.r, self.i = a(), a(), a()
        self.z = a() if gate else None
        self.dout = a()
        self.A = torch.from_numpy(-np.exp(rng.uniform(lo, hi, dim)).astype(np.float32)).to(device)
        self.rb, self.ib = (f32(rng, (dim,), device, 0.5), f32(rng, (dim,), device, 0.5)) if bias \
            else (None, None)
        self.h0 = f32(rng, (nstates, dim), device) if state else None
        self.dlast = f32(rng, (nstates, dim), device) if dlast else None

    def args(self):
        return (self.x, self.r, self.i, self.A)

    def kw(self):
        return dict(z=self.z, rgate_bias=self.rb, igate_bias=self.ib, normalize=self.normalize,
                    initial_state=self.h0)

    def host(self, s=None, t0=None, t1=None):
        """float64 copies; with s, of packed sequence s (tokens t0..t1) as a
        (1, len, dim) problem."""
        tok = lambda t: None if t is None else (np64(t) if s is None else np64(t)[None, t0:t1])
        st = lambda t: None if t is None else (np64(t) if s is None else np64(t)[s:s + 1])
        return dict(x=tok(self.x), r=tok(self.r), i=tok(self.i), z=tok(self.z), A=np64(self.A),
                    rb=np64(self.rb), ib=np64(self.ib), normalize=self.normalize, h0=st(self.h0)), \
            tok(self.dout), st(self.dlast)
