"""Thin Python binding of the C ABI in include/ssm_layer.h.

Argument marshalling only, in the manner of ``recurrent`` (whose helpers it
uses): the functions keep the C names, every step runs in the HIP kernels of
libssm_scan.so, PyTorch supplies device memory and the current HIP stream, and
a missing library fails loudly.  Tensors are on one HIP device, which need not
be the current one.  ``stream`` is a raw HIP stream handle (the tensors'
device's current stream by default); what is allocated here for a call on
another stream comes from that stream's memory, so the caller orders the two
streams for the inputs and the results alone.
"""
import ctypes

import torch

from . import ops
from .ops import _DTYPES
from .recurrent import _F32, _act, _buffers, _call, _heads, _in, _opt, _other, _out, _space

SSM_DELTA_CHUNK = 64

EXPORTS = ("ssm_delta_rule_fwd", "ssm_delta_rule_fwd_workspace_bytes", "ssm_delta_rule_fwd_varlen",
           "ssm_delta_rule_fwd_varlen_workspace_bytes", "ssm_delta_rule_bwd",
           "ssm_delta_rule_bwd_workspace_bytes", "ssm_delta_rule_bwd_varlen",
           "ssm_delta_rule_bwd_varlen_workspace_bytes", "ssm_delta_state_update",
           "ssm_layer_norm_fwd", "ssm_layer_norm_bwd", "ssm_layer_norm_bwd_workspace_bytes")

_lib = None


def _load():
    global _lib
    if _lib is not None:
        return _lib
    lib = ops.load_library()
    P, I, L, S, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    sig = {
        "ssm_delta_rule_fwd": [P] * 5 + [F] + [P] * 4 + [L] * 9 + [I, P, S, P],
        "ssm_delta_rule_fwd_varlen": [P] * 5 + [F] + [P] * 5 + [L] * 9 + [I, P, S, P],
        "ssm_delta_rule_bwd": [P] * 5 + [F] + [P] * 10 + [L] * 9 + [I, P, S, P],
        "ssm_delta_rule_bwd_varlen": [P] * 5 + [F] + [P] * 11 + [L] * 9 + [I, P, S, P],
        "ssm_delta_state_update": [P] * 6 + [F, P] + [L] * 8 + [I, P],
        "ssm_layer_norm_fwd": [P] * 4 + [F] + [P] * 2 + [L] * 4 + [I, P],
        "ssm_layer_norm_bwd": [P] * 2 + [F] + [P] * 5 + [L] * 3 + [I, P, S, P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = args, I
    for name, args in {"ssm_delta_rule_fwd_workspace_bytes": [L] * 6 + [I],
                       "ssm_delta_rule_fwd_varlen_workspace_bytes": [L] * 6 + [I],
                       "ssm_delta_rule_bwd_workspace_bytes": [L] * 6 + [I, I],
                       "ssm_delta_rule_bwd_varlen_workspace_bytes": [L] * 6 + [I, I],
                       "ssm_layer_norm_bwd_workspace_bytes": [L] * 2 + [I]}.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = args, S
    _lib = lib
    return lib


# ---------------------------------------------------------------------------
# gated delta rule
# ---------------------------------------------------------------------------
def ssm_delta_rule_fwd_workspace_bytes(batch, seqlen, nheads_k, nheads_v, headdim_k, headdim_v,
                                       dtype=torch.bfloat16):
    return int(_load().ssm_delta_rule_fwd_workspace_bytes(batch, seqlen, nheads_k, nheads_v, headdim_k, headdim_v,
                                                          _DTYPES[dtype]))


def ssm_delta_rule_fwd_varlen_workspace_bytes(nseq, total_len, nheads_k, nheads_v, headdim_k, headdim_v,
                                              dtype=torch.bfloat16):
    return int(_load().ssm_delta_rule_fwd_varlen_workspace_bytes(nseq, total_len, nheads_k, nheads_v, headdim_k,
                                                                 headdim_v, _DTYPES[dtype]))


def ssm_delta_rule_bwd_workspace_bytes(batch, seqlen, nheads_k, nheads_v, headdim_k, headdim_v,
                                       dtype=torch.bfloat16, with_chunk_states=True):
    return int(_load().ssm_delta_rule_bwd_workspace_bytes(batch, seqlen, nheads_k, nheads_v, headdim_k, headdim_v,
                                                          _DTYPES[dtype], int(bool(with_chunk_states))))


def ssm_delta_rule_bwd_varlen_workspace_bytes(nseq, total_len, nheads_k, nheads_v, headdim_k, headdim_v,
                                              dtype=torch.bfloat16, with_chunk_states=True):
    return int(_load().ssm_delta_rule_bwd_varlen_workspace_bytes(nseq, total_len, nheads_k, nheads_v, headdim_k,
                                                                 headdim_v, _DTYPES[dtype],
                                                                 int(bool(with_chunk_states))))


def _tokens(t, name, lead, D, like):
    """(heads, token stride) of a lead + (heads, D) tensor like ``like``."""
    shape = t.shape
    if t.dtype is like.dtype and shape[:-2] == lead and shape[-1] == D and t.get_device() == like.get_device() \
            and t.is_contiguous():
        return shape[-2], shape[-2] * D
    if len(lead) == 1:
        return _heads(t[None], name, 1, lead[0], D, like)
    return _heads(t, name, lead[0], lead[1], D, like)


def _scale(scale, K):
    if K < 1:
        raise ValueError("headdim_k must be at least 1")
    return K ** -0.5 if scale is None else float(scale)


class _Delta:
    """A delta rule call's inputs, checked: sizes, addresses, shapes."""

    def __init__(self, q, k, v, beta, g, scale, initial_state, cu_seqlens):
        self.packed = cu_seqlens is not None
        _, self.dt = _act(q, "q")
        if not (isinstance(k, torch.Tensor) and isinstance(v, torch.Tensor) and isinstance(beta, torch.Tensor)):
            raise TypeError("k, v and beta must be torch.Tensors")
        if self.packed:
            if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
                raise ValueError("q, k and v must be (total_len, heads, headdim)")
            if not isinstance(cu_seqlens, torch.Tensor):
                raise TypeError("cu_seqlens must be a torch.Tensor")
            if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
                raise ValueError("cu_seqlens must be (nseq + 1,) with nseq >= 1")
            lead, self.n = q.shape[:1], cu_seqlens.numel() - 1
            self.cu = _in(cu_seqlens, "cu_seqlens", (self.n + 1,), torch.int32, q)
            L = lead[0]
            chunks = (L // SSM_DELTA_CHUNK + self.n,)
        else:
            if q.dim() != 4 or k.dim() != 4 or v.dim() != 4:
                raise ValueError("q, k and v must be (batch, seqlen, heads, headdim)")
            lead, self.cu = q.shape[:2], None
            self.n, L = lead
            chunks = (self.n, (L + SSM_DELTA_CHUNK - 1) // SSM_DELTA_CHUNK)
        K, V = q.shape[-1], v.shape[-1]
        Hk, qs = _tokens(q, "q", lead, K, q)
        Hkk, ks = _tokens(k, "k", lead, K, q)
        Hv, vs = _tokens(v, "v", lead, V, q)
        if Hkk != Hk:
            raise ValueError("q has %d heads, k %d" % (Hk, Hkk))
        self.lead, self.like, self.gate = lead, q, lead + (Hv,)
        self.out, self.key = lead + (Hv, V), lead + (Hk, K)
        self.state, self.mids = (self.n, Hv, K, V), chunks + (Hv, K + SSM_DELTA_CHUNK, V)
        self.scale = _scale(scale, K)
        self.head = (q.data_ptr(), k.data_ptr(), v.data_ptr(), _in(beta, "beta", self.gate, _F32, q),
                     _opt(g, "g", self.gate, _F32, q), self.scale)
        self.h0 = _opt(initial_state, "initial_state", self.state, _F32, q)
        self.tail = ((self.cu,) if self.packed else ()) + (self.n, L, Hk, Hv, K, V, qs, ks, vs, _DTYPES[self.dt])
        self.sizes = (self.n, L, Hk, Hv, K, V, _DTYPES[self.dt])


def _ptr(t):
    return None if t is None else t.data_ptr()


def _delta_fwd(q, k, v, beta, cu_seqlens, g, scale, initial_state, return_last_state, return_chunk_states, out,
               last_state, chunk_states, workspace, stream):
    lib = _load()
    c = _Delta(q, k, v, beta, g, scale, initial_state, cu_seqlens)
    stream = _other(stream, q)
    out = _out(out, "out", c.out, c.dt, q, stream)
    if return_last_state or last_state is not None:
        last_state = _out(last_state, "last_state", c.state, _F32, q, stream)
    if return_chunk_states or chunk_states is not None:
        chunk_states = _out(chunk_states, "chunk_states", c.mids, _F32, q, stream)
    fn, need = (lib.ssm_delta_rule_fwd_varlen, lib.ssm_delta_rule_fwd_varlen_workspace_bytes) if c.packed else \
        (lib.ssm_delta_rule_fwd, lib.ssm_delta_rule_fwd_workspace_bytes)
    keep, ws, nbytes = _space(workspace, need(*c.sizes), q, stream)
    _call(fn, q, stream, *c.head, out.data_ptr(), _ptr(last_state), c.h0, _ptr(chunk_states), *c.tail, ws, nbytes)
    res = (out,) + tuple(t for t in (last_state, chunk_states) if t is not None)
    return res if len(res) > 1 else out


def ssm_delta_rule_fwd(q, k, v, beta, g=None, scale=None, initial_state=None, return_last_state=False,
                       return_chunk_states=False, out=None, last_state=None, chunk_states=None, workspace=None,
                       stream=None):
    """Gated delta rule over q, k (batch, seqlen, heads_k, headdim_k) and v
    (batch, seqlen, heads_v, headdim_v), which may be slices of wider rows;
    beta and the log decay g (batch, seqlen, heads_v), states (batch, heads_v,
    headdim_k, headdim_v) float32; ``scale`` defaults to headdim_k ** -0.5.

    Returns ``out`` (contiguous), followed by ``last_state`` and by
    ``chunk_states`` where they are asked for or passed (for the gradients:
    per chunk of 64 tokens the state before it and the tokens' v - S^T k, (batch,
    chunks, heads_v, headdim_k + 64, headdim_v) float32).
    """
    return _delta_fwd(q, k, v, beta, None, g, scale, initial_state, return_last_state, return_chunk_states, out,
                      last_state, chunk_states, workspace, stream)


def ssm_delta_rule_fwd_varlen(q, k, v, beta, cu_seqlens, g=None, scale=None, initial_state=None,
                              return_last_state=False, return_chunk_states=False, out=None, last_state=None,
                              chunk_states=None, workspace=None, stream=None):
    """The same over packed sequences: q, k, v (total_len, heads, headdim),
    beta and g (total_len, heads_v), ``cu_seqlens`` (nseq + 1) int32 offsets
    on the device, states (nseq, heads_v, headdim_k, headdim_v).  Rows of
    ``out`` behind the last sequence are not written."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    return _delta_fwd(q, k, v, beta, cu_seqlens, g, scale, initial_state, return_last_state, return_chunk_states, out,
                      last_state, chunk_states, workspace, stream)


_DELTA_GRADS = ("dq", "dk", "dv", "dbeta", "dg", "dinitial_state")


def _delta_bwd(q, k, v, beta, cu_seqlens, dout, g, scale, initial_state, dlast_state, chunk_states, grads, workspace,
               stream):
    lib = _load()
    c = _Delta(q, k, v, beta, g, scale, initial_state, cu_seqlens)
    r = _buffers(grads, _DELTA_GRADS, ("dg",) if g is None else ())
    stream = _other(stream, q)
    args = c.head + (c.h0, _opt(chunk_states, "chunk_states", c.mids, _F32, q), _in(dout, "dout", c.out, c.dt, q),
                     _opt(dlast_state, "dlast_state", c.state, _F32, q))
    for name, shape, dt in (("dq", c.key, c.dt), ("dk", c.key, c.dt), ("dv", c.out, c.dt), ("dbeta", c.gate, _F32),
                            ("dg", c.gate, _F32), ("dinitial_state", c.state, _F32)):
        r[name] = None if name == "dg" and g is None else _out(r.get(name), name, shape, dt, q, stream)
    args += tuple(_ptr(r[name]) for name in _DELTA_GRADS)
    fn, need = (lib.ssm_delta_rule_bwd_varlen, lib.ssm_delta_rule_bwd_varlen_workspace_bytes) if c.packed else \
        (lib.ssm_delta_rule_bwd, lib.ssm_delta_rule_bwd_workspace_bytes)
    keep, ws, nbytes = _space(workspace, need(*c.sizes, int(chunk_states is not None)), q, stream)
    _call(fn, q, stream, *args, *c.tail, ws, nbytes)
    return r


def ssm_delta_rule_bwd(q, k, v, beta, dout, g=None, scale=None, initial_state=None, dlast_state=None,
                       chunk_states=None, grads=None, workspace=None, stream=None):
    """Gradients of ``ssm_delta_rule_fwd`` for the loss sum(dout*out) +
    sum(dlast_state*last_state).  ``chunk_states``: what the forward returned
    for the same inputs (computed again without it).  Returns a dict: dq, dk,
    dv (contiguous, q's dtype); dbeta, dg (None without g), dinitial_state in
    float32.  ``grads`` may supply preallocated outputs under the same keys
    (other keys, or a dg without g, are refused)."""
    return _delta_bwd(q, k, v, beta, None, dout, g, scale, initial_state, dlast_state, chunk_states, grads, workspace,
                      stream)


def ssm_delta_rule_bwd_varlen(q, k, v, beta, cu_seqlens, dout, g=None, scale=None, initial_state=None,
                              dlast_state=None, chunk_states=None, grads=None, workspace=None, stream=None):
    """Gradients of ``ssm_delta_rule_fwd_varlen``, returned as
    ``ssm_delta_rule_bwd`` does.  Rows of the per-token gradients behind the
    last sequence are not written."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    return _delta_bwd(q, k, v, beta, cu_seqlens, dout, g, scale, initial_state, dlast_state, chunk_states, grads,
                      workspace, stream)


def ssm_delta_state_update(state, q, k, v, beta, g=None, scale=None, out=None, stream=None):
    """One decode step of the delta rule: ``state`` (batch, heads_v,
    headdim_k, headdim_v) float32 is updated in place; q, k (batch, heads_k,
    headdim_k) and v (batch, heads_v, headdim_v) may be slices of wider rows;
    returns ``out`` (batch, heads_v, headdim_v) in q's dtype."""
    lib = _load()
    _, dt = _act(q, "q")
    if not (isinstance(k, torch.Tensor) and isinstance(v, torch.Tensor)):
        raise TypeError("k and v must be torch.Tensors")
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3:
        raise ValueError("q, k and v must be (batch, heads, headdim)")
    lead, K, V = q.shape[:1], q.shape[2], v.shape[2]
    batch = lead[0]
    Hk, qs = _tokens(q, "q", lead, K, q)
    Hkk, ks = _tokens(k, "k", lead, K, q)
    Hv, vs = _tokens(v, "v", lead, V, q)
    if Hkk != Hk:
        raise ValueError("q has %d heads, k %d" % (Hk, Hkk))
    args = (_in(state, "state", (batch, Hv, K, V), _F32, q), q.data_ptr(), k.data_ptr(), v.data_ptr(),
            _in(beta, "beta", (batch, Hv), _F32, q), _opt(g, "g", (batch, Hv), _F32, q),
            _scale(scale, K))
    stream = _other(stream, q)
    out = _out(out, "out", (batch, Hv, V), dt, q, stream)
    _call(lib.ssm_delta_state_update, q, stream, *args, out.data_ptr(), batch, Hk, Hv, K, V, qs, ks, vs, _DTYPES[dt])
    return out


# ---------------------------------------------------------------------------
# layer norm
# ---------------------------------------------------------------------------
def _rows(t, name, shape, like):
    """(rows, row stride) of a (..., dim) tensor whose rows may lie apart (a
    slice of wider rows) at one stride."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dim() < 1 or t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype != like.dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, like.dtype))
    if t.get_device() != like.get_device():
        raise ValueError("%s is on %s, expected %s" % (name, t.device, like.device))
    dim = shape[-1]
    rows = 1
    for n in shape[:-1]:
        rows *= n
    if t.is_contiguous():
        return rows, dim
    step, run = None, 1  # every dimension with more than one row has to continue the stride of those behind it
    for n, st in zip(reversed(shape[:-1]), reversed(t.stride()[:-1])):
        if n > 1:
            if step is None:
                step = st
            elif st != run * step:
                step = -1
                break
            run *= n
    if (dim > 1 and t.stride(-1) != 1) or (step is not None and step < dim):
        raise ValueError("%s must hold a row's values together and its rows at one stride" % name)
    return rows, dim if step is None else step


def ssm_layer_norm_fwd(x, weight=None, bias=None, residual=None, eps=1e-5, return_residual=True, out=None,
                       residual_out=None, stream=None):
    """Layer norm over the last dimension of ``x`` (..., dim), weight and bias
    (dim,) float32.  With ``residual`` (x's shape) the sum x + residual, in
    x's dtype, is what is normalised.  x and residual may be slices of wider
    rows.

    Returns ``out`` (contiguous); with ``residual``, unless
    ``return_residual`` is false, ``(out, residual_out)``: the sum too.
    """
    lib = _load()
    _, dt = _act(x)
    if x.dim() < 1:
        raise ValueError("x must be (..., dim)")
    shape = x.shape
    rows, xs = _rows(x, "x", shape, x)
    dim, rs = shape[-1], shape[-1]
    if residual is not None:
        _, rs = _rows(residual, "residual", shape, x)
    elif residual_out is not None:
        raise ValueError("residual_out given without residual")
    args = (x.data_ptr(), _ptr(residual), _opt(weight, "weight", (dim,), _F32, x), _opt(bias, "bias", (dim,), _F32, x),
            eps)
    stream = _other(stream, x)
    out = _out(out, "out", x, dt, x, stream)
    both = residual is not None and (return_residual or residual_out is not None)
    if both:
        residual_out = _out(residual_out, "residual_out", x, dt, x, stream)
    _call(lib.ssm_layer_norm_fwd, x, stream, *args, out.data_ptr(), _ptr(residual_out), rows, dim, xs, rs, _DTYPES[dt])
    return (out, residual_out) if both else out


def ssm_layer_norm_bwd_workspace_bytes(rows, dim, dtype=torch.bfloat16):
    return int(_load().ssm_layer_norm_bwd_workspace_bytes(rows, dim, _DTYPES[dtype]))


def ssm_layer_norm_bwd(x, dout, weight=None, dresidual=None, eps=1e-5, grads=None, workspace=None, stream=None):
    """Gradients of ``ssm_layer_norm_fwd`` for the loss sum(dout*out) +
    sum(dresidual*residual_out).  ``x`` is what was normalised: the forward's
    ``residual_out``, or its x without a residual.  Returns a dict: dx (x's
    dtype; the gradient of x and of the residual alike), dweight, dbias
    (float32).  ``grads`` may supply preallocated outputs; keys that are no
    output of the call are refused."""
    lib = _load()
    _, dt = _act(x)
    if x.dim() < 1:
        raise ValueError("x must be (..., dim)")
    shape = x.shape
    rows, xs = _rows(x, "x", shape, x)
    dim = shape[-1]
    args = (x.data_ptr(), _opt(weight, "weight", (dim,), _F32, x), eps, _in(dout, "dout", shape, dt, x),
            _opt(dresidual, "dresidual", shape, dt, x))
    r = _buffers(grads, ("dx", "dweight", "dbias"), ())
    stream = _other(stream, x)
    r["dx"] = _out(r.get("dx"), "dx", x, dt, x, stream)
    for n in ("dweight", "dbias"):
        r[n] = _out(r.get(n), n, (dim,), _F32, x, stream)
    keep, ws, nbytes = _space(workspace, lib.ssm_layer_norm_bwd_workspace_bytes(rows, dim, _DTYPES[dt]), x, stream)
    _call(lib.ssm_layer_norm_bwd, x, stream, *args, r["dx"].data_ptr(), r["dweight"].data_ptr(), r["dbias"].data_ptr(),
          rows, dim, xs, _DTYPES[dt], ws, nbytes)
    return r
