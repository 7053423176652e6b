"""Thin Python binding of the C ABI in include/ssm_recurrent.h.

Argument marshalling only, in the manner of ``ops``: the functions keep the C
names, every step runs in the HIP kernels of libssm_scan.so, PyTorch supplies
device memory and the current HIP stream, and a missing library fails loudly.
Tensors are on one HIP device, which need not be the current one.  ``stream``
is a raw HIP stream handle (the tensors' device's current stream by default);
what is allocated here for a call on another stream is kept until that stream
is done with it.
"""
import ctypes

import torch

from . import ops
from .ops import _DTYPES, _check, _ptr, _raise

SSM_GATED_CHUNK = 16

EXPORTS = ("ssm_gated_scan_fwd", "ssm_gated_scan_fwd_workspace_bytes", "ssm_gated_scan_fwd_varlen",
           "ssm_gated_scan_fwd_varlen_workspace_bytes", "ssm_gated_scan_bwd",
           "ssm_gated_scan_bwd_workspace_bytes", "ssm_gated_scan_bwd_varlen",
           "ssm_gated_scan_bwd_varlen_workspace_bytes", "ssm_gated_state_update",
           "ssm_qk_norm_rotate_fwd", "ssm_qk_norm_rotate_bwd",
           "ssm_qk_norm_rotate_bwd_workspace_bytes", "ssm_causal_conv1d_bwd",
           "ssm_causal_conv1d_bwd_workspace_bytes")

_lib = None


def _load():
    global _lib
    if _lib is not None:
        return _lib
    lib = ops.load_library()
    P, I, L, S, F = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    sig = {
        "ssm_gated_scan_fwd": [P] * 6 + [I] + [P] * 5 + [L] * 3 + [I, P, S, P],
        "ssm_gated_scan_fwd_varlen": [P] * 6 + [I] + [P] * 6 + [L] * 3 + [I, P, S, P],
        "ssm_gated_scan_bwd": [P] * 6 + [I] + [P] * 13 + [L] * 3 + [I, P, S, P],
        "ssm_gated_scan_bwd_varlen": [P] * 6 + [I] + [P] * 14 + [L] * 3 + [I, P, S, P],
        "ssm_gated_state_update": [P] * 7 + [I] + [P] * 2 + [L] * 2 + [I, P],
        "ssm_qk_norm_rotate_fwd": [P] * 6 + [F, I] + [P] * 2 + [L] * 8 + [I, P],
        "ssm_qk_norm_rotate_bwd": [P] * 6 + [F, I] + [P] * 6 + [L] * 8 + [I, P, S, P],
        "ssm_causal_conv1d_bwd": [P] * 10 + [L] * 4 + [I, I, P, S, P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = args, I
    for name, args in {"ssm_gated_scan_fwd_workspace_bytes": [L] * 3 + [I],
                       "ssm_gated_scan_fwd_varlen_workspace_bytes": [L] * 3 + [I],
                       "ssm_gated_scan_bwd_workspace_bytes": [L] * 3 + [I, I],
                       "ssm_gated_scan_bwd_varlen_workspace_bytes": [L] * 3 + [I, I],
                       "ssm_qk_norm_rotate_bwd_workspace_bytes": [L] * 5,
                       "ssm_causal_conv1d_bwd_workspace_bytes": [L] * 4}.items():
        f = getattr(lib, name)
        f.argtypes, f.restype = args, S
    _lib = lib
    return lib


def _act(x, name="x"):
    if not isinstance(x, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if x.dtype not in _DTYPES:
        raise TypeError("activations must be float32 or bfloat16, got %s" % x.dtype)
    return x.device, x.dtype


def _buf(t, name, shape, dtype, dev, new):
    """The output buffer ``t``, checked, or a new one (noted in ``new``)."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=dev)
        new.append(t)
        return t
    _check(t, name, shape, dtype, dev)
    return t


def _space(workspace, need, dev, new):
    if workspace is None:
        if need == 0:
            return None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        new.append(workspace)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on %s" % dev)
    return workspace, workspace.numel() * workspace.element_size()


def _call(fn, dev, stream, new, *args):
    """fn(*args, stream) with ``dev`` current; ``new`` are the tensors
    allocated for the call."""
    if dev.type != "cuda":
        raise ValueError("tensors must be on a HIP device, got %s" % dev)
    current = torch.cuda.current_stream(dev).cuda_stream
    if stream is None:
        stream = current
    elif stream != current:
        ext = torch.cuda.ExternalStream(stream, device=dev)
        for t in new:
            t.record_stream(ext)
    if torch.cuda.current_device() == dev.index:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, stream)
    if rc != 0:
        _raise(rc)


# ---------------------------------------------------------------------------
# gated linear recurrence
# ---------------------------------------------------------------------------
def ssm_gated_scan_fwd_workspace_bytes(batch, seqlen, dim, dtype=torch.bfloat16):
    return int(_load().ssm_gated_scan_fwd_workspace_bytes(batch, seqlen, dim, _DTYPES[dtype]))


def ssm_gated_scan_fwd_varlen_workspace_bytes(nseq, total_len, dim, dtype=torch.bfloat16):
    return int(_load().ssm_gated_scan_fwd_varlen_workspace_bytes(nseq, total_len, dim,
                                                                 _DTYPES[dtype]))


def ssm_gated_scan_bwd_workspace_bytes(batch, seqlen, dim, dtype=torch.bfloat16,
                                       with_chunk_states=True):
    return int(_load().ssm_gated_scan_bwd_workspace_bytes(batch, seqlen, dim, _DTYPES[dtype],
                                                          int(bool(with_chunk_states))))


def ssm_gated_scan_bwd_varlen_workspace_bytes(nseq, total_len, dim, dtype=torch.bfloat16,
                                              with_chunk_states=True):
    return int(_load().ssm_gated_scan_bwd_varlen_workspace_bytes(nseq, total_len, dim,
                                                                 _DTYPES[dtype],
                                                                 int(bool(with_chunk_states))))


def _gated_check(x, rgate, igate, A, z, rgate_bias, igate_bias, initial_state, cu_seqlens):
    """Shapes of a gated scan's inputs: (packed, sequences, row length, dim)."""
    dev, dt = _act(x)
    if cu_seqlens is None:
        if x.dim() != 3:
            raise ValueError("x must be (batch, seqlen, dim)")
        n, L, dim = x.shape
    else:
        if x.dim() != 2:
            raise ValueError("x must be (total_len, dim)")
        if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
            raise ValueError("cu_seqlens must be (nseq + 1,) with nseq >= 1")
        L, dim = x.shape
        n = cu_seqlens.numel() - 1
        _check(cu_seqlens, "cu_seqlens", (n + 1,), torch.int32, dev)
    f32 = torch.float32
    for t, name in ((x, "x"), (rgate, "rgate"), (igate, "igate")):
        _check(t, name, x.shape, dt, dev)
    _check(z, "z", x.shape, dt, dev, optional=True)
    _check(A, "A", (dim,), f32, dev)
    _check(rgate_bias, "rgate_bias", (dim,), f32, dev, optional=True)
    _check(igate_bias, "igate_bias", (dim,), f32, dev, optional=True)
    _check(initial_state, "initial_state", (n, dim), f32, dev, optional=True)
    chunks = (L + SSM_GATED_CHUNK - 1) // SSM_GATED_CHUNK
    mid = (n, chunks, dim) if cu_seqlens is None else (chunks, dim)
    return dev, dt, n, L, dim, mid


def _gated_fwd(x, rgate, igate, A, cu_seqlens, z, rgate_bias, igate_bias, normalize, initial_state,
               return_last_state, return_chunk_states, out, last_state, chunk_states, workspace,
               stream):
    lib = _load()
    dev, dt, n, L, dim, mid = _gated_check(x, rgate, igate, A, z, rgate_bias, igate_bias,
                                           initial_state, cu_seqlens)
    new = []
    out = _buf(out, "out", x.shape, dt, dev, new)
    if return_last_state or last_state is not None:
        last_state = _buf(last_state, "last_state", (n, dim), torch.float32, dev, new)
    if return_chunk_states or chunk_states is not None:
        chunk_states = _buf(chunk_states, "chunk_states", mid, torch.float32, dev, new)
    head = (_ptr(x), _ptr(rgate), _ptr(igate), _ptr(A), _ptr(rgate_bias), _ptr(igate_bias),
            int(bool(normalize)), _ptr(z), _ptr(out), _ptr(last_state), _ptr(initial_state),
            _ptr(chunk_states))
    if cu_seqlens is None:
        need = lib.ssm_gated_scan_fwd_workspace_bytes(n, L, dim, _DTYPES[dt])
        ws, nbytes = _space(workspace, need, dev, new)
        _call(lib.ssm_gated_scan_fwd, dev, stream, new, *head, n, L, dim, _DTYPES[dt], _ptr(ws),
              nbytes)
    else:
        need = lib.ssm_gated_scan_fwd_varlen_workspace_bytes(n, L, dim, _DTYPES[dt])
        ws, nbytes = _space(workspace, need, dev, new)
        _call(lib.ssm_gated_scan_fwd_varlen, dev, stream, new, *head, _ptr(cu_seqlens), n, L, dim,
              _DTYPES[dt], _ptr(ws), nbytes)
    res = (out,) + tuple(t for t in (last_state, chunk_states) if t is not None)
    return res if len(res) > 1 else out


def ssm_gated_scan_fwd(x, rgate, igate, A, z=None, rgate_bias=None, igate_bias=None, normalize=True,
                       initial_state=None, return_last_state=False, return_chunk_states=False,
                       out=None, last_state=None, chunk_states=None, workspace=None, stream=None):
    """Gated linear recurrence over (batch, seqlen, dim) activations; A, the
    biases (dim,) and states (batch, dim) float32.

    Returns ``out``, followed by ``last_state`` and by ``chunk_states`` where
    they are asked for or passed (``chunk_states`` is for the gradients).
    """
    return _gated_fwd(x, rgate, igate, A, None, z, rgate_bias, igate_bias, normalize, initial_state,
                      return_last_state, return_chunk_states, out, last_state, chunk_states,
                      workspace, stream)


def ssm_gated_scan_fwd_varlen(x, rgate, igate, A, cu_seqlens, z=None, rgate_bias=None,
                              igate_bias=None, normalize=True, initial_state=None,
                              return_last_state=False, return_chunk_states=False, out=None,
                              last_state=None, chunk_states=None, workspace=None, stream=None):
    """The same over packed sequences: activations (total_len, dim),
    ``cu_seqlens`` (nseq + 1) int32 offsets on the device, states (nseq,
    dim).  Rows of ``out`` behind the last sequence are not written."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    return _gated_fwd(x, rgate, igate, A, cu_seqlens, z, rgate_bias, igate_bias, normalize,
                      initial_state, return_last_state, return_chunk_states, out, last_state,
                      chunk_states, workspace, stream)


def _gated_bwd(x, rgate, igate, A, cu_seqlens, dout, z, rgate_bias, igate_bias, normalize,
               initial_state, dlast_state, chunk_states, grads, workspace, stream):
    lib = _load()
    dev, dt, n, L, dim, mid = _gated_check(x, rgate, igate, A, z, rgate_bias, igate_bias,
                                           initial_state, cu_seqlens)
    f32, new = torch.float32, []
    _check(dout, "dout", x.shape, dt, dev)
    _check(dlast_state, "dlast_state", (n, dim), f32, dev, optional=True)
    _check(chunk_states, "chunk_states", mid, f32, dev, optional=True)
    g = dict(grads or {})
    for k in ("dx", "drgate", "digate", "dz"):
        g[k] = None if k == "dz" and z is None else _buf(g.get(k), k, x.shape, dt, dev, new)
    for k in ("dA", "drgate_bias", "digate_bias"):
        g[k] = _buf(g.get(k), k, (dim,), f32, dev, new)
    g["dinitial_state"] = _buf(g.get("dinitial_state"), "dinitial_state", (n, dim), f32, dev, new)
    head = (_ptr(x), _ptr(rgate), _ptr(igate), _ptr(A), _ptr(rgate_bias), _ptr(igate_bias),
            int(bool(normalize)), _ptr(z), _ptr(initial_state), _ptr(chunk_states), _ptr(dout),
            _ptr(dlast_state), _ptr(g["dx"]), _ptr(g["drgate"]), _ptr(g["digate"]), _ptr(g["dz"]),
            _ptr(g["dA"]), _ptr(g["drgate_bias"]), _ptr(g["digate_bias"]), _ptr(g["dinitial_state"]))
    have = int(chunk_states is not None)
    if cu_seqlens is None:
        need = lib.ssm_gated_scan_bwd_workspace_bytes(n, L, dim, _DTYPES[dt], have)
        ws, nbytes = _space(workspace, need, dev, new)
        _call(lib.ssm_gated_scan_bwd, dev, stream, new, *head, n, L, dim, _DTYPES[dt], _ptr(ws),
              nbytes)
    else:
        need = lib.ssm_gated_scan_bwd_varlen_workspace_bytes(n, L, dim, _DTYPES[dt], have)
        ws, nbytes = _space(workspace, need, dev, new)
        _call(lib.ssm_gated_scan_bwd_varlen, dev, stream, new, *head, _ptr(cu_seqlens), n, L, dim,
              _DTYPES[dt], _ptr(ws), nbytes)
    return g


def ssm_gated_scan_bwd(x, rgate, igate, A, dout, z=None, rgate_bias=None, igate_bias=None,
                       normalize=True, initial_state=None, dlast_state=None, chunk_states=None,
                       grads=None, workspace=None, stream=None):
    """Gradients of ``ssm_gated_scan_fwd`` for the loss sum(dout*out) +
    sum(dlast_state*last_state).  ``chunk_states``: what the forward returned
    for the same inputs (computed again without it).  Returns a dict: dx,
    drgate, digate, dz (None without z) in x's dtype; dA, drgate_bias,
    digate_bias, dinitial_state in float32.  ``grads`` may supply preallocated
    outputs under the same keys."""
    return _gated_bwd(x, rgate, igate, A, None, dout, z, rgate_bias, igate_bias, normalize,
                      initial_state, dlast_state, chunk_states, grads, workspace, stream)


def ssm_gated_scan_bwd_varlen(x, rgate, igate, A, cu_seqlens, dout, z=None, rgate_bias=None,
                              igate_bias=None, normalize=True, initial_state=None,
                              dlast_state=None, chunk_states=None, grads=None, workspace=None,
                              stream=None):
    """Gradients of ``ssm_gated_scan_fwd_varlen``, returned as
    ``ssm_gated_scan_bwd`` does.  Rows of the per-token gradients behind the
    last sequence are not written."""
    if cu_seqlens is None:
        raise ValueError("cu_seqlens is required")
    return _gated_bwd(x, rgate, igate, A, cu_seqlens, dout, z, rgate_bias, igate_bias, normalize,
                      initial_state, dlast_state, chunk_states, grads, workspace, stream)


def ssm_gated_state_update(state, x, rgate, igate, A, z=None, rgate_bias=None, igate_bias=None,
                           normalize=True, out=None, stream=None):
    """One decode step of the gated recurrence: ``state`` (batch, dim) float32
    is updated in place; returns ``out`` (batch, dim) in x's dtype."""
    lib = _load()
    dev, dt = _act(x)
    if x.dim() != 2:
        raise ValueError("x must be (batch, dim)")
    batch, dim = x.shape
    f32, new = torch.float32, []
    _check(state, "state", (batch, dim), f32, dev)
    for t, name in ((x, "x"), (rgate, "rgate"), (igate, "igate")):
        _check(t, name, x.shape, dt, dev)
    _check(z, "z", x.shape, dt, dev, optional=True)
    _check(A, "A", (dim,), f32, dev)
    _check(rgate_bias, "rgate_bias", (dim,), f32, dev, optional=True)
    _check(igate_bias, "igate_bias", (dim,), f32, dev, optional=True)
    out = _buf(out, "out", x.shape, dt, dev, new)
    _call(lib.ssm_gated_state_update, dev, stream, new, _ptr(state), _ptr(x), _ptr(rgate),
          _ptr(igate), _ptr(A), _ptr(rgate_bias), _ptr(igate_bias), int(bool(normalize)), _ptr(z),
          _ptr(out), batch, dim, _DTYPES[dt])
    return out


# ---------------------------------------------------------------------------
# norm and rotation of queries and keys
# ---------------------------------------------------------------------------
def _heads(t, name, batch, L, D, dt, dev):
    """(heads, token stride) of a (batch, seqlen, heads, headdim) tensor whose
    tokens may lie apart (a slice of wider rows) but nothing else."""
    if t.dim() != 4 or t.shape[0] != batch or t.shape[1] != L or t.shape[3] != D:
        raise ValueError("%s has shape %s, expected (%d, %d, heads, %d)"
                         % (name, tuple(t.shape), batch, L, D))
    if t.dtype != dt:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dt))
    if t.device != dev:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, dev))
    H = t.shape[2]
    sb, sl, sh, sd = t.stride()
    if L > 1:
        step = sl
    elif batch > 1:
        step = sb
    else:
        step = H * D
    if sd != 1 or (H > 1 and sh != D) or (batch > 1 and L > 0 and sb != L * step) or step < H * D:
        raise ValueError("%s must hold a token's heads together and its tokens at one stride" % name)
    return H, step


def _rot_check(q, k, inv_freq, q_weight, k_weight, positions):
    dev, dt = _act(q, "q")
    if q.dim() != 4:
        raise ValueError("q must be (batch, seqlen, heads, headdim)")
    batch, L, Hq, D = q.shape
    Hq, qs = _heads(q, "q", batch, L, D, dt, dev)
    Hk, ks = _heads(k, "k", batch, L, D, dt, dev) if k is not None else (0, 0)
    if k is not None and Hk == 0:
        raise ValueError("k has no heads: pass None")
    f32 = torch.float32
    if inv_freq is not None and (not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1):
        raise ValueError("inv_freq must be (rotary_dim / 2,)")
    R = 0 if inv_freq is None else 2 * inv_freq.numel()
    _check(inv_freq, "inv_freq", (R // 2,), f32, dev, optional=True)
    _check(q_weight, "q_weight", (D,), f32, dev, optional=True)
    _check(k_weight, "k_weight", (D,), f32, dev, optional=True)
    _check(positions, "positions", (batch, L), torch.int32, dev, optional=True)
    return dev, dt, batch, L, Hq, Hk, D, R, qs, ks


def ssm_qk_norm_rotate_fwd(q, k, inv_freq, q_weight=None, k_weight=None, positions=None, eps=1e-6,
                           interleaved=False, q_out=None, k_out=None, stream=None):
    """RMS norm of each head's row of q (batch, seqlen, heads_q, headdim) and
    k (.., heads_k, ..), then the position rotation of its first 2 *
    len(inv_freq) values.  q and k may be slices of wider rows (a fused
    projection); ``k`` may be None, ``inv_freq`` None leaves the norm alone,
    ``positions`` (batch, seqlen) int32 defaults to the token's index.

    Returns ``(q_out, k_out)``, contiguous (k_out None without k)."""
    lib = _load()
    dev, dt, batch, L, Hq, Hk, D, R, qs, ks = _rot_check(q, k, inv_freq, q_weight, k_weight, positions)
    new = []
    q_out = _buf(q_out, "q_out", (batch, L, Hq, D), dt, dev, new)
    if k is not None:
        k_out = _buf(k_out, "k_out", (batch, L, Hk, D), dt, dev, new)
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out or k_weight given without k")
    _call(lib.ssm_qk_norm_rotate_fwd, dev, stream, new, _ptr(q), _ptr(k), _ptr(q_weight),
          _ptr(k_weight), _ptr(inv_freq), _ptr(positions), eps, int(bool(interleaved)), _ptr(q_out),
          _ptr(k_out), batch, L, Hq, Hk, D, R, qs, ks, _DTYPES[dt])
    return q_out, k_out


def ssm_qk_norm_rotate_bwd_workspace_bytes(batch, seqlen, nheads_q, nheads_k, headdim):
    return int(_load().ssm_qk_norm_rotate_bwd_workspace_bytes(batch, seqlen, nheads_q, nheads_k,
                                                              headdim))


def ssm_qk_norm_rotate_bwd(q, k, inv_freq, dq_out, dk_out, q_weight=None, k_weight=None,
                           positions=None, eps=1e-6, interleaved=False, grads=None, workspace=None,
                           stream=None):
    """Gradients of ``ssm_qk_norm_rotate_fwd`` for the loss sum(dq_out*q_out)
    + sum(dk_out*k_out): a dict of dq, dk (contiguous, q's dtype; dk None
    without k) and dq_weight, dk_weight (float32; None without the weight)."""
    lib = _load()
    dev, dt, batch, L, Hq, Hk, D, R, qs, ks = _rot_check(q, k, inv_freq, q_weight, k_weight, positions)
    f32, new = torch.float32, []
    if k is None and (dk_out is not None or k_weight is not None):
        raise ValueError("dk_out or k_weight given without k")
    _check(dq_out, "dq_out", (batch, L, Hq, D), dt, dev)
    if k is not None:
        _check(dk_out, "dk_out", (batch, L, Hk, D), dt, dev)
    g = dict(grads or {})
    g["dq"] = _buf(g.get("dq"), "dq", (batch, L, Hq, D), dt, dev, new)
    g["dk"] = None if k is None else _buf(g.get("dk"), "dk", (batch, L, Hk, D), dt, dev, new)
    for n, w in (("dq_weight", q_weight), ("dk_weight", k_weight)):
        g[n] = None if w is None else _buf(g.get(n), n, (D,), f32, dev, new)
    need = lib.ssm_qk_norm_rotate_bwd_workspace_bytes(batch, L, Hq, Hk, D)
    ws, nbytes = _space(workspace, need, dev, new)
    _call(lib.ssm_qk_norm_rotate_bwd, dev, stream, new, _ptr(q), _ptr(k), _ptr(q_weight),
          _ptr(k_weight), _ptr(inv_freq), _ptr(positions), eps, int(bool(interleaved)), _ptr(dq_out),
          _ptr(dk_out), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dq_weight"]), _ptr(g["dk_weight"]),
          batch, L, Hq, Hk, D, R, qs, ks, _DTYPES[dt], _ptr(ws), nbytes)
    return g


# ---------------------------------------------------------------------------
# gradients of the causal convolution
# ---------------------------------------------------------------------------
def ssm_causal_conv1d_bwd_workspace_bytes(batch, seqlen, dim, width):
    return int(_load().ssm_causal_conv1d_bwd_workspace_bytes(batch, seqlen, dim, width))


def ssm_causal_conv1d_bwd(x, weight, dout, bias=None, initial_conv_state=None,
                          dfinal_conv_state=None, silu=True, grads=None, workspace=None,
                          stream=None):
    """Gradients of ``ssm_causal_conv1d_fwd`` for the loss sum(dout*out) +
    sum(dfinal_conv_state*final_conv_state): a dict of dx and
    dinitial_conv_state (x's dtype; the latter None without
    ``initial_conv_state``), dweight and dbias (float32; None without
    ``bias``).  ``grads`` may supply preallocated outputs."""
    lib = _load()
    dev, dt = _act(x)
    if x.dim() != 3:
        raise ValueError("x must be (batch, seqlen, dim)")
    batch, L, dim = x.shape
    if weight.dim() != 2:
        raise ValueError("weight must be (dim, width)")
    W = weight.shape[1]
    f32, new, st = torch.float32, [], (batch, dim, W - 1)
    _check(x, "x", x.shape, dt, dev)
    _check(dout, "dout", x.shape, dt, dev)
    _check(weight, "weight", (dim, W), f32, dev)
    _check(bias, "bias", (dim,), f32, dev, optional=True)
    _check(initial_conv_state, "initial_conv_state", st, dt, dev, optional=True)
    _check(dfinal_conv_state, "dfinal_conv_state", st, dt, dev, optional=True)
    g = dict(grads or {})
    g["dx"] = _buf(g.get("dx"), "dx", x.shape, dt, dev, new)
    g["dweight"] = _buf(g.get("dweight"), "dweight", (dim, W), f32, dev, new)
    g["dbias"] = None if bias is None else _buf(g.get("dbias"), "dbias", (dim,), f32, dev, new)
    g["dinitial_conv_state"] = None if initial_conv_state is None else \
        _buf(g.get("dinitial_conv_state"), "dinitial_conv_state", st, dt, dev, new)
    need = lib.ssm_causal_conv1d_bwd_workspace_bytes(batch, L, dim, W)
    ws, nbytes = _space(workspace, need, dev, new)
    _call(lib.ssm_causal_conv1d_bwd, dev, stream, new, _ptr(x), _ptr(weight), _ptr(bias),
          _ptr(initial_conv_state), _ptr(dout), _ptr(dfinal_conv_state), _ptr(g["dx"]),
          _ptr(g["dweight"]), _ptr(g["dbias"]), _ptr(g["dinitial_conv_state"]), batch, L, dim, W,
          int(bool(silu)), _DTYPES[dt], _ptr(ws), nbytes)
    return g
