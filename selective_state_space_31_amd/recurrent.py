"""Thin Python binding of the C ABI in include/ssm_recurrent.h.

Argument marshalling only, in the manner of ``ops``: the functions keep the C
names, every step runs in the HIP kernels of libssm_scan.so, PyTorch supplies
device memory and the current HIP stream, and a missing library fails loudly.
Tensors are on one HIP device, which need not be the current one.  ``stream``
is a raw HIP stream handle (the tensors' device's current stream by default);
what is allocated here for a call on another stream comes from that stream's
memory, so the caller orders the two streams for the inputs and the results
alone.
"""
import ctypes

import torch

from . import ops
from .ops import _DTYPES, _check, _raise

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


# the current stream's handle of a device index, without building a Stream object where torch lets one
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_F32, _Tensor, _empty_like = torch.float32, torch.Tensor, torch.empty_like


def _act(x, name="x"):
    if not isinstance(x, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if x.dtype not in _DTYPES:
        raise TypeError("activations must be float32 or bfloat16, got %s" % x.dtype)
    return x.get_device(), x.dtype


def _in(t, name, shape, dtype, like):
    """The address of input ``t``, which has to have this shape and type and
    be contiguous on ``like``'s device (``ops._check`` says what is wrong)."""
    if not (type(t) is _Tensor and t.dtype is dtype and t.shape == shape
            and t.get_device() == like.get_device() and t.is_contiguous()):
        _check(t, name, shape, dtype, like.device)
    return t.data_ptr()


def _opt(t, name, shape, dtype, like):
    if t is None:
        return None
    return _in(t, name, shape, dtype, like)


def _new(like, shape, dtype, stream):
    """A new tensor for a call on ``stream`` (None: the current one), on
    ``like``'s device; ``shape`` may be ``like`` itself (its shape and type)."""
    if stream is None:
        # (empty_like is the quickest; it would keep the strides of a slice)
        if (shape is like or (dtype is like.dtype and shape == like.shape)) and like.is_contiguous():
            return _empty_like(like)
        if shape is like:
            shape = like.shape
        return like.new_empty(shape, dtype=dtype)
    # On another stream the memory has to come from that stream's pool: a block
    # of the current stream may still be in use by work queued there.  The
    # caller will read it from the current stream, which the pool has to know.
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, device=like.device)):
        t = like.new_empty(like.shape if shape is like else shape, dtype=dtype)
    t.record_stream(torch.cuda.current_stream(like.device))
    return t


def _out(t, name, shape, dtype, like, stream):
    """The output buffer ``t``, checked, or a new one."""
    if t is None:
        return _new(like, shape, dtype, stream)
    _in(t, name, like.shape if shape is like else shape, dtype, like)
    return t


def _space(workspace, need, like, stream):
    """(the caller's workspace or a new one, its address, its bytes)."""
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = _new(like, (need,), torch.uint8, stream)
        return workspace, workspace.data_ptr(), need
    if workspace.device != like.device or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous and on %s" % like.device)
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _buffers(grads, names, absent):
    """A copy of ``grads``, whose keys have to be among ``names``; buffers for
    outputs that this call does not have (``absent``) are refused."""
    if not grads:
        return {}
    for k, t in grads.items():
        if k not in names:
            raise ValueError("grads: %r is none of %s" % (k, ", ".join(names)))
        if t is not None and k in absent:
            raise ValueError("grads: %s is given, but this call has no such output" % k)
    return dict(grads)


def _other(stream, like):
    """``stream`` where it is another one than ``like``'s device's current
    stream, else None."""
    index = like.get_device()
    if index < 0 or not like.is_cuda:
        raise ValueError("tensors must be on a HIP device, got %s" % like.device)
    return None if stream is None or stream == _raw_stream(index) else stream


def _call(fn, like, stream, *args):
    """fn(*args, stream) with ``like``'s device current."""
    index = like.get_device()
    if stream is None:
        stream = _raw_stream(index)
    if _current_device() == index:
        rc = fn(*args, stream)
    else:
        with torch.cuda.device(index):
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


def _gated_inputs(x, rgate, igate, A, z, rgate_bias, igate_bias, normalize, initial_state, cu_seqlens):
    """Sizes and addresses of a gated scan's inputs: (type, sequences, row
    length, dim, shape of the chunk states, the C call's first arguments, the
    initial state, the offsets)."""
    _, dt = _act(x)
    cu = None
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
        cu = _in(cu_seqlens, "cu_seqlens", (n + 1,), torch.int32, x)
    head = (_in(x, "x", x.shape, dt, x), _in(rgate, "rgate", x.shape, dt, x), _in(igate, "igate", x.shape, dt, x),
            _in(A, "A", (dim,), _F32, x), _opt(rgate_bias, "rgate_bias", (dim,), _F32, x),
            _opt(igate_bias, "igate_bias", (dim,), _F32, x), int(bool(normalize)), _opt(z, "z", x.shape, dt, x))
    h0 = _opt(initial_state, "initial_state", (n, dim), _F32, x)
    chunks = (L + SSM_GATED_CHUNK - 1) // SSM_GATED_CHUNK
    return dt, n, L, dim, (n, chunks, dim) if cu_seqlens is None else (chunks, dim), head, h0, cu


def _gated_fwd(x, rgate, igate, A, cu_seqlens, z, rgate_bias, igate_bias, normalize, initial_state,
               return_last_state, return_chunk_states, out, last_state, chunk_states, workspace,
               stream):
    lib = _load()
    dt, n, L, dim, mid, head, h0, cu = _gated_inputs(x, rgate, igate, A, z, rgate_bias, igate_bias, normalize,
                                                     initial_state, cu_seqlens)
    stream, code = _other(stream, x), _DTYPES[dt]
    out = _out(out, "out", x, dt, x, stream)
    if return_last_state or last_state is not None:
        last_state = _out(last_state, "last_state", (n, dim), _F32, x if initial_state is None else initial_state,
                          stream)
    if return_chunk_states or chunk_states is not None:
        chunk_states = _out(chunk_states, "chunk_states", mid, _F32, x, stream)
    args = head + (out.data_ptr(), None if last_state is None else last_state.data_ptr(), h0,
                   None if chunk_states is None else chunk_states.data_ptr())
    if cu is None:
        keep, ws, nbytes = _space(workspace, lib.ssm_gated_scan_fwd_workspace_bytes(n, L, dim, code), x, stream)
        _call(lib.ssm_gated_scan_fwd, x, stream, *args, n, L, dim, code, ws, nbytes)
    else:
        keep, ws, nbytes = _space(workspace, lib.ssm_gated_scan_fwd_varlen_workspace_bytes(n, L, dim, code), x, stream)
        _call(lib.ssm_gated_scan_fwd_varlen, x, stream, *args, cu, n, L, dim, code, ws, nbytes)
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


_GATED_GRADS = ("dx", "drgate", "digate", "dz", "dA", "drgate_bias", "digate_bias", "dinitial_state")


def _gated_bwd(x, rgate, igate, A, cu_seqlens, dout, z, rgate_bias, igate_bias, normalize,
               initial_state, dlast_state, chunk_states, grads, workspace, stream):
    lib = _load()
    dt, n, L, dim, mid, head, h0, cu = _gated_inputs(x, rgate, igate, A, z, rgate_bias, igate_bias, normalize,
                                                     initial_state, cu_seqlens)
    g = _buffers(grads, _GATED_GRADS, ("dz",) if z is None else ())
    stream, code = _other(stream, x), _DTYPES[dt]
    args = head + (h0, _opt(chunk_states, "chunk_states", mid, _F32, x), _in(dout, "dout", x.shape, dt, x),
                   _opt(dlast_state, "dlast_state", (n, dim), _F32, x))
    for k in _GATED_GRADS[:4]:
        g[k] = None if k == "dz" and z is None else _out(g.get(k), k, x, dt, x, stream)
    for k in ("dA", "drgate_bias", "digate_bias"):
        g[k] = _out(g.get(k), k, (dim,), _F32, A, stream)
    g["dinitial_state"] = _out(g.get("dinitial_state"), "dinitial_state", (n, dim), _F32,
                               x if initial_state is None else initial_state, stream)
    args += tuple(None if g[k] is None else g[k].data_ptr() for k in _GATED_GRADS)
    have = int(chunk_states is not None)
    if cu is None:
        keep, ws, nbytes = _space(workspace, lib.ssm_gated_scan_bwd_workspace_bytes(n, L, dim, code, have), x, stream)
        _call(lib.ssm_gated_scan_bwd, x, stream, *args, n, L, dim, code, ws, nbytes)
    else:
        keep, ws, nbytes = _space(workspace, lib.ssm_gated_scan_bwd_varlen_workspace_bytes(n, L, dim, code, have), x, stream)
        _call(lib.ssm_gated_scan_bwd_varlen, x, stream, *args, cu, n, L, dim, code, ws, nbytes)
    return g


def ssm_gated_scan_bwd(x, rgate, igate, A, dout, z=None, rgate_bias=None, igate_bias=None,
                       normalize=True, initial_state=None, dlast_state=None, chunk_states=None,
                       grads=None, workspace=None, stream=None):
    """Gradients of ``ssm_gated_scan_fwd`` for the loss sum(dout*out) +
    sum(dlast_state*last_state).  ``chunk_states``: what the forward returned
    for the same inputs (computed again without it).  Returns a dict: dx,
    drgate, digate, dz (None without z) in x's dtype; dA, drgate_bias,
    digate_bias, dinitial_state in float32.  ``grads`` may supply preallocated
    outputs under the same keys (other keys, or a dz without z, are refused)."""
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
    _, dt = _act(x)
    if x.dim() != 2:
        raise ValueError("x must be (batch, dim)")
    shape = x.shape
    batch, dim = shape
    args = (_in(state, "state", shape, _F32, x), _in(x, "x", shape, dt, x), _in(rgate, "rgate", shape, dt, x),
            _in(igate, "igate", shape, dt, x), _in(A, "A", (dim,), _F32, x),
            _opt(rgate_bias, "rgate_bias", (dim,), _F32, x), _opt(igate_bias, "igate_bias", (dim,), _F32, x),
            int(bool(normalize)), _opt(z, "z", shape, dt, x))
    stream = _other(stream, x)
    out = _out(out, "out", x, dt, x, stream)
    _call(lib.ssm_gated_state_update, x, stream, *args, out.data_ptr(), batch, dim, _DTYPES[dt])
    return out


# ---------------------------------------------------------------------------
# norm and rotation of queries and keys
# ---------------------------------------------------------------------------
def _heads(t, name, batch, L, D, like):
    """(heads, token stride) of a (batch, seqlen, heads, headdim) tensor whose
    tokens may lie apart (a slice of wider rows) but nothing else."""
    if t.dim() != 4 or t.shape[0] != batch or t.shape[1] != L or t.shape[3] != D:
        raise ValueError("%s has shape %s, expected (%d, %d, heads, %d)"
                         % (name, tuple(t.shape), batch, L, D))
    if t.dtype != like.dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, like.dtype))
    if t.get_device() != like.get_device():
        raise ValueError("%s is on %s, expected %s" % (name, t.device, like.device))
    H = t.shape[2]
    if t.is_contiguous():
        return H, H * D
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


def _rot_inputs(q, k, inv_freq, q_weight, k_weight, positions, eps, interleaved):
    """Sizes and the C call's first arguments."""
    _act(q, "q")
    if q.dim() != 4:
        raise ValueError("q must be (batch, seqlen, heads, headdim)")
    batch, L, Hq, D = q.shape
    Hq, qs = _heads(q, "q", batch, L, D, q)
    Hk, ks = _heads(k, "k", batch, L, D, q) if k is not None else (0, 0)
    if k is not None and Hk == 0:
        raise ValueError("k has no heads: pass None")
    if inv_freq is not None and (not isinstance(inv_freq, torch.Tensor) or inv_freq.dim() != 1):
        raise ValueError("inv_freq must be (rotary_dim / 2,)")
    R = 0 if inv_freq is None else 2 * inv_freq.numel()
    head = (q.data_ptr(), None if k is None else k.data_ptr(), _opt(q_weight, "q_weight", (D,), _F32, q),
            _opt(k_weight, "k_weight", (D,), _F32, q), _opt(inv_freq, "inv_freq", (R // 2,), _F32, q),
            _opt(positions, "positions", (batch, L), torch.int32, q), eps, int(bool(interleaved)))
    return head, (batch, L, Hq, Hk, D, R, qs, ks, _DTYPES[q.dtype])


def ssm_qk_norm_rotate_fwd(q, k, inv_freq, q_weight=None, k_weight=None, positions=None, eps=1e-6,
                           interleaved=False, q_out=None, k_out=None, stream=None):
    """RMS norm of each head's row of q (batch, seqlen, heads_q, headdim) and
    k (.., heads_k, ..), then the position rotation of its first 2 *
    len(inv_freq) values.  q and k may be slices of wider rows (a fused
    projection); ``k`` may be None, ``inv_freq`` None leaves the norm alone,
    ``positions`` (batch, seqlen) int32 defaults to the token's index.

    Returns ``(q_out, k_out)``, contiguous (k_out None without k)."""
    lib = _load()
    head, sizes = _rot_inputs(q, k, inv_freq, q_weight, k_weight, positions, eps, interleaved)
    if k is None and (k_out is not None or k_weight is not None):
        raise ValueError("k_out or k_weight given without k")
    stream = _other(stream, q)
    q_out = _out(q_out, "q_out", q, q.dtype, q, stream)
    if k is not None:
        k_out = _out(k_out, "k_out", k, q.dtype, k, stream)
    _call(lib.ssm_qk_norm_rotate_fwd, q, stream, *head, q_out.data_ptr(),
          None if k is None else k_out.data_ptr(), *sizes)
    return q_out, k_out


def ssm_qk_norm_rotate_bwd_workspace_bytes(batch, seqlen, nheads_q, nheads_k, headdim):
    return int(_load().ssm_qk_norm_rotate_bwd_workspace_bytes(batch, seqlen, nheads_q, nheads_k,
                                                              headdim))


def ssm_qk_norm_rotate_bwd(q, k, inv_freq, dq_out, dk_out, q_weight=None, k_weight=None,
                           positions=None, eps=1e-6, interleaved=False, grads=None, workspace=None,
                           stream=None):
    """Gradients of ``ssm_qk_norm_rotate_fwd`` for the loss sum(dq_out*q_out)
    + sum(dk_out*k_out): a dict of dq, dk (contiguous, q's dtype; dk None
    without k) and dq_weight, dk_weight (float32; None without the weight).
    ``grads`` may supply preallocated outputs; keys that are no output of the
    call are refused."""
    lib = _load()
    head, sizes = _rot_inputs(q, k, inv_freq, q_weight, k_weight, positions, eps, interleaved)
    batch, L, Hq, Hk, D = sizes[:5]
    if k is None and (dk_out is not None or k_weight is not None):
        raise ValueError("dk_out or k_weight given without k")
    head += (_in(dq_out, "dq_out", q.shape, q.dtype, q),
             None if k is None else _in(dk_out, "dk_out", k.shape, q.dtype, q))
    g = _buffers(grads, ("dq", "dk", "dq_weight", "dk_weight"),
                 [n for n, t in (("dk", k), ("dq_weight", q_weight), ("dk_weight", k_weight)) if t is None])
    stream = _other(stream, q)
    g["dq"] = _out(g.get("dq"), "dq", q, q.dtype, q, stream)
    g["dk"] = None if k is None else _out(g.get("dk"), "dk", k, q.dtype, k, stream)
    for n, w in (("dq_weight", q_weight), ("dk_weight", k_weight)):
        g[n] = None if w is None else _out(g.get(n), n, (D,), _F32, w, stream)
    head += tuple(None if g[n] is None else g[n].data_ptr() for n in ("dq", "dk", "dq_weight", "dk_weight"))
    keep, ws, nbytes = _space(workspace, lib.ssm_qk_norm_rotate_bwd_workspace_bytes(batch, L, Hq, Hk, D), q, stream)
    _call(lib.ssm_qk_norm_rotate_bwd, q, stream, *head, *sizes, ws, nbytes)
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
    ``bias``).  ``grads`` may supply preallocated outputs; keys that are no
    output of the call are refused."""
    lib = _load()
    _, dt = _act(x)
    if x.dim() != 3:
        raise ValueError("x must be (batch, seqlen, dim)")
    batch, L, dim = x.shape
    if weight.dim() != 2:
        raise ValueError("weight must be (dim, width)")
    W = weight.shape[1]
    st = (batch, dim, W - 1)
    args = (_in(x, "x", x.shape, dt, x), _in(weight, "weight", (dim, W), _F32, x), _opt(bias, "bias", (dim,), _F32, x),
            _opt(initial_conv_state, "initial_conv_state", st, dt, x), _in(dout, "dout", x.shape, dt, x),
            _opt(dfinal_conv_state, "dfinal_conv_state", st, dt, x))
    g = _buffers(grads, ("dx", "dweight", "dbias", "dinitial_conv_state"),
                 [n for n, t in (("dbias", bias), ("dinitial_conv_state", initial_conv_state)) if t is None])
    stream = _other(stream, x)
    g["dx"] = _out(g.get("dx"), "dx", x, dt, x, stream)
    g["dweight"] = _out(g.get("dweight"), "dweight", (dim, W), _F32, weight, stream)
    g["dbias"] = None if bias is None else _out(g.get("dbias"), "dbias", (dim,), _F32, bias, stream)
    g["dinitial_conv_state"] = None if initial_conv_state is None else \
        _out(g.get("dinitial_conv_state"), "dinitial_conv_state", st, dt, initial_conv_state, stream)
    args += tuple(None if g[k] is None else g[k].data_ptr() for k in ("dx", "dweight", "dbias", "dinitial_conv_state"))
    keep, ws, nbytes = _space(workspace, lib.ssm_causal_conv1d_bwd_workspace_bytes(batch, L, dim, W), x, stream)
    _call(lib.ssm_causal_conv1d_bwd, x, stream, *args, batch, L, dim, W, int(bool(silu)), _DTYPES[dt], ws, nbytes)
    return g
