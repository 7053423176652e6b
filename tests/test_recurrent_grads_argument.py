"""The ``grads`` argument of the recurrent operators' gradients: names that
are no output, and buffers for outputs that the call does not have, are
refused (CPU: on the host, before the device is looked at)."""
import pytest
import torch

import selective_state_space_31_amd as pkg

X, A = torch.zeros(2, 5, 6), torch.zeros(6)
CU = torch.tensor([0, 2, 5], dtype=torch.int32)
Q, K, F, W = torch.zeros(1, 5, 2, 8), torch.zeros(1, 5, 1, 8), torch.zeros(4), torch.zeros(8)


def scan(**kw):
    return pkg.ssm_gated_scan_bwd(X, X, X, A, X, **kw)


def packed(**kw):
    return pkg.ssm_gated_scan_bwd_varlen(X[0], X[0], X[0], A, CU, X[0], **kw)


def rotate(k=None, **kw):
    return pkg.ssm_qk_norm_rotate_bwd(Q, k, F, Q, k, **kw)


def conv(**kw):
    return pkg.ssm_causal_conv1d_bwd(X, torch.zeros(6, 4), X, **kw)


@pytest.mark.parametrize("call,grads", [
    (scan, dict(dX=X)), (scan, dict(drgate_bais=A)), (scan, dict(dX=None)), (scan, dict(dz=X)), (packed, dict(dcu=X[0])),
    (packed, dict(dz=X[0])), (rotate, dict(dw=W)), (rotate, dict(dk=K)), (rotate, dict(dq_weight=W)),
    (rotate, dict(dk_weight=W)), (conv, dict(dw=torch.zeros(6, 4))), (conv, dict(dbias=A)),
    (conv, dict(dinitial_conv_state=torch.zeros(2, 6, 3)))])
def test_refused(call, grads):
    with pytest.raises(ValueError, match=list(grads)[0]):
        call(grads=grads)


@pytest.mark.parametrize("call,grads", [(scan, dict(dz=None, dx=X)), (packed, dict(dA=A)), (rotate, dict(dk=None, dq=Q)),
                                        (conv, dict(dbias=None, dx=X))])
def test_not_refused_for_its_names(call, grads):
    """None stands for an output that is not there; the refusal that comes is
    the device's."""
    with pytest.raises(ValueError, match="HIP device"):
        call(grads=grads)
