"""Packed batches of many short sequences, empty ones among them, in chunks and
token by token (GPU)."""
import numpy as np
import pytest
import torch

import selective_state_space_31_amd as pkg
from tests._layer import Delta, check_forward, check_grads

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("n,hk,hv,K,V,lengths", [
    (40, 8, 16, 64, 24, [1]),               # one token each
    (40, 8, 16, 64, 24, [1, 0, 1, 1]),      # the odd one empty
    (20, 32, 64, 40, 33, [2, 5, 1, 4]),     # a few each
    (20, 32, 64, 40, 33, [0] * 19 + [66]),  # all in one, beyond a chunk
    (30, 8, 16, 64, 24, [0] * 9 + [1] + [0, 0] + [4] + [0] * 17)], ids=str)  # token by token
def test_many_short(n, hk, hv, K, V, lengths, dtype):
    """Outputs, states, chunk states (and their unused places), the rows behind
    the last sequence, and the gradients from those states."""
    lengths = (lengths * n)[:n]
    cu = np.concatenate([[0], np.cumsum(lengths)])
    end, T = int(cu[-1]), int(cu[-1]) + 3
    by_token = T <= 8
    assert by_token == (pkg.ssm_delta_rule_fwd_varlen_workspace_bytes(n, T, hk, hv, K, V) == 0)
    p = Delta((T,), n, hk, hv, K, V, dtype, DEV, seed=T, fused=True)
    off = torch.tensor(cu, dtype=torch.int32, device=DEV)
    out = torch.full((T, hv, V), 5.0, dtype=p.v.dtype, device=DEV)
    mids = torch.full((T // 64 + n, hv, K + 64, V), 7.0, device=DEV)
    _, last, _ = pkg.ssm_delta_rule_fwd_varlen(*p.args(), off, return_last_state=True, out=out, chunk_states=mids, **p.kw())
    r = pkg.ssm_delta_rule_bwd_varlen(*p.args(), off, p.dout, dlast_state=p.dlast, chunk_states=mids, **p.kw())
    torch.cuda.synchronize()
    assert (out[end:] == 5.0).all()
    used = torch.zeros(T // 64 + n, dtype=torch.bool)
    for s in range(n):
        a, z = int(cu[s]), int(cu[s + 1])
        at, c = a // 64 + s, (z - a + 63) // 64
        used[at:at + c] = True
        if s % 5 and z - a < 60:
            continue
        check_forward(p, out[a:z], last[s], s, a, z, what="sequence %d" % s, mids=mids[at:at + c])
        check_grads(p, {k: t[s] if k == "dinitial_state" else t[a:z] for k, t in r.items()}, s, a, z, what="sequence %d" % s)
    assert (mids[~used.to(DEV)] == 7.0).all()
