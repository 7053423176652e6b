"""Packed sequences of many heads, which as whole ones would go by two column
blocks a workgroup, and the results of which do not depend on that (GPU)."""
import numpy as np
import pytest
import torch

import selective_state_space_31_amd as pkg
from tests._layer import Delta, check_forward, check_grads

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
LENGTHS = [70, 0, 1, 129, 64, 30, 9]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hk,hv,K,V", [(16, 48, 64, 77), (60, 60, 32, 60), (14, 56, 128, 80), (40, 40, 32, 60), (2, 2, 128, 96),
                                       (18, 18, 64, 129)])
def test_packed_many_heads(hk, hv, K, V, dtype):
    """Outputs, states and gradients of every sequence."""
    cu = np.concatenate([[0], np.cumsum(LENGTHS)])
    n, T = len(LENGTHS), int(cu[-1])
    p = Delta((T,), n, hk, hv, K, V, dtype, DEV, seed=hv, fused=True)
    off = torch.tensor(cu, dtype=torch.int32, device=DEV)
    out, last, mids = pkg.ssm_delta_rule_fwd_varlen(*p.args(), off, return_last_state=True, return_chunk_states=True, **p.kw())
    only = pkg.ssm_delta_rule_fwd_varlen(*p.args(), off, **p.kw())
    r = pkg.ssm_delta_rule_bwd_varlen(*p.args(), off, p.dout, dlast_state=p.dlast, chunk_states=mids, **p.kw())
    torch.cuda.synchronize()
    assert torch.equal(only, out)
    for s in range(n):
        a, z = int(cu[s]), int(cu[s + 1])
        at = a // 64 + s
        check_forward(p, out[a:z], last[s], s, a, z, what="sequence %d" % s, mids=mids[at:at + (z - a + 63) // 64])
        check_grads(p, {k: t[s] if k == "dinitial_state" else t[a:z] for k, t in r.items()}, s, a, z, what="sequence %d" % s)


def test_a_sequence_is_the_same_alone():
    """Bit for bit the results of packed and whole calls with this sequence and
    two of the heads alone, and of a whole call with all heads."""
    cu = np.concatenate([[0], np.cumsum(LENGTHS)])
    p = Delta((int(cu[-1]),), len(LENGTHS), 40, 40, 64, 77, "bf16", DEV, seed=3)
    off = torch.tensor(cu, dtype=torch.int32, device=DEV)
    out, last = pkg.ssm_delta_rule_fwd_varlen(*p.args(), off, return_last_state=True, **p.kw())
    a, z = int(cu[3]), int(cu[4])
    cut = lambda t: t[a:z, 7:9].contiguous()
    one = torch.tensor([0, z - a], dtype=torch.int32, device=DEV)
    o2, l2 = pkg.ssm_delta_rule_fwd_varlen(*(cut(t) for t in p.args()), one, g=cut(p.g), initial_state=p.h0[3:4, 7:9].contiguous(),
                                           return_last_state=True)
    o3, l3 = pkg.ssm_delta_rule_fwd(*(t[a:z][None].contiguous() for t in p.args()), g=p.g[a:z][None].contiguous(),
                                    initial_state=p.h0[3:4], return_last_state=True)
    o4, l4 = pkg.ssm_delta_rule_fwd(*(torch.cat([cut(t)[None]] * 40) for t in p.args()), g=torch.cat([cut(p.g)[None]] * 40),
                                    initial_state=torch.cat([p.h0[3:4, 7:9]] * 40), return_last_state=True)
    torch.cuda.synchronize()
    assert torch.equal(out[a:z, 7:9], o2) and torch.equal(last[3, 7:9], l2[0])
    assert torch.equal(out[a:z], o3[0]) and torch.equal(last[3], l3[0])
    for i in (0, 39):  # (80 heads of five column blocks: two blocks a workgroup)
        assert torch.equal(o2, o4[i]) and torch.equal(l2[0], l4[i])
