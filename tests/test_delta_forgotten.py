"""dg where the decay rounds to 0: exactly 0, whatever the sums that it is the
rest of leave (GPU)."""
import pytest
import torch

import selective_state_space_31_amd as pkg
from tests._layer import Delta, check_grads

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
GONE = ((0, -105.0), (3, -106.0), (40, -200.0), (63, -1e30), (64, float("-inf")), (100, float("-inf")), (101, -1000.0),
        (149, -110.0))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("hk,hv,K,V", [(2, 2, 64, 64), (1, 3, 80, 33), (32, 64, 64, 20), (1, 2, 256, 40)])
@pytest.mark.parametrize("packed", [False, True])
def test_no_slope(packed, hk, hv, K, V, dtype):
    b = 1 if packed else 2
    p = Delta((150,) if packed else (b, 150), b, hk, hv, K, V, dtype, DEV, seed=K)
    g = p.g if packed else p.g[b - 1]
    for t, x in GONE:
        g[t] = x
    if packed:
        cu = torch.tensor([0, 150], dtype=torch.int32, device=DEV)
        r = pkg.ssm_delta_rule_bwd_varlen(*p.args(), cu, p.dout, dlast_state=p.dlast, **p.kw())
        one = {n: t if n != "dinitial_state" else t[0] for n, t in r.items()}
    else:
        r = pkg.ssm_delta_rule_bwd(*p.args(), p.dout, dlast_state=p.dlast, **p.kw())
        one = {n: t[b - 1] for n, t in r.items()}
    torch.cuda.synchronize()
    for t, _ in GONE:
        assert (one["dg"][t] == 0).all(), t
    kept = [t for t in range(150) if t not in dict(GONE)]
    assert (one["dg"][kept] != 0).all()
    if packed:
        check_grads(p, one, 0, 0, 150)
    else:
        check_grads(p, one, b - 1)
