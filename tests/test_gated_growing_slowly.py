"""Factors just above 1 (A > 0): their rounding must not line up (GPU)."""
import pytest

import selective_state_space_31_amd as pkg
from oracle import gated as og
from tests import _gated_bound as gb
from tests._recurrent import Gated, within

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("A", [0.147, 0.08, 0.01])
@pytest.mark.parametrize("b,L,d", [(2, 60, 70), (2, 500, 70), (300, 301, 66)])
def test_growth_within_its_bound(b, L, d, A, normalize):
    """With r = 2, -la log2 e reaches -0.187, -0.102 and -0.013."""
    p = Gated((b, L), b, d, "fp32", "cuda:0", 51, gate=False, bias=False, normalize=normalize)
    p.r.fill_(2.0)
    p.A.fill_(A)
    out, last, mid = pkg.ssm_gated_scan_fwd(*p.args(), return_last_state=True, return_chunk_states=True, **p.kw())
    h, dout, dl = p.host()
    ref, rl, _ = og.gated_scan(**h)
    bo, bl, _, _ = gb.forward(**h)
    within(out, ref, bo, "out")
    within(last, rl, bl, "last")
    g = pkg.ssm_gated_scan_bwd(*p.args(), p.dout, dlast_state=p.dlast, chunk_states=mid, **p.kw())
    rg, bg = og.gated_scan_bwd(dout=dout, dlast=dl, **h), gb.backward(dout=dout, dlast=dl, **h)
    for k in rg:
        if k != "dz":
            within(g[k], rg[k], bg[k], k)
