"""dg is the rest of larger sums that cancel: its error against float64 stays
below that of the same chunked form in plain float32 products and sums (GPU).

The kernels sum dg's long sums in float64 and round a chunk's addition to a
state once, so of the plain form's errors those of single products are left; the
mean ratio of the two errors (geometric, over the shapes below, whose ratios
scatter by about a quarter to either side) has to stay below 0.95, which the
form with float32 sums throughout does not reach (1.1).
"""
import numpy as np
import pytest
import torch

import selective_state_space_31_amd as pkg
from oracle import delta
from tests._layer import Delta
from tests._recurrent import np64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
C = 64


def plain_dg(p, s):
    """dg of sequence s (L a multiple of 64): the chunked form in float32 torch operations on the CPU."""
    q, k, v, beta, g, do = (getattr(p, n)[s].float().cpu().movedim(1, 0) for n in ("q", "k", "v", "beta", "g", "dout"))
    hv, L, V = v.shape
    K, r = q.shape[-1], hv // q.shape[0]
    cut = lambda t: t.unflatten(1, (L // C, C))
    q, k = cut(q.repeat_interleave(r, 0)) * K ** -0.5, cut(k.repeat_interleave(r, 0))
    v, do, beta, g = cut(v), cut(do), cut(beta), cut(g)
    tr = lambda t: t.transpose(-1, -2)
    G = torch.cumsum(g.double(), -1)
    low = torch.ones(C, C, dtype=torch.bool).tril()
    D = torch.exp(torch.where(low, G[..., :, None] - G[..., None, :], -np.inf).float())
    gam, d = torch.exp(G.float())[..., None], torch.exp((G[..., -1:] - G).float())[..., None]
    kk, P = D.tril(-1) * (k @ tr(k)), D * (q @ tr(k))
    T = torch.linalg.solve_triangular(torch.eye(C) + beta[..., None] * kk, torch.eye(C).expand_as(kk), upper=False)
    b = beta[..., None]
    W, Uv, kd, n = T @ (b * gam * k), T @ (b * v), d * k, L // C
    S, before, U = p.h0[s].cpu(), [], []
    for c in range(n):
        before.append(S)
        U.append(Uv[:, c] - W[:, c] @ S)
        S = gam[:, c, -1:] * S + tr(kd[:, c]) @ U[-1]
    before, U, last = torch.stack(before, 1), torch.stack(U, 1), S
    dS, behind, dU = p.dlast[s].cpu(), [], []
    for c in range(n - 1, -1, -1):
        behind.append(dS)
        dU.append(tr(P[:, c]) @ do[:, c] + kd[:, c] @ dS)
        dS = gam[:, c, -1:] * dS + tr(gam[:, c] * q[:, c]) @ do[:, c] - tr(W[:, c]) @ dU[-1]
    behind, dU = torch.stack(behind[::-1], 1), torch.stack(dU[::-1], 1)
    Y = tr(T) @ dU
    E, F = -b * (Y @ tr(U)).tril(-1) * D, (do @ tr(U)) * D
    read = (q * (gam * (do @ tr(before)) + F @ k) + k * (E @ k - gam * ((b * Y) @ tr(before)))).sum(-1)
    dG = read - (k * (tr(E) @ k + tr(F) @ q + d * (U @ tr(behind)))).sum(-1)
    dG[..., -1] += (torch.cat([before[:, 1:], last[:, None]], 1) * behind).sum((-1, -2))
    return dG.flip(-1).cumsum(-1).flip(-1).flatten(1).movedim(0, 1)


def test_dg_against_the_plain_form():
    ratios = []
    for L, hk, hv, K, V in ((320, 1, 2, 64, 64), (192, 2, 4, 128, 40), (640, 1, 1, 32, 48), (128, 1, 1, 256, 64), (256, 3, 3, 80, 77)):
        p = Delta((2, L), 2, hk, hv, K, V, "fp32", DEV, seed=L)
        got = pkg.ssm_delta_rule_bwd(*p.args(), p.dout, dlast_state=p.dlast, **p.kw())["dg"]
        torch.cuda.synchronize()
        for s in range(2):
            h, dout, dlast = p.host(s)
            ref = delta.delta_rule_bwd(dout=dout, dlast=dlast, **h)["dg"]
            rms = lambda x: np.sqrt(((np64(x) - ref) ** 2).mean())
            ratios.append(rms(got[s]) / rms(plain_dg(p, s)))
    mean = np.exp(np.mean(np.log(ratios)))
    print("dg's error over the plain form's:", np.round(ratios, 2), "mean %.2f" % mean)
    assert mean <= 0.95, ratios
