"""Outputs of the delta rule where states are large against them: a key's old
value is a hundred or a thousand times the new one, which the rule replaces it
by (GPU).

Every key has 64 entries of +-1/8, so |k|^2 = 1 and its products with a state
are exact up to the sums.  With beta = 1, q = k, scale 1 and no decay a token
reads what it has just written: the exact output is v, a value of the output's
type.  A float32 sum that comes within E of v is rounded to v itself where E is
below half of v's step, and is off by at most 2 E where it is not: the result's
own rounding adds nothing else.

E, by root mean square: a chunk's output goes through four products one after
another (state by key, the triangular solve, query by state, the triangle by the
solution), of at most 8, 2, 8 and 2 matrix instructions of 32 terms by at most
six partial products each: 120 roundings of at most half a step of a sum whose
size is that of S^T k, which a state of size s gives as s in root mean square.
Half a step is 2^-24, a uniform error in it 2^-24 / sqrt(3), and independent
ones add up by their squares: sqrt(120 / 3) 2^-24 s a chunk, and what a chunk
leaves in the state reaches the next ones undiminished at most.
"""
import numpy as np
import pytest
import torch

import selective_state_space_31_amd as pkg
from oracle import delta
from tests._recurrent import DT, np64

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def keys(rng, shape, K):
    k = np.zeros(shape + (K,), np.float32)
    flat = k.reshape(-1, K)
    for row in flat:
        row[rng.permutation(K)[:64]] = rng.choice([-0.125, 0.125], 64)
    return k


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("size", [100.0, 1000.0])
@pytest.mark.parametrize("b,L,hk,hv,K,V", [(1, 64, 1, 2, 128, 128), (2, 150, 2, 2, 64, 77), (1, 90, 1, 1, 256, 40),
                                           (4, 64, 16, 64, 128, 33), (3, 17, 1, 1, 128, 128)], ids=str)
@pytest.mark.parametrize("packed", [False, True])
def test_a_large_old_value_is_replaced(packed, b, L, hk, hv, K, V, size, dtype):
    rng = np.random.default_rng(int(size) + L + K)
    t = lambda a, dt=torch.float32: torch.from_numpy(np.ascontiguousarray(a)).to(dt).to(DEV)
    k = t(keys(rng, (b, L, hk), K), DT[dtype])
    v = t(rng.standard_normal((b, L, hv, V)).astype(np.float32), DT[dtype])
    h0 = t((size * rng.standard_normal((b, hv, K, V))).astype(np.float32))
    beta = torch.ones(b, L, hv, device=DEV)
    if packed:
        cu = torch.arange(0, b * L + 1, L, dtype=torch.int32, device=DEV)
        f = lambda a: a.flatten(0, 1)
        out = pkg.ssm_delta_rule_fwd_varlen(f(k), f(k), f(v), f(beta), cu, scale=1.0, initial_state=h0).view(b, L, hv, V)
    else:
        out = pkg.ssm_delta_rule_fwd(k, k, v, beta, scale=1.0, initial_state=h0)
    torch.cuda.synchronize()
    got, want = np64(out), np64(v)
    ref, _, _ = delta.delta_rule(np64(k[0]), np64(k[0]), np64(v[0]), np64(beta[0]), None, 1.0, np64(h0[0]))
    assert np.abs(ref - want[0]).max() < 1e-9 * size  # (the exact output is v)
    chunks = (L + 63) // 64
    rms = np.sqrt(((got - want) ** 2).mean())
    assert rms <= 2.0 * np.sqrt(chunks * 120 / 3.0) * 2.0 ** -24 * size, rms
