"""Pins of the float64 references of the delta rule and of layer norm: closed
forms, independent forms, automatic gradients and differences (CPU)."""
import numpy as np
import pytest
import torch

from oracle import delta, layer_norm


def problem(seed, L=9, hk=2, hv=4, K=5, V=3, decay=True):
    r = np.random.default_rng(seed)
    k = r.standard_normal((L, hk, K))
    return dict(q=r.standard_normal((L, hk, K)), k=k / np.sqrt((k * k).sum(-1, keepdims=True)), v=r.standard_normal((L, hv, V)),
                beta=r.uniform(0, 1, (L, hv)), g=-np.exp(r.standard_normal((L, hv))) if decay else None,
                h0=r.standard_normal((hv, K, V)))


@pytest.mark.parametrize("decay", [True, False])
def test_states_are_the_unrolled_products(decay):
    """S_t = sum_j beta_j a_j+1..t P_t .. P_j+1 k_j v_j^T + a_1..t P_t .. P_1 S_0 with
    P = I - beta k k^T, whatever the order the update is written in."""
    p = problem(1, decay=decay)
    out, last, before = delta.delta_rule(**p)
    L, hv = p["beta"].shape
    for h in range(hv):
        S = p["h0"][h]
        for t in range(L):
            np.testing.assert_allclose(before[t, h], S, rtol=1e-12, atol=1e-13)
            k = p["k"][t, h // 2]
            a = 1.0 if p["g"] is None else np.exp(p["g"][t, h])
            S = a * (np.eye(5) - p["beta"][t, h] * np.outer(k, k)) @ S + p["beta"][t, h] * np.outer(k, p["v"][t, h])
            np.testing.assert_allclose(out[t, h], 5 ** -0.5 * S.T @ p["q"][t, h // 2], rtol=1e-12, atol=1e-13)
        np.testing.assert_allclose(last[h], S, rtol=1e-12, atol=1e-13)


def test_all_tokens_as_one_triangular_system():
    """(I + A) E = V - gamma K S0 with A_ij = beta_j D_ij k_i . k_j for j < i."""
    p = problem(2, hk=1, hv=1)
    G = np.cumsum(p["g"][:, 0])
    k, b, S0 = p["k"][:, 0], p["beta"][:, 0], p["h0"][0]
    D = np.tril(np.exp(G[:, None] - G[None, :]))
    E = np.linalg.solve(np.eye(9) + np.tril(b[None] * D * (k @ k.T), -1), p["v"][:, 0] - np.exp(G)[:, None] * (k @ S0))
    np.testing.assert_allclose(delta.missing(**p)[:, 0], E, rtol=1e-11, atol=1e-12)
    out, last, _ = delta.delta_rule(**p)
    q = p["q"][:, 0]
    np.testing.assert_allclose(out[:, 0], 5 ** -0.5 * (np.exp(G)[:, None] * (q @ S0) + (b[None] * D * (q @ k.T)) @ E), rtol=1e-11)
    np.testing.assert_allclose(last[0], np.exp(G[-1]) * S0 + k.T @ ((b * np.exp(G[-1] - G))[:, None] * E), rtol=1e-11)


def test_limits():
    """beta 1 and a unit key: what was written reads back.  beta 0: nothing is
    written.  Orthogonal keys: plain linear attention.  g = -inf: forgotten."""
    p = problem(3, decay=False)
    p["beta"][:] = 1.0
    _, _, before = delta.delta_rule(**dict(p, q=p["k"], scale=1.0))
    out, _, _ = delta.delta_rule(**dict(p, q=p["k"], scale=1.0))
    np.testing.assert_allclose(out, p["v"], rtol=1e-12, atol=1e-12)
    p["beta"][:] = 0.0
    _, last, _ = delta.delta_rule(**p)
    np.testing.assert_array_equal(last, p["h0"])
    o = problem(4, L=5, hk=1, hv=1, decay=False)
    o["k"][:, 0] = np.linalg.qr(np.random.default_rng(5).standard_normal((5, 5)))[0]
    out, _, _ = delta.delta_rule(**dict(o, h0=None))
    s = np.tril(o["q"][:, 0] @ o["k"][:, 0].T) * 5 ** -0.5
    np.testing.assert_allclose(out[:, 0], s @ (o["beta"] * o["v"][:, 0]), rtol=1e-11, atol=1e-12)
    f = problem(6)
    f["g"][4] = -np.inf
    _, a, _ = delta.delta_rule(**f)
    _, b, _ = delta.delta_rule(**{n: (t[4:] if n not in ("h0",) else None) for n, t in f.items()})
    np.testing.assert_allclose(a, b, rtol=1e-14, atol=1e-15)


def test_delta_gradients_are_the_automatic_ones():
    p = problem(7)
    t = {n: torch.tensor(a, requires_grad=True) for n, a in p.items()}
    r = np.random.default_rng(8)
    dout, dlast = r.standard_normal((9, 4, 3)), r.standard_normal((4, 5, 3))
    S, loss = t["h0"], 0.0
    for i in range(9):
        q, k = t["q"][i].repeat_interleave(2, 0), t["k"][i].repeat_interleave(2, 0)
        S = S * torch.exp(t["g"][i])[:, None, None]
        u = t["beta"][i][:, None] * (t["v"][i] - (S * k[:, :, None]).sum(1))
        S = S + k[:, :, None] * u[:, None, :]
        loss = loss + ((S * q[:, :, None]).sum(1) * 5 ** -0.5 * torch.tensor(dout[i])).sum()
    (loss + (S * torch.tensor(dlast)).sum()).backward()
    got = delta.delta_rule_bwd(dout=dout, dlast=dlast, **p)
    for n in ("q", "k", "v", "beta", "g"):
        np.testing.assert_allclose(got["d" + n], t[n].grad.numpy(), rtol=1e-10, atol=1e-11, err_msg=n)
    np.testing.assert_allclose(got["dinitial_state"], t["h0"].grad.numpy(), rtol=1e-10, atol=1e-11)


def test_delta_gradients_by_differences():
    p = problem(9)
    r = np.random.default_rng(10)
    dout, dlast = r.standard_normal((9, 4, 3)), r.standard_normal((4, 5, 3))
    got = delta.delta_rule_bwd(dout=dout, dlast=dlast, **p)

    def loss(v):
        o, l, _ = delta.delta_rule(**v)
        return (o * dout).sum() + (l * dlast).sum()
    for n, grad in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("beta", "dbeta"), ("g", "dg"), ("h0", "dinitial_state")):
        way, e = r.standard_normal(p[n].shape), 1e-5
        want = (loss(dict(p, **{n: p[n] + e * way})) - loss(dict(p, **{n: p[n] - e * way}))) / (2 * e)
        np.testing.assert_allclose((got[grad] * way).sum(), want, rtol=1e-7, atol=1e-8, err_msg=n)


@pytest.mark.parametrize("affine", [True, False])
def test_layer_norm_is_torchs_in_float64(affine):
    r = np.random.default_rng(11)
    x, dy, dres = r.standard_normal((4, 7)) + 3, r.standard_normal((4, 7)), r.standard_normal((4, 7))
    w, b = (r.standard_normal(7), r.standard_normal(7)) if affine else (None, None)
    t = [None if a is None else torch.tensor(a, requires_grad=True) for a in (x, w, b)]
    y = torch.nn.functional.layer_norm(t[0], (7,), t[1], t[2], 1e-5)
    got, _, _ = layer_norm.layer_norm(x, w, b, 1e-5)
    np.testing.assert_allclose(got, y.detach().numpy(), rtol=1e-11, atol=1e-12)
    ((y * torch.tensor(dy)).sum() + (t[0] * torch.tensor(dres)).sum()).backward()
    dx, dw, db = layer_norm.layer_norm_bwd(x, w, 1e-5, dy, dres)
    np.testing.assert_allclose(dx, t[0].grad.numpy(), rtol=1e-10, atol=1e-11)
    if affine:
        np.testing.assert_allclose(dw, t[1].grad.numpy(), rtol=1e-10, atol=1e-11)
        np.testing.assert_allclose(db, t[2].grad.numpy(), rtol=1e-10, atol=1e-11)
