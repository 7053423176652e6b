"""Plain float64 forms of the gated delta rule and its gradients (numpy), token
after token as the formulas say:

    S <- e^g S;  u = beta (v - S^T k);  S <- S + k u^T;  o = scale S^T q

q, k (L, Hk, K); v (L, Hv, V); beta, g (L, Hv); states (Hv, K, V), for one
sequence.  Value head h reads key head h // (Hv // Hk).
"""
import numpy as np


def _heads(q, k, hv):
    r = hv // q.shape[1]
    return np.repeat(q, r, axis=1), np.repeat(k, r, axis=1)


def delta_rule(q, k, v, beta, g=None, scale=None, h0=None):
    """(out, last state, the states before every token)."""
    L, hv, V = v.shape
    K = q.shape[-1]
    scale = K ** -0.5 if scale is None else scale
    q, k = _heads(q, k, hv)
    S = np.zeros((hv, K, V)) if h0 is None else np.array(h0, np.float64)
    out, before = np.zeros(v.shape), np.zeros((L, hv, K, V))
    for t in range(L):
        before[t] = S
        if g is not None:
            S = np.exp(g[t])[:, None, None] * S
        u = beta[t][:, None] * (v[t] - np.einsum("hkv,hk->hv", S, k[t]))
        S = S + k[t][:, :, None] * u[:, None, :]
        out[t] = scale * np.einsum("hkv,hk->hv", S, q[t])
    return out, S, before


def missing(q, k, v, beta, g=None, scale=None, h0=None):
    """v - S^T k of every token (L, Hv, V)."""
    _, last, before = delta_rule(q, k, v, beta, g, scale, h0)
    _, kh = _heads(q, k, v.shape[1])
    S = before if g is None else np.exp(g)[:, :, None, None] * before
    return v - np.einsum("thkv,thk->thv", S, kh)


def delta_rule_bwd(q, k, v, beta, dout, g=None, scale=None, h0=None, dlast=None):
    """Gradients of sum(dout * out) + sum(dlast * last), a dict."""
    L, hv, V = v.shape
    hk, K = q.shape[1:]
    scale = K ** -0.5 if scale is None else scale
    _, _, before = delta_rule(q, k, v, beta, g, scale, h0)
    qh, kh = _heads(q, k, hv)
    dS = np.zeros((hv, K, V)) if dlast is None else np.array(dlast, np.float64)
    r = dict(dq=np.zeros(qh.shape), dk=np.zeros(qh.shape), dv=np.zeros(v.shape), dbeta=np.zeros(beta.shape),
             dg=np.zeros(beta.shape))
    for t in range(L - 1, -1, -1):
        a = np.ones(hv) if g is None else np.exp(g[t])
        S = a[:, None, None] * before[t]
        e = v[t] - np.einsum("hkv,hk->hv", S, kh[t])
        u = beta[t][:, None] * e
        new = S + kh[t][:, :, None] * u[:, None, :]
        r["dq"][t] = scale * np.einsum("hkv,hv->hk", new, dout[t])
        dS = dS + scale * qh[t][:, :, None] * dout[t][:, None, :]
        du = np.einsum("hkv,hk->hv", dS, kh[t])
        r["dbeta"][t] = (du * e).sum(-1)
        de = beta[t][:, None] * du
        r["dv"][t] = de
        r["dk"][t] = np.einsum("hkv,hv->hk", dS, u) - np.einsum("hkv,hv->hk", S, de)
        dS = dS - kh[t][:, :, None] * de[:, None, :]
        r["dg"][t] = (dS * S).sum((-1, -2))
        dS = a[:, None, None] * dS
    r["dinitial_state"] = dS
    for n in ("dq", "dk"):
        r[n] = r[n].reshape(L, hk, hv // hk, K).sum(2)
    return r


def grad_sizes(q, k, v, beta, dout, g=None, scale=None, h0=None, dlast=None):
    """What the gradients' rounding errors are measured against, per head: the
    largest norm of the factors that each one is a product of, over the tokens
    (dq, dk per key head, (1, Hk, 1); dv (1, Hv, 1); dbeta, dg (1, Hv); dstate
    (Hv, 1, 1))."""
    L, hv, V = v.shape
    hk, K = q.shape[1:]
    scale = K ** -0.5 if scale is None else scale
    _, last, before = delta_rule(q, k, v, beta, g, scale, h0)
    qh, kh = _heads(q, k, hv)
    norm = lambda x, ax: np.sqrt((x * x).sum(ax))
    dS = np.zeros((hv, K, V)) if dlast is None else np.array(dlast, np.float64)
    top = dict(S=norm(last, (1, 2)), dS=norm(dS, (1, 2)), u=np.zeros(hv), e=np.zeros(hv), du=np.zeros(hv), do=np.zeros(hv))
    for t in range(L - 1, -1, -1):
        a = np.ones(hv) if g is None else np.exp(g[t])
        S = a[:, None, None] * before[t]
        e = v[t] - np.einsum("hkv,hk->hv", S, kh[t])
        dS = dS + scale * qh[t][:, :, None] * dout[t][:, None, :]
        du = np.einsum("hkv,hk->hv", dS, kh[t])
        for n, x in (("S", norm(before[t], (1, 2))), ("dS", norm(dS, (1, 2))), ("u", beta[t] * norm(e, 1)), ("e", norm(e, 1)),
                     ("du", norm(du, 1)), ("do", scale * norm(dout[t], 1))):
            top[n] = np.maximum(top[n], x)
        dS = a[:, None, None] * (dS - kh[t][:, :, None] * (beta[t][:, None] * du)[:, None, :])
    join = lambda x: x.reshape(hk, hv // hk).sum(1)[None, :, None]
    size = top["S"] + top["u"]
    return dict(dq=join(size * top["do"]), dk=join(top["dS"] * top["u"] + size * top["du"]), dv=top["du"][None, :, None],
                dbeta=(top["du"] * top["e"])[None], dg=(top["dS"] * size)[None], dstate=top["dS"][:, None, None])
