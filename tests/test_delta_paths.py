"""The delta rule where its calls take another way through the kernels: many
heads (two column blocks a workgroup; shared key heads), few tokens (token by token), two graphs
at once, and offsets that pass 2^31 (GPU)."""
import numpy as np
import pytest
import torch

import selective_state_space_31_amd as pkg
from tests._layer import Delta, check_forward, check_grads

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def train(p, cu=None):
    """Forward with states, then the gradients."""
    off = () if cu is None else (cu,)
    f, b = (pkg.ssm_delta_rule_fwd, pkg.ssm_delta_rule_bwd) if cu is None else \
        (pkg.ssm_delta_rule_fwd_varlen, pkg.ssm_delta_rule_bwd_varlen)
    out, last, mids = f(*p.args(), *off, return_last_state=True, return_chunk_states=True, **p.kw())
    grads = b(*p.args(), *off, p.dout, dlast_state=p.dlast, chunk_states=mids, **p.kw())
    torch.cuda.synchronize()
    return out, last, mids, grads


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(2, 70, 16, 64, 32, 77), (1, 66, 64, 64, 128, 96), (3, 65, 32, 64, 64, 33)], ids=str)
def test_many_heads(shape, dtype):
    b, L, hk, hv, K, V = shape
    p = Delta((b, L), b, hk, hv, K, V, dtype, DEV, seed=L, fused=L % 2 == 1)
    out, last, mids, grads = train(p)
    for s in range(b):
        check_forward(p, out[s], last[s], s, what="sequence %d" % s, mids=mids[s])
        check_grads(p, {k: t[s] for k, t in grads.items()}, s, what="sequence %d" % s)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("K,V", [(16, 9), (64, 20), (128, 33), (200, 9)])
def test_shared_heads_together(K, V, dtype):
    """Key heads enough to fill the device: a workgroup goes through all value
    heads of one."""
    p = Delta((4, 65), 4, 32, 64, K, V, dtype, DEV, seed=K)
    _, _, _, grads = train(p)
    for s in (0, 3):
        check_grads(p, {k: t[s] for k, t in grads.items()}, s, what="sequence %d" % s)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_many_packed_heads(dtype):
    lengths = [0, 1, 64, 3, 65, 0, 30] * 4
    cu = np.concatenate([[0], np.cumsum(lengths)])
    n = len(lengths)
    p = Delta((int(cu[-1]),), n, 5, 10, 40, 48, dtype, DEV, seed=n)
    out, last, mids, grads = train(p, torch.tensor(cu, dtype=torch.int32, device=DEV))
    for s in range(n):
        a, z = int(cu[s]), int(cu[s + 1])
        check_forward(p, out[a:z], last[s], s, a, z, what="sequence %d" % s)
        check_grads(p, {k: t[s] if k == "dinitial_state" else t[a:z] for k, t in grads.items()}, s, a, z,
                    what="sequence %d" % s)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("shape", [(1, 3, 1, 1, 64, 64), (2, 8, 2, 4, 128, 40), (1, 8, 1, 2, 250, 7), (70, 9, 4, 4, 16, 20),
                                   (9, 16, 16, 32, 64, 33), (2, 12, 2, 2, 64, 64), (2, 5, 1, 1, 128, 128)], ids=str)
def test_few_tokens(shape, dtype):
    """Outputs, states, and the gradients from the states that the walk left."""
    b, L, hk, hv, K, V = shape
    p = Delta((b, L), b, hk, hv, K, V, dtype, DEV, seed=L + b, fused=b % 2 == 1)
    out, last, mids, grads = train(p)
    again = pkg.ssm_delta_rule_bwd(*p.args(), p.dout, dlast_state=p.dlast, **p.kw())
    torch.cuda.synchronize()
    for s in sorted({0, b // 2, b - 1}):
        check_forward(p, out[s], last[s], s, what="sequence %d" % s, mids=mids[s])
        check_grads(p, {k: t[s] for k, t in grads.items()}, s, what="sequence %d" % s)
        check_grads(p, {k: t[s] for k, t in again.items()}, s, what="sequence %d, states computed here" % s)


def test_few_packed_tokens():
    """All sequences together have 8 tokens: empty ones, and rows behind the last
    that stay as they were."""
    cu = [0, 0, 3, 3, 4, 7]
    p = Delta((8,), 5, 2, 4, 64, 24, "bf16", DEV, seed=21)
    off = torch.tensor(cu, dtype=torch.int32, device=DEV)
    out = torch.full((8, 4, 24), 5.0, dtype=torch.bfloat16, device=DEV)
    mids = torch.full((5, 4, 64 + 64, 24), 7.0, device=DEV)
    _, last, _ = pkg.ssm_delta_rule_fwd_varlen(*p.args(), off, return_last_state=True, out=out, chunk_states=mids, **p.kw())
    torch.cuda.synchronize()
    assert (out[7:] == 5.0).all() and (mids[0] == 7.0).all() and (mids[2] == 7.0).all()
    for s in range(5):
        a, z = cu[s], cu[s + 1]
        check_forward(p, out[a:z], last[s], s, a, z, what="sequence %d" % s, mids=mids[s:s + (z > a)])


@pytest.mark.parametrize("L", [8, 9, 63, 64, 65])
def test_a_decay_that_ends_at_a_chunk(L):
    """The last token of a sequence forgets everything; the one behind a chunk's
    end too."""
    p = Delta((1, L), 1, 1, 2, 64, 32, "fp32", DEV, seed=L)
    p.g[0, L - 1] = float("-inf")
    out, last, mids, grads = train(p)
    check_forward(p, out[0], last[0], 0, mids=mids[0])
    check_grads(p, {k: t[0] for k, t in grads.items()}, 0)


def test_two_graphs_and_two_streams():
    """Two captured training steps with workspaces of their own, replayed at the
    same time on two streams, several times, with eager work between."""
    ps = [Delta((2, 130), 2, 2, 4, 64, 64, "bf16", DEV, seed=s) for s in (31, 32)]

    def step(p):
        out, last, mids = pkg.ssm_delta_rule_fwd(*p.args(), return_last_state=True, return_chunk_states=True, **p.kw())
        g = pkg.ssm_delta_rule_bwd(*p.args(), p.dout, dlast_state=p.dlast, chunk_states=mids, **p.kw())
        return [out, last] + [g[k] for k in sorted(g)]

    want = [[t.clone() for t in step(p)] for p in ps]
    torch.cuda.synchronize()
    graphs, res = [], []
    for p in ps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res.append(step(p))
        graphs.append(g)
    streams = [torch.cuda.Stream(DEV) for _ in ps]
    for _ in range(4):
        for r in res:
            for t in r:
                t.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for w, r in zip(want, res):
            assert all(torch.equal(a, b) for a, b in zip(w, r))
        eager = step(ps[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want[0], eager))


@pytest.fixture
def big():
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    yield lambda seed, *shape: torch.empty(shape, device=DEV, dtype=torch.bfloat16).normal_(
        generator=torch.Generator(device=DEV).manual_seed(seed))
    torch.cuda.empty_cache()


def same(a, b):
    assert torch.equal(a, b)


@pytest.mark.parametrize("packed", [False, True])
def test_past_32_bits(packed, big):
    """The last sequence of a call whose v, out and states have more than 2^31
    values, against a call of its own (the same kernels: bit for bit)."""
    L, hv, K, V, tail = 33000, 256, 16, 256, 200
    n = [L, tail]
    T = sum(n)
    q, k = big(1, T, 1, K) * 0.2, big(2, T, 1, K) * 0.2
    v, dout = big(3, T, hv, V), big(4, T, hv, V)
    assert v.numel() > 1 << 31
    beta = torch.rand(T, hv, device=DEV, generator=torch.Generator(device=DEV).manual_seed(5))
    g = -0.01 * beta
    if packed:
        cu = torch.tensor([0, L, T], dtype=torch.int32, device=DEV)
        one = torch.tensor([0, tail], dtype=torch.int32, device=DEV)
        out, last, mids = pkg.ssm_delta_rule_fwd_varlen(q, k, v, beta, cu, g=g, return_last_state=True, return_chunk_states=True)
        grads = pkg.ssm_delta_rule_bwd_varlen(q, k, v, beta, cu, dout, g=g, chunk_states=mids)
        e = slice(L, T)
        o2, l2, m2 = pkg.ssm_delta_rule_fwd_varlen(q[e], k[e], v[e], beta[e], one, g=g[e], return_last_state=True,
                                                   return_chunk_states=True)
        g2 = pkg.ssm_delta_rule_bwd_varlen(q[e], k[e], v[e], beta[e], one, dout[e], g=g[e], chunk_states=m2)
        same(out[e], o2), same(last[1], l2[0]), same(mids[L // 64 + 1:L // 64 + 5], m2[:4])
        for name in ("dq", "dk", "dv", "dbeta", "dg"):
            same(grads[name][e], g2[name])
        same(grads["dinitial_state"][1], g2["dinitial_state"][0])
    else:
        half = T // 2
        lay = lambda t: t[:2 * half].view(2, half, *t.shape[1:])
        q, k, v, dout, beta, g = (lay(t) for t in (q, k, v, dout, beta, g))
        out, last, mids = pkg.ssm_delta_rule_fwd(q, k, v, beta, g=g, return_last_state=True, return_chunk_states=True)
        assert out.numel() > 1 << 31 and mids.numel() > 1 << 31
        grads = pkg.ssm_delta_rule_bwd(q, k, v, beta, dout, g=g, chunk_states=mids)
        e = slice(1, 2)
        o2, l2, m2 = pkg.ssm_delta_rule_fwd(q[e], k[e], v[e], beta[e], g=g[e], return_last_state=True, return_chunk_states=True)
        g2 = pkg.ssm_delta_rule_bwd(q[e], k[e], v[e], beta[e], dout[e], g=g[e], chunk_states=m2)
        same(out[e], o2), same(last[e], l2), same(mids[e], m2)
        for name in ("dq", "dk", "dv", "dbeta", "dg", "dinitial_state"):
            same(grads[name][e], g2[name])


def test_wide_rows_past_32_bits(big):
    """Tokens 2^17 values apart, the last ones behind 2^31 values."""
    T, hv, V, K = 20000, 2, 64, 32
    rows = big(6, T, 1 << 17)
    q, k = rows[..., 5:5 + K].unflatten(-1, (1, K)), rows[..., 100:100 + K].unflatten(-1, (1, K))
    v = rows[..., 1000:1000 + hv * V].unflatten(-1, (hv, V))
    beta = torch.full((1, T, hv), 0.02, device=DEV)
    out, last = pkg.ssm_delta_rule_fwd(q[None], k[None], v[None], beta, return_last_state=True)
    o2, l2 = pkg.ssm_delta_rule_fwd(q[None].contiguous(), k[None].contiguous(), v[None].contiguous(), beta,
                                    return_last_state=True)
    same(out, o2), same(last, l2)
    state, s2 = last.clone(), last.clone()
    b = beta[0, :1].contiguous()
    x = pkg.ssm_delta_state_update(state, q[-1:], k[-1:], v[-1:], b)
    same(x, pkg.ssm_delta_state_update(s2, q[-1:].contiguous(), k[-1:].contiguous(), v[-1:].contiguous(), b))
    same(state, s2)


def test_layer_norm_past_32_bits(big):
    rows, dim = 140000, 16384
    x, r, dy = (big(s, rows, dim) for s in (7, 8, 9))
    w = torch.linspace(0.5, 1.5, dim, device=DEV)
    out, total = pkg.ssm_layer_norm_fwd(x, w, w, residual=r)
    e = slice(rows - 3000, rows)
    o2, t2 = pkg.ssm_layer_norm_fwd(x[e], w, w, residual=r[e])
    same(out[e], o2), same(total[e], t2)
    g = pkg.ssm_layer_norm_bwd(total, dy, w)
    g2 = pkg.ssm_layer_norm_bwd(total[e], dy[e], w)
    same(g["dx"][e], g2["dx"])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("K,V,hv", [(64, 77, 4), (128, 33, 2), (40, 16, 2), (200, 50, 2)])
@pytest.mark.parametrize("packed", [False, True])
def test_what_buffers_held_before(packed, K, V, hv, dtype):
    """Workspaces and outputs full of NaN change nothing: nothing is read before
    it is written, also of chunks that are not full."""
    T, cu = 170, torch.tensor([0, 70, 70, 71, 165], dtype=torch.int32, device=DEV)
    p = Delta((T,) if packed else (2, T), 4 if packed else 2, 2, hv, K, V, dtype, DEV, seed=K)
    off = (cu,) if packed else ()
    f, b = (pkg.ssm_delta_rule_fwd_varlen, pkg.ssm_delta_rule_bwd_varlen) if packed else \
        (pkg.ssm_delta_rule_fwd, pkg.ssm_delta_rule_bwd)
    size = (4, T, 2, hv, K, V, p.v.dtype) if packed else (2, T, 2, hv, K, V, p.v.dtype)
    fb, bb = (pkg.ssm_delta_rule_fwd_varlen_workspace_bytes, pkg.ssm_delta_rule_bwd_varlen_workspace_bytes) if packed else \
        (pkg.ssm_delta_rule_fwd_workspace_bytes, pkg.ssm_delta_rule_bwd_workspace_bytes)
    res = []
    for fill in (0, 0xFF):
        raw = lambda n: torch.full((max(n, 256),), fill, dtype=torch.uint8, device=DEV)
        buf = lambda t: raw(t.numel() * t.element_size())[:t.numel() * t.element_size()].view(t.dtype).view(t.shape)
        like = f(*p.args(), *off, return_last_state=True, return_chunk_states=True, **p.kw())
        out, last, mids = (buf(t) for t in like)
        f(*p.args(), *off, out=out, last_state=last, chunk_states=mids, workspace=raw(fb(*size)), **p.kw())
        got = [out, last]
        for have in (True, False):
            grads = {k: buf(t) for k, t in b(*p.args(), *off, p.dout, dlast_state=p.dlast, **p.kw()).items()}
            b(*p.args(), *off, p.dout, dlast_state=p.dlast, chunk_states=mids if have else None, grads=grads,
              workspace=raw(bb(*size, with_chunk_states=have)), **p.kw())
            got += [grads[k] for k in sorted(grads)]
        torch.cuda.synchronize()
        end = 165 if packed else T
        res.append([t[:end] if packed and t.shape[0] == T else t for t in got])
    for a, z in zip(*res):
        assert torch.isfinite(a.float()).all() and torch.equal(a, z)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("off", [1, 2, 3])
def test_outputs_at_any_element(off, dtype):
    """Outputs, states and gradients in buffers that start `off` elements behind an
    aligned address: the same values."""
    p = Delta((2, 100), 2, 2, 4, 48, 32, dtype, DEV, seed=off)
    out, last, mids, grads = train(p)

    def buf(t):
        return torch.empty(t.numel() + 8, dtype=t.dtype, device=DEV)[off:off + t.numel()].view(t.shape)
    o, l, m = buf(out), buf(last), buf(mids)
    pkg.ssm_delta_rule_fwd(*p.args(), out=o, last_state=l, chunk_states=m, **p.kw())
    g = {k: buf(t) for k, t in grads.items()}
    pkg.ssm_delta_rule_bwd(*p.args(), p.dout, dlast_state=p.dlast, chunk_states=m, grads=g, **p.kw())
    torch.cuda.synchronize()
    assert torch.equal(o, out) and torch.equal(l, last) and torch.equal(m, mids)
    assert all(torch.equal(g[k], grads[k]) for k in grads)
