"""The recurrent operators where element offsets pass 2^31: the end of a large
call against a call on that end alone (GPU)."""
import pytest
import torch

import selective_state_space_31_amd as pkg
from selective_state_space_31_amd.recurrent import SSM_GATED_CHUNK as CHUNK

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
L, D, TAIL = 1100000, 2048, 5000  # 2.25e9 values a tensor
BF16 = 2.0 ** -8


@pytest.fixture(autouse=True)
def _memory():
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    yield
    torch.cuda.empty_cache()


def act(seed, *shape):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.empty(shape, device=DEV, dtype=torch.bfloat16).normal_(generator=g)


def near(got, ref):
    """Two float32 computations of the same values, each rounded to bf16 once
    (2 * 2^-8 of the value between them); what the float32 part may differ by
    is far below 2^-8 of the largest value."""
    lim = 2 * BF16 * ref.float().abs() + BF16 * 2.0 ** -4 * float(ref.float().abs().max())
    assert bool(((got.float() - ref.float()).abs() <= lim).all())


def test_gated_scan_past_32_bits():
    x, r, i, dout = (act(k, 1, L, D) for k in range(4))
    A = -torch.linspace(0.05, 3.0, D, device=DEV)
    out, last, mid = pkg.ssm_gated_scan_fwd(x, r, i, A, return_last_state=True, return_chunk_states=True)
    # the state before the tail is one that the forward left
    cut = (L - TAIL) // CHUNK
    t0 = cut * CHUNK
    h0 = mid[:, cut].contiguous()
    end = [v[:, t0:].contiguous() for v in (x, r, i)]
    o2, l2, m2 = pkg.ssm_gated_scan_fwd(*end, A, initial_state=h0, return_last_state=True, return_chunk_states=True)
    near(out[:, t0:], o2)
    torch.testing.assert_close(last, l2, rtol=1e-4, atol=1e-4)
    torch.testing.assert_close(mid[:, cut:], m2, rtol=1e-4, atol=1e-4)
    g = pkg.ssm_gated_scan_bwd(x, r, i, A, dout, chunk_states=mid)
    g2 = pkg.ssm_gated_scan_bwd(*end, A, dout[:, t0:].contiguous(), initial_state=h0, chunk_states=m2)
    for k in ("dx", "drgate", "digate"):
        near(g[k][:, t0:], g2[k])


def test_norm_rotate_past_32_bits():
    T, H, K = 140000, 128, 128
    q = act(5, 1, T, H, K)
    pos = torch.arange(T, dtype=torch.int32, device=DEV)[None]
    freq = 10000.0 ** (-torch.arange(K // 2, device=DEV) / (K // 2))
    w = torch.linspace(0.5, 1.5, K, device=DEV)
    end = q[:, -100:].contiguous()
    out, _ = pkg.ssm_qk_norm_rotate_fwd(q, None, freq, q_weight=w, positions=pos)
    ref, _ = pkg.ssm_qk_norm_rotate_fwd(end, None, freq, q_weight=w, positions=pos[:, -100:].contiguous())
    assert torch.equal(out[:, -100:], ref)
    g = pkg.ssm_qk_norm_rotate_bwd(q, None, freq, out, None, q_weight=w, positions=pos)
    g2 = pkg.ssm_qk_norm_rotate_bwd(end, None, freq, ref, None, q_weight=w, positions=pos[:, -100:].contiguous())
    assert torch.equal(g["dq"][:, -100:], g2["dq"])


def test_conv1d_gradients_past_32_bits():
    x, dout = act(6, 1, L, D), act(7, 1, L, D)
    w, bias = torch.linspace(-1, 1, D * 4, device=DEV).view(D, 4).contiguous(), torch.linspace(-1, 1, D, device=DEV)
    g = pkg.ssm_causal_conv1d_bwd(x, w, dout, bias=bias)
    t0 = L - TAIL
    before = x[:, t0 - 3:t0].transpose(1, 2).contiguous()
    g2 = pkg.ssm_causal_conv1d_bwd(x[:, t0:].contiguous(), w, dout[:, t0:].contiguous(), bias=bias,
                                   initial_conv_state=before)
    assert torch.equal(g["dx"][:, t0:], g2["dx"])


def test_largest_dim():
    """dim = 2^22: a wave's rows span the most bytes that are allowed.  Each
    end of the channels against a call on those channels alone."""
    dim, n, tok = 1 << 22, 70, 100
    g = torch.Generator(device=DEV).manual_seed(8)
    new = lambda *s: torch.empty(s, device=DEV).normal_(generator=g)
    x, r, i, dout = (new(1, tok, dim) for _ in range(4))
    A, h0 = -torch.rand(dim, device=DEV, generator=g), new(1, dim)
    out, last = pkg.ssm_gated_scan_fwd(x, r, i, A, z=dout, initial_state=h0, return_last_state=True)
    grads = pkg.ssm_gated_scan_bwd(x, r, i, A, dout, z=r, initial_state=h0)
    w = new(dim, 4)
    conv = pkg.ssm_causal_conv1d_bwd(x, w, dout, bias=A)
    for s in (slice(0, n), slice(dim - n, dim)):
        c = lambda t: t[..., s].contiguous()
        o2, l2 = pkg.ssm_gated_scan_fwd(c(x), c(r), c(i), c(A), z=c(dout), initial_state=c(h0), return_last_state=True)
        g2 = pkg.ssm_gated_scan_bwd(c(x), c(r), c(i), c(A), c(dout), z=c(r), initial_state=c(h0))
        c2 = pkg.ssm_causal_conv1d_bwd(c(x), w[s].contiguous(), c(dout), bias=c(A))
        # two foldings of 100 tokens: each value within 100 roundings of the largest there
        close = lambda a, b: torch.testing.assert_close(a, b, rtol=0, atol=200 * 2.0 ** -24 * float(b.abs().max()))
        close(out[..., s], o2)
        close(last[..., s], l2)
        for k in g2:
            close(grads[k][..., s], g2[k])
        assert torch.equal(conv["dx"][..., s], c2["dx"])
        assert torch.equal(conv["dweight"][s], c2["dweight"]) and torch.equal(conv["dbias"][s], c2["dbias"])


def test_largest_step():
    batch, dim = 1023, 1 << 21  # just below the limit of 2^31 - 2048
    x, r, i = (act(9 + k, batch, dim) for k in range(3))
    A = -torch.linspace(0.05, 3.0, dim, device=DEV)
    state = torch.ones(batch, dim, device=DEV)
    row = state[-1:].clone()
    out = pkg.ssm_gated_state_update(state, x, r, i, A)
    ref = pkg.ssm_gated_state_update(row, x[-1:].contiguous(), r[-1:].contiguous(), i[-1:].contiguous(), A)
    assert torch.equal(out[-1:], ref) and torch.equal(state[-1:], row)


def test_packed_offsets_up_to_int32():
    """One channel, sequences that end just below the largest offset."""
    total, cut = 2 ** 31 - 1000, 2 ** 31 - 7001
    x, r, i = (act(20 + k, total, 1) for k in range(3))
    A = torch.full((1,), -0.5, device=DEV)
    cu = torch.tensor([0, 5, cut, cut, total], dtype=torch.int32, device=DEV)
    out, last = pkg.ssm_gated_scan_fwd_varlen(x, r, i, A, cu, return_last_state=True)
    end = [v[cut:].contiguous() for v in (x, r, i)]
    o2, l2 = pkg.ssm_gated_scan_fwd_varlen(*end, A, torch.tensor([0, total - cut], dtype=torch.int32, device=DEV),
                                           return_last_state=True)
    near(out[cut:], o2)
    torch.testing.assert_close(last[3], l2[0], rtol=1e-5, atol=1e-5)
    assert last[2] == 0 and bool(torch.isfinite(last).all()) and bool(torch.isfinite(out[cut - 100:]).all())
    # the long sequence's end: decays around 0.78 leave nothing of what is 3000 tokens back
    o3, l3 = pkg.ssm_gated_scan_fwd_varlen(*(v[cut - 5000:cut].contiguous() for v in (x, r, i)), A,
                                           torch.tensor([0, 5000], dtype=torch.int32, device=DEV), return_last_state=True)
    near(out[cut - 2000:cut], o3[-2000:])
    torch.testing.assert_close(last[1], l3[0], rtol=1e-5, atol=1e-5)
