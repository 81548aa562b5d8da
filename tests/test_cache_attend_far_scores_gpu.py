"""Scores so large that fp32 holds them in steps of more than one: the best key takes all, rows stay finite."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("batch,nq", [(2, 1), (3, 12), (40, 1), (150, 2)])
@pytest.mark.parametrize("scale", [1e8, 1e12, -1e12, 1e30])
def test_the_best_key_takes_all(batch, nq, hd, scale):
    """Keys whose scores are exact in fp32 (a whole number each, one a position), so that the best one is known."""
    import auto_regressive_decode_b200.mk as mk
    g = torch.Generator("cuda").manual_seed(hd + nq)
    T, P, n = 300, 200, 280
    k = torch.zeros((1, batch, 1, T, hd), device="cuda")
    k[..., 3] = torch.stack([torch.randperm(T, generator=g, device="cuda") for _ in range(batch)])[None, :, None].float() - T // 2
    k = k.bfloat16()                                   # whole numbers of up to 150
    v = torch.randn((1, batch, 1, T, hd), generator=g, device="cuda").bfloat16()
    q = torch.zeros((batch, nq, hd), device="cuda")
    q[..., 3] = torch.arange(1, batch * nq + 1, device="cuda").view(batch, nq) % 7 + 1.0
    c = mk.Cache(k, v, n_q_heads=nq, batch=batch, max_ctx=T)
    lens = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    out, lse = c.attend(0, q.bfloat16(), lens, scale=scale, prefix_len=P)
    kk, vv = (torch.cat([t[0, :1, 0, :P].expand(batch, P, hd), t[0, :, 0, P:n]], 1).double() for t in (k, v))
    s = torch.einsum("bnd,bhd->bhn", kk, q.double()) * scale
    top = s.amax(-1, keepdim=True)
    w = (s == top).double()
    w /= w.sum(-1, keepdim=True)                       # a whole number may come once in the prefix and once behind it
    want = w @ vv
    # outputs and probabilities round to bf16
    assert ((out.double() - want).abs() <= 2 ** -8 * (want.abs() + w @ vv.abs()) + 2 ** -12).all()
    # scale, its product with log2 e and that with a score are rounded, the way back likewise: six roundings of 2^-24
    assert ((lse.double() - torch.logsumexp(s, -1)).abs() <= 6 * 2 ** -24 * top[..., 0].abs()).all()
    assert c.status() == mk.MK_OK
