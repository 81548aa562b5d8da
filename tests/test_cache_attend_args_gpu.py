"""Scales that fp32 cannot hold, and none: refused, not replaced by the default."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [1e-50, -1e-46, 1e39, 3e38, -3e38, float("inf"), "0.1", None])
def test_scales_that_do_not_fit(scale):
    import auto_regressive_decode_b200.mk as mk
    k = torch.zeros((1, 2, 1, 8, 64), dtype=torch.bfloat16, device="cuda")
    c = mk.Cache(k, k.clone(), n_q_heads=1, batch=2, max_ctx=8)
    q, lens = torch.zeros((2, 1, 64), dtype=torch.bfloat16, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7)
    with pytest.raises(mk.MkError) as e:
        c.attend(0, q, lens, scale=scale, out=out)
    assert e.value.code == mk.MK_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert (out == 7).all()


@pytest.mark.parametrize("scale", [1e-30, -1e-38])
@pytest.mark.parametrize("batch", [2, 40])
def test_small_scales_that_fit(batch, scale):
    """Next to no difference between scores: the mean of the values."""
    import auto_regressive_decode_b200.mk as mk
    g = torch.Generator("cuda").manual_seed(0)
    k = torch.randn((1, batch, 1, 200, 64), generator=g, device="cuda").bfloat16()
    v = torch.randn((1, batch, 1, 200, 64), generator=g, device="cuda").bfloat16()
    c = mk.Cache(k, v, n_q_heads=1, batch=batch, max_ctx=200)
    q, lens = torch.randn((batch, 1, 64), generator=g, device="cuda").bfloat16(), torch.full((batch,), 150, dtype=torch.int32, device="cuda")
    out, lse = c.attend(0, q, lens, scale=scale, prefix_len=100)
    kk, vv = (torch.cat([t[0, :1, 0, :100].expand(batch, 100, 64), t[0, :, 0, 100:150]], 1).double() for t in (k, v))
    s = torch.einsum("bnd,bd->bn", kk, q[:, 0].double())
    want = vv.mean(1)
    # outputs and probabilities round to bf16; the sum's fp32 error is far below
    assert ((out[:, 0].double() - want).abs() <= 2 ** -8 * (want.abs() + vv.abs().amax(1)) + 2 ** -12).all()
    size = torch.einsum("bnd,bd->bn", kk.abs(), q[:, 0].double().abs()).amax(1) * abs(scale)
    assert ((lse[:, 0].double() - torch.logsumexp(s * scale, 1)).abs() <= 66 * 2 ** -24 * size + 2 ** -18).all()
    assert c.status() == mk.MK_OK
