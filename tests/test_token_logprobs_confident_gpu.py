"""Scores of tokens that are all but certain: small log probabilities and entropies keep their value and their sign.

A row holds a logit 0 at its start and p > 0 far behind it, in another chunk of the same thread, and nothing else: with
r = e^-p, z = 1 + r is off by two exponentials of 2^-22 (the maximum's own, and the move of its rounded reference),
three roundings of 2^-24, and r times 2^-19 (an exponent of up to 23 is rounded at 2^-20, two more exponentials); the logarithm
adds 2^-23 of itself.  The entropy ln z + r p / (1 + r) has besides r p times 2^-19.
"""
import math

import pytest
import torch

from tests.test_token_logprobs_gpu import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,late", [(torch.float32, 4096), (torch.bfloat16, 8192)])
@pytest.mark.parametrize("rows", [64, 200, 500])
@pytest.mark.parametrize("k", [0, 3])
def test_two_logits(rows, k, dtype, late):
    import auto_regressive_decode_b200.mk as mk
    x = torch.full((rows, 20000), -math.inf, dtype=dtype, device="cuda")
    x[:, 0] = 0
    x[:, late] = torch.linspace(0.25, 15.9, rows, device="cuda")
    logp, ent, ids, best = mk.token_logprobs(x, torch.full((rows,), late, dtype=torch.int32, device="cuda"), top_k=k)
    p = x[:, late].double()
    r = torch.exp(-p)
    lnz = torch.log1p(r)
    tol = 11 * 2 ** -24 + 2 ** -19 * r + 2 ** -23 * lnz
    err = (logp.double() + lnz).abs()
    assert (err <= tol).all(), float((err / tol).max())
    assert (logp <= 0).all() and (ent >= 0).all()
    h = lnz + r * p / (1 + r)
    err, tol = (ent.double() - h).abs(), tol + 2 ** -19 * r * p + 2 ** -24 * h
    assert (err <= tol).all(), float((err / tol).max())
    if k:
        assert torch.equal(ids[:, 0], torch.full_like(ids[:, 0], late)) and torch.equal(best[:, 0], logp) and (best <= 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", [(3, 128256), (60, 20000), (200, 20011), (500, 20000), (500, 333)])
@pytest.mark.parametrize("above", [5, 15, 25])
def test_a_late_peak_above_the_rest(rows, vocab, above, dtype):
    """No log probability above 0, no entropy below, wherever the peak is."""
    import auto_regressive_decode_b200.mk as mk
    g = torch.Generator("cuda").manual_seed(above)
    x = torch.randn((rows, vocab), generator=g, device="cuda")
    tok = (vocab - 1 - torch.randint(vocab // 2, (rows,), generator=g, device="cuda")).int()
    x.scatter_(1, tok.long()[:, None], x.amax(-1, keepdim=True) + above)
    x = x.to(dtype)
    for k in (0, 4):
        got = mk.token_logprobs(x, tok, top_k=k)
        assert (got[0] <= 0).all() and (got[1] >= 0).all() and (got[3] <= 0).all()
        check(x, tok, k, got)
