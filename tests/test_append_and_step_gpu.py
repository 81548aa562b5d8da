"""The row that the decode step writes for its token, and the row that the append writes from the same projections.

Both are the same numbers rounded to bf16 once (2^-8 of each), from fp32 products of `hidden` terms: those are off by
(hidden + 2) 2^-24 of the sum of their magnitudes, and a rotation adds the errors of its pair.  A norm divides value and
error by the head's root mean square, whose own error is below 2^-20 of it.
"""
import numpy as np
import pytest
import torch
import torch.nn.functional as F

import fixtures as fx
from fixtures.device import device_caches, device_model

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ctx", [1, 127, 3001])
@pytest.mark.parametrize("qk_norm", [False, True])
@pytest.mark.parametrize("kw", [{}, {"head_dim": 128, "rope_theta": 5e5}, {"n_kv_heads": 4}])
def test_the_appended_row_is_the_steps(kw, qk_norm, ctx):
    import auto_regressive_decode_b200.mk as mk
    cfg = fx.CONFIGS["tiny"].replace(ctx=ctx, qk_norm=qk_norm, **kw)
    w = device_model(cfg, gains="random")
    S0 = fx.context_lengths(cfg)
    kc, vc = device_caches(cfg, S0)
    dec = mk.Decoder(cfg, w, kc, vc)
    S = torch.from_numpy(S0.astype(np.int32)).cuda()
    tok = torch.from_numpy(fx.tokens(cfg)[0].copy()).cuda()
    dec.step(tok, S, S, torch.empty((1, cfg.vocab), device="cuda"))
    assert dec.status() == mk.MK_OK
    at = int(S0[0])
    step = [c[0, 0, :, at].double() for c in (kc, vc)]                  # [n_kv][hd] of layer 0

    lw = w["layers"][0]
    x = F.rms_norm(w["embed"][tok.long()].double(), (cfg.hidden,), lw["attn_norm"].double(), eps=cfg.rms_eps)
    k, v, k_size, v_size = [(y @ m.double().t()).view(1, cfg.n_kv_heads, cfg.head_dim)
                            for y, m in ((x, lw["wk"]), (x, lw["wv"]), (x.abs(), lw["wk"].abs()), (x.abs(), lw["wv"].abs()))]
    cache = dec.cache()
    kc[:, :, :, at] = vc[:, :, :, at] = float("nan")
    cache.append(0, k.float().contiguous(), v.float().contiguous(), S, k_norm=lw["k_norm"] if qk_norm else None)
    assert cache.status() == mk.MK_OK
    mine = [c[0, 0, :, at].double() for c in (kc, vc)]

    unit = (cfg.hidden + 2) * 2 ** -24
    k_size, v_size = k_size[0], v_size[0]
    if qk_norm:
        k_size = (k_size / k[0].square().mean(-1, keepdim=True).sqrt() + 16 * k[0].abs()) * lw["k_norm"].double().abs()
    pair = k_size + k_size.roll(cfg.head_dim // 2, -1)
    for a, b, size in ((step[0], mine[0], pair), (step[1], mine[1], v_size)):
        err, tol = (a - b).abs(), 2 ** -8 * (a.abs() + b.abs()) + 2 * unit * size
        assert (err <= tol).all(), float((err / tol).max())
        assert a.abs().max() > 0.1
