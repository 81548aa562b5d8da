"""What mk_decode_greedy_scored refuses of its description, whose sizes the buffers have to be of."""
import numpy as np
import pytest
import torch

import fixtures as fx
from fixtures.device import device_caches, device_model

pytestmark = pytest.mark.gpu


def decoder(**kw):
    import auto_regressive_decode_b200.mk as mk
    cfg = fx.CONFIGS["tiny"].replace(batch=4, ffn_dim=704, ctx=0, ctx_lo=5, ctx_hi=100, **kw)
    S0 = fx.context_lengths(cfg)
    kc, vc = device_caches(cfg, S0)
    tok = torch.from_numpy(fx.tokens(cfg)[0].copy()).cuda()
    return cfg, mk.Decoder(cfg, device_model(cfg), kc, vc), tok, torch.from_numpy(S0.astype(np.int32)).cuda()


def test_descriptions_that_differ_from_the_handles():
    """Another vocabulary, and sizes whose product of layers, batch and width is the handle's."""
    import auto_regressive_decode_b200.mk as mk
    cfg, dec, tok, lens = decoder()
    right = dec.desc
    others = [{"vocab": cfg.vocab * 2}, {"vocab": cfg.vocab // 2}, {"batch": 2, "hidden": 2 * cfg.hidden}, {"batch": 8, "hidden": cfg.hidden // 2}]
    picks = torch.full((3, 8), -5, dtype=torch.int32, device="cuda")
    logits = torch.full((8, 2 * cfg.vocab), 3.0, device="cuda")       # large enough for each of them
    for kw in others:
        d = mk.mk_model_desc.from_buffer_copy(right)
        for name, value in kw.items():
            setattr(d, name, value)
        dec.desc = d
        with pytest.raises(mk.MkError) as e:
            dec.greedy_scored(3, tok, lens, picks, logits=logits)
        assert e.value.code == mk.MK_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert (picks == -5).all() and (logits == 3.0).all()
    dec.desc = right
    dec.greedy_scored(3, tok, lens, picks)
    assert dec.status() == mk.MK_OK and (picks.view(-1)[:3 * cfg.batch] >= 0).all()


@pytest.mark.parametrize("bad", ["tokens type", "tokens length", "tokens host", "lens type", "lens strides", "picks type", "picks length",
                                 "logits type", "logits length", "logits none", "steps", "top_k"])
def test_wrong_tensors(bad):
    import auto_regressive_decode_b200.mk as mk
    cfg, dec, tok, lens = decoder()
    B, V = cfg.batch, cfg.vocab
    picks = torch.full((2, B), -5, dtype=torch.int32, device="cuda")
    a = dict(n_steps=2, tokens=tok, seq_lens=lens, out_tokens=picks, top_k=3, logits=torch.full((B, V), 3.0, device="cuda"))
    a.update({"tokens type": {"tokens": tok.long()}, "tokens length": {"tokens": tok[:3]}, "tokens host": {"tokens": tok.cpu()},
              "lens type": {"seq_lens": lens.float()}, "lens strides": {"seq_lens": lens.repeat_interleave(2)[::2]},
              "picks type": {"out_tokens": picks.long()}, "picks length": {"out_tokens": picks[:1]},
              "logits type": {"logits": a["logits"].bfloat16()}, "logits length": {"logits": a["logits"][1:]},
              "logits none": {"logits": 5}, "steps": {"n_steps": -1}, "top_k": {"top_k": -1}}[bad])
    with pytest.raises(mk.MkError) as e:
        dec.greedy_scored(**a)
    assert e.value.code == mk.MK_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert (picks == -5).all() and dec.status() == mk.MK_OK


def test_larger_buffers_and_a_stream_of_its_own():
    """Room for more steps than are run is fine, and the results are those of the current stream's call."""
    cfg, dec, tok, lens = decoder()
    B = cfg.batch
    a, b = (torch.full((5, B), -5, dtype=torch.int32, device="cuda") for _ in range(2))
    first = dec.greedy_scored(3, tok, lens, a, top_k=2)
    _, dec, _, _ = decoder()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    second = dec.greedy_scored(3, tok, lens, b, top_k=2, stream=st)
    st.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(a, b) and (a[3:] == -5).all() and all(torch.equal(x, y) for x, y in zip(first, second))


def test_refused_within_a_capture():
    """The steps carry their numbers, so that a replay would be wrong; the capture goes on without the call."""
    import auto_regressive_decode_b200.mk as mk
    cfg, dec, tok, lens = decoder()
    picks = torch.full((2, cfg.batch), -5, dtype=torch.int32, device="cuda")
    x = torch.zeros(3, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.add_(1)
        with pytest.raises(mk.MkError) as e:
            dec.greedy_scored(2, tok, lens, picks)
        x.add_(1)
    assert e.value.code == mk.MK_ERR_UNSUPPORTED
    graph.replay()
    torch.cuda.synchronize()
    assert (x == 2).all() and (picks == -5).all()
    dec.greedy_scored(2, tok, lens, picks)
    assert dec.status() == mk.MK_OK and (picks >= 0).all()
