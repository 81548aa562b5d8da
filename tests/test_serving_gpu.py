"""The operators together, and with the decode step: prefill a cache, attend over a shared prefix, score tokens."""
import numpy as np
import pytest
import torch

import fixtures as fx
from fixtures.device import device_caches, device_model
from tests.test_cache_append_gpu import rotate
from tests.test_token_logprobs_gpu import check as check_scores

pytestmark = pytest.mark.gpu


def test_a_layer_over_a_shared_prompt():
    """Prompt appended once, then steps of one token a sequence: append, attend, project, score; against 64 bits."""
    import auto_regressive_decode_b200.mk as mk
    g = torch.Generator("cuda").manual_seed(0)
    B, nq, nkv, hd, page, P, steps, V = 5, 8, 2, 64, 16, 75, 3, 1000
    max_ctx = P + steps
    stride = -(-max_ctx // page)
    # the prompt's whole pages belong to everyone; the page where it ends is each sequence's own
    shared = P // page
    pool = shared + B * (stride - shared)
    order = torch.randperm(pool, generator=g, device="cuda").int()
    table = torch.cat([order[:shared].expand(B, shared), order[shared:].view(B, -1)], 1).contiguous()
    k, v = (torch.full((1, pool, nkv, page, hd), float("nan"), device="cuda").bfloat16() for _ in range(2))
    cache = mk.Cache(k, v, n_q_heads=nq, batch=B, max_ctx=max_ctx, block_table=table, page_size=page)
    qkv = torch.randn((P, nq + 2 * nkv, hd), generator=g, device="cuda")
    starts = torch.tensor([0] + [P] * B, dtype=torch.int32, device="cuda")          # all of it is sequence 0's
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    cache.append(0, qkv[:, nq:nq + nkv], qkv[:, nq + nkv:], zero, starts=starts)
    bf = lambda t: t.bfloat16().double()  # noqa: E731
    pos = torch.arange(P, device="cuda")
    ks = [[bf(rotate(qkv[:, nq:nq + nkv], None, pos)[0])] for _ in range(B)]
    vs = [[bf(qkv[:, nq + nkv:])] for _ in range(B)]
    head = torch.randn((nq * hd, V), generator=g, device="cuda") * 0.05
    for t in range(steps):
        x = torch.randn((B, nq + 2 * nkv, hd), generator=g, device="cuda")
        lens = torch.full((B,), P + t, dtype=torch.int32, device="cuda")
        q = cache.append(0, x[:, nq:nq + nkv], x[:, nq + nkv:], lens, q=x[:, :nq])
        out, lse = cache.attend(0, q, lens + 1, prefix_len=P)
        logits = out.view(B, -1).float() @ head
        tok = logits.argmax(-1).int()
        check_scores(logits, tok, 5, mk.token_logprobs(logits, tok, top_k=5))
        kk = bf(rotate(x[:, nq:nq + nkv], None, lens)[0])
        for b in range(B):
            ks[b].append(kk[b:b + 1])
            vs[b].append(bf(x[b:b + 1, nq + nkv:]))
            K, W = torch.cat(ks[b]).transpose(0, 1), torch.cat(vs[b]).transpose(0, 1)
            a = torch.softmax(q[b].double().view(nkv, -1, hd) @ K.transpose(1, 2) * hd ** -0.5, -1)
            o, size = a @ W, a @ W.abs()
            err = (out[b].double().view(o.shape) - o).abs()
            # the tolerance of the attention tests, and a half bf16 step for a key whose rounding falls on the other side
            assert (err <= 2 ** -8 * (o.abs() + size) + 2 ** -8 * size).all()
    assert cache.status() == mk.MK_OK


@pytest.mark.parametrize("kw", [{}, {"batch": 3, "ffn_dim": 704, "ctx": 0, "ctx_lo": 5, "ctx_hi": 100}])
@pytest.mark.parametrize("paged", [False, True])
def test_rows_appended_through_the_decoders_cache_are_the_ones_it_attends(kw, paged):
    import auto_regressive_decode_b200.mk as mk
    cfg = fx.CONFIGS["tiny"].replace(**kw)
    S0 = fx.context_lengths(cfg)
    w = device_model(cfg)
    kc, vc = device_caches(cfg, S0)
    table, page = None, 0
    if paged:
        page = 256
        stride = -(-cfg.max_ctx // page)
        table = torch.arange(cfg.batch * stride, dtype=torch.int32, device="cuda").flip(0).view(cfg.batch, stride).contiguous()
        shape = (cfg.n_layers, cfg.batch * stride, cfg.n_kv_heads, page, cfg.head_dim)
    else:
        shape = kc.shape
    k2, v2 = torch.zeros(shape, dtype=torch.bfloat16, device="cuda"), torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    a = mk.Decoder(cfg, w, kc, vc)
    b = mk.Decoder(cfg, w, k2, v2, block_table=table, page_size=page)
    cache = b.cache()
    # the same rows, appended in two calls at rotation position 0 (they count as rotated already)
    for part in (0, 1):
        counts = [int(s) // 2 if part == 0 else int(s) - int(s) // 2 for s in S0]
        held = [0 if part == 0 else int(s) // 2 for s in S0]
        starts = torch.tensor(np.cumsum([0] + counts), dtype=torch.int32, device="cuda")
        lens = torch.tensor(held, dtype=torch.int32, device="cuda")
        at = torch.zeros(sum(counts), dtype=torch.int32, device="cuda")
        for layer in range(cfg.n_layers):
            rows = [torch.cat([c[layer, i, :, h:h + n].transpose(0, 1) for i, (h, n) in enumerate(zip(held, counts))]) for c in (kc, vc)]
            cache.append(layer, rows[0], rows[1], lens, starts=starts, positions=at)
    assert cache.status() == mk.MK_OK
    la, lb = (torch.empty((cfg.batch, cfg.vocab), dtype=torch.float32, device="cuda") for _ in range(2))
    S = torch.from_numpy(S0.astype(np.int32)).cuda()
    tok = torch.from_numpy(fx.tokens(cfg)[0].copy()).cuda()
    a.step(tok, S, S, la)
    b.step(tok, S, S, lb)
    assert a.status() == mk.MK_OK and b.status() == mk.MK_OK
    assert torch.equal(la, lb)


@pytest.mark.parametrize("kw", [{}, {"batch": 4, "ffn_dim": 704, "ctx": 0, "ctx_lo": 5, "ctx_hi": 100}])
def test_scored_greedy_loop(kw):
    """The picks of greedy(), and the scores of each step's logits."""
    import auto_regressive_decode_b200.mk as mk
    cfg = fx.CONFIGS["tiny"].replace(**kw)
    steps = 6
    S0 = fx.context_lengths(cfg)
    w = device_model(cfg, gains="random")
    tok = torch.from_numpy(fx.tokens(cfg)[0].copy()).cuda()
    lens = torch.from_numpy(S0.astype(np.int32)).cuda()
    runs = []
    for scored in (False, True):
        kc, vc = device_caches(cfg, S0)
        dec = mk.Decoder(cfg, w, kc, vc)
        picks = torch.empty((steps, cfg.batch), dtype=torch.int32, device="cuda")
        if scored:
            scores = dec.greedy_scored(steps, tok, lens, picks, top_k=4)
        else:
            last = torch.empty((cfg.batch, cfg.vocab), dtype=torch.float32, device="cuda")
            dec.greedy(steps, tok, lens, picks, last)
        assert dec.status() == mk.MK_OK
        runs.append((picks, kc, vc))
    for x, y in zip(*runs):
        assert torch.equal(x, y)
    logprob, entropy, ids, tops, end = scores
    assert torch.equal(end, lens + steps) and torch.equal(ids[:, :, 0], runs[0][0]) and torch.equal(tops[:, :, 0], logprob)
    check_scores(last, picks[-1], 4, (logprob[-1], entropy[-1], ids[-1], tops[-1]))
    # every step's scores are those of its logits, replayed on the picked tokens
    kc, vc = device_caches(cfg, S0)
    rep = mk.Decoder(cfg, w, kc, vc)
    x = tok
    for t in range(steps):
        s = lens + t
        rep.step(x, s, s, last)
        check_scores(last, picks[t], 4, (logprob[t], entropy[t], ids[t], tops[t]))
        x = picks[t].contiguous()
    assert rep.status() == mk.MK_OK


def test_scored_loop_that_runs_out_of_the_cache():
    import auto_regressive_decode_b200.mk as mk
    cfg = fx.CONFIGS["tiny"]
    S0 = fx.context_lengths(cfg)
    kc, vc = device_caches(cfg, S0)
    dec = mk.Decoder(cfg, device_model(cfg), kc, vc)
    steps = cfg.max_ctx - int(S0[0]) + 2
    picks = torch.empty((steps, 1), dtype=torch.int32, device="cuda")
    tok = torch.from_numpy(fx.tokens(cfg)[0].copy()).cuda()
    logprob, _, _, _, _ = dec.greedy_scored(steps, tok, torch.from_numpy(S0.astype(np.int32)).cuda(), picks)
    assert dec.status() == mk.MK_ERR_RANGE
    assert (picks[-2:] == -1).all() and torch.isnan(logprob[-2:]).all() and torch.isfinite(logprob[:-2]).all()


def test_scored_loop_refuses_what_does_not_fit():
    import auto_regressive_decode_b200.mk as mk
    cfg = fx.CONFIGS["tiny"].replace(batch=4, ffn_dim=704, ctx=0, ctx_lo=5, ctx_hi=100)
    S0 = fx.context_lengths(cfg)
    kc, vc = device_caches(cfg, S0)
    dec = mk.Decoder(cfg, device_model(cfg), kc, vc)
    tok = torch.from_numpy(fx.tokens(cfg)[0].copy()).cuda()
    lens = torch.from_numpy(S0.astype(np.int32)).cuda()
    picks = torch.full((2, 4), -5, dtype=torch.int32, device="cuda")
    for kw, code in (({"batch": 3}, mk.MK_ERR_INVALID_ARG), ({"hidden": 512}, mk.MK_ERR_INVALID_ARG), ({"n_layers": 1}, mk.MK_ERR_INVALID_ARG)):
        dec.desc, right = mk.model_desc(cfg.replace(**kw)), dec.desc
        with pytest.raises(mk.MkError) as e:
            dec.greedy_scored(2, tok, lens, picks)
        assert e.value.code == code
        dec.desc = right
    for k in (-1, 33):
        with pytest.raises((mk.MkError, RuntimeError)):
            dec.greedy_scored(2, tok, lens, picks, top_k=k)
    torch.cuda.synchronize()
    assert (picks == -5).all()
    *_, end = dec.greedy_scored(0, tok, lens, picks[:0])
    assert torch.equal(end, lens)


def test_a_closed_cache_refuses():
    import auto_regressive_decode_b200.mk as mk
    k = torch.zeros((1, 2, 1, 8, 64), dtype=torch.bfloat16, device="cuda")
    c = mk.Cache(k, k.clone(), n_q_heads=1, batch=2, max_ctx=8)
    q, lens = torch.zeros((2, 1, 64), dtype=torch.bfloat16, device="cuda"), torch.ones(2, dtype=torch.int32, device="cuda")
    c.attend(0, q, lens)
    c.close()
    c.close()
    for f in (lambda: c.attend(0, q, lens), lambda: c.append(0, q, q, lens)):
        with pytest.raises(mk.MkError):
            f()


@pytest.mark.parametrize("bad", ["layer", "q type", "q shape", "q strides", "lens type", "lens length", "prefix", "out", "workspace", "scale"])
def test_attend_refuses(bad):
    import auto_regressive_decode_b200.mk as mk
    k = torch.zeros((2, 3, 2, 40, 64), dtype=torch.bfloat16, device="cuda")
    c = mk.Cache(k, k.clone(), n_q_heads=4, batch=3, max_ctx=40)
    a = dict(layer=1, q=torch.zeros((3, 4, 64), dtype=torch.bfloat16, device="cuda"), seq_lens=torch.ones(3, dtype=torch.int32, device="cuda"))
    c.attend(**a)
    a.update({"layer": {"layer": 2}, "q type": {"q": a["q"].float()}, "q shape": {"q": a["q"][:, :2].contiguous()},
              "q strides": {"q": a["q"].transpose(0, 1).contiguous().transpose(0, 1)}, "lens type": {"seq_lens": a["seq_lens"].long()},
              "lens length": {"seq_lens": a["seq_lens"][:2]}, "prefix": {"prefix_len": 41}, "out": {"out": a["q"].float()},
              "workspace": {"workspace": torch.empty(c.workspace_bytes - 1, dtype=torch.uint8, device="cuda")},
              "scale": {"scale": float("nan")}}[bad])
    with pytest.raises(mk.MkError):
        c.attend(**a)


@pytest.mark.parametrize("bad", ["layer", "type", "heads", "mixed types", "tokens", "starts", "stride", "gain", "q_out", "lens"])
def test_append_refuses(bad):
    import auto_regressive_decode_b200.mk as mk
    kc = torch.zeros((2, 3, 2, 40, 64), dtype=torch.bfloat16, device="cuda")
    c = mk.Cache(kc, kc.clone(), n_q_heads=4, batch=3, max_ctx=40)
    x = torch.zeros((3, 8, 64), device="cuda")
    odd = torch.zeros((3, 2 * 64 + 1), device="cuda")[:, :128].view(3, 2, 64) if bad == "stride" else None
    a = dict(layer=0, k=x[:, 4:6], v=x[:, 6:], q=x[:, :4], seq_lens=torch.zeros(3, dtype=torch.int32, device="cuda"))
    c.append(**a)
    a.update({"layer": {"layer": -1}, "type": {"k": a["k"].double(), "v": a["v"].double(), "q": a["q"].double()}, "heads": {"k": x[:, 3:6]},
              "mixed types": {"v": a["v"].bfloat16()}, "tokens": {"k": x[:2, 4:6], "v": x[:2, 6:], "q": x[:2, :4]},
              "starts": {"starts": torch.zeros(3, dtype=torch.int32, device="cuda")}, "stride": {"k": odd},
              "gain": {"k_norm": torch.ones(64, device="cuda")}, "q_out": {"q_out": torch.empty((3, 4, 64), device="cuda")},
              "lens": {"seq_lens": a["seq_lens"].cpu()}}[bad])
    with pytest.raises(mk.MkError):
        c.append(**a)


@pytest.mark.parametrize("batch", [4, 30])
def test_far_pages_of_a_large_pool_equal_near_ones(batch):
    """Rows whose element offsets pass 2^32, against the same rows in a small pool: bit for bit."""
    import auto_regressive_decode_b200.mk as mk
    g = torch.Generator("cuda").manual_seed(9)
    nq, nkv, hd, page, far = 16, 8, 128, 64, 68000
    P, own = 200, 70
    stride = -(-(P + own) // page)
    max_ctx = stride * page
    small = torch.randperm(batch * stride, generator=g, device="cuda").int().view(batch, stride).contiguous()
    outs = []
    x = torch.randn((P + batch * own, nq + 2 * nkv, hd), generator=g, device="cuda").bfloat16()
    for pool, table in ((batch * stride, small), (far + batch * stride, small + far)):
        k, v = (torch.empty((1, pool, nkv, page, hd), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        assert pool < far or k.numel() > 2 ** 32
        c = mk.Cache(k, v, n_q_heads=nq, batch=batch, max_ctx=max_ctx, block_table=table.contiguous(), page_size=page)
        zero = torch.zeros(batch, dtype=torch.int32, device="cuda")
        first = torch.tensor([0] + [P] * batch, dtype=torch.int32, device="cuda")
        c.append(0, x[:P, nq:nq + nkv], x[:P, nq + nkv:], zero, starts=first)
        rest = torch.arange(batch + 1, dtype=torch.int32, device="cuda") * own
        q = c.append(0, x[P:, nq:nq + nkv], x[P:, nq + nkv:], zero + P, q=x[P:, :nq], starts=rest)
        outs.append((q, *c.attend(0, q.view(batch, own, nq, hd)[:, -1].contiguous(), zero + P + own, prefix_len=P)))
        assert c.status() == mk.MK_OK
        c.close()
        del k, v
    for a, b in zip(*outs):
        assert torch.equal(a, b) and not torch.isnan(a).any()


FIRST_CALLS = """
import torch
import auto_regressive_decode_b200.mk as mk
g = torch.Generator("cuda").manual_seed(0)
B, nq, nkv, hd, T = 40, 8, 2, 64, 400
k, v = (torch.randn((1, B, nkv, T, hd), generator=g, device="cuda").bfloat16() for _ in range(2))
c = mk.Cache(k, v, n_q_heads=nq, batch=B, max_ctx=T)
x = torch.randn((B, nq + 2 * nkv, hd), generator=g, device="cuda")
lens = torch.full((B,), 300, dtype=torch.int32, device="cuda")
more = lens + 1
logits, tok = torch.randn((3, 50000), generator=g, device="cuda"), torch.zeros(3, dtype=torch.int32, device="cuda")

def calls():
    q = c.append(0, x[:, nq:nq + nkv], x[:, nq + nkv:], lens, q=x[:, :nq])
    return (q, *c.attend(0, q, more, prefix_len=200), *c.attend(0, q, more), *mk.token_logprobs(logits, tok, top_k=5))

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    inside = calls()
graph.replay()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(inside, calls())) and c.status() == 0
"""


def test_the_first_calls_of_a_process_can_be_captured():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0, r.stderr[-2000:]
