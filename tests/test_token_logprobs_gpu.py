"""mk_token_logprobs against log_softmax in 64 bits.

A log probability is x - m - ln z in fp32: two roundings of 2^-24 of at most
|x - m| + ln z, and z off by at most 2^-16 of itself (a thread sums under 512
terms in a row, the rest is a tree: 512 roundings of 2^-24 and 2^-21 of the
exponential, whose argument is rounded at 2^-24 of at most 150), so 2^-15 + 2^-22 |x - m| covers it;
the entropy, a weighted mean of terms of at most ln z + |x - m|, likewise with ln(vocab).
Ids are compared exactly: the largest logit first, the lowest id first among equals.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def expect(x, tokens, k):
    x = x.double()
    lp = torch.log_softmax(x, -1)
    given = torch.gather(lp, 1, tokens.long()[:, None])[:, 0]
    ent = torch.special.entr(lp.exp()).sum(-1)
    v, i = torch.sort(x, dim=-1, descending=True, stable=True)
    best, ids = torch.gather(lp, 1, i)[:, :k], i[:, :k].int()
    ids = torch.where(v[:, :k] == -math.inf, -1, ids)
    short = k - ids.shape[1]
    if short > 0:
        ids, best = torch.nn.functional.pad(ids, (0, short), value=-1), torch.nn.functional.pad(best, (0, short), value=-math.inf)
    return given, ent, ids, best


def check(x, tokens, k, got=None):
    import auto_regressive_decode_b200.mk as mk
    got = got or mk.token_logprobs(x, tokens, top_k=k)
    want = expect(x, tokens, k)
    assert torch.equal(got[2], want[2])
    for g, w in ((got[0], want[0]), (got[3], want[3])):
        inf = torch.isinf(w)
        assert torch.equal(torch.isinf(g), inf) and (g[inf] < 0).all()
        err, tol = (g.double() - w).abs()[~inf], 2 ** -15 + 2 ** -22 * w.abs()[~inf]
        assert (err <= tol).all(), float((err / tol).max())
    err = (got[1].double() - want[1]).abs()
    assert (err <= 2 ** -15 * (1 + math.log(x.shape[1]))).all(), float(err.max())


@pytest.mark.parametrize("rows,vocab,k", [
    (1, 1, 1), (1, 2, 32), (3, 7, 5), (2, 50, 0), (5, 127, 20), (1, 4096, 32), (2, 4097, 8), (4, 8191, 1), (1, 32000, 32), (2, 50257, 20),
    (1, 128256, 5), (8, 151936, 20), (40, 9001, 10), (300, 20000, 3), (1000, 61, 4),
])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_scores_match_the_definition(rows, vocab, k, dtype):
    g = torch.Generator("cuda").manual_seed(rows * 7 + vocab)
    x = (torch.randn((rows, vocab), generator=g, device="cuda") * 3).to(dtype)
    check(x, torch.randint(vocab, (rows,), generator=g, device="cuda", dtype=torch.int32), k)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset,extra", [(1, 0), (3, 5), (0, 1), (7, 9)])
def test_rows_of_any_alignment_and_stride(dtype, offset, extra):
    g = torch.Generator("cuda").manual_seed(1)
    rows, vocab = 6, 5003
    big = torch.full((rows * (vocab + extra) + offset + 16,), 1000.0, dtype=dtype, device="cuda")   # neighbours that would win
    x = big[offset:].as_strided((rows, vocab), (vocab + extra, 1))
    x.copy_(torch.randn((rows, vocab), generator=g, device="cuda"))
    check(x, torch.randint(vocab, (rows,), generator=g, device="cuda", dtype=torch.int32), 9)


def special(kind, rows, vocab, g):
    x = torch.randn((rows, vocab), generator=g, device="cuda")
    n = torch.arange(vocab, device="cuda")
    if kind == "equal":
        x.fill_(1.5)
    elif kind == "ascending":
        x = (n * 1e-3).repeat(rows, 1)
    elif kind == "descending":
        x = (-n * 1e-3).repeat(rows, 1)
    elif kind == "two values":
        x = (n % 2).float().repeat(rows, 1)
    elif kind == "zeros of both signs":
        x = torch.where(n % 3 == 0, -0.0, 0.0).repeat(rows, 1) + torch.where(n == vocab // 2, -1.0, 0.0)
    elif kind == "few allowed":
        keep = torch.zeros(vocab, dtype=torch.bool, device="cuda")
        keep[[0, vocab - 1, vocab // 2]] = True
        x.masked_fill_(~keep, -math.inf)
    elif kind == "tail allowed":
        x[:, :vocab * 3 // 4] = -math.inf
    elif kind == "lowest masks":
        x[:, ::2] = torch.finfo(torch.float32).min
    elif kind == "huge":
        x = x * 1e37
    elif kind == "far":
        x[:, 1] = 3e4
    elif kind == "one":
        x.fill_(-math.inf)
        x[:, vocab // 3] = -7.0
    return x


@pytest.mark.parametrize("kind", ["equal", "ascending", "descending", "two values", "zeros of both signs", "few allowed", "tail allowed",
                                  "lowest masks", "far", "one"])
@pytest.mark.parametrize("rows,vocab", [(2, 30011), (200, 30011), (3, 900)])
def test_special_rows(kind, rows, vocab):
    g = torch.Generator("cuda").manual_seed(2)
    x = special(kind, rows, vocab, g)
    check(x, torch.randint(vocab, (rows,), generator=g, device="cuda", dtype=torch.int32), 20)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("order", ["up", "down", "equal", "random", "pairs", "late pair"])
@pytest.mark.parametrize("rows,vocab,step", [(5, 151936, 8192), (5, 70003, 4096), (300, 70003, 4096), (7, 3500, 1024)])
def test_the_best_lie_a_fixed_step_apart(order, rows, vocab, step, dtype):
    """All of them in the share of few threads."""
    g = torch.Generator("cuda").manual_seed(5)
    x = torch.randn((rows, vocab), generator=g, device="cuda")
    at = torch.arange(41, vocab, step, device="cuda")
    n = torch.arange(len(at), device="cuda")
    value = {"up": n, "down": -n, "equal": n * 0, "random": torch.randint(0, 4, (len(at),), generator=g, device="cuda"), "pairs": -(n // 2),
             "late pair": (n >= len(at) - 2).int()}[order]
    x[:, at] = 50 + value.float()
    x[1::2] = x[1::2].roll(3, 1)
    check(x.to(dtype), torch.randint(vocab, (rows,), generator=g, device="cuda", dtype=torch.int32), 20)


@pytest.mark.parametrize("kind", ["equal", "ascending", "descending", "two values", "zeros of both signs", "few allowed", "tail allowed", "far", "one"])
def test_special_rows_of_bf16(kind):
    g = torch.Generator("cuda").manual_seed(6)
    x = special(kind, 3, 100003, g).bfloat16()
    check(x, torch.randint(100003, (3,), generator=g, device="cuda", dtype=torch.int32), 32)


def test_huge_logits_do_not_overflow():
    import auto_regressive_decode_b200.mk as mk
    g = torch.Generator("cuda").manual_seed(3)
    x = special("huge", 4, 10000, g)
    tok = x.argmax(-1).int()
    logp, ent, ids, best = mk.token_logprobs(x, tok, top_k=4)
    assert torch.equal(ids, expect(x, tok, 4)[2])
    assert (logp == 0).all() and (ent == 0).all() and (best[:, 0] == 0).all() and (best[:, 1:] < -1e30).all()


@pytest.mark.parametrize("rows,vocab", [(4, 40000), (200, 20000), (4, 100)])
def test_rows_without_a_distribution_are_nan_and_leave_the_others(rows, vocab):
    import auto_regressive_decode_b200.mk as mk
    g = torch.Generator("cuda").manual_seed(4)
    x = torch.randn((rows, vocab), generator=g, device="cuda")
    x[0] = -math.inf
    x[1, vocab - 1] = math.nan
    x[2, 5] = math.inf
    tok = torch.randint(vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
    logp, ent, ids, best = mk.token_logprobs(x, tok, top_k=6)
    for t in (logp[:3], ent[:3], best[:3]):
        assert torch.isnan(t).all()
    assert (ids[:3] == -1).all()
    check(x[3:], tok[3:], 6, (logp[3:], ent[3:], ids[3:], best[3:]))


def test_tokens_out_of_range_are_nan():
    import auto_regressive_decode_b200.mk as mk
    x = torch.randn((3, 700), device="cuda")
    logp, ent, ids, best = mk.token_logprobs(x, torch.tensor([-1, 700, 699], dtype=torch.int32, device="cuda"), top_k=2)
    assert torch.isnan(logp[:2]).all() and torch.isfinite(logp[2]) and torch.isfinite(ent).all() and (ids >= 0).all()


def test_no_rows_and_captured_calls():
    import auto_regressive_decode_b200.mk as mk
    x = torch.randn((5, 20000), device="cuda")
    tok = torch.tensor([1, 2, 3, 4, 5], dtype=torch.int32, device="cuda")
    out = mk.token_logprobs(x[:0], tok[:0], top_k=3)
    assert [tuple(t.shape) for t in out] == [(0,), (0,), (0, 3), (0, 3)]
    g = torch.cuda.CUDAGraph()
    mk.token_logprobs(x, tok, top_k=3)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        out = mk.token_logprobs(x, tok, top_k=3)
    x.copy_(torch.randn((5, 20000), device="cuda"))
    tok.copy_(tok.flip(0))
    g.replay()
    torch.cuda.synchronize()
    check(x, tok, 3, out)


def test_calls_on_several_streams_and_the_same_bits_every_time():
    import auto_regressive_decode_b200.mk as mk
    g = torch.Generator("cuda").manual_seed(7)
    work = []
    for rows, vocab, dtype in ((1, 128256, torch.float32), (600, 5000, torch.bfloat16), (20, 151936, torch.bfloat16), (5, 333, torch.float32)):
        x = (torch.randn((rows, vocab), generator=g, device="cuda") * 3).to(dtype)
        tok = torch.randint(vocab, (rows,), generator=g, device="cuda", dtype=torch.int32)
        work.append((x, tok, mk.token_logprobs(x, tok, top_k=17)))
        check(x, tok, 17, work[-1][2])
    streams = [torch.cuda.Stream() for _ in work]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for st, (x, tok, _) in zip(streams, work):
            got.append(mk.token_logprobs(x, tok, top_k=17, stream=st))
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        for a, b in zip(r, work[i % len(work)][2]):
            assert torch.equal(a, b)


def test_a_row_read_many_times_and_rows_of_one_buffer():
    """Row stride 0, and rows that overlap: they are only read."""
    g = torch.Generator("cuda").manual_seed(8)
    x = torch.randn(9000, generator=g, device="cuda")
    tok = torch.randint(8000, (6,), generator=g, device="cuda", dtype=torch.int32)
    check(x[:8000].expand(6, 8000), tok, 5)
    check(x.as_strided((6, 8000), (100, 1)), tok, 5)
