"""mk_cache_attend against attention in 64 bits.

Tolerance of an output o = sum p v / l with A = sum p |v| / l: the result is
rounded to bf16 (2^-8 |o|) and so is every probability (2^-8 A).  In fp32, a
score sums head_dim exact products: it is off by at most (head_dim + 2) 2^-24
of scale sum |q k| = S, which moves every p by that much of itself, p and l by
2^-21 of the exponential, and the output's sum by 2^-24 per term of a run of
tiles: 2^-12 A + 2 (head_dim + 2) 2^-24 S A covers them.  lse moves by (head_dim + 2) 2^-24 S + 2^-18.

Every cache row that the operator has no business reading holds NaN.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


def make(batch, nq, nkv, hd, page, prefix, lens, seed=0, n_layers=2, layer=1, max_ctx=None, q_scale=1.0):
    g = torch.Generator("cuda").manual_seed(seed)
    max_ctx = max_ctx or max(max(lens), prefix, 1) + 5
    nan = float("nan")

    def rows():  # each sequence's own rows; NaN behind its length, and below the prefix (sequence 0 apart)
        r = torch.randn((batch, nkv, max_ctx, hd), generator=g, device="cuda").bfloat16()
        for b, n in enumerate(lens):
            r[b, :, n if b else max(n, min(prefix, max(lens))):] = nan
            if b:
                r[b, :, :prefix] = nan
        if lens[0] <= prefix:
            r[0, :, min(prefix, max(lens)):] = nan
        return r
    s = dict(batch=batch, nq=nq, nkv=nkv, hd=hd, page=page, prefix=prefix, lens=lens, max_ctx=max_ctx, layer=layer, kr=rows(), vr=rows())
    s["q"] = (torch.randn((batch, nq, hd), generator=g, device="cuda") * q_scale).bfloat16()
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["table"] = None
    for w in ("k", "v"):
        src = s[w + "r"]
        if page:
            stride = -(-max_ctx // page)
            pool = batch * stride + 3
            if s["table"] is None:
                table = torch.randperm(pool, generator=g, device="cuda").int()[:batch * stride].view(batch, stride).contiguous()
                s["table"] = table
            t = torch.full((n_layers, pool, nkv, page, hd), nan, dtype=torch.bfloat16, device="cuda")
            for b in range(batch):
                for j in range(stride):
                    part = src[b, :, j * page:(j + 1) * page]
                    t[layer, int(s["table"][b, j]), :, :part.shape[1]] = part
        else:
            t = torch.full((n_layers, batch, nkv, max_ctx, hd), nan, dtype=torch.bfloat16, device="cuda")
            t[layer] = src
        s[w] = t
    if page:  # pages a sequence has no business with are outside the pool
        for b, n in enumerate(lens):
            for j in range(s["table"].shape[1]):
                lo, hi = j * page, (j + 1) * page
                if not (b == 0 and lo < min(prefix, max(lens)) or n > prefix and lo < n and hi > prefix):
                    s["table"][b, j] = -1
    return s


def handle(s):
    import auto_regressive_decode_b200.mk as mk
    return mk.Cache(s["k"], s["v"], n_q_heads=s["nq"], batch=s["batch"], max_ctx=s["max_ctx"], block_table=s["table"], page_size=s["page"])


def check(s, out, lse, scale=None):
    hd, g, p = s["hd"], s["nq"] // s["nkv"], s["prefix"]
    scale = scale or hd ** -0.5
    assert not torch.isnan(out).any() and not torch.isnan(lse).any()
    for b, n in enumerate(s["lens"]):
        if n == 0:
            assert (out[b] == 0).all() and (lse[b] == -math.inf).all()
            continue
        q = s["q"][b].double().view(s["nkv"], g, hd)
        k, v = (torch.cat([s[w][0, :, :min(n, p)], s[w][b, :, p:max(n, p)]], 1).double() for w in ("kr", "vr"))
        sc = q @ k.transpose(1, 2) * scale
        size = ((q.abs() @ k.abs().transpose(1, 2)) * abs(scale)).amax(-1, keepdim=True)
        w = torch.softmax(sc, -1)
        o, a = w @ v, w @ v.abs()
        tol = 2 ** -8 * (o.abs() + a) + 2 ** -12 * a + 2 * (hd + 2) * 2 ** -24 * size * a
        err = (out[b].double().view(o.shape) - o).abs()
        assert (err <= tol).all(), (b, float((err / tol).max()))
        le = (lse[b].double().view(o.shape[:2]) - torch.logsumexp(sc, -1)).abs()
        assert (le <= (hd + 2) * 2 ** -24 * size[..., 0] + 2 ** -18).all(), (b, float(le.max()))


CASES = [
    # batch, nq, nkv, hd, page, prefix, lens
    (1, 1, 1, 64, 0, 0, [1]),
    (1, 4, 2, 128, 0, 0, [129]),
    (1, 16, 8, 128, 16, 100, [101]),
    (1, 8, 1, 128, 128, 128, [128]),                                   # the prefix is all
    (2, 4, 2, 64, 0, 5, [6, 5]),                                       # one has nothing of its own
    (3, 6, 2, 64, 48, 50, [0, 51, 200]),                               # an idle slot 0: the prefix is still its rows
    (3, 8, 8, 128, 16, 130, [130, 7, 300]),                            # shorter than the prefix
    (4, 32, 4, 128, 32, 17, [18, 400, 17, 145]),
    (5, 10, 2, 128, 128, 640, [641, 700, 0, 1000, 640]),
    (2, 64, 1, 128, 16, 33, [40, 1000]),                               # 64 heads on one KV head
    (2, 17, 1, 64, 0, 200, [201, 333]),
    (8, 40, 40, 128, 128, 300, [301, 1024, 555, 310, 900, 301, 777, 428]),
    (33, 16, 4, 64, 16, 1000, [1000 + i for i in range(33)]),          # 132 rows of a KV head share the prefix
    (40, 8, 1, 128, 0, 500, [500 + 13 * i for i in range(40)]),
    (130, 4, 2, 128, 64, 257, [i * 3 for i in range(130)]),            # many shorter than the prefix
    (300, 2, 2, 64, 16, 31, [i % 47 for i in range(300)]),
    (4, 8, 2, 128, 64, 1000, [0, 300, 299, 10]),                       # the prefix is longer than every sequence
    (3, 4, 4, 64, 16, 64, [0, 0, 0]),
    (2, 8, 2, 64, 384, 5000, [5001, 9000]),
]


@pytest.mark.parametrize("case", CASES)
def test_attend_matches_the_definition(case):
    s = make(*case, seed=1)
    c = handle(s)
    out, lse = c.attend(s["layer"], s["q"], s["seq_lens"], prefix_len=s["prefix"])
    assert c.status() == 0
    check(s, out, lse)


@pytest.mark.parametrize("case", [
    (600, 2, 1, 128, 128, 700, [(700 + i * 7 % 91) * (i % 5 > 0) for i in range(600)]),   # 1200 rows a KV head, some idle
    (385, 4, 2, 64, 128, 1500, [1500 + i % 9 for i in range(385)]),                       # the last two rows by themselves
    (160, 64, 1, 64, 0, 300, [300 + i % 3 for i in range(160)]),                          # 10240 rows a KV head
    (257, 1, 1, 128, 16, 129, [100 + i % 60 for i in range(257)]),
], ids=lambda c: "%d rows" % (c[0] * c[1] // c[2]))
def test_many_rows_share_a_prefix(case):
    s = make(*case, seed=8)
    c = handle(s)
    out, lse = c.attend(s["layer"], s["q"], s["seq_lens"], prefix_len=s["prefix"])
    assert c.status() == 0
    check(s, out, lse)


def test_sharing_changes_nothing_but_roundings():
    """The same sequences with the prefix read from sequence 0, and each with its own copy of it."""
    s = make(6, 16, 4, 128, 16, 600, [600 + 50 * i + 1 for i in range(6)], seed=2)
    c = handle(s)
    out, lse = c.attend(1, s["q"], s["seq_lens"], prefix_len=600)
    check(s, out, lse)
    full = torch.cat([s["kr"][:1, :, :600].expand(6, -1, -1, -1), s["kr"][:, :, 600:]], 2), \
        torch.cat([s["vr"][:1, :, :600].expand(6, -1, -1, -1), s["vr"][:, :, 600:]], 2)
    t = dict(s, page=0, table=None, prefix=0, kr=full[0], vr=full[1],
             k=torch.stack([full[0]] * 2).contiguous(), v=torch.stack([full[1]] * 2).contiguous())
    out2, lse2 = handle(t).attend(1, s["q"], s["seq_lens"])
    check(t, out2, lse2)


@pytest.mark.parametrize("scale", [0.5, 3.0, -0.1])
def test_scale_and_large_scores(scale):
    s = make(3, 8, 2, 64, 16, 100, [101, 180, 340], seed=3, q_scale=4.0)
    out, lse = handle(s).attend(1, s["q"], s["seq_lens"], prefix_len=100, scale=scale)
    check(s, out, lse, scale)


def test_equal_keys_give_the_mean_value():
    s = make(2, 4, 2, 64, 0, 128, [129, 400], seed=4)
    for w in ("k", "kr"):
        s[w].copy_(torch.where(torch.isnan(s[w]), s[w], torch.ones_like(s[w])))
    out, lse = handle(s).attend(1, s["q"], s["seq_lens"], prefix_len=128)
    check(s, out, lse)


def test_infinite_and_nan_rows_that_are_attended_spread():
    s = make(2, 4, 2, 64, 0, 10, [11, 40], seed=5)
    s["v"][1, 1, 0, 20, 3] = float("inf")
    s["v"][1, 0, 1, 4, 5] = float("nan")          # in the prefix: both sequences attend it
    out, lse = handle(s).attend(1, s["q"], s["seq_lens"], prefix_len=10)
    o = out.view(2, 2, 2, 64)
    assert torch.isinf(o[1, 0, :, 3]).all() and torch.isnan(o[:, 1, :, 5]).all()
    o = o.clone()
    o[1, 0, :, 3] = 0
    o[:, 1, :, 5] = 0
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


def test_bad_lengths_and_pages_are_reported():
    import auto_regressive_decode_b200.mk as mk
    s = make(3, 4, 2, 64, 16, 20, [30, 41, 25], seed=6)
    c = handle(s)
    for bad in (-1, s["max_ctx"] + 1):
        lens = s["seq_lens"].clone()
        lens[1] = bad
        full = s["table"].clone()
        s["table"].clamp_(min=0)                   # every page readable: only the length is wrong
        out, lse = c.attend(1, s["q"], lens, prefix_len=20)
        assert c.status() == mk.MK_ERR_RANGE and c.status() == mk.MK_OK
        s["table"].copy_(full)
        ok = {w: s[w] for w in s}
        for b in (0, 2):                           # the others are as ever
            check(dict(ok, lens=[s["lens"][x] if x == b else 0 for x in range(3)]),
                  torch.where(torch.arange(3, device="cuda")[:, None, None] == b, out, 0),
                  torch.where(torch.arange(3, device="cuda")[:, None] == b, lse, -math.inf))
    s["table"][1, 2] = s["k"].shape[1]             # rows 32..47 of sequence 1
    c.attend(1, s["q"], s["seq_lens"], prefix_len=20)
    assert c.status() == mk.MK_ERR_RANGE


def test_overlapping_calls_and_captured_graphs():
    s = make(4, 8, 2, 128, 16, 200, [201, 300, 0, 250], seed=7)
    c = handle(s)
    q2 = (s["q"].float() * 0.5).bfloat16()
    want = [c.attend(1, q, s["seq_lens"], prefix_len=200) for q in (s["q"], q2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(20):
        got += [c.attend(1, q, s["seq_lens"], prefix_len=200, stream=st) for q, st in zip((s["q"], q2), streams)]
    graphs = []
    for q in (s["q"], q2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, c.attend(1, q, s["seq_lens"], prefix_len=200)))
    for _ in range(5):
        for (g, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    got += [graphs[0][1], graphs[1][1]]
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, want[i % 2][0]) and torch.equal(lse, want[i % 2][1]), i
    # a captured call follows lengths rewritten between replays
    s["lens"] = [201, 240, 0, 215]
    s["seq_lens"].copy_(torch.tensor(s["lens"], dtype=torch.int32))
    graphs[0][0].replay()
    torch.cuda.synchronize()
    check(s, *graphs[0][1])
    assert c.status() == 0


def test_caller_buffers_and_same_bits_every_time():
    s = make(9, 16, 2, 64, 32, 400, [401 + 37 * i for i in range(9)], seed=9)
    c = handle(s)
    out = torch.empty_like(s["q"])
    lse = torch.empty((9, 16), device="cuda")
    ws = torch.full((c.workspace_bytes,), 0xFF, dtype=torch.uint8, device="cuda")    # NaN everywhere
    a = c.attend(1, s["q"], s["seq_lens"], prefix_len=400, out=out, lse=lse, workspace=ws)
    assert a[0] is out and a[1] is lse
    check(s, out, lse)
    first = out.clone(), lse.clone()
    for _ in range(10):
        c.attend(1, s["q"], s["seq_lens"], prefix_len=400, out=out, lse=lse, workspace=ws)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


# ---- many rows over a shared prefix: another kernel

@pytest.mark.parametrize("scale", [0.5, 3.0, -0.1])
@pytest.mark.parametrize("batch", [20, 50])
def test_scale_and_large_scores_of_many_rows(batch, scale):
    s = make(batch, 8, 2, 64, 16, 300, [301 + i * 11 % 80 for i in range(batch)], seed=10, q_scale=4.0)
    out, lse = handle(s).attend(1, s["q"], s["seq_lens"], prefix_len=300, scale=scale)
    check(s, out, lse, scale)


def test_scores_that_grow_along_the_prefix():
    """Every row's maximum is raised again and again: keys grow with the position."""
    s = make(40, 4, 1, 128, 0, 1000, [1000 + i % 3 for i in range(40)], seed=11)
    ramp = torch.linspace(0.05, 3, s["max_ctx"], device="cuda")[:, None]
    s["kr"].copy_((s["kr"].abs() * ramp).bfloat16())
    s["k"][1] = s["kr"]
    s["q"].copy_(s["q"].abs())
    out, lse = handle(s).attend(1, s["q"], s["seq_lens"], prefix_len=1000)
    check(s, out, lse)


def test_infinite_and_nan_rows_that_many_attend_spread():
    s = make(40, 4, 2, 64, 0, 200, [201] * 40, seed=12)
    s["v"][1, 7, 0, 200, 3] = float("inf")          # sequence 7's own
    s["v"][1, 0, 1, 150, 5] = float("nan")          # everyone's
    s["k"][1, 0, 0, 60, 1] = float("nan")           # everyone's scores of one KV head
    out, lse = handle(s).attend(1, s["q"], s["seq_lens"], prefix_len=200)
    o = out.view(40, 2, 2, 64).clone()
    assert torch.isnan(o[:, 0]).all() and torch.isnan(lse.view(40, 2, 2)[:, 0]).all()
    assert torch.isnan(o[:, 1, :, 5]).all() and torch.isfinite(lse.view(40, 2, 2)[:, 1]).all()
    o[:, 1, :, 5] = 0
    assert torch.isfinite(o[:, 1]).all()


def test_bad_pages_of_a_prefix_that_many_share_are_reported():
    import auto_regressive_decode_b200.mk as mk
    s = make(40, 4, 2, 64, 16, 200, [201] * 40, seed=13)
    c = handle(s)
    s["table"][0, 5] = s["k"].shape[1]
    c.attend(1, s["q"], s["seq_lens"], prefix_len=200)
    assert c.status() == mk.MK_ERR_RANGE
    s["table"][0, 5] = -7
    c.attend(1, s["q"], s["seq_lens"], prefix_len=200)
    assert c.status() == mk.MK_ERR_RANGE and c.status() == mk.MK_OK


def test_overlapping_calls_and_captured_graphs_of_many_rows():
    s = make(70, 8, 2, 128, 64, 700, [700 + i % 50 for i in range(70)], seed=14)
    c = handle(s)
    q2 = (s["q"].float() * 0.5).bfloat16()
    want = [c.attend(1, q, s["seq_lens"], prefix_len=700) for q in (s["q"], q2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        got += [c.attend(1, q, s["seq_lens"], prefix_len=700, stream=st) for q, st in zip((s["q"], q2), streams)]
    torch.cuda.synchronize()
    # one workspace for the calls of a graph: they follow one another; replayed next to calls with their own
    ws = torch.empty(c.workspace_bytes, dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        inside = [c.attend(1, q, s["seq_lens"], prefix_len=700, workspace=ws) for q in (s["q"], q2)]
    for _ in range(5):
        with torch.cuda.stream(streams[0]):
            g.replay()
        got += [c.attend(1, q, s["seq_lens"], prefix_len=700, stream=streams[1]) for q in (s["q"], q2)]
    torch.cuda.synchronize()
    for i, (out, lse) in enumerate(got + inside):
        assert torch.equal(out, want[i % 2][0]) and torch.equal(lse, want[i % 2][1]), i
    check(s, *want[0])
    assert c.status() == 0


def test_a_call_right_behind_what_writes_its_inputs():
    """Queries, lengths and rows written by the kernels just ahead on the stream, with no pause in between."""
    s = make(40, 8, 2, 64, 0, 300, [301 + i for i in range(40)], seed=15)
    c = handle(s)
    want = [c.attend(1, (s["q"] * f).contiguous(), s["seq_lens"], prefix_len=300) for f in (1, 0.5, 0.25)]
    for small in (False, True):
        t, cc = (s, c)
        if small:                                   # few rows: no prefix kernel
            t = make(3, 8, 2, 64, 0, 300, [301, 305, 340], seed=16)
            cc = handle(t)
            want = [cc.attend(1, (t["q"] * f).contiguous(), t["seq_lens"], prefix_len=300) for f in (1, 0.5, 0.25)]
        q, lens = torch.empty_like(t["q"]), torch.empty_like(t["seq_lens"])
        for _ in range(20):
            for f, w in zip((1, 0.5, 0.25), want):
                q.copy_(t["q"]).mul_(f)
                lens.zero_().add_(t["seq_lens"])
                out, lse = cc.attend(1, q, lens, prefix_len=300)
                q.zero_()                           # behind the call: not seen by it
                lens.zero_()
                assert torch.equal(out, w[0]) and torch.equal(lse, w[1])


@pytest.mark.parametrize("batch", [3, 40])
def test_inputs_from_another_stream_and_from_copies(batch):
    """What is ahead of the call: a wait for another stream's kernels, a copy; on the stream and in a captured graph."""
    s = make(batch, 8, 2, 64, 16, 300, [301 + 3 * i for i in range(batch)], seed=17)
    c = handle(s)
    factors = (1, 0.5, 0.25, 2)
    want = [c.attend(1, (s["q"] * f).contiguous(), s["seq_lens"], prefix_len=300) for f in factors]
    src, q, lens = s["q"].clone(), torch.empty_like(s["q"]), torch.empty_like(s["seq_lens"])
    big = torch.zeros(1 << 24, device="cuda")
    side = torch.cuda.Stream()

    def call():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            big.add_(1)                             # long enough that a missing wait would show
            lens.copy_(s["seq_lens"])
            q.copy_(src)
        big[:1 << 20].mul_(0.5)
        main.wait_stream(side)
        first = c.attend(1, q, lens, prefix_len=300)
        q.zero_()
        q.copy_(src)                                # a copy just ahead
        return first, c.attend(1, q, lens, prefix_len=300)

    def compare(got, i):
        for out, lse in got:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1]), i
    for i, f in enumerate(factors):
        src.copy_(s["q"]).mul_(f)
        lens.zero_()
        compare(call(), i)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        inside = call()
    for _ in range(3):
        for i, f in enumerate(factors):
            src.copy_(s["q"]).mul_(f)
            lens.zero_()
            q.zero_()
            g.replay()
            torch.cuda.synchronize()
            compare(inside, i)
    assert c.status() == 0


@pytest.mark.parametrize("case", [
    (1, 16, 8, 128, 0, 1000, [1024]), (7, 12, 4, 64, 16, 777, [800 + 40 * i for i in range(7)]), (9, 32, 8, 128, 64, 600, [601] * 9),
    (33, 64, 2, 128, 0, 130, [200] * 33), (300, 4, 4, 64, 32, 65, [66 + i % 40 for i in range(300)]), (200, 8, 2, 128, 128, 2000, [2001] * 200),
], ids=lambda c: "%d of %d/%d heads" % c[:3])
def test_nothing_is_written_outside_the_callers_buffers(case):
    s = make(*case, seed=18)
    c = handle(s)
    batch, nq, hd = s["q"].shape

    def fenced(nbytes):
        whole = torch.full((nbytes + 2 * 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        return whole, whole[4096:4096 + nbytes]
    parts = [fenced(n) for n in (c.workspace_bytes, batch * nq * hd * 2, batch * nq * 4)]
    k0, v0 = s["k"].clone(), s["v"].clone()
    out, lse = parts[1][1].view(torch.bfloat16).view(batch, nq, hd), parts[2][1].view(torch.float32).view(batch, nq)
    for _ in range(2):
        c.attend(s["layer"], s["q"], s["seq_lens"], prefix_len=s["prefix"], out=out, lse=lse, workspace=parts[0][1])
    check(s, out, lse)
    for whole, _ in parts:
        assert (whole[:4096] == 0xA5).all() and (whole[-4096:] == 0xA5).all()
    assert torch.equal(s["k"].view(torch.int16), k0.view(torch.int16)) and torch.equal(s["v"].view(torch.int16), v0.view(torch.int16))
