"""mk_cache_append against its definition in 64 bits.

Every value of the result is one fp32 expression a cos - b sin (or the value
itself) rounded once to bf16: off by half a bf16 step (2^-8 of the value) and
by fp32 roundings of its two products (at most 2^-21 (|a| + |b|): the norm,
the table's cos and sin, two products and their sum, under eight roundings of 2^-24 each).
Everything the call must not touch is compared bit for bit.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

THETA, EPS = 1e4, 1e-5


def make(batch, nq, nkv, hd, page, lens, counts, dtype, seed=0, n_layers=2, norm=False, pad=0, positions=False):
    g = torch.Generator("cuda").manual_seed(seed)
    n = sum(counts) + pad
    max_ctx = max(a + b for a, b in zip(lens, counts)) + 3
    s = dict(batch=batch, nq=nq, nkv=nkv, hd=hd, page=page, max_ctx=max_ctx, n=n, counts=counts, lens=lens)
    if page:
        stride = -(-max_ctx // page)
        pool = batch * stride + 2
        s["table"] = torch.randperm(pool, generator=g, device="cuda").int()[:batch * stride].view(batch, stride).contiguous()
        shape = (n_layers, pool, nkv, page, hd)
    else:
        s["table"], shape = None, (n_layers, batch, nkv, max_ctx, hd)
    s["k"], s["v"] = (torch.randn(shape, generator=g, device="cuda").bfloat16() for _ in range(2))
    s["x"] = torch.randn((n, nq + 2 * nkv, hd), generator=g, device="cuda").to(dtype)
    s["starts"] = torch.tensor([0] + list(torch.tensor(counts).cumsum(0)), dtype=torch.int32, device="cuda")
    s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["q_norm"], s["k_norm"] = ((torch.rand(hd, generator=g, device="cuda") + 0.5).bfloat16() for _ in range(2)) if norm else (None, None)
    s["positions"] = torch.randint(max_ctx, (n,), generator=g, device="cuda", dtype=torch.int32) if positions else None
    return s


def handle(s):
    import auto_regressive_decode_b200.mk as mk
    return mk.Cache(s["k"], s["v"], n_q_heads=s["nq"], batch=s["batch"], max_ctx=s["max_ctx"], block_table=s["table"], page_size=s["page"],
                    rope_theta=THETA, rms_eps=EPS)


def rotate(x, gain, pos):
    """(value, |a| + |b|) of rows [n][heads][hd] in 64 bits."""
    x = x.double()
    hd = x.shape[-1]
    if gain is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * gain.double()
    i = torch.arange(hd // 2, device="cuda", dtype=torch.float64)
    ang = pos.double()[:, None, None] * THETA ** (-2 * i / hd)
    a, b = x[..., :hd // 2], x[..., hd // 2:]
    size = (a.abs() + b.abs()).repeat(1, 1, 2)
    return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1), size


def expect(s, layer, skip=()):
    """The caches after the call, the tolerance, and the rotated queries of every placed token."""
    nq, nkv = s["nq"], s["nkv"]
    k, v = s["k"].double(), s["v"].double()
    tol = torch.zeros_like(k)
    q, qt = torch.zeros((s["n"], nq, s["hd"]), dtype=torch.float64, device="cuda"), None
    qt = torch.zeros_like(q)
    t = 0
    for b, cnt in enumerate(s["counts"]):
        for i in range(cnt):
            row = s["lens"][b] + i
            if t not in skip:
                pos = s["positions"][t:t + 1] if s["positions"] is not None else torch.tensor([row], device="cuda")
                q[t:t + 1], size = rotate(s["x"][t:t + 1, :nq], s["q_norm"], pos)
                qt[t:t + 1] = q[t:t + 1].abs() * 2 ** -8 + size * 2 ** -21
                kk, size = rotate(s["x"][t:t + 1, nq:nq + nkv], s["k_norm"], pos)
                at = (layer, int(s["table"][b, row // s["page"]]), slice(None), row % s["page"]) if s["page"] else (layer, b, slice(None), row)
                k[at], tol[at] = kk[0], kk[0].abs() * 2 ** -8 + size[0] * 2 ** -21
                v[at] = s["x"][t, nq + nkv:].bfloat16().double()
            t += 1
    return k, v, tol, q, qt




CASES = [
    # batch, nq, nkv, hd, page, lens, counts
    (1, 1, 1, 64, 0, [0], [1]),
    (1, 16, 8, 128, 16, [15], [3]),                          # crosses a page
    (3, 4, 2, 64, 0, [5, 0, 100], [7, 0, 1]),                # an empty sequence
    (3, 8, 2, 128, 48, [47, 1, 0], [2, 50, 96]),
    (4, 40, 40, 128, 128, [127, 0, 300, 4], [1, 130, 2, 0]),
    (2, 7, 7, 64, 32, [31, 32], [33, 1]),                    # odd heads
    (2, 32, 1, 128, 16, [0, 3], [257, 5]),                   # one KV head
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("norm", [False, True])
def test_append_matches_the_definition(case, dtype, norm):
    s = make(*case, dtype, seed=3, norm=norm, positions=case[4] == 48)
    k0, v0 = s["k"].clone(), s["v"].clone()
    c = handle(s)
    nq, nkv = s["nq"], s["nkv"]
    x = s["x"]
    q = c.append(1, x[:, nq:nq + nkv], x[:, nq + nkv:], s["seq_lens"], q=x[:, :nq], starts=s["starts"], positions=s["positions"],
                 q_norm=s["q_norm"], k_norm=s["k_norm"])
    assert c.status() == 0
    k, v, tol, qe, qt = expect(dict(s, k=k0, v=v0), 1)
    assert ((s["k"].double() - k).abs() <= tol).all()        # zero tolerance on every row not written
    assert torch.equal(s["v"].double(), v)
    assert ((q.double() - qe).abs() <= qt).all()


def test_one_token_a_sequence_without_starts_equals_the_ragged_call():
    s = make(5, 8, 4, 128, 16, [0, 15, 16, 31, 200], [1] * 5, torch.float32, seed=4)
    c, x = handle(s), s["x"]
    k0, v0 = s["k"].clone(), s["v"].clone()
    qa = c.append(0, x[:, 8:12], x[:, 12:], s["seq_lens"], q=x[:, :8], starts=s["starts"])
    ka, va = s["k"].clone(), s["v"].clone()
    s["k"].copy_(k0)
    s["v"].copy_(v0)
    qb = c.append(0, x[:, 8:12], x[:, 12:], s["seq_lens"], q=x[:, :8])
    assert torch.equal(qa, qb) and torch.equal(ka, s["k"]) and torch.equal(va, s["v"])


def test_no_queries_separate_buffers_and_strides():
    s = make(2, 8, 4, 64, 0, [2, 0], [3, 4], torch.bfloat16, seed=5)
    k0, v0 = s["k"].clone(), s["v"].clone()
    c, x = handle(s), s["x"]
    wide = torch.full((7, 4 * 64 + 40), float("nan"), device="cuda").bfloat16()   # rows padded by 40 values
    wide[:, :256] = x[:, 8:12].reshape(7, 256)
    kk = wide[:, :256].unflatten(1, (4, 64))
    assert c.append(1, kk, x[:, 12:].contiguous(), s["seq_lens"], starts=s["starts"]) is None
    k, v, tol, _, _ = expect(dict(s, k=k0, v=v0), 1)
    assert ((s["k"].double() - k).abs() <= tol).all() and torch.equal(s["v"].double(), v)


def test_tokens_behind_the_last_sequence_are_left_out():
    s = make(2, 4, 2, 64, 16, [3, 9], [2, 3], torch.float32, seed=6, pad=4)
    k0, v0 = s["k"].clone(), s["v"].clone()
    c, x = handle(s), s["x"]
    q_out = torch.full((9, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    c.append(0, x[:, 4:6], x[:, 6:], s["seq_lens"], q=x[:, :4], starts=s["starts"], q_out=q_out)
    assert c.status() == 0
    k, v, tol, qe, qt = expect(dict(s, k=k0, v=v0), 0)
    assert ((s["k"].double() - k).abs() <= tol).all() and torch.equal(s["v"].double(), v)
    assert ((q_out[:5].double() - qe[:5]).abs() <= qt[:5]).all()
    assert (q_out[5:] == 7.0).all()


@pytest.mark.parametrize("what", ["row", "page", "position", "negative"])
def test_values_out_of_range_are_left_out_and_reported(what):
    import auto_regressive_decode_b200.mk as mk
    s = make(2, 4, 2, 64, 16, [3, 9], [2, 3], torch.float32, seed=7, positions=True)
    skip = {"row": (4,), "page": (2, 3, 4), "position": (1,), "negative": (0, 1)}[what]
    if what == "row":                      # the last token's row is max_ctx
        s["max_ctx"] = 11
        s["table"] = s["table"][:, :1].contiguous()
        s["positions"].clamp_(max=10)
    if what == "page":
        s["table"][1, 0] = s["k"].shape[1]
    if what == "position":
        s["positions"][1] = s["max_ctx"]
    if what == "negative":
        s["seq_lens"][0] = -2
    k0, v0 = s["k"].clone(), s["v"].clone()
    c, x = handle(s), s["x"]
    q_out = torch.full((5, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    c.append(0, x[:, 4:6], x[:, 6:], s["seq_lens"], q=x[:, :4], starts=s["starts"], positions=s["positions"], q_out=q_out)
    assert c.status() == mk.MK_ERR_RANGE
    assert c.status() == mk.MK_OK
    k, v, tol, qe, qt = expect(dict(s, k=k0, v=v0), 0, skip)
    assert ((s["k"].double() - k).abs() <= tol).all() and torch.equal(s["v"].double(), v)
    for t in range(5):
        assert (q_out[t] == 7.0).all() if t in skip else ((q_out[t].double() - qe[t]).abs() <= qt[t]).all()


def test_starts_out_of_order_are_reported():
    import auto_regressive_decode_b200.mk as mk
    s = make(2, 4, 2, 64, 0, [3, 9], [2, 3], torch.float32, seed=8)
    c, x = handle(s), s["x"]
    c.append(0, x[:, 4:6], x[:, 6:], s["seq_lens"], starts=torch.tensor([0, 4, 2], dtype=torch.int32, device="cuda"))
    assert c.status() == mk.MK_ERR_RANGE


def test_no_tokens_is_no_work():
    s = make(2, 4, 2, 64, 0, [3, 9], [2, 3], torch.float32, seed=9)
    c, x = handle(s), s["x"][:0]
    k0 = s["k"].clone()
    q = c.append(0, x[:, 4:6], x[:, 6:], s["seq_lens"], q=x[:, :4], starts=torch.zeros(3, dtype=torch.int32, device="cuda"))
    assert q.shape == (0, 4, 64) and torch.equal(s["k"], k0) and c.status() == 0


def test_many_sequences():
    counts = [i % 3 for i in range(300)]
    s = make(300, 2, 1, 64, 16, [(7 * i) % 40 for i in range(300)], counts, torch.bfloat16, seed=10)
    k0, v0 = s["k"].clone(), s["v"].clone()
    c, x = handle(s), s["x"]
    q = c.append(1, x[:, 2:3], x[:, 3:], s["seq_lens"], q=x[:, :2], starts=s["starts"])
    k, v, tol, qe, qt = expect(dict(s, k=k0, v=v0), 1)
    assert ((s["k"].double() - k).abs() <= tol).all() and torch.equal(s["v"].double(), v)
    assert ((q.double() - qe).abs() <= qt).all()


def test_captured_and_replayed_on_another_stream():
    s = make(2, 4, 2, 128, 16, [3, 9], [2, 3], torch.float32, seed=11)
    c, x = handle(s), s["x"]
    k0, v0 = s["k"].clone(), s["v"].clone()
    q_eager = c.append(0, x[:, 4:6], x[:, 6:], s["seq_lens"], q=x[:, :4], starts=s["starts"])
    want = s["k"].clone(), s["v"].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        q_graph = c.append(0, x[:, 4:6], x[:, 6:], s["seq_lens"], q=x[:, :4], starts=s["starts"])
    s["k"].copy_(k0)
    s["v"].copy_(v0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g.replay()
    side.synchronize()
    assert torch.equal(s["k"], want[0]) and torch.equal(s["v"], want[1]) and torch.equal(q_graph, q_eager)
