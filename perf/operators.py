"""Cases, plain forms and definitions of the cache and scoring operators.

Three operators of a serving loop:

  append    the keys and values of new tokens into a contiguous or paged KV cache, rotated by their positions
            (after a per-head RMS norm where the model has one), and the rotated queries
  attend    one query token a sequence over a cache whose first positions all sequences share
  logprobs  log probabilities of given tokens, the entropy and the most likely alternatives, from logits

`run` computes them in plain torch operations, or, where `own` is set, through this package.
"""
import math

import torch

own = False

THETA = 5e5
EPS = 1e-6
LAYERS, LAYER = 2, 1  # the caches hold two layers; the operators work on the second
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one decode step's rows of eight sequences (13B heads), fp32 projections as the decode step makes them: latency
        dict(name="append decode 8", op="append", tokens=8, batch=8, q_heads=40, kv_heads=40, head_dim=128, dtype="fp32", page=128,
             cached=4000, norm=False),
        # a chunk of ragged prompts of the 0.6B heads with query/key norms, contiguous cache, odd count
        dict(name="append chunk 509 norm", op="append", tokens=509, batch=5, q_heads=16, kv_heads=8, head_dim=128, dtype="bf16", page=0,
             cached=700, norm=True),
        # prefill of a ragged batch, 8B heads, small pages
        dict(name="append prefill 4100", op="append", tokens=4100, batch=8, q_heads=32, kv_heads=8, head_dim=128, dtype="bf16", page=16,
             cached=300, norm=False),
        # the largest: a long prefill of the 13B heads from fp32 projections
        dict(name="append prefill 16384", op="append", tokens=16384, batch=12, q_heads=40, kv_heads=40, head_dim=128, dtype="fp32", page=128,
             cached=2000, norm=False),
        # one sequence over a short context (0.6B heads): latency
        dict(name="attend single 1024", op="attend", batch=1, q_heads=16, kv_heads=8, head_dim=128, prefix=1000, own_lo=24, own_hi=24, page=0,
             idle=False),
        # small heads, odd lengths, pages of 16, an idle slot
        dict(name="attend hd64 ragged", op="attend", batch=7, q_heads=12, kv_heads=4, head_dim=64, prefix=777, own_lo=1, own_hi=333, page=16,
             idle=True),
        # the 13B batch: as many key/value heads as query heads, a system prompt shared, ragged answers: memory
        dict(name="attend batch 8", op="attend", batch=8, q_heads=40, kv_heads=40, head_dim=128, prefix=2048, own_lo=100, own_hi=2048, page=128,
             idle=False),
        # a long document asked about by 64 sequences (8B heads)
        dict(name="attend doc 32768 x 64", op="attend", batch=64, q_heads=32, kv_heads=8, head_dim=128, prefix=32768, own_lo=16, own_hi=300, page=64,
             idle=False),
        # the largest: many samples of one long prompt, compute bound
        dict(name="attend doc 16384 x 256", op="attend", batch=256, q_heads=32, kv_heads=8, head_dim=128, prefix=16384, own_lo=1, own_hi=255,
             page=128, idle=True),
        # the step's own logits of one sequence (8B vocabulary): latency
        dict(name="logprobs 1", op="logprobs", rows=1, vocab=128256, dtype="fp32", top=5, masked=False),
        # a small batch of the 0.6B vocabulary, part of it masked away
        dict(name="logprobs 8 masked", op="logprobs", rows=8, vocab=151936, dtype="fp32", top=20, masked=True),
        # scoring a whole prompt from bf16 logits
        dict(name="logprobs 2047 bf16", op="logprobs", rows=2047, vocab=128256, dtype="bf16", top=20, masked=False),
    ]


def _log(rng, lo, hi):
    return min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


HEADS = [(16, 8), (32, 8), (40, 40), (32, 4), (4, 2), (7, 7), (8, 1), (6, 2), (32, 1), (12, 4), (16, 16), (10, 2)]
PAGES = [0, 16, 32, 48, 64, 128, 256, 384]


def draw(rng):
    top = {op: {k: max(work(c)[k] for c in listed() if c["op"] == op) for k in ("bytes", "flops")} for op in ("append", "attend", "logprobs")}
    op = rng.choice(["append", "attend", "attend", "logprobs"])
    while True:
        heads = rng.choice(HEADS)
        common = dict(q_heads=heads[0], kv_heads=heads[1], head_dim=rng.choice([64, 128, 128]), page=rng.choice(PAGES))
        if op == "append":
            batch = _log(rng, 1, 64)
            decode = rng.random() < 0.3
            c = dict(op=op, tokens=batch if decode else _log(rng, 1, 16384), batch=batch, dtype=rng.choice(["bf16", "fp32"]), cached=_log(rng, 1, 4000),
                     norm=rng.random() < 0.4, **common)
            room = common["page"] > 0 or batch * common["kv_heads"] * common["head_dim"] * (c["cached"] + c["tokens"]) * 8 < 8e9
        elif op == "attend":
            hi = _log(rng, 1, 4096)
            batch = _log(rng, 1, 256)
            c = dict(op=op, batch=batch, prefix=rng.choice([0, _log(rng, 1, 65536), _log(rng, 1, 65536)]), own_lo=rng.randint(1, hi), own_hi=hi,
                     idle=batch > 1 and rng.random() < 0.3, **common)
            # what the plain form holds: the scores, and each sequence's own rows
            room = c["batch"] * (c["q_heads"] * (c["prefix"] + hi) + c["kv_heads"] * hi * common["head_dim"] * 2) * 4 < 4e9
            if common["page"] == 0:
                room = room and c["batch"] * (c["prefix"] + hi) * c["kv_heads"] * common["head_dim"] * 8 < 24e9
        else:
            c = dict(op=op, rows=_log(rng, 1, 2047), vocab=_log(rng, 50, 151936), dtype=rng.choice(["bf16", "fp32"]), top=rng.choice([0, 1, 5, 8, 20, 32]),
                     masked=rng.random() < 0.4)
            room = True
        w = work(c)
        if room and w["bytes"] <= top[op]["bytes"] and w["flops"] <= top[op]["flops"]:
            return c


def work(case):
    c = case
    if c["op"] == "append":
        n = c["tokens"] * (c["q_heads"] + 2 * c["kv_heads"]) * c["head_dim"]
        turned = c["tokens"] * (c["q_heads"] + c["kv_heads"]) * c["head_dim"]
        return {"bytes": n * (2 + TYPES[c["dtype"]].itemsize), "flops": turned * (3 + (4 if c["norm"] else 0))}
    if c["op"] == "attend":
        lens = _attend_lens(c)
        own_rows = sum(max(0, x - c["prefix"]) for x in lens)
        io = c["batch"] * c["q_heads"] * (c["head_dim"] * 4 + 4)
        return {"bytes": (c["prefix"] + own_rows) * c["kv_heads"] * c["head_dim"] * 4 + io, "flops": 4 * c["q_heads"] * c["head_dim"] * sum(lens)}
    n = c["rows"] * c["vocab"]
    return {"bytes": n * TYPES[c["dtype"]].itemsize + c["rows"] * (12 + 8 * c["top"]), "flops": 5 * n}


def _attend_lens(c):
    """Positions that each sequence attends over, before a seed's permutation."""
    b, lo, hi = c["batch"], c["own_lo"], c["own_hi"]
    lens = [c["prefix"] + (hi if b == 1 else lo + (hi - lo) * i // (b - 1)) for i in range(b)]
    if c["idle"]:
        lens[0] = 0
    return lens


def _pages(c, g, s):
    """A table of shuffled pages and the pool's size: a sequence holds the pages it needs, its other entries are -1."""
    b, page = c["batch"], c["page"]
    stride = -(-s["max_ctx"] // page)
    j = torch.arange(stride, device="cuda", dtype=torch.int32)
    if c["op"] == "attend":  # the prefix's whole pages are the same for every sequence
        shared = c["prefix"] // page
        pool = shared + b * (stride - shared) + 3
        at = torch.where(j < shared, j, j + torch.arange(b, device="cuda", dtype=torch.int32)[:, None] * (stride - shared))
        used = torch.ones_like(at, dtype=torch.bool)
    else:
        pool = (b * c["cached"] + c["tokens"]) // page + b + 3
        new = 1 if s["starts"] is None else s["starts"].diff()
        need = (s["seq_lens"] + new + page - 1) // page
        at = (need.cumsum(0) - need)[:, None] + j
        used = j < need[:, None]
    order = torch.randperm(pool, generator=g, device="cuda").int()
    return torch.where(used, order[torch.where(used, at, 0).long()], -1).contiguous(), pool


def _caches(c, g, s):
    """Random caches of LAYERS layers: contiguous, or a pool of pages with spare ones and its table."""
    n, d, page = c["kv_heads"], c["head_dim"], c["page"]
    s["table"], shape = None, (LAYERS, c["batch"], n, s["max_ctx"], d)
    if page:
        s["table"], pool = _pages(c, g, s)
        shape = (LAYERS, pool, n, page, d)
    s["k_cache"], s["v_cache"] = (torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g) for _ in range(2))


def prepare(case, seed):
    c = case
    g = torch.Generator("cuda")
    g.manual_seed(seed)
    s = {"case": c}
    if c["op"] == "logprobs":
        n, v, t = c["rows"], c["vocab"], TYPES[c["dtype"]]
        x = torch.empty((n, v), dtype=torch.float32, device="cuda").normal_(generator=g).mul_(3.0)
        if c["masked"]:  # a grammar that allows a part of the vocabulary
            keep = torch.rand((n, 1), generator=g, device="cuda") * 0.9 + 0.05
            x.masked_fill_(torch.rand((n, v), generator=g, device="cuda") > keep, -math.inf)
            x[:, v // 2] = 1.0
        s["logits"] = x.to(t)
        s["tokens"] = torch.randint(v, (n,), generator=g, device="cuda", dtype=torch.int32)
    elif c["op"] == "append":
        b, n = c["batch"], c["tokens"]
        lens = (torch.rand(b, generator=g, device="cuda") * (c["cached"] + 1)).int()
        max_ctx = c["cached"] + n
        if n == b:  # one token a sequence
            s["starts"] = None
            max_ctx = c["cached"] + 1
        else:  # ragged: any cut of the tokens, empty sequences among them
            cuts = torch.randint(n + 1, (b - 1,), generator=g, device="cuda", dtype=torch.int32).sort()[0]
            zero = torch.zeros(1, dtype=torch.int32, device="cuda")
            s["starts"] = torch.cat([zero, cuts, zero + n])
        t = TYPES[c["dtype"]]
        width = (c["q_heads"] + 2 * c["kv_heads"]) * c["head_dim"]
        s["qkv"] = torch.empty((n, width), dtype=t, device="cuda").normal_(generator=g)
        if c["norm"]:
            s["q_norm"], s["k_norm"] = (torch.empty(c["head_dim"], device="cuda").uniform_(0.5, 1.5, generator=g).bfloat16() for _ in range(2))
        else:
            s["q_norm"] = s["k_norm"] = None
        s["seq_lens"] = lens
        s["max_ctx"] = max_ctx
        _caches(c, g, s)
    else:
        lens = torch.tensor(_attend_lens(c), dtype=torch.int32, device="cuda")
        s["seq_lens"] = lens[torch.randperm(c["batch"], generator=g, device="cuda")].contiguous()
        s["max_ctx"] = c["prefix"] + c["own_hi"]
        s["q"] = torch.empty((c["batch"], c["q_heads"], c["head_dim"]), device="cuda").normal_(generator=g).mul_(1.5).bfloat16()
        _caches(c, g, s)
    if own and c["op"] != "logprobs":
        import auto_regressive_decode_b200.mk as mk
        s["cache"] = mk.Cache(s["k_cache"], s["v_cache"], n_q_heads=c["q_heads"], batch=c["batch"], max_ctx=s["max_ctx"], block_table=s["table"],
                              page_size=c["page"], rope_theta=THETA, rms_eps=EPS)
    return s


def run(state):
    op = state["case"]["op"]
    if own:
        return {"append": _own_append, "attend": _own_attend, "logprobs": _own_logprobs}[op](state)
    return {"append": _append, "attend": _attend, "logprobs": _logprobs}[op](state)


# ---- the framework's calls -----------------------------------------------------------------------

def _own_append(s):
    c = s["case"]
    nq, nkv, d = c["q_heads"], c["kv_heads"], c["head_dim"]
    x = s["qkv"].view(c["tokens"], nq + 2 * nkv, d)
    q = s["cache"].append(LAYER, x[:, nq:nq + nkv], x[:, nq + nkv:], s["seq_lens"], q=x[:, :nq], starts=s["starts"], q_norm=s["q_norm"],
                          k_norm=s["k_norm"])
    return [q, s["k_cache"], s["v_cache"]]


def _own_attend(s):
    return s["cache"].attend(LAYER, s["q"], s["seq_lens"], prefix_len=s["case"]["prefix"])


def _own_logprobs(s):
    import auto_regressive_decode_b200.mk as mk
    return mk.token_logprobs(s["logits"], s["tokens"], top_k=s["case"]["top"])


# ---- plain forms ---------------------------------------------------------------------------------

def _token_places(s, n):
    """Sequence and cache index of each of the n tokens."""
    b, dev = s["case"]["batch"], s["seq_lens"].device
    if s["starts"] is None:
        return torch.arange(b, device=dev), s["seq_lens"].long()
    starts = s["starts"].long()
    t = torch.arange(n, device=dev)
    seq = torch.searchsorted(starts, t, right=True) - 1
    return seq, s["seq_lens"].long()[seq] + t - starts[seq]


def _append(s):
    c = s["case"]
    n, nq, nkv, d = c["tokens"], c["q_heads"], c["kv_heads"], c["head_dim"]
    seq, slot = _token_places(s, n)
    x = s["qkv"].view(n, nq + 2 * nkv, d)
    turned = []
    freq = THETA ** (-torch.arange(0, d, 2, device=x.device, dtype=torch.float64) / d)
    angle = slot.double()[:, None] * freq
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    for y, gain in ((x[:, :nq].float(), s["q_norm"]), (x[:, nq:nq + nkv].float(), s["k_norm"])):
        if gain is not None:
            y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * gain.float()
        a, b = y[..., :d // 2], y[..., d // 2:]
        turned.append(torch.cat([a * cos - b * sin, b * cos + a * sin], -1).bfloat16())
    _rows(s, "k_cache", seq, slot, turned[1])
    _rows(s, "v_cache", seq, slot, x[:, nq + nkv:].float().bfloat16())
    return [turned[0], s["k_cache"], s["v_cache"]]


def _rows(s, which, seq, pos, put=None):
    """The cache's rows [..., kv head, head_dim] at (sequence, position), read or written."""
    pool, page = s[which][LAYER], s["case"]["page"]
    first, second = (s["table"].long()[seq, pos // page], pos % page) if page else (seq, pos)
    if put is None:
        return pool[first, :, second]
    pool[first, :, second] = put


def _attend(s):
    c = s["case"]
    b, n, d, p = c["batch"], c["kv_heads"], c["head_dim"], c["prefix"]
    q = s["q"].float().view(b, n, c["q_heads"] // n, d) / math.sqrt(d)
    dev = q.device
    shared = torch.arange(p, device=dev)
    later = torch.arange(p, p + c["own_hi"], device=dev)
    at = torch.arange(b, device=dev)[:, None], later[None].expand(b, -1)
    kp, ko = _rows(s, "k_cache", torch.zeros_like(shared), shared).float(), _rows(s, "k_cache", *at).float()
    vp, vo = _rows(s, "v_cache", torch.zeros_like(shared), shared).float(), _rows(s, "v_cache", *at).float()
    score = torch.cat([torch.einsum("bngd,pnd->bngp", q, kp), torch.einsum("bngd,bwnd->bngw", q, ko)], -1)
    seen = torch.cat([shared, later]) < s["seq_lens"][:, None]
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(score - top)
    z = e.sum(-1, keepdim=True)
    o = torch.einsum("bngp,pnd->bngd", e[..., :p], vp) + torch.einsum("bngw,bwnd->bngd", e[..., p:], vo)
    o = torch.where(z == 0, 0.0, o / z)
    return [o.bfloat16().view(b, -1, d), (top + z.log()).view(b, -1)]


def _logprobs(s):
    c = s["case"]
    x = s["logits"].float()
    top = x.amax(-1, keepdim=True)
    e = torch.exp(x - top)
    z = e.sum(-1, keepdim=True)
    gap = torch.where(e == 0, 0.0, top - x)
    entropy = (z.log() + (e * gap).sum(-1, keepdim=True) / z)[:, 0]
    given = torch.gather(x, 1, s["tokens"].long()[:, None])
    logp = (given - top - z.log())[:, 0]
    # the largest first, the lowest index first among equals
    k = min(c["top"], c["vocab"])
    bits = x.view(torch.int32).long()
    key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * 2 ** 32 - torch.arange(c["vocab"], device=x.device)
    ids = torch.topk(key, k, dim=1)[1]
    best = torch.gather(x, 1, ids) - top - z.log()
    ids = torch.where(best == -math.inf, -1, ids).int()
    if k < c["top"]:  # fewer words than alternatives asked for
        ids = torch.cat([ids, ids.new_full((c["rows"], c["top"] - k), -1)], 1)
        best = torch.cat([best, best.new_full((c["rows"], c["top"] - k), -math.inf)], 1)
    return [logp, entropy, ids, best]


# ---- the definitions in 64 bits ------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "logprobs": _exact_logprobs}[case["op"]](s)


def _exact_append(s):
    c = s["case"]
    n, nq, nkv, d = c["tokens"], c["q_heads"], c["kv_heads"], c["head_dim"]
    starts = list(range(c["batch"] + 1)) if s["starts"] is None else s["starts"].tolist()
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    x = s["qkv"].view(n, nq + 2 * nkv, d)
    q_out = torch.empty((n, nq, d), dtype=torch.float64, device=x.device)
    for b, cached in enumerate(s["seq_lens"].tolist()):
        lo, hi = starts[b], starts[b + 1]
        if lo == hi:
            continue
        pos = torch.arange(cached, cached + hi - lo, device=x.device)
        i = torch.arange(d // 2, device=x.device, dtype=torch.float64)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device), pos.double()[:, None] * torch.exp(-2 * i / d * math.log(THETA)))
        part = x[lo:hi].double()
        out = []
        for y, gain in ((part[:, :nq], s["q_norm"]), (part[:, nq:nq + nkv], s["k_norm"])):
            if gain is not None:
                y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / d + EPS) * gain.double()
            z = torch.complex(y[..., :d // 2].contiguous(), y[..., d // 2:].contiguous()) * turn[:, None]
            out.append(torch.cat([z.real, z.imag], -1))
        q_out[lo:hi] = out[0]
        for pool, rows in ((kc, out[1]), (vc, part[:, nq + nkv:])):
            if c["page"]:
                pages = s["table"][b].long()
                pool[LAYER][pages[pos // c["page"]], :, pos % c["page"]] = rows
            else:
                pool[LAYER, b, :, pos] = rows.transpose(0, 1)
    return [q_out, kc, vc]


def _exact_attend(s):
    c = s["case"]
    p, d, page = c["prefix"], c["head_dim"], c["page"]
    g = c["q_heads"] // c["kv_heads"]
    out = torch.zeros((c["batch"], c["q_heads"], d), dtype=torch.float64, device="cuda")
    lse = torch.full((c["batch"], c["q_heads"]), -math.inf, dtype=torch.float64, device="cuda")

    def rows(pool, b, lo, hi):  # [kv head, positions, head_dim]
        if not page:
            return pool[LAYER, b, :, lo:hi].double()
        pos = torch.arange(lo, hi, device="cuda")
        return pool[LAYER][s["table"][b].long()[pos // page], :, pos % page].transpose(0, 1).double()

    kp, vp = rows(s["k_cache"], 0, 0, p), rows(s["v_cache"], 0, 0, p)
    for b, n in enumerate(s["seq_lens"].tolist()):
        if n == 0:
            continue
        q = s["q"][b].double().view(c["kv_heads"], g, d)
        k, v = (torch.cat([x[:, :min(n, p)], rows(s[w], b, p, max(n, p))], 1) for x, w in ((kp, "k_cache"), (vp, "v_cache")))
        a = torch.bmm(q, k.transpose(1, 2)) * d ** -0.5
        out[b] = torch.bmm(torch.softmax(a, -1), v).reshape(-1, d)
        lse[b] = torch.logsumexp(a, -1).reshape(-1)
    return [out, lse]


def _exact_logprobs(s):
    c = s["case"]
    logp, entropy, ids, best = [], [], [], []
    for x, t in zip(s["logits"].split(256), s["tokens"].split(256)):
        lp = torch.log_softmax(x.double(), -1)
        logp.append(torch.gather(lp, 1, t.long()[:, None])[:, 0])
        entropy.append(torch.special.entr(lp.exp()).sum(-1))
        v, i = torch.sort(lp, dim=-1, descending=True, stable=True)
        best.append(v[:, :c["top"]])
        ids.append(torch.where(v == -math.inf, -1, i)[:, :c["top"]].int())
    logp, entropy, ids, best = (torch.cat(x) for x in (logp, entropy, ids, best))
    short = c["top"] - ids.shape[1]
    if short > 0:
        ids = torch.nn.functional.pad(ids, (0, short), value=-1)
        best = torch.nn.functional.pad(best, (0, short), value=-math.inf)
    return [logp, entropy, ids, best]
