"""When a cache handle is destroyed: never by a Cache that is merely dropped, which may happen within a stream capture."""
import gc

import pytest
import torch

import auto_regressive_decode_b200.mk as mk


@pytest.fixture
def destroyed(monkeypatch):
    calls = []
    monkeypatch.setattr(mk, "mk_cache_destroy", lambda h: calls.append(h) or 0)
    monkeypatch.setattr(mk, "_dropped", [])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)     # a host without a GPU cannot be asked
    return calls


def fake(h):
    c = object.__new__(mk.Cache)
    c.h, c.torch = h, torch
    return c


def test_a_dropped_cache_leaves_its_handle(destroyed):
    c = fake(1 << 20)
    del c
    gc.collect()
    assert destroyed == [] and mk._dropped == [1 << 20]
    mk._destroy_dropped()
    assert destroyed == [1 << 20] and mk._dropped == []


def test_close_destroys_once_and_what_was_dropped_before(destroyed):
    a, b = fake(1), fake(2)
    del a
    gc.collect()
    b.close()
    b.close()
    del b
    gc.collect()
    assert sorted(destroyed) == [1, 2] and mk._dropped == []


def test_close_within_a_capture_waits(destroyed, monkeypatch):
    c = fake(7)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    c.close()
    assert destroyed == [] and mk._dropped == [7] and c.h == 0


def test_a_cache_that_was_never_made(destroyed):
    c = object.__new__(mk.Cache)
    del c
    gc.collect()
    assert destroyed == [] and mk._dropped == []


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["drop", "close", "make"])
def test_captures_survive(how):
    """A cache dropped, closed or asked for within a capture; the graph's own cache goes on."""
    g = torch.Generator("cuda").manual_seed(0)
    k, v = (torch.randn((1, 2, 1, 40, 64), generator=g, device="cuda").bfloat16() for _ in range(2))
    q, lens = torch.randn((2, 4, 64), generator=g, device="cuda").bfloat16(), torch.tensor([30, 7], dtype=torch.int32, device="cuda")

    def make():
        return mk.Cache(k, v, n_q_heads=4, batch=2, max_ctx=40)
    kept, other = make(), make()
    want = other.attend(0, q, lens)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = kept.attend(0, q, lens)
        if how == "drop":
            del other
            gc.collect()
        elif how == "close":
            other.close()
        else:
            with pytest.raises(mk.MkError):
                make()
        again = kept.attend(0, q, lens)
    graph.replay()
    torch.cuda.synchronize()
    for r in (out, again):
        assert torch.equal(r[0], want[0]) and torch.equal(r[1], want[1])
    more = make()
    assert not mk._dropped
    assert torch.equal(more.attend(0, q, lens)[0], want[0])


@pytest.mark.gpu
def test_memory_of_closed_handles_goes_back():
    """Tables of 512 MB in all; 64 MB may stay with the library, and the driver's own blocks are of some MB."""
    T = 1 << 18
    k = torch.zeros((1, 1, 1, T, 128), dtype=torch.bfloat16, device="cuda")
    table = 8 * T * 64

    def make():
        return mk.Cache(k, k, n_q_heads=1, batch=1, max_ctx=T)
    make().close()
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0]
    handles = [make() for _ in range(4)]
    torch.cuda.synchronize()
    held = before - torch.cuda.mem_get_info()[0]
    assert held >= 4 * table - (64 << 20)
    for h in handles:
        h.close()
    torch.cuda.synchronize()
    assert before - torch.cuda.mem_get_info()[0] <= (64 << 20) + (32 << 20)


@pytest.mark.gpu
def test_handles_of_many_sizes_come_and_go():
    k = torch.randn((1, 1, 1, 1 << 15, 64), device="cuda").bfloat16()
    q, n = torch.randn((1, 1, 64), device="cuda").bfloat16(), torch.ones(1, dtype=torch.int32, device="cuda")
    for i in range(40):
        T = 1 + (i * 7919) % (1 << 15)
        part = k.view(-1)[:T * 64].view(1, 1, 1, T, 64)
        c = mk.Cache(part, part, n_q_heads=1, batch=1, max_ctx=T)
        assert torch.equal(c.attend(0, q, n)[0], part[0, :, :, 0])
        if i % 3:
            c.close()
