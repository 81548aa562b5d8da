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
