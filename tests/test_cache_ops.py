"""Refusals of the cache and scoring operators, on the host (no GPU): every check comes before a CUDA call."""
import ctypes

import pytest

import auto_regressive_decode_b200.mk as mk

FAKE = 1 << 20      # a pointer that is never followed


def create(kv=None, **kw):
    d = dict(n_layers=2, batch=4, n_q_heads=8, n_kv_heads=2, head_dim=64, max_ctx=100, rms_eps=1e-6, rope_theta=1e4)
    d.update(kw)
    kv = kv or mk.mk_kv(FAKE, FAKE, None, 0, 0)
    h = ctypes.c_void_p()
    rc = mk.mk_cache_create(ctypes.byref(mk.mk_cache_desc(*d.values())), ctypes.byref(kv), ctypes.byref(h))
    assert not h.value
    return rc


@pytest.mark.parametrize("kw", [{"n_layers": 0}, {"batch": -1}, {"n_q_heads": 0}, {"n_kv_heads": 0}, {"head_dim": -64}, {"max_ctx": 0},
                                {"rms_eps": -1.0}, {"rms_eps": float("nan")}, {"rope_theta": 0.0}])
def test_malformed_descriptions(kw):
    assert create(**kw) == mk.MK_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [{"head_dim": 96}, {"head_dim": 256}, {"n_q_heads": 9}, {"n_q_heads": 130}, {"batch": 1025},
                                {"n_layers": 2000, "batch": 1000, "max_ctx": 1000}, {"max_ctx": 1 << 30}])
def test_unsupported_shapes(kw):
    assert create(**kw) == mk.MK_ERR_UNSUPPORTED


@pytest.mark.parametrize("kv,rc", [
    ((None, FAKE, None, 0, 0), mk.MK_ERR_INVALID_ARG), ((FAKE, None, None, 0, 0), mk.MK_ERR_INVALID_ARG),
    ((FAKE + 2, FAKE, None, 0, 0), mk.MK_ERR_UNSUPPORTED), ((FAKE, FAKE + 8, None, 0, 0), mk.MK_ERR_UNSUPPORTED),
    ((FAKE, FAKE, FAKE, 0, 5), mk.MK_ERR_INVALID_ARG), ((FAKE, FAKE, FAKE, 16, 0), mk.MK_ERR_INVALID_ARG),
    ((FAKE, FAKE, FAKE, 24, 5), mk.MK_ERR_UNSUPPORTED), ((FAKE, FAKE, FAKE + 1, 16, 5), mk.MK_ERR_UNSUPPORTED),
    ((FAKE, FAKE, FAKE, 1 << 20, 1 << 20), mk.MK_ERR_UNSUPPORTED),
])
def test_caches(kv, rc):
    assert create(mk.mk_kv(*kv)) == rc


def test_null_arguments():
    assert mk.mk_cache_create(None, None, None) == mk.MK_ERR_INVALID_ARG
    assert mk.mk_cache_destroy(None) == mk.MK_OK
    assert mk.mk_cache_get_status(None, None) == mk.MK_ERR_INVALID_ARG
    assert mk.mk_cache_append(None, 0, None, None) == mk.MK_ERR_INVALID_ARG
    assert mk.mk_cache_attend(None, 0, None, None, 0, 0.0, None, None, None, 0, None) == mk.MK_ERR_INVALID_ARG
    assert mk.mk_cache_attend_bytes(None) == 0
    assert mk.mk_decode_greedy_scored(None, None, 1, None, None, None, None, None, None, None, None, 0, None, None) == mk.MK_ERR_INVALID_ARG


def scores(logits=FAKE, dtype=mk.MK_DTYPE_FP32, stride=10, rows=1, vocab=10, tokens=FAKE, logprob=FAKE, entropy=FAKE, k=2, ids=FAKE, tops=FAKE):
    return mk.mk_token_logprobs(logits, dtype, stride, rows, vocab, tokens, logprob, entropy, k, ids, tops, -1, None)


@pytest.mark.parametrize("kw,rc", [
    ({"rows": 0, "logits": None, "tokens": None}, mk.MK_OK),
    ({"rows": -1}, mk.MK_ERR_INVALID_ARG), ({"vocab": 0}, mk.MK_ERR_INVALID_ARG), ({"k": -1}, mk.MK_ERR_INVALID_ARG),
    ({"dtype": 7}, mk.MK_ERR_INVALID_ARG), ({"logits": None}, mk.MK_ERR_INVALID_ARG), ({"tokens": None}, mk.MK_ERR_INVALID_ARG),
    ({"logprob": None}, mk.MK_ERR_INVALID_ARG), ({"ids": None}, mk.MK_ERR_INVALID_ARG), ({"tops": None}, mk.MK_ERR_INVALID_ARG),
    ({"stride": -10}, mk.MK_ERR_INVALID_ARG), ({"k": 33}, mk.MK_ERR_UNSUPPORTED), ({"logits": FAKE + 2}, mk.MK_ERR_UNSUPPORTED),
    ({"logits": FAKE + 1, "dtype": mk.MK_DTYPE_BF16}, mk.MK_ERR_UNSUPPORTED), ({"tokens": FAKE + 2}, mk.MK_ERR_UNSUPPORTED),
    ({"logprob": FAKE + 2}, mk.MK_ERR_UNSUPPORTED), ({"ids": FAKE + 3}, mk.MK_ERR_UNSUPPORTED),
])
def test_scores(kw, rc):
    assert scores(**kw) == rc


def test_the_binding_refuses_host_tensors_and_wrong_shapes():
    import torch
    x, tok = torch.zeros(2, 5), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(mk.MkError):
        mk.token_logprobs(x, tok)
    k = torch.zeros((1, 2, 1, 8, 64), dtype=torch.bfloat16)
    with pytest.raises(mk.MkError):
        mk.Cache(k, k, n_q_heads=1, batch=2, max_ctx=8)


def test_a_stream_of_another_device_is_refused():
    import types

    import torch
    with pytest.raises(mk.MkError, match="stream of cpu"):
        mk.token_logprobs(torch.zeros(2, 5), torch.zeros(2, dtype=torch.int32), stream=types.SimpleNamespace(device=torch.device("cuda:1")))
