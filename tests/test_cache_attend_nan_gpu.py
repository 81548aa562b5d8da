"""Rows whose scores are NaN: the output and its log-sum-exp both say so; -infinity is left to rows without positions."""
import math

import pytest
import torch

from tests.test_cache_attend_gpu import check, handle, make

pytestmark = pytest.mark.gpu

SHAPES = [(3, 8, 2, 64, 16), (2, 32, 2, 128, 0), (40, 4, 1, 128, 0), (50, 8, 2, 64, 16)]     # few rows over a prefix, and many


def attend(s):
    out, lse = handle(s).attend(s["layer"], s["q"], s["seq_lens"], prefix_len=s["prefix"])
    return out, lse


def compare(s, out, lse, bad):
    """`bad` [B][n_q]: NaN all through; the others are as ever."""
    assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all()
    t = dict(s, **{w: s[w + "0"] for w in ("q", "k", "v")})
    clean = attend(t)
    check(t, *clean)
    assert torch.equal(out[~bad], clean[0][~bad]) and torch.equal(lse[~bad], clean[1][~bad])


def keep(s):
    for w in ("q", "k", "v"):
        s[w + "0"] = s[w].clone()
    return s


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("prefix", [0, 150])
def test_a_query_of_nan(shape, prefix):
    B, nq = shape[:2]
    s = keep(make(*shape, prefix, [prefix + 1 + 30 * (i % 3) for i in range(B)], seed=30))
    bad = torch.zeros((B, nq), dtype=torch.bool, device="cuda")
    bad[B // 2, 1] = bad[B - 1] = True
    s["q"][bad] = math.nan
    compare(s, *attend(s), bad)


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("prefix", [90, 150])
def test_a_bad_key_of_the_prefix_alone(shape, prefix, value):
    """Sequences that end with the prefix: nothing but the prefix's pieces, or its only one, speak for them."""
    B, nq, nkv, hd, page = shape
    s = keep(make(*shape, prefix, [prefix if i % 2 else 0 for i in range(B)] if B > 2 else [prefix, prefix], seed=31))
    where = (s["layer"], int(s["table"][0, 60 // page]), 0, 60 % page, 3) if page else (s["layer"], 0, 0, 60, 3)
    s["k"][where] = value
    if value == math.inf:      # a score of +infinity for positive queries there, -infinity (no part) for negative ones
        s["q"][:, :, 3] = s["q0"][:, :, 3] = s["q"][:, :, 3].abs() + 0.5
    bad = torch.zeros((B, nq), dtype=torch.bool, device="cuda")
    bad[:, :nq // nkv] = (s["seq_lens"] > 60)[:, None]
    compare(s, *attend(s), bad)


@pytest.mark.parametrize("shape", SHAPES)
def test_a_single_position_whose_key_is_nan(shape):
    B, nq, nkv, hd, page = shape
    s = keep(make(*shape, 0, [1 + (i % 2) * 70 for i in range(B)], seed=32))
    at = (s["layer"], int(s["table"][0, 0]), nkv - 1, 0) if page else (s["layer"], 0, nkv - 1, 0)
    s["k"][at] = math.nan
    bad = torch.zeros((B, nq), dtype=torch.bool, device="cuda")
    bad[0, -(nq // nkv):] = True
    compare(s, *attend(s), bad)


def test_idle_sequences_stay_zero_and_minus_infinity():
    s = make(40, 4, 1, 128, 0, 100, [0 if i % 3 else 100 + i for i in range(40)], seed=33)
    check(s, *attend(s))
