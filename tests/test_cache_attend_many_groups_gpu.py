"""Short prefixes under so many sequences that a block of the prefix kernel ends several groups of rows, each with a
partial last tile; against attention in 64 bits, with the tolerance of the attention tests."""
import pytest
import torch

from tests.test_cache_attend_gpu import check, handle, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,nq,nkv,hd,page,prefix", [
    (1024, 64, 8, 128, 0, 100), (1024, 64, 8, 128, 16, 127), (1024, 64, 8, 128, 0, 128), (1024, 64, 8, 128, 0, 129), (1000, 80, 8, 128, 0, 100),
    (1000, 80, 8, 128, 0, 1), (1000, 40, 40, 128, 0, 100), (1024, 128, 8, 128, 0, 300), (1024, 64, 8, 64, 0, 200), (1000, 80, 8, 64, 16, 300),
    (1024, 128, 8, 64, 0, 383), (1000, 128, 8, 64, 0, 100),
], ids=lambda v: str(v))
def test_blocks_that_end_several_groups(batch, nq, nkv, hd, page, prefix):
    lens = [prefix + (i % 4) * (i % 7 > 0) - (i % 11 == 3) for i in range(batch)]      # some end with the prefix or before it
    s = make(batch, nq, nkv, hd, page, prefix, lens, seed=20, n_layers=1, layer=0)
    c = handle(s)
    got = [c.attend(0, s["q"], s["seq_lens"], prefix_len=prefix) for _ in range(3)]
    assert c.status() == 0
    check(s, *got[0])
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
