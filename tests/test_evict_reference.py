"""The 64-bit reference of the gathered weights, the eviction and the trees, pinned on the CPU:
against the oracle's decode and causal chunk, and by hand."""
import math

import torch

import oracle
from tests import evict_reference as ref

BF = torch.bfloat16


def test_weighted_decode_is_the_oracles_decode_and_its_weights_add_up():
    lens = [0, 1, 37, 130]
    k, v, w, bt, ctx = ref.pool(lens, 2, 64, BF, 1)
    q = torch.randn((4, 6, 64), generator=torch.Generator().manual_seed(2)).to(BF)
    out, _, new, _ = ref.weighted_decode(q, k, v, w, bt, ctx, 0.1, 10 ** 6)
    want = oracle.decode(q, k, v, bt, ctx, 0.1, 0)
    # (the oracle's results are fp32-rounded or better)
    assert (out - torch.from_numpy(want).double()).abs().max() < 1e-6
    for b, t in enumerate(lens):
        page, slot = ref.places(bt, b, torch.arange(t))
        total = new[page, :, slot].sum(0)
        assert torch.allclose(total, torch.full_like(total, 3.0 if t else 0.0), atol=1e-12)


def test_a_chain_is_the_oracles_chunk():
    lens, n = [20, 0, 7], 9
    k, v, _, bt, _ = ref.pool([t + n for t in lens], 2, 64, BF, 3)
    ctx = torch.tensor(lens, dtype=torch.int32)
    q = torch.randn((3, n, 4, 64), generator=torch.Generator().manual_seed(4)).to(BF)
    chain = torch.ones((3, n, n), dtype=torch.bool).tril()
    out, _ = ref.tree(q, k, v, bt, ctx, chain, 0.2)
    want = oracle.prefill(q, k, v, bt, ctx, 0.2, 0)
    assert (out - torch.from_numpy(want).double()).abs().max() < 1e-6


def test_kept_by_hand():
    w = torch.tensor([9.0, 1.0, math.nan, 2.0, 2.0, -0.0, 0.0, math.inf, 5.0, 0.1])
    assert ref.keep_list(w, 10, 10, 1, 1).tolist() == list(range(10))
    assert ref.keep_list(w, 10, 4, 1, 1).tolist() == [0, 7, 8, 9]
    assert ref.keep_list(w, 10, 5, 1, 1).tolist() == [0, 3, 7, 8, 9]       # ties: the lowest
    assert ref.keep_list(w, 10, 8, 1, 1).tolist() == [0, 1, 3, 4, 5, 7, 8, 9]
    assert ref.keep_list(w, 10, 9, 1, 1).tolist() == [0, 1, 3, 4, 5, 6, 7, 8, 9]  # NaN last
    assert ref.keep_list(w, 10, 3, 1, 2).tolist() == [0, 8, 9]


def test_bits():
    seen = torch.zeros((1, 33, 33), dtype=torch.bool)
    seen[0, 0, 0] = seen[0, 1, 31] = seen[0, 2, 32] = True
    words = ref.bits(seen)
    assert words[0, 0].tolist() == [1, 0] and words[0, 1].tolist() == [-2 ** 31, 0]
    assert words[0, 2].tolist() == [0, 1]
