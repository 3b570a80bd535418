"""Rows of one warp that go different ways: maxima that move in some rows only, drafted values
that only some rows add back."""
import math

import pytest
import torch

import paged_kv_cache_171_gb300 as pa
from tests import evict_reference as ref
from tests.test_tree_gpu import _built, _case, _parents, _run, _seen  # noqa: F401

pytestmark = pytest.mark.gpu


def _slopes(lens, n, hq, hkv, d, dt):
    """A case whose scores rise with the key in some rows, fall in others, and stay level in the
    rest, by 32 over 64 keys, beside noise."""
    q, k, v, bt, ctx = _case(lens, n, hq, hkv, d, dt, 5)
    for b, t in enumerate(lens):
        pos = torch.arange(t + n)
        page, slot = ref.places(bt, b, pos)
        k[page, :, slot, 0] = (pos % 128 * 0.5).to(dt)[:, None]
    way = torch.arange(n * hq).view(n, hq) % 3 - 1
    q[..., 0] = way * 10.0
    return q, k, v, bt, ctx


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,hq", [(3, 8), (20, 8), (30, 8), (150, 8)])
def test_maxima_that_move_in_some_rows(n, hq, dt):
    lens = [0, 700, 129]
    q, k, v, bt, ctx = _slopes(lens, n, hq, 1, 64, dt)
    w = torch.full((k.shape[0], 1, 16), 0.5)
    gw = w.cuda()
    pa.prefill_weights(q.cuda(), k.cuda(), gw, bt.cuda(), ctx.cuda(), 0.1)
    assert pa.pa_last_device_error() == 0
    want, bound = ref.chunk_weights(q, k, w, bt, ctx, 0.1, n)
    assert ((gw.cpu().double() - want).abs() <= bound).all()
    seen, _ = _seen(_parents(3, n, n))
    got = _run(q, k, v, bt, ctx, ref.bits(seen), 0.1)
    want, bound = ref.tree(q, k, v, bt, ctx, seen, 0.1)
    assert ((got.double() - want).abs() <= bound).all()


@pytest.mark.parametrize("lens,n,hq", [([20], 8, 8), ([300, 5], 16, 8), ([128, 1000], 60, 4),
                                       ([0, 500], 200, 8), ([5000], 33, 8)])
def test_drafted_values_added_back_by_some_rows(lens, n, hq):
    """Every third drafted token has an infinite value, in a dimension of its own."""
    seen, _ = _seen(_parents(len(lens), n, 2))
    q, k, v, bt, ctx = _case(lens, n, hq, 1, 64, torch.bfloat16, 8)
    bad = torch.arange(0, n, 3)
    for b, c in enumerate(lens):
        page, slot = ref.places(bt, b, c + bad)
        v[page, 0, slot, bad % 64] = math.inf
    got = _run(q, k, v, bt, ctx, ref.bits(seen), 0.1)
    want, bound = ref.tree(q, k, v, bt, ctx, seen, 0.1)
    hit = torch.zeros((len(lens), n, 64), dtype=torch.bool)
    for j in bad.tolist():
        hit[:, :, j % 64] |= seen[:, :, j]
    hit = hit[:, :, None].expand(got.shape)
    assert (got[hit] == math.inf).all()
    assert ((got.double() - want).abs() <= bound)[~hit].all()
