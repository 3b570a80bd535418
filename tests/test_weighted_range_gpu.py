"""Gathered weights of keys with values that are not finite: a key that every query scores -inf
weighs nothing, one that some query scores +inf or NaN weighs NaN, the others what they would
without it."""
import math

import pytest
import torch

import paged_kv_cache_171_gb300 as pa
from tests import evict_reference as ref
from tests.test_weighted_gpu import _built  # noqa: F401

pytestmark = pytest.mark.gpu


def _case(n, hq, hkv, d, dt, lens, value):
    """Queries whose dimension 0 is positive; keys 7, 150 and the last but one hold `value`
    there."""
    k, v, w, bt, _ = ref.pool([t + n for t in lens], hkv, d, dt, n + hq)
    q = torch.randn((len(lens), n, hq, d), generator=torch.Generator().manual_seed(n)).to(dt)
    q[..., 0] = q[..., 0].abs() + 0.25
    odd = []
    for b, t in enumerate(lens):
        at = torch.tensor(sorted({min(x, t + n - 1) for x in (7, 150, t + n - 2)}))
        page, slot = ref.places(bt, b, at)
        k[page, :, slot, 0] = value
        odd.append((page, slot))
    return q, k, v, w, bt, torch.tensor(lens, dtype=torch.int32), odd


def _without(q, k, w, bt, ctx, odd, scale):
    """(weights, bound), all of them set, where the keys in `odd` are not there: the bound is
    ref.chunk_weights' (scores, exponentials, the rows' statistics, the sums)."""
    B, n, hq, d = q.shape
    hkv = k.shape[1]
    G = hq // hkv
    new, wb = w.double().clone(), torch.zeros(w.shape).double()
    for b, c in enumerate(ctx.tolist()):
        t = c + n
        kk = torch.nan_to_num(ref.rows(k, bt, b, t), 0, 0, 0)
        page, slot = ref.places(bt, b, torch.arange(t))
        seen = torch.arange(t)[None, :] <= c + torch.arange(n)[:, None]
        for p2, s2 in zip(*odd[b]):
            seen &= ~((page == p2) & (slot == s2))
        for g in range(hkv):
            qq = q[b, :, g * G:(g + 1) * G].double()
            p, l, err = ref.attention(qq, kk[g], seen, scale)
            s = (torch.einsum("nhd,td->nht", qq, kk[g]) * scale).masked_fill(~seen[:, None], 0.0)
            lse = s.abs().amax(-1, keepdim=True) + l.log().abs()
            err = err + 4 * ref.H32 * lse + 2 * ref.H32 * (n * G / 4 + 16)
            new[page, g, slot] = p.sum((0, 1))
            wb[page, g, slot] = (err * p).sum((0, 1)) + 2 * ref.H32 * p.sum((0, 1))
    return new, wb


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,hq,hkv", [(1, 1, 1), (3, 8, 1), (20, 8, 1), (33, 8, 1), (5, 10, 1),
                                      (90, 8, 1), (150, 10, 1), (70, 14, 2), (600, 3, 1)])
@pytest.mark.parametrize("scale", [0.1, -0.1])
def test_keys_that_score_minus_infinity_weigh_nothing(n, hq, hkv, dt, scale):
    value = -math.inf if scale > 0 else math.inf
    q, k, _, w, bt, ctx, odd = _case(n, hq, hkv, 64, dt, [400, 100, 3], value)
    gw = w.cuda()
    pa.prefill_weights(q.cuda(), k.cuda(), gw, bt.cuda(), ctx.cuda(), scale, fresh=10 ** 9)
    assert pa.pa_last_device_error() == 0
    want, bound = _without(q, k, w, bt, ctx, odd, scale)
    for page, slot in odd:
        assert (gw.cpu()[page, :, slot] == 0).all()
    assert ((gw.cpu().double() - want).abs() <= bound).all()


@pytest.mark.parametrize("n,hq", [(3, 8), (5, 10), (150, 10), (40, 8)])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_keys_that_score_otherwise_weigh_nan(n, hq, value):
    q, k, _, w, bt, ctx, odd = _case(n, hq, 1, 64, torch.bfloat16, [400], value)
    gw = w.cuda()
    pa.prefill_weights(q.cuda(), k.cuda(), gw, bt.cuda(), ctx.cuda(), 0.1)
    assert pa.pa_last_device_error() == 0
    page, slot = odd[0]
    assert gw.cpu()[page, :, slot].isnan().all()


@pytest.mark.parametrize("hq", [1, 4, 10])
def test_decode_too(hq):
    q, k, v, w, bt, ctx, odd = _case(1, hq, 1, 64, torch.bfloat16, [400, 100], -math.inf)
    gw = w.cuda()
    pa.decode_weighted(q[:, 0].contiguous().cuda(), k.cuda(), v.cuda(), gw, bt.cuda(),
                       (ctx + 1).cuda(), 0.1, fresh=10 ** 9)
    assert pa.pa_last_device_error() == 0
    for page, slot in odd:
        assert (gw.cpu()[page, :, slot] == 0).all()
    assert gw.isfinite().all()
