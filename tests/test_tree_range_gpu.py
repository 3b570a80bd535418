"""Tree attention where a query's weights span a wide range: a key far above all the others whose
value is nothing, as an attention sink's is, so that the others make up the result."""
import math

import pytest
import torch

import paged_kv_cache_171_gb300 as pa
from tests import evict_reference as ref
from tests.test_tree_gpu import _built, _case, _parents, _run, _seen  # noqa: F401

pytestmark = pytest.mark.gpu


COPIES = 160  # CTAs enough that no sequence's keys are cut into ranges


def _sink(t, n, hq, dt, above, at, seed):
    """One sequence of t keys whose key `at` scores `above` (scale 0.1) over the others, which
    score nearly the same, so that the roundings of their weights do not average out; its value
    is 0."""
    q, k, v, bt, ctx = _case([t], n, hq, 1, 64, dt, seed)
    k[..., 1:] *= 0.02
    k[..., 0] = 0
    v += 0.5  # the others' contributions add up
    page, slot = ref.places(bt, 0, torch.tensor([at]))
    k[page, 0, slot] = 0
    k[page, 0, slot, 0] = above
    v[page, 0, slot] = 0
    q[..., 0] = 10
    return q, k, v, bt, ctx


def _bound(q, k, v, bt, ctx, seen, scale):
    """(out, bound).  The weights' and the result's roundings, half a step of q's type each; fp32's
    part: the scores, the exponential, and sums of which each of t / 128 tiles and 32 partial
    sums of a tile takes half a step (ref.tree's).  P is 2^7 p in fp16, so below 2^-14 its half
    step is 2^-25, of a weight 2^-32 of the row's reference, which is no larger than its
    largest: 2^-32 sum |v| / l in place of the 2^-25 of weights held as they are."""
    want, loose = ref.tree(q, k, v, bt, ctx, seen, scale)
    B, n, hq, _ = q.shape
    off = torch.zeros_like(want)
    for b, c in enumerate(ctx.tolist()):
        kk, vv = ref.rows(k, bt, b, c + n)[0], ref.rows(v, bt, b, c + n)[0]
        vis = torch.cat((torch.ones((n, c), dtype=torch.bool), seen[b]), 1)
        _, l, _ = ref.attention(q[b].double(), kk, vis, scale)
        size = torch.einsum("nt,td->nd", vis.double(), vv.abs())[:, None]
        off[b] = size / torch.where(l > 0, l, 1.0)
    return want, loose - (2.0 ** -25 - 2.0 ** -32) * off


@pytest.mark.parametrize("above", [6, 12, 14, 16, 17.5])
@pytest.mark.parametrize("n,hq", [(4, 8), (12, 8), (20, 8)])
@pytest.mark.parametrize("at", [0, 9000])
def test_the_others_beside_a_sink(above, n, hq, at):
    t = 16000
    seen, _ = _seen(_parents(1, n, n))
    case = _sink(t, n, hq, torch.float16, above, at, 3)
    q, k, v, bt, ctx = case
    many = [x.expand(COPIES, *x.shape[1:]).contiguous() for x in (q, bt, ctx, ref.bits(seen))]
    all_of_them = _run(many[0], k, v, many[1], many[2], many[3], 0.1)
    got = all_of_them[:1]
    assert (all_of_them == got).all()
    want, bound = _bound(*case, seen, 0.1)
    off = (got.double() - want).abs() - bound
    assert (off <= 0).all(), (off.max().item(), (off / want.abs()).max().item())
