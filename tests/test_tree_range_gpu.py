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


@pytest.mark.parametrize("n", [4, 12, 20])
def test_small_weights_count_beside_a_large_one(n):
    """262144 keys 15 nats below a sink: each weighs 2.57 of the last places of a running sum that
    holds the sink's, so added one by one they would count as 3."""
    t, dt, hq, scale = 262144, torch.float16, 8, 0.1
    q, k, v, bt, ctx = _sink(t, n, hq, dt, 15, 0, 4)
    k[..., 1:] *= 0.25
    seen, _ = _seen(_parents(1, n, n))
    many = [x.expand(COPIES, *x.shape[1:]).contiguous() for x in (q, bt, ctx, ref.bits(seen))]
    got = _run(many[0], k, v, many[1], many[2], many[3], scale)[0].double()
    kk, vv = ref.rows(k, bt, 0, t + n)[0], ref.rows(v, bt, 0, t + n)[0]
    half = torch.finfo(dt).eps / 2
    for i in (0, n - 1):
        vis = torch.cat((torch.ones(t, dtype=torch.bool), seen[0, i]))[None]
        p, l, err = ref.attention(q[0, i:i + 1].double(), kk, vis, scale)
        want, size = p[0] @ vv, p[0] @ vv.abs()
        # Roundings of the result and of the weights; fp32's scores, exponentials and sums (a
        # half step a tile of 128 keys, and 32 for the tile's own); the tensor cores', which cut
        # the running sum off after each 16 keys, 2^-23 of it; fp16's last places of 2^7 p.
        bound = half * want.abs() + size * (half * 1.01 + err[0] + 2 * ref.H32 * (t / 128 + 32)
                                            + t / 16 * 2.0 ** -23)
        bound += 2.0 ** -32 * vv[vis[0]].abs().sum(0) / l[0]
        off = (got[i] - want).abs() - bound
        assert (off <= 0).all(), (off.max().item(), ((got[i] - want) / want).mean().item())
