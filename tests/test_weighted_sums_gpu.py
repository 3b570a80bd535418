"""Weighted decode's normaliser where one key outweighs many: the others have to count for what
they are, however long the run of pages that a warp sums up."""
import pytest
import torch

import paged_kv_cache_171_gb300 as pa
from tests import evict_reference as ref
from tests.test_weighted_gpu import _built  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_small_weights_count_beside_a_large_one(dt):
    """16384 keys 15 nats below a sink: each weighs 2.57 last places of a sum that holds the
    sink's, so added to it one by one they would count as 3.  As many such sequences as give
    each warp one of them."""
    t, d, hq, scale = 16384, 64, 2, 0.1
    copies = torch.cuda.get_device_properties(0).multi_processor_count * 8
    gen = torch.Generator().manual_seed(1)
    k = torch.zeros((t // 16, 1, 16, d))
    k[..., 1:] = torch.randn(k[..., 1:].shape, generator=gen) * 0.005
    k[0, 0, 0] = 0
    k[0, 0, 0, 0] = 15
    v = torch.randn(k.shape, generator=gen) * 0.3 + 0.5
    v[0, 0, 0] = 0
    q = torch.randn((1, hq, d), generator=gen)
    q[..., 0] = 10
    k, v, q = k.to(dt), v.to(dt), q.to(dt)
    pages = k.shape[0]
    bt = torch.arange(copies * pages, dtype=torch.int32, device="cuda").view(copies, pages)
    w = torch.zeros((copies * pages, 1, 16), device="cuda")
    got = pa.decode_weighted(q.cuda().expand(copies, -1, -1).contiguous(),
                             *(x.cuda().repeat(copies, 1, 1, 1) for x in (k, v)), w, bt,
                             torch.full((copies,), t, dtype=torch.int32, device="cuda"), scale)
    assert pa.pa_last_device_error() == 0
    kk, vv = k[:, 0].reshape(-1, d).double(), v[:, 0].reshape(-1, d).double()
    p, _, err = ref.attention(q.double(), kk, torch.ones((1, t), dtype=torch.bool), scale)
    # ref.attention's bound of the scores and exponentials; half a step of each sum: of 16 pages'
    # two weights a lane, of the t / 256 of those, of eight lanes and of the partial states, and
    # of a page's products in the result
    adds = 2 * ref.H32 * (32 + t / 256 + 16)
    out = p[0] @ vv
    own = 2 * ref.H32 * t / 16  # the result's sum over pages, relative to it
    bound = (err[0] + adds + own) * (p[0] @ vv.abs())
    some = torch.tensor([0, 1, copies // 2, copies - 1])
    assert ((got[some].cpu().double() - out).abs() <= bound).all()
    # the weights have no sum over pages but the normaliser's
    add, wb = p[0].sum(0), ((err[0] + adds) * p[0]).sum(0) + 2 * ref.H32 * p[0].sum(0)
    for c in some.tolist():
        gw = w[c * pages:(c + 1) * pages, 0].reshape(-1).cpu().double()
        assert ((gw - add).abs() <= wb).all(), ((gw - add).abs() / add).max().item()


@pytest.mark.parametrize("above", [15, 17, 18.5])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_a_result_made_up_of_small_weights(above, dt):
    """32768 keys far below a sink that has no value: the result is theirs alone, so it has the
    relative error that their weights are held with."""
    t, d, hq, scale = 32768, 64, 2, 0.1
    gen = torch.Generator().manual_seed(2)
    k = torch.zeros((t // 16, 1, 16, d))
    k[..., 1:] = torch.randn(k[..., 1:].shape, generator=gen) * 0.005
    v = torch.randn(k.shape, generator=gen) * 0.3 + 0.5
    for page in range(0, t // 16, 8):  # one a part of the sequence, wherever it is cut
        k[page, 0, 0] = 0
        k[page, 0, 0, 0] = above
        v[page, 0, 0] = 0
    q = torch.randn((1, hq, d), generator=gen)
    q[..., 0] = 10
    k, v, q = k.to(dt), v.to(dt), q.to(dt)
    bt = torch.arange(t // 16, dtype=torch.int32)[None]
    w = torch.zeros((t // 16, 1, 16))
    ctx = torch.tensor([t], dtype=torch.int32)
    got = pa.decode_weighted(q.cuda(), k.cuda(), v.cuda(), w.cuda(), bt.cuda(), ctx.cuda(), scale)
    assert pa.pa_last_device_error() == 0
    out, bound, _, _ = ref.weighted_decode(q, k, v, w, bt, ctx, scale, 1)
    assert ((got.cpu().double() - out).abs() <= bound).all(), ((got.cpu() - out) / out).abs().max()
