"""GPU parity of tree attention and of the trees' masks against the definition in 64 bits."""
import math

import pytest
import torch

import paged_kv_cache_171_gb300 as pa
from tests import evict_reference as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_171_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert pa.pa_last_device_error() == 0


def _parents(B, n, seed, reach=9):
    gen = torch.Generator().manual_seed(seed)
    p = torch.full((B, n), -1, dtype=torch.int32)
    for i in range(1, n):
        p[:, i] = i - 1 - torch.randint(0, min(i, reach) + 1, (B,), generator=gen).clamp(max=i)
    return p.clamp(min=-1)


def _seen(parents):
    B, n = parents.shape
    seen = torch.zeros((B, n, n), dtype=torch.bool)
    depth = torch.zeros((B, n), dtype=torch.int32)
    for b in range(B):
        for i in range(n):
            p = int(parents[b, i])
            if p >= 0:
                seen[b, i] = seen[b, p]
                depth[b, i] = depth[b, p] + 1
            seen[b, i, i] = True
    return seen, depth


def _case(lens, n, hq, hkv, d, dt, seed, blocks=None, mul=1.0):
    k, v, _, bt, _ = ref.pool([t + n for t in lens], hkv, d, dt, seed, fill=math.nan, blocks=blocks)
    q = (torch.randn((len(lens), n, hq, d), generator=torch.Generator().manual_seed(seed + 1))
         * mul).to(dt)
    return q, k, v, bt, torch.tensor(lens, dtype=torch.int32)


def _run(q, k, v, bt, ctx, words, scale):
    got = pa.prefill_tree(q.cuda(), k.cuda(), v.cuda(), bt.cuda(), ctx.cuda(), words.cuda(), scale)
    assert pa.pa_last_device_error() == 0
    return got.cpu()


def _check(case, seen, scale, words=None):
    got = _run(*case, ref.bits(seen) if words is None else words, scale)
    want, bound = ref.tree(*case, seen, scale)
    assert torch.isfinite(got).all()
    off = (got.double() - want).abs() - bound
    assert (off <= 0).all(), (off.max().item(), (off > 0).sum().item())
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,n", [(4, 4, 5), (4, 2, 33), (6, 2, 64), (8, 2, 60), (10, 2, 26),
                                      (7, 1, 37), (8, 1, 16), (8, 1, 17), (33, 3, 12), (24, 2, 22),
                                      (16, 1, 40), (2, 2, 130)])
def test_trees(hq, hkv, n, d, dtype):
    parents = _parents(3, n, n)
    _check(_case([0, 100, 300], n, hq, hkv, d, DT[dtype], hq * n), _seen(parents)[0],
           1 / math.sqrt(d))


@pytest.mark.parametrize("lens,n", [([0], 1), ([0], 128), ([127], 1), ([128], 3), ([120], 20),
                                    ([112, 128, 129], 33), ([4000], 16), ([6000, 1], 64),
                                    ([1000], 260), ([700, 0, 40], 31), ([15, 16, 17], 32)])
@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 128), (4, 2, 64), (5, 1, 128)])
def test_tree_lengths(lens, n, hq, hkv, d):
    _check(_case(lens, n, hq, hkv, d, torch.bfloat16, n, mul=2.0),
           _seen(_parents(len(lens), n, n))[0], 1 / math.sqrt(d))


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.6])
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_any_mask(scale, dtype):
    """Random bits: queries that do not see themselves, that see later ones, that see nothing
    (their rows are zeros where there is no context)."""
    n = 70
    seen = torch.rand((3, n, n), generator=torch.Generator().manual_seed(3)) < 0.2
    seen[:, 5] = False
    seen[:, 69] = True
    got = _check(_case([0, 50, 1000], n, 8, 2, 128, DT[dtype], 4), seen, scale)
    assert (got[0, 5] == 0).all()


def test_bits_behind_the_last_token_are_not_used():
    n = 37
    seen, _ = _seen(_parents(2, n, 1))
    case = _case([9, 200], n, 4, 1, 64, torch.bfloat16, 6)
    words = ref.bits(seen)
    more = words.clone()
    more[..., 1] |= -(1 << 5)
    assert torch.equal(_run(*case, words, 0.1), _run(*case, more, 0.1))


@pytest.mark.parametrize("where", ["k", "v"])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("lens,n,hq", [([20], 40, 4), ([128, 1000], 40, 4), ([0, 500], 200, 8)])
def test_what_is_not_finite_stays_with_those_who_see_it(where, value, lens, n, hq):
    seen, _ = _seen(_parents(len(lens), n, 2))
    q, k, v, bt, ctx = _case(lens, n, hq, 1, 64, torch.bfloat16, 8)
    bad = 7
    for b, c in enumerate(lens):
        page, slot = ref.places(bt, b, torch.tensor([c + bad]))
        (k if where == "k" else v)[page, 0, slot, 3] = value
    got = _run(q, k, v, bt, ctx, ref.bits(seen), 0.1)
    want, bound = ref.tree(q, k, v, bt, ctx, seen, 0.1)
    free = ~seen[:, :, bad]
    assert ((got.double() - want).abs() <= bound)[free].all()
    hit = got[~free]
    if where == "v":  # the one dimension
        col = hit[..., 3].float()
        assert (col.isnan() if math.isnan(value) else col == value).all()
        assert torch.isfinite(hit[..., :3]).all() and torch.isfinite(hit[..., 4:]).all()
    elif math.isnan(value):
        assert hit.isnan().all()


def test_a_chain_is_the_causal_chunk():
    n = 45
    case = _case([0, 130, 2000], n, 8, 2, 128, torch.bfloat16, 9)
    chain = torch.ones((3, n, n), dtype=torch.bool).tril()
    got = _check(case, chain, 0.1)
    q, k, v, bt, ctx = (x.cuda() for x in case)
    other = pa.prefill(q, k.nan_to_num(), v.nan_to_num(), bt, ctx, 0.1).cpu()
    # the chunk's own bound, and a tree's two roundings (of its weights and of its output) of
    # values up to 4, 2 x 2^-8 x 4, taken a little short
    assert (got.float() - other).abs().max() < 2e-3 + 3e-2


def test_a_wide_table_and_many_sequences():
    _check(_case([5, 3000], 20, 8, 1, 128, torch.bfloat16, 10, blocks=2000),
           _seen(_parents(2, 20, 3))[0], 0.1)
    _check(_case([33] * 90, 6, 4, 2, 64, torch.float16, 11), _seen(_parents(90, 6, 4))[0], 0.1)


def test_bad_pages_lengths_and_nothing():
    q, k, v, bt, ctx = _case([100, 100], 8, 4, 1, 64, torch.bfloat16, 12)
    k, v = k.nan_to_num(), v.nan_to_num()
    seen, _ = _seen(_parents(2, 8, 5))
    words = ref.bits(seen)
    bad = bt.clone()
    bad[0, 1] = -9
    got = pa.prefill_tree(q.cuda(), k.cuda(), v.cuda(), bad.cuda(), ctx.cuda(), words.cuda(), 0.1)
    assert pa.pa_last_device_error() == -11
    want, bound = ref.tree(q, k, v, bt, ctx, seen, 0.1)
    assert ((got.cpu().double() - want).abs() <= bound)[1].all()
    c = ctx.clone()
    c[0] = 105  # the tree would leave the table
    pa.prefill_tree(q.cuda(), k.cuda(), v.cuda(), bt.cuda(), c.cuda(), words.cuda(), 0.1)
    assert pa.pa_last_device_error() == -12
    none = pa.prefill_tree(q[:, :0].contiguous().cuda(), k.cuda(), v.cuda(), bt.cuda(), ctx.cuda(),
                           words[:, :0, :0].contiguous().cuda(), 0.1)
    assert none.shape == (2, 0, 4, 64) and pa.pa_last_device_error() == 0


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 64, 65, 200, 1000])
@pytest.mark.parametrize("reach", [1, 9, 2000])
def test_masks(n, reach):
    parents = _parents(3, n, n + reach, reach)
    parents[2] = torch.arange(-1, n - 1)  # a chain
    mask, depth = pa.tree_mask(parents.cuda())
    assert pa.pa_last_device_error() == 0
    seen, want = _seen(parents)
    assert torch.equal(mask.cpu(), ref.bits(seen)) and torch.equal(depth.cpu(), want)


@pytest.mark.parametrize("parent", [5, 6, 40, -2, 2 ** 31 - 1, -2 ** 31])
def test_masks_bad_parents(parent):
    parents = torch.arange(-1, 39, dtype=torch.int32)[None].clone()
    parents[0, 5] = parent
    mask, depth = pa.tree_mask(parents.cuda())
    assert pa.pa_last_device_error() == -14
    parents[0, 5] = -1  # the branch ends there
    seen, want = _seen(parents)
    assert torch.equal(mask.cpu(), ref.bits(seen)) and torch.equal(depth.cpu(), want)
