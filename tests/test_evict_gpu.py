"""GPU parity of eviction and compaction: which tokens stay and where they lie, bit for bit."""
import math

import pytest
import torch

import paged_kv_cache_171_gb300 as pa
from tests import evict_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_171_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert pa.pa_last_device_error() == 0


def _same(a, b):
    a, b = a.cpu().contiguous(), b.contiguous()
    view = {2: torch.int16, 4: torch.int32}[a.element_size()]
    return torch.equal(a.view(view), b.view(view))


def _evict(lens, hkv, d, dt, budget, sink, recent, seed, kind="rand", place="in"):
    k, v, w, bt, ctx = ref.pool(lens, hkv, d, dt, seed, spare=2 + sum(-(-t // 16) for t in lens))
    gen = torch.Generator().manual_seed(seed + 5)
    if kind == "ties":
        w = torch.randint(0, 3, w.shape, generator=gen).float()
    elif kind == "same":
        w = torch.full_like(w, 0.25)
    elif kind == "odd":  # NaN, infinities, both zeros, negative, subnormal
        odd = torch.tensor([math.nan, math.inf, -math.inf, 0.0, -0.0, -1.0, 1e-41, 2.0, 2.0])
        w = odd[torch.randint(0, 9, w.shape, generator=gen)]
    elif kind == "close":  # equal but for the last bits
        w = 1.0 + torch.randint(0, 40, w.shape, generator=gen).float() * 2.0 ** -23
    dst = bt
    if place == "out":  # pages that no sequence uses
        free = sorted(set(range(k.shape[0])) - set(bt[bt >= 0].tolist()))
        dst, at = torch.full_like(bt, -1), 0
        for b, t in enumerate(lens):
            n = -(-min(t, budget) // 16)
            dst[b, :n] = torch.tensor(free[at:at + n], dtype=torch.int32)
            at += n
    want = ref.evict(k, v, w, bt, dst, ctx, budget, sink, recent)
    gk, gv, gw = k.cuda(), v.cuda(), w.cuda()
    table = bt.cuda()
    to = None if place == "in" else table.clone() if place == "copy" else dst.cuda()
    got = pa.evict_kv(gk, gv, gw, table, ctx.cuda(), budget, sink, recent, dst_table=to)
    assert pa.pa_last_device_error() == 0
    assert torch.equal(got.cpu(), want[3])
    for a, b, name in ((gw, want[2], "weights"), (gk, want[0], "k"), (gv, want[1], "v")):
        assert _same(a, b), name


@pytest.mark.parametrize("place", ["in", "out", "copy"])
@pytest.mark.parametrize("kind", ["rand", "ties", "same", "odd", "close"])
@pytest.mark.parametrize("budget,sink,recent", [(100, 4, 30), (1, 0, 0), (17, 17, 0), (33, 0, 33),
                                                (299, 0, 5)])
def test_eviction(kind, budget, sink, recent, place):
    _evict([300, 0, 99, 100, 101, 299], 3, 64, torch.bfloat16, budget, sink, recent, budget, kind,
           place)


@pytest.mark.parametrize("lens,hkv,d,budget", [([1], 1, 128, 0), ([1], 1, 64, 1), ([2], 1, 64, 1),
                                               ([16, 17], 2, 128, 16), ([5000], 1, 128, 700),
                                               ([3000] * 40, 4, 64, 500), ([7000, 9], 8, 128, 6999),
                                               ([4096] * 3, 2, 128, 2048)])
@pytest.mark.parametrize("place", ["in", "out"])
def test_eviction_sizes(lens, hkv, d, budget, place):
    _evict(lens, hkv, d, torch.float16, budget, min(4, budget), budget // 3, 3, place=place)


@pytest.mark.parametrize("t,budget", [(60001, 20000), (400001, 1000)])
def test_eviction_long(t, budget):
    """More keys than shared memory holds (the second), several CTAs a list (both)."""
    for kind in ("rand", "ties"):
        _evict([t], 1, 64, torch.bfloat16, budget, 4, 100, 4, kind)


def test_eviction_again_and_again():
    """Each eviction works on what the one before it left, in place."""
    k, v, w, bt, ctx = ref.pool([900, 640], 2, 64, torch.bfloat16, 21)
    gk, gv, gw, gbt, gctx = (x.cuda() for x in (k, v, w, bt, ctx))
    for budget in (800, 500, 499, 20):
        k, v, w, ctx = ref.evict(k, v, w, bt, bt, ctx, budget, 3, 9)
        gctx = pa.evict_kv(gk, gv, gw, gbt, gctx, budget, 3, 9)
        assert torch.equal(gctx.cpu(), ctx) and _same(gk, k) and _same(gv, v) and _same(gw, w)


def test_eviction_bad_pages_and_lengths():
    k, v, w, bt, ctx = ref.pool([100, 100], 2, 64, torch.bfloat16, 22)
    bad = bt.clone()
    bad[0, 3] = 10 ** 6
    gk, gv, gw = k.cuda(), v.cuda(), w.cuda()
    pa.evict_kv(gk, gv, gw, bad.cuda(), ctx.cuda(), 50, 4, 10)
    assert pa.pa_last_device_error() == -11
    k2, v2, w2, _ = ref.evict(k, v, w, bt, bt, ctx, 50, 4, 10)
    used = bt[1].long()
    assert _same(gk.cpu()[used], k2[used]) and _same(gw.cpu()[used], w2[used])
    for length in (-3, 113):
        c = ctx.clone()
        c[0] = length
        pa.evict_kv(k.cuda(), v.cuda(), w.cuda(), bt.cuda(), c.cuda(), 50, 4, 10)
        assert pa.pa_last_device_error() == -12
    # a table for the kept rows that is too short for them
    pa.evict_kv(k.cuda(), v.cuda(), w.cuda(), bt.cuda(), ctx.cuda(), 50, 4, 10,
                dst_table=bt[:, :2].contiguous().cuda())
    assert pa.pa_last_device_error() == -11
    with pytest.raises(pa.PAError):
        c = ctx.cuda()
        pa.evict_kv(k.cuda(), v.cuda(), w.cuda(), bt.cuda(), c, 50, new_lens=c)


def _compacted(x, bt, b, first, keep):
    out = x.clone()
    sp, sl = ref.places(bt, b, first + keep)
    dp, dl = ref.places(bt, b, first + torch.arange(len(keep)))
    out[dp, :, dl] = x[sp, :, sl]
    return out


@pytest.mark.parametrize("d,dt", [(64, torch.float16), (128, torch.bfloat16)])
@pytest.mark.parametrize("weights", [False, True])
@pytest.mark.parametrize("first,keeps", [([0], [[0, 2, 3]]), ([37, 15, 0], [[1, 5, 6, 40], [], [19]]),
                                         ([100], [list(range(1, 900, 3))]),
                                         ([16, 9], [list(range(50)), [49]])])
def test_compaction(first, keeps, weights, d, dt):
    n = max(max(k, default=0) for k in keeps) + 1
    k, v, w, bt, _ = ref.pool([t + n for t in first], 3, d, dt, n)
    most = max(len(x) for x in keeps)
    keep = torch.tensor([x + [-7] * (most - len(x)) for x in keeps], dtype=torch.int32)
    n_keep = torch.tensor([len(x) for x in keeps], dtype=torch.int32)
    ctx = torch.tensor(first, dtype=torch.int32)
    gk, gv, gw = k.cuda(), v.cuda(), w.cuda()
    got = pa.compact_kv(gk, gv, bt.cuda(), ctx.cuda(), keep.cuda(), n_keep.cuda(),
                        weights=gw if weights else None)
    assert pa.pa_last_device_error() == 0
    assert torch.equal(got.cpu(), ctx + n_keep)
    for b, x in enumerate(keeps):
        at = torch.tensor(x, dtype=torch.int64)
        k, v = _compacted(k, bt, b, first[b], at), _compacted(v, bt, b, first[b], at)
        if weights:
            w = _compacted(w, bt, b, first[b], at)
    assert _same(gk, k) and _same(gv, v) and _same(gw, w)


@pytest.mark.parametrize("keep,n_keep,first", [([3, 2, 5], 3, 10), ([2, 2, 5], 3, 10),
                                               ([-1, 2, 5], 3, 10), ([1, 2, 54], 3, 10),
                                               ([1, 2, 3], 4, 10), ([1, 2, 3], -1, 10),
                                               ([1, 2, 3], 2, -1), ([1, 2, 3], 2, 65)])
def test_compaction_refuses_a_bad_list(keep, n_keep, first):
    k, v, w, bt, _ = ref.pool([64, 64], 2, 64, torch.bfloat16, 31)
    gk, gv, gw = k.cuda(), v.cuda(), w.cuda()
    ctx = torch.tensor([first, 5], dtype=torch.int32, device="cuda")
    lists = torch.tensor([keep, [1, 4, 9]], dtype=torch.int32, device="cuda")
    got = pa.compact_kv(gk, gv, bt.cuda(), ctx, lists,
                        torch.tensor([n_keep, 3], dtype=torch.int32, device="cuda"), weights=gw)
    assert pa.pa_last_device_error() == (-12 if first < 0 or first > 64 else -14)
    assert got.tolist() == [min(max(first, 0), 64), 8]  # nothing kept; the other one as asked
    at = torch.tensor([1, 4, 9])
    assert _same(gk, _compacted(k, bt, 1, 5, at)) and _same(gw, _compacted(w, bt, 1, 5, at))
