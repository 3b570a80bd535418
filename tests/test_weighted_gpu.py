"""GPU parity of weighted decode and of a chunk's gathered weights against the definition in
64 bits."""
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


def _within(got, want, bound, what):
    assert torch.isfinite(got).all(), what
    off = (got.double().cpu() - want).abs() - bound
    assert (off <= 0).all(), (what, off.max().item(), (off > 0).sum().item())


def _decode(lens, hq, hkv, d, dt, seed, scale, fresh, blocks=None, mul=1.0):
    k, v, w, bt, ctx = ref.pool(lens, hkv, d, dt, seed, fill=math.nan, blocks=blocks)
    q = (torch.randn((len(lens), hq, d), generator=torch.Generator().manual_seed(seed + 1))
         * mul).to(dt)
    gw = w.cuda()
    got = pa.decode_weighted(q.cuda(), k.cuda(), v.cuda(), gw, bt.cuda(), ctx.cuda(), scale, fresh)
    assert pa.pa_last_device_error() == 0
    out, ob, new, wb = ref.weighted_decode(q, k, v, w, bt, ctx, scale, fresh)
    _within(got, out, ob, "out")
    _within(gw, new, wb, "weights")  # (the bound is 0 where nothing is written)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(4, 4), (4, 2), (6, 2), (8, 2), (10, 2), (7, 1), (8, 1), (9, 1),
                                    (16, 1), (33, 1), (24, 2)])
def test_decode_groups(hq, hkv, d, dtype):
    _decode([0, 1, 15, 16, 17, 33, 300], hq, hkv, d, DT[dtype], hq * d, 1 / math.sqrt(d), 1)


@pytest.mark.parametrize("lens", [[1], [5000], [16] * 70, [0, 0, 0], [0, 2049, 0, 1], [1023, 1025],
                                  [12000, 3, 700]])
@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 128), (8, 2, 64)])
def test_decode_lengths(lens, hq, hkv, d):
    _decode(lens, hq, hkv, d, torch.bfloat16, sum(lens), 1 / math.sqrt(d), 1, mul=2.0)


@pytest.mark.parametrize("scale", [0.0, -0.07, 1.0])
@pytest.mark.parametrize("fresh", [0, 1, 5, 10 ** 9])
def test_decode_scales_and_fresh(scale, fresh):
    _decode([3, 40, 700], 8, 2, 128, torch.float16, 5, scale, fresh)


def test_decode_wide_table():
    _decode([5, 900], 8, 2, 128, torch.bfloat16, 6, 0.1, 1, blocks=3000)


def test_decode_same_bits_and_other_calls_between():
    k, v, w, bt, ctx = (x.cuda() for x in ref.pool([3000, 700], 2, 128, torch.bfloat16, 7))
    q = torch.randn((2, 8, 128), device="cuda").bfloat16()
    ws = torch.empty(pa.pa_decode_weighted_workspace_size(2, 8, 2, 128, 16, bt.shape[1]),
                     dtype=torch.uint8, device="cuda")
    got = []
    for i in range(20):
        gw = w.clone()
        ws.fill_(i)  # contents on entry do not matter
        got.append((pa.decode_weighted(q, k, v, gw, bt, ctx, 0.1, workspace=ws), gw))
    for o, gw in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(gw, got[0][1])


def test_decode_bad_pages_and_lengths():
    k, v, w, bt, ctx = ref.pool([40, 40, 40], 2, 64, torch.bfloat16, 8)
    q = torch.randn((3, 4, 64), generator=torch.Generator().manual_seed(9)).bfloat16()
    bad = bt.clone()
    bad[1, 1] = k.shape[0]
    gw = w.cuda()
    got = pa.decode_weighted(q.cuda(), k.cuda(), v.cuda(), gw, bad.cuda(), ctx.cuda(), 0.1)
    assert pa.pa_last_device_error() == -11
    out, ob, new, wb = ref.weighted_decode(q, k, v, w, bt, ctx, 0.1, 1)
    for b in (0, 2):
        _within(got[b], out[b], ob[b], b)
        pages = bt[b].long()
        _within(gw.cpu()[pages], new[pages], wb[pages], b)
    assert torch.equal(gw.cpu()[bt[1, 1].long()], w[bt[1, 1].long()])  # not written
    for length in (-1, 10 ** 6):
        c = ctx.clone()
        c[1] = length
        pa.decode_weighted(q.cuda(), k.cuda(), v.cuda(), w.cuda(), bt.clamp(min=0).cuda(), c.cuda(),
                           0.1)
        assert pa.pa_last_device_error() == -12


def _chunk(lens, n, hq, hkv, d, dt, seed, scale, fresh, view=False, blocks=None, mul=1.0):
    k, _, w, bt, _ = ref.pool([t + n for t in lens], hkv, d, dt, seed, fill=math.nan, blocks=blocks)
    ctx = torch.tensor(lens, dtype=torch.int32)
    gen = torch.Generator().manual_seed(seed + 1)
    wide = (torch.randn((len(lens), n + 3, hq + 2, d), generator=gen) * mul).to(dt)
    q = wide[:, 3:, 1:hq + 1]
    gw = w.cuda()
    gq = wide.cuda()[:, 3:, 1:hq + 1]
    pa.prefill_weights(gq if view else gq.contiguous(), k.cuda(), gw, bt.cuda(), ctx.cuda(), scale,
                       fresh)
    assert pa.pa_last_device_error() == 0
    new, wb = ref.chunk_weights(q, k, w, bt, ctx, scale, n if fresh is None else fresh)
    _within(gw, new, wb, "weights")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,n", [(4, 4, 5), (4, 4, 130), (6, 2, 44), (10, 2, 26), (7, 1, 19),
                                      (8, 1, 70), (130, 1, 5), (131, 1, 2), (33, 3, 12),
                                      (8, 2, 200), (256, 1, 3)])
def test_chunk_groups(hq, hkv, n, d, dtype):
    _chunk([0, 100, 257], n, hq, hkv, d, DT[dtype], hq + n, 1 / math.sqrt(d), None, view=n % 2 == 0)


@pytest.mark.parametrize("lens,n", [([0], 1), ([0], 128), ([127], 1), ([128, 0], 1), ([255], 2),
                                    ([4000], 16), ([3000, 5], 33), ([1], 600), ([900, 77, 0], 300)])
@pytest.mark.parametrize("hq,hkv,d", [(8, 1, 128), (4, 2, 64)])
def test_chunk_lengths(lens, n, hq, hkv, d):
    _chunk(lens, n, hq, hkv, d, torch.bfloat16, n, 1 / math.sqrt(d), None, mul=2.0)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
@pytest.mark.parametrize("fresh", [0, 3, 10 ** 9])
@pytest.mark.parametrize("n", [6, 150])
def test_chunk_scales_and_fresh(scale, fresh, n):
    _chunk([30, 200], n, 8, 2, 128, torch.float16, 5, scale, fresh)


def test_chunk_wide_table():
    _chunk([30, 2000], 40, 8, 2, 128, torch.bfloat16, 5, 0.1, None, blocks=2500)
    _chunk([30, 2000], 300, 8, 2, 64, torch.bfloat16, 6, 0.1, None, blocks=2500)


def test_chunk_of_one_agrees_with_decode():
    k, v, w, bt, ctx = ref.pool([1, 90, 2000], 2, 128, torch.bfloat16, 11)
    q = torch.randn((3, 8, 128), generator=torch.Generator().manual_seed(12)).bfloat16()
    a, b = w.cuda(), w.cuda()
    pa.decode_weighted(q.cuda(), k.cuda(), v.cuda(), a, bt.cuda(), ctx.cuda(), 0.1)
    pa.prefill_weights(q[:, None].cuda(), k.cuda(), b, bt.cuda(), (ctx - 1).cuda(), 0.1)
    _, _, new, wb = ref.weighted_decode(q, k, v, w, bt, ctx, 0.1, 1)
    _, cb = ref.chunk_weights(q[:, None], k, w, bt, ctx - 1, 0.1, 1)
    _within(a, new, wb, "decode")
    _within(b, new, cb, "chunk")


def test_nothing_to_do_and_bad_pages():
    k, _, w, bt, ctx = (x.cuda() for x in ref.pool([40], 2, 64, torch.bfloat16, 13))
    gw = w.clone()
    pa.prefill_weights(torch.empty((1, 0, 4, 64), dtype=torch.bfloat16, device="cuda"), k, gw, bt,
                       ctx, 0.1)
    assert torch.equal(gw, w)
    bad = bt.clone()
    bad[0, 2] = -5
    pa.prefill_weights(torch.randn((1, 4, 4, 64), device="cuda").bfloat16(), k, gw, bad, ctx - 4, 0.1)
    assert pa.pa_last_device_error() == -11
    assert torch.equal(gw[bt[0, 2].long()], w[bt[0, 2].long()])
