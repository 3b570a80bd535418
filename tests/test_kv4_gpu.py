"""GPU parity of the 4-bit cache: append (bytes exact), read, page copy, decode and
prefill attention against the definition in 64 bits; rows with no key, pages that
end inside a tile, rows behind a sequence, non-finite rows, far page offsets,
streams and graphs."""
import math

import pytest
import torch

import paged_kv_cache_171_gb300 as pa
from tests import kv4_reference as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_171_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert pa.pa_last_device_error() == 0


def tokens_of(lens):
    seq = torch.cat([torch.full((t,), b, dtype=torch.int32) for b, t in enumerate(lens)])
    pos = torch.cat([torch.arange(t, dtype=torch.int32) for t in lens])
    return seq, pos


def make_pool(lens, hkv, d, dt, gen, spread=1.0, junk=True):
    """A pool with N(0, spread) rows for every token of `lens`, in shuffled pages;
    everything else (rows behind a sequence, spare pages) random codes and NaN
    scales and zeros."""
    blocks = [-(-t // 16) for t in lens]
    pages = sum(blocks) + 2
    perm = torch.randperm(pages, generator=gen).to(torch.int32)
    bt = torch.full((len(lens), max(1, max(blocks))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(blocks):
        bt[b, :n] = perm[at:at + n]
        at += n
    shape = (pages, hkv, ref.block_bytes(d))
    pool = torch.zeros(shape, dtype=torch.uint8)
    if junk:
        pool.copy_(torch.randint(0, 256, shape, generator=gen, dtype=torch.uint8))
        pool[:, :, 16 * d:] = 255
    seq, pos = tokens_of(lens)
    k = torch.randn((seq.numel(), hkv, d), generator=gen) * spread
    v = torch.randn((seq.numel(), hkv, d), generator=gen) * spread
    ref.store(pool, bt, seq, pos, k, v, dt)
    return pool, bt


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def check_decode(lens, hq, hkv, d, dtype, seed=0, q_mul=1.0, spread=1.0, scale=None):
    dt, gen = DT[dtype], torch.Generator().manual_seed(seed)
    pool, bt = make_pool(lens, hkv, d, dt, gen, spread)
    q = (torch.randn((len(lens), hq, d), generator=gen) * q_mul).to(dt)
    scale = 1 / math.sqrt(d) if scale is None else scale
    want, bound = ref.attention(q[:, None].cuda(), pool.cuda(), bt, [[t] for t in lens], scale, dt)
    got = pa.decode_kv4(q.cuda(), pool.cuda(), bt.cuda(), i32(*lens), scale)
    torch.cuda.synchronize()
    assert pa.pa_last_device_error() == 0
    assert got.dtype == torch.float32 and torch.isfinite(got).all()
    err = (got.double() - want[:, 0]).abs()
    assert (err <= bound[:, 0, :, None]).all(), (err.max(), bound.min())
    rel = float((got.double() - want[:, 0]).norm() / want.norm().clamp(min=1e-300))
    assert rel < 1e-5 or want.norm() == 0, rel
    for b, t in enumerate(lens):
        if t == 0:
            assert (got[b] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (4, 2), (8, 2), (7, 1), (12, 4), (10, 2),
                                    (16, 2), (9, 1), (24, 1), (33, 3)])
def test_decode_head_layouts(hq, hkv, d, dtype):
    check_decode([1, 0, 15, 16, 17, 300], hq, hkv, d, dtype, seed=hq * 100 + d)


@pytest.mark.parametrize("lens", [[1], [0], [0, 0, 0], [2], [63, 64, 65], [1025], [5000, 3],
                                  [1] * 70, list(range(40)), [0] * 33 + [700] + [0] * 9])
def test_decode_lengths(lens):
    check_decode(lens, 8, 2, 128, "bf16", seed=len(lens))


@pytest.mark.parametrize("lens,hq,hkv,d,dtype", [
    ([32768, 1, 20000, 777], 64, 8, 128, "bf16"),
    ([4096] * 3, 32, 32, 128, "fp16"),
    ([9000, 128, 8192, 5], 28, 4, 64, "bf16")])
def test_decode_long(lens, hq, hkv, d, dtype):
    check_decode(lens, hq, hkv, d, dtype, seed=5, q_mul=2.0)


@pytest.mark.parametrize("dtype,q_mul,spread,scale", [
    ("bf16", 1e-20, 1.0, None), ("bf16", 1e20, 1e-18, 0.01), ("bf16", 1.0, 1e15, 1e-16),
    ("bf16", 1.0, 1e-20, None), ("fp16", 100.0, 0.01, None), ("fp16", 0.001, 100.0, None),
    ("bf16", 1.0, 1.0, 0.0), ("bf16", 1.0, 1.0, -0.1), ("fp16", 0.0, 1.0, None),
    ("bf16", 20.0, 1.0, None)])
def test_decode_magnitudes(dtype, q_mul, spread, scale):
    """Very small and very large queries and values, negative and zero scales."""
    check_decode([40, 1, 333], 8, 2, 128, dtype, seed=9, q_mul=q_mul, spread=spread, scale=scale)


def test_decode_equal_values_are_exact():
    """A constant row quantises to scale 0: every output is that constant."""
    dt, n = torch.bfloat16, 50
    kv = pa.kv4_cache(4, 2, 128)
    bt = i32(0, 1, 2, 3)[None]
    k = torch.randn((n, 2, 128), device="cuda").to(dt)
    v = torch.full((n, 2, 128), 1.5, dtype=dt, device="cuda")
    pa.append_kv4(k, v, kv, bt, torch.zeros(n, dtype=torch.int32, device="cuda"),
                  torch.arange(n, dtype=torch.int32, device="cuda"))
    q = torch.randn((1, 8, 128), device="cuda").to(dt)
    out = pa.decode_kv4(q, kv, bt, i32(n), 0.09)
    # z and l are sums of the same 50 weights: a rounding a term, and the merges'
    assert (out - 1.5).abs().max() <= 1.5 * 64 * ref.EPS32


def test_decode_scales_that_grow():
    """V rows whose scales grow, or shrink, by powers of ten along the sequence."""
    dt, gen = torch.bfloat16, torch.Generator().manual_seed(3)
    for order in (1, -1):
        pool, bt = make_pool([200], 1, 128, dt, gen, junk=False)
        k = torch.randn((200, 1, 128), generator=gen)
        v = torch.randn((200, 1, 128), generator=gen)
        v *= 10.0 ** (order * torch.linspace(-3, 3, 200))[:, None, None]
        ref.store(pool, bt, *tokens_of([200]), k, v, dt)
        q = torch.randn((1, 4, 128), generator=gen).to(dt)
        want, bound = ref.attention(q[:, None], pool, bt, [[200]], 0.088, dt)
        got = pa.decode_kv4(q.cuda(), pool.cuda(), bt.cuda(), i32(200), 0.088)
        err = (got.cpu().double() - want[:, 0]).abs()
        assert (err <= bound[:, 0, :, None]).all()


def check_prefill(hq, hkv, n_new, ctx, d, dtype, q_mul=1.0, spread=1.0, scale=None, seed=0):
    dt, gen = DT[dtype], torch.Generator().manual_seed(n_new + hq + seed)
    pool, bt = make_pool([t + n_new for t in ctx], hkv, d, dt, gen, spread)
    q = (torch.randn((len(ctx), n_new, hq, d), generator=gen) * q_mul).to(dt)
    scale = 1 / math.sqrt(d) if scale is None else scale
    seen = [[t + i + 1 for i in range(n_new)] for t in ctx]
    want, bound = ref.attention(q.cuda(), pool.cuda(), bt, seen, scale, dt)
    got = pa.prefill_kv4(q.cuda(), pool.cuda(), bt.cuda(), i32(*ctx), scale)
    torch.cuda.synchronize()
    assert pa.pa_last_device_error() == 0
    assert got.dtype == dt and torch.isfinite(got).all()
    # The weights may enter the tensor cores as one bf16 term, off by at most half a
    # step (2^-8) each, so a row by 2^-8 vmax (N(0, spread) values stay below
    # 8 spread); then the result's own rounding.
    err = (got.double() - want).abs()
    half = torch.finfo(dt).eps / 2
    assert (err <= bound[..., None] + 8 * spread * 2.0 ** -8 + half * want.abs()).all(), err.max()
    rel = float((got.double() - want).norm() / want.norm())
    assert rel < 5e-3, rel


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,n_new,ctx", [
    (8, 2, 1, [0, 5, 100]), (8, 2, 4, [0, 15, 16, 1000]), (4, 4, 17, [3, 200]),
    (16, 2, 3, [50, 0]), (7, 1, 5, [129, 1]), (12, 4, 33, [0, 31]), (24, 1, 2, [77]),
    (8, 1, 130, [0, 260]), (32, 8, 64, [500]), (7, 1, 150, [0, 127, 128]), (10, 2, 300, [1]),
    (2, 2, 257, [0, 1000])])
def test_prefill_matches_definition(hq, hkv, n_new, ctx, d, dtype):
    check_prefill(hq, hkv, n_new, ctx, d, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n_new,ctx", [
    (6, [5000, 0, 130, 9000, 64, 2, 127, 128] + [40] * 60), (8, [100] * 90), (16, [20000, 3]),
    (20, [5000, 0, 130, 9000, 64]), (70, [3000, 0, 130, 1, 6000]), (6, [7] * 3 + [4000])])
def test_prefill_items_cut_between_runs(n_new, ctx, dtype):
    """Many short items a run, long ones over many runs, both in one call: chunks of 24
    to 280 rows a kv head."""
    check_prefill(16, 4, n_new, ctx, 128, dtype, seed=3)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n_new", [8, 9, 16, 17, 24, 25, 32, 33, 64, 65, 128, 129, 256, 257])
def test_prefill_rows_at_every_border(n_new, dtype):
    """One row a query: the kernels' row counts, one on either side."""
    check_prefill(2, 2, n_new, [300, 0, 1000], 128, dtype, seed=1)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_items_cut_between_runs(d):
    """More items than teams of warps, short and long ones mixed."""
    gen = torch.Generator().manual_seed(6)
    lens = torch.randint(0, 400, (150,), generator=gen).tolist() + [9000, 1, 3000]
    check_decode(lens, 32, 8, d, "bf16", seed=6)


@pytest.mark.parametrize("dtype,q_mul,spread,scale", [
    ("bf16", 1.0, 1e15, 1e-16), ("bf16", 1.0, 1e-20, None), ("fp16", 100.0, 0.01, None),
    ("fp16", 0.001, 100.0, None), ("bf16", 1.0, 1.0, 0.0), ("bf16", 1.0, 1.0, -0.1),
    ("bf16", 20.0, 1.0, None)])
@pytest.mark.parametrize("n_new", [3, 140])
def test_prefill_magnitudes(n_new, dtype, q_mul, spread, scale):
    check_prefill(8, 2, n_new, [0, 333], 128, dtype, q_mul, spread, scale)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("order", [1, -1])
@pytest.mark.parametrize("n_new,ctx", [(6, 5000), (300, 4000)])
def test_prefill_magnitudes_along_the_context(n_new, ctx, order, dtype):
    """K and V whose magnitude grows, or shrinks, along a long context: each tile of
    keys with scales of its own."""
    dt, gen, n = DT[dtype], torch.Generator().manual_seed(8), n_new + ctx
    pool, bt = make_pool([n], 1, 128, dt, gen, junk=False)
    by = 4.0 ** (order * torch.linspace(-2, 2, n))[:, None, None]
    k = torch.randn((n, 1, 128), generator=gen) * by
    v = torch.randn((n, 1, 128), generator=gen) * by
    ref.store(pool, bt, *tokens_of([n]), k, v, dt)
    q = (torch.randn((1, n_new, 4, 128), generator=gen) * 0.1).to(dt)
    seen = [[ctx + i + 1 for i in range(n_new)]]
    want, _ = ref.attention(q.cuda(), pool.cuda(), bt, seen, 0.09, dt)
    got = pa.prefill_kv4(q.cuda(), pool.cuda(), bt.cuda(), i32(ctx), 0.09)
    rel = float((got.double() - want).norm() / want.norm())
    # four roundings of half a step each at most: K, V, the weights and the result
    assert rel < 4 * torch.finfo(dt).eps / 2, rel


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n_new", [5, 40, 200])
def test_prefill_rows_that_are_not_finite_reach_only_their_queries(n_new, dtype):
    """A key or value row that is not finite makes the queries that see it NaN, and
    leaves the ones before it as they are."""
    dt, gen, ctx, at = DT[dtype], torch.Generator().manual_seed(6), 30, 3
    pool, bt = make_pool([ctx + n_new], 1, 128, dt, gen)
    q = torch.randn((1, n_new, 4, 128), generator=gen).to(dt).cuda()
    clean = pa.prefill_kv4(q, pool.cuda(), bt.cuda(), i32(ctx), 0.09)
    page, slot = int(bt[0, (ctx + at) // 16]), (ctx + at) % 16
    for which in (0, 1):
        bad = pool.clone()
        bad[page, 0, 16 * 128 + (which * 16 + slot) * 4:][:4] = 255  # NaN scale and zero
        got = pa.prefill_kv4(q, bad.cuda(), bt.cuda(), i32(ctx), 0.09)
        assert torch.equal(got[:, :at], clean[:, :at])
        assert torch.isnan(got[:, at:]).all()


@pytest.mark.parametrize("rot,inter", [(None, False), (1, False), (1, True), (2, False), (2, True),
                                       (16, False), (48, True)])
@pytest.mark.parametrize("hq,hkv,d,dtype,lens", [
    (8, 2, 128, "bf16", [1, 0, 37]), (0, 3, 64, "fp16", [20, 5]), (4, 4, 64, "bf16", [1]),
    (12, 4, 128, "fp16", [16, 17]), (32, 8, 128, "bf16", [900, 1700])])
def test_append_bytes_match_the_definition(hq, hkv, d, dtype, lens, rot, inter):
    """Codes, scales and zeros are those of the documented fp32 steps, bit for bit;
    rows not written keep their bytes."""
    dt, gen = DT[dtype], torch.Generator().manual_seed(d + hkv)
    pool, bt = make_pool(lens, hkv, d, dt, gen)
    seq, pos = tokens_of(lens)
    n = seq.numel()
    wide = torch.randn((n, hq + 2 * hkv + 1, d), generator=gen).to(dt)  # one row of slack
    q, k, v = wide[:, :hq], wide[:, hq:hq + hkv], wide[:, hq + hkv:hq + 2 * hkv]
    cos_sin = None
    k32 = k.float()
    if rot is not None:
        rot = d // rot if rot < 16 else rot
        cos_sin = pa.rope_table(max(lens) + 3, rot, device="cpu")
        k32 = ref.rotate(k, pos, cos_sin, inter, torch.float32)
    want = pool.clone()
    ref.store(want, bt, seq, pos, k32, v.float(), dt)
    dev, w = pool.cuda(), wide.cuda()
    q_out = pa.append_kv4(
        w[:, hq:hq + hkv], w[:, hq + hkv:hq + 2 * hkv], dev, bt.cuda(), seq.cuda(), pos.cuda(),
        cos_sin=None if cos_sin is None else cos_sin.cuda(),
        q=w[:, :hq] if hq else None, interleaved=inter)
    torch.cuda.synchronize()
    assert pa.pa_last_device_error() == 0
    assert torch.equal(dev.cpu(), want)
    if hq:
        want_q = q if cos_sin is None else ref.rotate(q, pos, cos_sin, inter, torch.float32).to(dt)
        assert torch.equal(q_out.cpu(), want_q)
    # read them back: the values the bytes stand for, rounded once
    order = torch.randperm(n, generator=gen)
    rows = pa.read_kv4(dev, bt.cuda(), seq[order].cuda(), pos[order].cuda(), dtype=dt)
    page = bt[seq[order].long(), (pos[order] // 16).long()].long()
    slot = (pos[order] % 16).long()
    kk, vv, _ = ref.values(want, dt)
    assert torch.equal(rows[0].cpu(), kk[page, :, slot].float().to(dt))
    assert torch.equal(rows[1].cpu(), vv[page, :, slot].float().to(dt))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_append_special_rows(dtype):
    """Constant, zero, tiny, huge and non-finite rows, and ties between codes."""
    dt, d = DT[dtype], 128
    big = float(torch.finfo(dt).max)
    rows = torch.randn((12, 1, d), generator=torch.Generator().manual_seed(1))
    rows[0] = 0.0
    rows[1] = -3.25
    rows[2] *= 2.0 ** -20
    rows[3] = torch.where(rows[3] > 0, big, -big)
    rows[4, 0, 7] = math.inf
    rows[5, 0, 100] = -math.inf
    rows[6, 0, 0] = math.nan
    rows[7] = torch.arange(d) * 0.5                   # many exact halves
    rows[8] = torch.arange(d) % 16
    rows[9] = torch.finfo(dt).tiny * (torch.arange(d) % 3)
    rows[10] = 1000.0 + torch.arange(d) * 0.25
    rows = rows.to(dt)
    n = rows.shape[0]
    bt = torch.tensor([[0]], dtype=torch.int32)
    seq, pos = tokens_of([n])
    want = torch.zeros((1, 1, ref.block_bytes(d)), dtype=torch.uint8)
    ref.store(want, bt, seq, pos, rows.float(), rows.flip(0).float(), dt)
    dev = pa.kv4_cache(1, 1, d)
    pa.append_kv4(rows.cuda(), rows.flip(0).contiguous().cuda(), dev, bt.cuda(), seq.cuda(), pos.cuda())
    got = dev.cpu()
    assert torch.equal(got[..., :16 * d], want[..., :16 * d])
    a = got[..., 16 * d:].contiguous().view(dt).float()
    b = want[..., 16 * d:].contiguous().view(dt).float()
    assert torch.equal(torch.isnan(a), torch.isnan(b))
    assert torch.equal(a[~torch.isnan(a)], b[~torch.isnan(b)])
    # attention over a NaN row is NaN, without it finite
    q = torch.ones((1, 2, d), dtype=dt, device="cuda")
    assert torch.isnan(pa.decode_kv4(q, dev, bt.cuda(), i32(8), 1e-30)).all()
    assert torch.isnan(pa.prefill_kv4(q[:, None], dev, bt.cuda(), i32(7), 1e-30)).all()
    clean = pa.kv4_cache(1, 1, d)
    pa.append_kv4(rows[:3].cuda(), rows[:3].cuda(), clean, bt.cuda(), seq[:3].cuda(), pos[:3].cuda())
    assert torch.isfinite(pa.decode_kv4(q, clean, bt.cuda(), i32(3), 0.1)).all()


def test_bad_tokens_are_skipped_and_reported():
    d, hkv = 128, 2
    pool = torch.full((3, hkv, ref.block_bytes(d)), 7, dtype=torch.uint8, device="cuda")
    bt = torch.tensor([[0, 99], [1, -1]], dtype=torch.int32, device="cuda")
    x = torch.randn((6, hkv, d), device="cuda").bfloat16()
    # good, past the table, no such sequence, negative, bad page, unmapped
    seq, pos = i32(0, 0, 2, 0, 0, 1), i32(3, 32, 0, -1, 16, 17)
    out = torch.full((6, 4, d), 5.0, dtype=torch.bfloat16, device="cuda")
    q = torch.randn((6, 4, d), device="cuda").bfloat16()
    pa.append_kv4(x, x, pool, bt, seq, pos, q=q, q_out=out)
    assert pa.pa_last_device_error() in (-11, -14)
    assert torch.equal(out[0], q[0]) and (out[1:] == 5.0).all()
    touched = (pool != 7).flatten(1).any(1)
    assert touched.tolist() == [True, False, False]
    k, v = torch.full_like(x, 9.0), torch.full_like(x, 9.0)
    pa.read_kv4(pool, bt, seq, pos, k_out=k, v_out=v)
    assert pa.pa_last_device_error() in (-11, -14)
    assert (k[1:] == 9).all() and not (k[0] == 9).all()
    # positions beyond the rotation's table
    before = pool.clone()
    pa.append_kv4(x[:1], x[:1], pool, bt, seq[:1], pos[:1], cos_sin=pa.rope_table(2, 128))
    assert pa.pa_last_device_error() == -14
    assert torch.equal(pool, before)
    # attention: bad page ids and lengths are reported, nothing faults
    qd = torch.randn((2, 4, d), device="cuda").bfloat16()
    for n_new in (1, 24):
        qc = qd[:, None].expand(2, n_new, 4, d).contiguous()
        pa.decode_kv4(qd, pool, bt, i32(20, 3), 0.1)
        assert pa.pa_last_device_error() == -11
        pa.decode_kv4(qd, pool, bt, i32(16, 33), 0.1)
        assert pa.pa_last_device_error() in (-11, -12)
        pa.decode_kv4(qd, pool, bt, i32(16, -1), 0.1)
        assert pa.pa_last_device_error() == -12
        pa.prefill_kv4(qc, pool, bt, i32(32, 0), 0.1)
        assert pa.pa_last_device_error() in (-11, -12)
        pa.prefill_kv4(qc, pool, bt, i32(8, 0), 0.1)
        assert pa.pa_last_device_error() == (0 if n_new == 1 else -11)
        pa.prefill_kv4(qc, pool, bt, i32(-5, -2 ** 31), 0.1)
        assert pa.pa_last_device_error() in (-11, -12)
        pa.prefill_kv4(qc, pool, bt, i32(2 ** 31 - 1, 0), 0.1)
        assert pa.pa_last_device_error() in (-11, -12)


def test_copy_pages():
    pool = torch.randint(0, 256, (9, 3, ref.block_bytes(64)), device="cuda").to(torch.uint8)
    want = pool.clone()
    want[[4, 0]] = pool[[7, 2]]
    pa.copy_pages_kv4(pool, i32(7, 2), i32(4, 0))
    assert torch.equal(pool, want)
    pa.copy_pages_kv4(pool, i32(9, 1), i32(1, 8))
    want[8] = want[1]
    assert torch.equal(pool, want)
    assert pa.pa_last_device_error() == -11


def test_page_offsets_past_32_bits():
    """Pages whose byte offsets need more than 32 bits."""
    d, n = 128, 2_100_000  # 4.57 GB
    pool = torch.empty((n, 1, ref.block_bytes(d)), dtype=torch.uint8, device="cuda")
    pages = i32(n - 1, 5, 1_990_000)[None]
    small, sb = pa.kv4_cache(3, 1, d), i32(2, 0, 1)[None]
    x = torch.randn((40, 1, d), device="cuda").half()
    y = torch.randn((40, 1, d), device="cuda").half()
    q = torch.randn((1, 4, d), device="cuda").half()
    seq = torch.zeros(40, dtype=torch.int32, device="cuda")
    pos = torch.arange(40, dtype=torch.int32, device="cuda")
    outs = []
    for kv, bt in ((pool, pages), (small, sb)):
        pa.append_kv4(x, y, kv, bt, seq, pos)
        rows = pa.read_kv4(kv, bt, seq, pos, dtype=torch.float16)
        outs.append((rows[0], rows[1], pa.decode_kv4(q, kv, bt, i32(40), 0.1),
                     pa.prefill_kv4(q[:, None], kv, bt, i32(39), 0.1),
                     pa.prefill_kv4(q.expand(40, 4, d)[None].contiguous(), kv, bt, i32(0), 0.1)))
    assert pa.pa_last_device_error() == 0
    for a, b in zip(*outs):
        assert torch.equal(a, b)


def test_serving_run_together():
    """A prompt stored in 4 bits with rotation, then decode steps: append and
    attend, a fork whose shared page is copied first; every step against the
    definition on the bytes stored, and the bytes against the definition."""
    dt, hq, hkv, d = torch.bfloat16, 8, 2, 128
    gen = torch.Generator().manual_seed(11)
    pool = pa.kv4_cache(32, hkv, d)
    shadow = torch.zeros(pool.shape, dtype=torch.uint8)
    bt = torch.full((2, 8), -1, dtype=torch.int32)
    bt[0, :6] = torch.tensor([9, 3, 30, 1, 20, 7])
    cs = pa.rope_table(128, d)

    def step(seq, pos):
        qkv = torch.randn((len(seq), hq + 2 * hkv, d), generator=gen).to(dt)
        s, p = torch.tensor(seq, dtype=torch.int32), torch.tensor(pos, dtype=torch.int32)
        g = qkv.cuda()
        q = pa.append_kv4(g[:, hq:hq + hkv], g[:, hq + hkv:], pool, bt.cuda(), s.cuda(), p.cuda(),
                          cos_sin=cs, q=g[:, :hq])
        k32 = ref.rotate(qkv[:, hq:hq + hkv], p, cs.cpu(), False, torch.float32)
        ref.store(shadow, bt, s, p, k32, qkv[:, hq + hkv:].float(), dt)
        assert torch.equal(pool.cpu(), shadow)
        return q

    def attend(q, lens):
        got = pa.decode_kv4(q, pool, bt.cuda(), i32(*lens), 0.09)
        want, bound = ref.attention(q[:, None].cpu(), shadow, bt, [[t] for t in lens], 0.09, dt)
        assert ((got.cpu().double() - want[:, 0]).abs() <= bound[:, 0, :, None]).all()

    n = 45
    q = step([0] * n, list(range(n)))
    chunk = pa.prefill_kv4(q[None], pool, bt[:1].cuda(), i32(0), 0.09)
    want, bound = ref.attention(q[None].cpu(), shadow, bt, [[i + 1 for i in range(n)]], 0.09, dt)
    tol = bound[..., None] + 8 * 2.0 ** -8 + 2.0 ** -8 * want.abs()
    assert ((chunk.cpu().double() - want).abs() <= tol).all()
    # fork: sequence 1 shares pages 9 and 3, and gets a copy of the page it writes
    bt[1, :3] = torch.tensor([9, 3, 12])
    pa.copy_pages_kv4(pool, i32(30), i32(12))
    shadow[12] = shadow[30]
    for t in range(n, n + 3):
        attend(step([0, 1], [t, t]), [t + 1, t + 1])
    assert pa.pa_last_device_error() == 0


def test_streams_and_graphs():
    """On a stream of its own; captured once and replayed on new data, two graphs
    sharing a workspace; every replay like the eager call."""
    dt, gen = torch.bfloat16, torch.Generator().manual_seed(2)
    lens = [700, 33, 1, 250]
    pool, bt = make_pool(lens, 2, 128, dt, gen)
    pool, bt = pool.cuda(), bt.cuda()
    q = torch.randn((4, 8, 128), generator=gen).to(dt).cuda()
    qs = q.clone()
    ctx = i32(*lens)
    before = ctx - 1
    eager = pa.decode_kv4(q, pool, bt, ctx, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = pa.decode_kv4(q, pool, bt, ctx, 0.1, stream=side)
    by_handle = pa.decode_kv4(q, pool, bt, ctx, 0.1, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(other, eager) and torch.equal(by_handle, eager)
    ws = torch.empty(pa.pa_decode_kv4_workspace_size(128), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(eager) for _ in range(2)]
    chunk = torch.empty((4, 1, 8, 128), dtype=dt, device="cuda")
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    torch.cuda.synchronize()
    with torch.cuda.graph(graphs[0]):
        pa.decode_kv4(qs, pool, bt, ctx, 0.1, out=outs[0], workspace=ws)
    with torch.cuda.graph(graphs[1]):
        pa.prefill_kv4(qs[:, None], pool, bt, before, 0.1, out=chunk)
        pa.decode_kv4(qs, pool, bt, ctx, 0.2, out=outs[1], workspace=ws)
    for k in range(3):
        qs.copy_(q * (1 + k))
        graphs[k % 2].replay()
        graphs[(k + 1) % 2].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], pa.decode_kv4(qs, pool, bt, ctx, 0.1))
        assert torch.equal(outs[1], pa.decode_kv4(qs, pool, bt, ctx, 0.2))
        assert torch.equal(chunk, pa.prefill_kv4(qs[:, None], pool, bt, before, 0.1))
    assert pa.pa_last_device_error() == 0


def test_repeated_calls_are_bit_identical():
    gen = torch.Generator().manual_seed(4)
    pool, bt = make_pool([3000, 100, 2777], 4, 128, torch.bfloat16, gen)
    pool, bt = pool.cuda(), bt.cuda()
    q = torch.randn((3, 16, 128), generator=gen).bfloat16().cuda()
    ctx = i32(3000, 100, 2777)
    first = pa.decode_kv4(q, pool, bt, ctx, 0.1)
    for _ in range(20):
        assert torch.equal(pa.decode_kv4(q, pool, bt, ctx, 0.1), first)
    for n_new in (3, 10, 30, 80):  # of 4 rows a query
        qc = torch.randn((3, n_new, 16, 128), generator=gen).bfloat16().cuda()
        first = pa.prefill_kv4(qc, pool, bt, ctx - n_new, 0.1)
        for _ in range(10):
            assert torch.equal(pa.prefill_kv4(qc, pool, bt, ctx - n_new, 0.1), first)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_chunk_graphs_share_a_workspace(dtype):
    """Chunks of 6, 40 and 160 rows a kv head captured in graphs that share one
    workspace, replayed in turn on new queries: like the eager calls."""
    dt, gen = DT[dtype], torch.Generator().manual_seed(12)
    lens = [1500, 90, 200]
    pool, bt = make_pool(lens, 2, 128, dt, gen)
    pool, bt = pool.cuda(), bt.cuda()
    sizes = [3, 20, 80]
    ws = torch.empty(max(pa.pa_prefill_kv4_workspace_size(3, n, 4, 2, 128, 16, bt.shape[1])
                         for n in sizes), dtype=torch.uint8, device="cuda")
    qs = [torch.randn((3, n, 4, 128), generator=gen).to(dt).cuda() for n in sizes]
    ctx = [i32(*[t - n for t in lens]) for n in sizes]
    outs = [torch.empty_like(q) for q in qs]
    graphs = [torch.cuda.CUDAGraph() for _ in sizes]
    for q, c in zip(qs, ctx):
        pa.prefill_kv4(q, pool, bt, c, 0.1)
    torch.cuda.synchronize()
    for g, q, c, o in zip(graphs, qs, ctx, outs):
        with torch.cuda.graph(g):
            pa.prefill_kv4(q, pool, bt, c, 0.1, out=o, workspace=ws)
    for k in range(3):
        for q in qs:
            q.mul_(1.5)
        for g in graphs[k:] + graphs[:k]:
            g.replay()
        torch.cuda.synchronize()
        for q, c, o in zip(qs, ctx, outs):
            assert torch.isfinite(o).all()
            assert torch.equal(o, pa.prefill_kv4(q, pool, bt, c, 0.1))
    assert pa.pa_last_device_error() == 0
