"""The 4-bit cache's attention where weights, rows and queries span a wide range: a key
that takes nearly all of the weight, rows far larger than their neighbours, very large
and very small queries, runs that a worker walks over many windows of page ids.  Every
row is checked by itself against the definition in 64 bits.

The sequences of a call share one set of pages, so that each has a long run of its own
on the GPU without a large cache."""
import math

import pytest
import torch

import paged_kv_cache_171_gb300 as pa
from tests import kv4_reference as ref

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
U = 2.0 ** -11  # half a step of fp16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_171_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert pa.pa_last_device_error() == 0


def randn(*shape, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=gen, device="cuda")


def stored(k, v, dt):
    """One sequence's rows k, v [n, Hkv, D] in a cache of shuffled pages: the cache and
    the block table [1, blocks]."""
    n, hkv, d = k.shape
    blocks = -(-n // 16)
    gen = torch.Generator(device="cuda").manual_seed(n)
    bt = torch.randperm(blocks + 1, generator=gen, device="cuda")[:blocks].to(torch.int32)[None]
    pool = torch.zeros((blocks + 1, hkv, ref.block_bytes(d)), dtype=torch.uint8, device="cuda")
    pos = torch.arange(n, device="cuda")
    ref.store(pool, bt, torch.zeros_like(pos), pos, k, v, dt)
    return pool, bt.contiguous()


def attend(q, pool, bt, seen, scale, dt):
    """softmax(q K^T scale) V in 64 bits, q [nq, Hq, D], query i over seen[i] keys; and
    R = sqrt(sum p^2 |v|^2) a row: what independent relative errors of the terms p v add
    up to, a unit of error each."""
    nq, hq, d = q.shape
    k, v, _ = ref.values(pool[bt[0].long()], dt)
    k = k.transpose(0, 1).reshape(pool.shape[1], -1, d)[:, :max(seen)]
    v = v.transpose(0, 1).reshape(pool.shape[1], -1, d)[:, :max(seen)]
    out, r = torch.empty(q.shape, dtype=torch.float64, device="cuda"), torch.empty(nq, hq, device="cuda")
    group = hq // pool.shape[1]
    late = torch.arange(max(seen), device="cuda")[None, :] >= torch.tensor(seen, device="cuda")[:, None]
    for h in range(hq):
        s = (q[:, h].double() @ k[h // group].T * scale).masked_fill_(late, -math.inf)
        p = s.softmax(-1)
        out[:, h] = p @ v[h // group]
        r[:, h] = (p.square() @ v[h // group].square().sum(-1)).sqrt()
    return out, r


def assert_rows(got, want, r, dt):
    """A chunk's rows [nq, Hq, D] against `attend`'s.  A row's error, in the norm: half a step
    of the result's type of the row; and, a key, the roundings of its terms, each at most U =
    2^-11 relatively: of the weight, and in bf16 of V, twice, the second time of its row's
    least value, up to 3 times a typical one.  (Scores are good to fp32's last bits.)
    Independent ones add up to sqrt(1 + 1 + 9) U R / sqrt(3) < 2 U R, for fp16 U R / sqrt(3);
    3 and 2.5 times that are allowed.  An element below the type's normal range is off by up
    to half a step there, smallest_normal eps / 2, whatever its size: sqrt(D) of them."""
    half, most = torch.finfo(dt).eps / 2, (6 if dt is torch.bfloat16 else 1.5) * U
    err, size = (got.double() - want).norm(dim=-1), want.norm(dim=-1)
    tol = half * (size + math.sqrt(want.shape[-1]) * torch.finfo(dt).smallest_normal) + most * r
    assert (err <= tol).all(), (float((err / size).max()), float((err / tol).max()))


def check_chunk(q, pool, bt, ctx, scale, dt, look):
    """q [B, n_new, Hq, D] over the one sequence of `bt`, in B sequences; those of `look`
    are compared."""
    B, n_new, hq, d = q.shape
    tokens = torch.full((B,), ctx, dtype=torch.int32, device="cuda")
    got = pa.prefill_kv4(q, pool, bt.expand(B, -1).contiguous(), tokens, scale)
    assert pa.pa_last_device_error() == 0
    for b in look:
        want, r = attend(q[b], pool, bt, [ctx + i + 1 for i in range(n_new)], scale, dt)
        assert_rows(got[b], want, r, dt)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n_new,hq,d,keys", [
    (7, 4, 128, 131072), (40, 4, 128, 32768), (14, 4, 64, 32768), (300, 1, 64, 16384)])
def test_chunk_over_a_long_run(n_new, hq, d, keys, dtype):
    """One item a CTA: the sums of a whole context in one accumulator.  28, 56, 160 and 300
    rows a kv head."""
    dt = DT[dtype]
    pool, bt = stored(randn(keys, 1, d, seed=1), randn(keys, 1, d, seed=2), dt)
    q = randn(152, n_new, hq, d, seed=3).to(dt)
    check_chunk(q, pool, bt, keys - n_new, 1 / math.sqrt(d), dt, (0, 77, 151))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,d,keys", [(4, 128, 32768), (8, 128, 131072), (3, 64, 131072)])
def test_decode_over_a_long_run(hq, d, keys, dtype):
    """One item a team of warps.  A score is off by at most 8 roundings of a partial sum, 4 in
    powers of two (2.6e-6 of a weight), a weight's two terms and its exponential by 2^-21, and
    the sums, a few times the result, by as much as a plain fp32 evaluation's (1e-6)."""
    dt, scale = DT[dtype], 1 / math.sqrt(d)
    pool, bt = stored(randn(keys, 1, d, seed=1), randn(keys, 1, d, seed=2), dt)
    q = randn(608, hq, d, seed=3).to(dt)
    tokens = torch.full((608,), keys, dtype=torch.int32, device="cuda")
    got = pa.decode_kv4(q, pool, bt.expand(608, -1).contiguous(), tokens, scale)
    assert pa.pa_last_device_error() == 0
    for b in (0, 300, 607):
        want, _ = attend(q[b:b + 1], pool, bt, [keys], scale, dt)
        err = (got[b].double() - want[0]).norm(dim=-1) / want[0].norm(dim=-1)
        assert err.max() <= 5e-6, (b, float(err.max()))


def sink_case(keys, weight, at, d, dt, shape, seed):
    """Keys of N(0, 1) scores and values, and one, whose value is 0, that takes `weight` of
    every query's softmax: along dimension 0 of q, where the others are 0."""
    scale = 1 / math.sqrt(d)
    k, v = randn(keys, 1, d, seed=seed), randn(keys, 1, d, seed=seed + 1)
    k[:, :, 0] = 0
    v[at] = 0
    k[at] = 0
    k[at, :, 0] = math.log(weight / (1 - weight) * keys * math.exp(0.5)) / (8 * scale)
    q = randn(*shape, d, seed=seed + 2)
    q[..., 0] = 8
    pool, bt = stored(k, v, dt)
    return q.to(dt), pool, bt, scale


# one item a CTA at least, so that a run holds the sink and many other keys; 28, 56 and
# 160 rows a kv head: one row tile, the same, and two
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n_new,hq,d,keys,weight,at", [
    (7, 4, 128, 32768, 0.99, 0), (7, 4, 128, 32768, 0.999, 9000), (14, 4, 64, 131072, 0.99, 0),
    (7, 4, 128, 131072, 0.999, 0), (40, 4, 128, 32768, 0.999, 0), (40, 4, 64, 8192, 0.99, 5000),
    (300, 1, 128, 32768, 0.99, 3)])
def test_chunk_below_a_sink(n_new, hq, d, keys, weight, at, dtype):
    dt = DT[dtype]
    q, pool, bt, scale = sink_case(keys, weight, at, d, dt, (152, n_new, hq), seed=n_new)
    check_chunk(q, pool, bt, keys - n_new, scale, dt, (0, 77, 151))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,d,keys,weight,at", [
    (4, 128, 32768, 0.99, 0), (8, 128, 32768, 0.99, 7000), (3, 64, 131072, 0.99, 0),
    (8, 64, 131072, 0.999, 0), (1, 128, 32768, 0.999, 5), (12, 128, 32768, 0.999, 20000)])
def test_decode_below_a_sink(hq, d, keys, weight, at, dtype):
    """One item a team of warps.  Scores whose terms add up to at most 16 in powers of two
    are off by at most 12 roundings of 2^-23 of that, 1.6e-5 of a weight; a weight's two
    terms and its exponential by 2^-21; the sums of a row, whose middles add up to some 60
    times the result while it cancels, by about that times 2^-23 (7e-6): 2.4e-5 in all."""
    dt = DT[dtype]
    q, pool, bt, scale = sink_case(keys, weight, at, d, dt, (608, hq), seed=hq)
    tokens = torch.full((608,), keys, dtype=torch.int32, device="cuda")
    got = pa.decode_kv4(q, pool, bt.expand(608, -1).contiguous(), tokens, scale)
    assert pa.pa_last_device_error() == 0
    for b in (0, 300, 607):
        want, _ = attend(q[b:b + 1], pool, bt, [keys], scale, dt)
        err = (got[b].double() - want[0]).norm(dim=-1) / want[0].norm(dim=-1)
        assert err.max() <= 2.4e-5, (b, float(err.max()))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n_new,hq,d,keys,weight", [
    (2, 4, 128, 131072, 0.99), (1, 1, 64, 131072, 0.999), (3, 5, 128, 65536, 0.999)])
def test_short_chunk_below_a_sink(n_new, hq, d, keys, weight, dtype):
    """Up to 16 rows a kv head, which take the decode's kernel."""
    dt = DT[dtype]
    q, pool, bt, scale = sink_case(keys, weight, 11, d, dt, (608, n_new, hq), seed=n_new)
    check_chunk(q, pool, bt, keys - n_new, scale, dt, (0, 300, 607))


@pytest.mark.parametrize("n_new,hq,d,keys,every", [
    (7, 4, 128, 1000, 32), (14, 4, 64, 5000, 32), (40, 4, 128, 3000, 500), (160, 2, 64, 700, 32),
    (2, 4, 128, 1000, 32)])
@pytest.mark.parametrize("dtype,what,factor", [
    ("bf16", "kv", 64), ("bf16", "kv", 1024), ("bf16", "kv", 8192), ("bf16", "k", 2 ** 20),
    ("bf16", "v", 4096), ("fp16", "kv", 1024), ("fp16", "kv", 8192)])
def test_chunk_beside_rows_far_larger(n_new, hq, d, keys, every, dtype, what, factor):
    """Rows `factor` times the others, of no weight (every query's score for them is far below
    the others): their neighbours keep their digits.  The last is a token of the chunk that no
    query but the last one sees.  28, 56, 160 and 320 rows a kv head, and 8, which take the
    decode's kernel."""
    dt, scale = DT[dtype], 1 / math.sqrt(d)
    k, v = randn(keys, 1, d, seed=1), randn(keys, 1, d, seed=2)
    k[..., 0] = 0
    big = torch.arange(5, keys, every, device="cuda")
    big = torch.cat((big, torch.tensor([keys - 1], device="cuda")))
    # q . k = -8 f + 0.1 f N(0, D), f = `factor`, or 64 where only the values are larger
    f = factor if "k" in what else 64
    k[big] = k[big] * 0.1 * f
    k[big, :, 0] = -f
    if "v" in what:
        v[big] *= factor
    pool, bt = stored(k, v, dt)
    q = randn(2, n_new, hq, d, seed=3)
    q[..., 0] = 8
    check_chunk(q.to(dt), pool, bt, keys - n_new, scale, dt, (0, 1))


@pytest.mark.parametrize("n_new,hq,d,keys", [(7, 4, 128, 2000), (40, 4, 64, 3000)])
@pytest.mark.parametrize("dtype,by", [("bf16", 2.0 ** -e) for e in (4, 5, 6, 7, 12, 30)] +
                         [("fp16", 2.0 ** -12)])
def test_chunk_beside_rows_far_smaller(n_new, hq, d, keys, dtype, by):
    """One key and value in 32 much smaller than the others, which keep their digits."""
    dt = DT[dtype]
    k, v = randn(keys, 1, d, seed=1), randn(keys, 1, d, seed=2)
    k[7::32] *= by
    v[7::32] *= by
    pool, bt = stored(k, v, dt)
    q = randn(2, n_new, hq, d, seed=3).to(dt)
    check_chunk(q, pool, bt, keys - n_new, 1 / math.sqrt(d), dt, (0, 1))


@pytest.mark.parametrize("q_mul,k_mul,scale", [
    (1e34, 1e-33, 0.01), (1e36, 1e-30, 1e-7), (1e-36, 1e33, 100.0), (1e-38, 1e30, 1e7)])
@pytest.mark.parametrize("n_new,hq", [(0, 4), (0, 8), (2, 4), (7, 4), (60, 4)])
def test_queries_near_the_ends_of_the_range(n_new, hq, q_mul, k_mul, scale):
    """Products of bf16 queries and keys far outside fp16's range, of ordinary scores: decode
    (n_new = 0), 8, 28 and 240 rows a kv head."""
    dt, d, keys = torch.bfloat16, 128, 500
    pool, bt = stored(randn(keys, 1, d, seed=1) * k_mul, randn(keys, 1, d, seed=2), dt)
    q = (randn(2, max(n_new, 1), hq, d, seed=3) * q_mul).to(dt)
    if n_new:
        check_chunk(q, pool, bt, keys - n_new, scale, dt, (0, 1))
        return
    got = pa.decode_kv4(q[:, 0].contiguous(), pool, bt.expand(2, -1).contiguous(),
                        torch.full((2,), keys, dtype=torch.int32, device="cuda"), scale)
    for b in (0, 1):
        want, _ = attend(q[b], pool, bt, [keys], scale, dt)
        # 12 roundings of 2^-23 of a score whose terms add up to at most 200 in powers of two
        err = (got[b].double() - want[0]).norm(dim=-1) / want[0].norm(dim=-1)
        assert err.max() <= 12 * 200 * 2.0 ** -23, float(err.max())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("hq,hkv,n_new,ctx,d", [
    (8, 2, 4, [0, 15, 16, 1000], 128), (8, 2, 7, [100, 0], 128), (4, 4, 17, [3, 200], 64),
    (7, 1, 5, [129, 1, 127], 128), (12, 4, 33, [0, 31], 64), (24, 1, 2, [77, 500], 128),
    (8, 1, 130, [0, 260], 128), (32, 8, 64, [500], 64), (7, 1, 150, [0, 127, 128], 128),
    (2, 2, 257, [0, 1000], 64), (16, 4, 6, [5000, 0, 130, 9000, 64, 2, 127, 128] + [40] * 60, 128),
    (16, 4, 70, [3000, 0, 130, 1, 6000], 128), (16, 4, 20, [20000, 3], 64)])
def test_every_row_of_a_chunk(hq, hkv, n_new, ctx, d, dtype):
    """Head layouts, ragged batches and items cut between runs, row by row."""
    dt, scale = DT[dtype], 1 / math.sqrt(d)
    lens = [t + n_new for t in ctx]
    blocks = [-(-t // 16) for t in lens]
    gen = torch.Generator(device="cuda").manual_seed(n_new)
    perm = torch.randperm(sum(blocks) + 2, generator=gen, device="cuda").to(torch.int32)
    bt = torch.full((len(lens), max(blocks)), -1, dtype=torch.int32, device="cuda")
    for b, n in enumerate(blocks):
        bt[b, :n] = perm[sum(blocks[:b]):sum(blocks[:b]) + n]
    # what no token has written: any codes, NaN scales and zeros
    pool = torch.randint(0, 256, (sum(blocks) + 2, hkv, ref.block_bytes(d)), generator=gen,
                         device="cuda").to(torch.uint8)
    pool[:, :, 16 * d:] = 255
    seq = torch.cat([torch.full((t,), b, device="cuda") for b, t in enumerate(lens)])
    pos = torch.cat([torch.arange(t, device="cuda") for t in lens])
    ref.store(pool, bt, seq, pos, randn(len(pos), hkv, d, seed=1), randn(len(pos), hkv, d, seed=2), dt)
    q = randn(len(lens), n_new, hq, d, seed=3).to(dt)
    got = pa.prefill_kv4(q, pool, bt, torch.tensor(ctx, dtype=torch.int32, device="cuda"), scale)
    assert pa.pa_last_device_error() == 0
    for b, t in enumerate(ctx):
        seen = [t + i + 1 for i in range(n_new)]
        want, r = attend(q[b], pool, bt[b:b + 1, :blocks[b]], seen, scale, dt)
        assert_rows(got[b], want, r, dt)


@pytest.mark.parametrize("n_new", [7, 40, 100])
def test_rows_that_are_not_finite_beside_far_larger_ones(n_new):
    """A NaN row of the chunk among 32 keys that span a wide range: the queries before it are
    as without it, the others NaN."""
    dt, d, ctx, at = torch.bfloat16, 128, 60, 3
    k, v = randn(ctx + n_new, 1, d, seed=1), randn(ctx + n_new, 1, d, seed=2)
    k[50] *= 2000
    v[40] *= 3e4
    v[52] = 0
    pool, bt = stored(k, v, dt)
    q = randn(1, n_new, 4, d, seed=3).to(dt)
    tokens = torch.full((1,), ctx, dtype=torch.int32, device="cuda")
    clean = pa.prefill_kv4(q, pool, bt, tokens, 0.09)
    assert torch.isfinite(clean).all()
    page, slot = int(bt[0, (ctx + at) // 16]), (ctx + at) % 16
    for which in (0, 1):
        bad = pool.clone()
        bad[page, 0, 16 * d + (which * 16 + slot) * 4:][:4] = 255  # NaN scale and zero
        got = pa.prefill_kv4(q, bad, bt, tokens, 0.09)
        assert torch.equal(got[:, :at], clean[:, :at])
        assert torch.isnan(got[:, at:]).all()
    assert pa.pa_last_device_error() == 0


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n_new,hq,d", [(2, 4, 128), (12, 4, 128), (64, 4, 64), (64, 4, 128),
                                        (300, 1, 128)])
@pytest.mark.parametrize("q_mul,spread", [(10, 0), (40, 0), (1, 1)])
def test_chunk_of_large_scores(q_mul, spread, n_new, hq, d, dtype):
    """Scores of N(0, 10) and N(0, 40), and rows whose sizes are spread by e^N(0, 1) (K) and
    e^N(0, 2) (V): few keys share the weight, and an error in a score is one of the row."""
    dt, keys = DT[dtype], 3000
    k, v = randn(keys, 1, d, seed=1), randn(keys, 1, d, seed=2)
    k *= torch.exp(spread * randn(keys, 1, 1, seed=5))
    v *= torch.exp(2 * spread * randn(keys, 1, 1, seed=6))
    pool, bt = stored(k, v, dt)
    q = (randn(2, n_new, hq, d, seed=3) * q_mul).to(dt)
    check_chunk(q, pool, bt, keys - n_new, 1 / math.sqrt(d), dt, (0, 1))
