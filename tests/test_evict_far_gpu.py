"""Weighted decode, prompt weights, eviction, compaction and trees where offsets pass 32 bits,
and queries laid out token by token."""
import pytest
import torch

import paged_kv_cache_171_gb300 as pa
from tests import evict_reference as ref
from tests.test_evict_flow_gpu import WRITTEN, _built, _loop, _results  # noqa: F401

pytestmark = pytest.mark.gpu


def test_pages_at_the_far_end_of_a_large_pool():
    """The loop's step over the last pages of pools of 2^32 and more values, bit for bit that of
    a small pool."""
    near, step = _loop(21)
    far, far_step = _loop(21)
    small = near["k"].shape[0]
    many = (1 << 32) // near["k"][0].numel() + small
    for x in ("k", "v", "w"):
        big = torch.empty((many,) + near[x].shape[1:], dtype=near[x].dtype, device="cuda")
        big[many - small:] = near[x]
        far[x] = big
    far["bt"] = torch.where(near["bt"] >= 0, near["bt"] + (many - small), near["bt"])
    step()
    far_step()
    assert pa.pa_last_device_error() == 0
    for x in WRITTEN:
        got = far[x][many - small:] if x in ("k", "v", "w") else far[x]
        assert torch.equal(got, near[x]), x


def test_a_table_of_more_scores_than_32_bits_count():
    near, _ = _loop(22)
    far, _ = _loop(22)
    blocks = 8 << 20  # 24 rows x 2^27 tokens
    far["bt"] = torch.full((3, blocks), -1, dtype=torch.int32, device="cuda")
    far["bt"][:, :near["bt"].shape[1]] = near["bt"]
    a, b = (pa.decode_weighted(s["q"], s["k"], s["v"], s["w"], s["bt"], s["ctx"], 0.1)
            for s in (near, far))
    assert pa.pa_last_device_error() == 0
    assert torch.equal(a, b) and torch.equal(near["w"], far["w"])


def test_queries_token_by_token():
    """q [n][B][heads][D] seen as [B, n, heads, D]: a batch stride smaller than a token's."""
    a, _ = _loop(23)
    b, _ = _loop(23)
    pa.prefill_weights(a["qs"], a["k"], a["w"], a["bt"], a["ctx"], 0.1)
    q = b["qs"].transpose(0, 1).contiguous().transpose(0, 1)
    assert q.stride(0) < q.stride(1)
    pa.prefill_weights(q, b["k"], b["w"], b["bt"], b["ctx"], 0.1)
    assert pa.pa_last_device_error() == 0
    assert torch.equal(a["w"], b["w"])


def test_one_query_for_a_whole_batch_is_refused():
    s, _ = _loop(24)
    w = s["w"].clone()
    with pytest.raises(pa.PAError):
        pa.prefill_weights(s["qs"][:1].expand(3, -1, -1, -1), s["k"], s["w"], s["bt"], s["ctx"], 0.1)
    assert torch.equal(s["w"], w)


@pytest.mark.parametrize("n", [1, 4, 16, 24, 32, 40, 64])
def test_few_queries_over_many_key_tiles(n):
    """One to four row tiles (8 n rows) beside which every CTA has some twenty key tiles, so that
    each of its buffers goes round several times; twice, with the same bits."""
    lens = [20000, 18901]
    dt = torch.bfloat16
    k, _, w, bt, _ = ref.pool([t + n for t in lens], 8, 64, dt, n)
    ctx = torch.tensor(lens, dtype=torch.int32)
    q = torch.randn((2, n, 64, 64), generator=torch.Generator().manual_seed(n + 1)).to(dt)
    got = []
    for _ in range(2):
        gw = w.cuda()
        pa.prefill_weights(q.cuda(), k.cuda(), gw, bt.cuda(), ctx.cuda(), 0.2)
        got.append(gw.cpu())
    assert pa.pa_last_device_error() == 0
    new, bound = ref.chunk_weights(q, k, w, bt, ctx, 0.2, n)
    assert ((got[0].double() - new).abs() <= bound).all()
    assert torch.equal(*got)
