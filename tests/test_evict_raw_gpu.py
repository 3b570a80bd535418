"""The bindings of the C calls around eviction and trees, argument by argument, give what the
tensor forms give."""
import pytest
import torch

import paged_kv_cache_171_gb300 as pa
from tests.test_evict_flow_gpu import WRITTEN, _built, _loop, _results  # noqa: F401

pytestmark = pytest.mark.gpu


def test_the_loop_by_its_c_calls():
    a, step = _loop(31)
    step()
    want = _results(a)
    s, _ = _loop(31)
    (pages, hkv, P, d), (B, n, hq, _), mb = s["k"].shape, s["qs"].shape, s["bt"].shape[1]
    heads, table = (hq, hkv, d, P), (B, mb, pages, pa.BF16)
    ws, size = s["ws"], s["ws"].nbytes
    assert 0 < pa.pa_decode_weighted_workspace_size(B, *heads, mb) <= size
    pa.pa_decode_weighted(s["q"], s["k"], s["v"], s["w"], s["bt"], s["ctx"], s["out"], 0.1, 1,
                          *heads, *table, ws, size)
    pa.pa_tree_mask(s["parents"], s["mask"], s["depth"], B, n)
    assert 0 <= pa.pa_prefill_tree_workspace_size(B, n, *heads, mb) <= size
    pa.pa_prefill_tree(s["qs"], s["k"], s["v"], s["bt"], s["ctx"], s["mask"], n, s["tree"], 0.1,
                       *heads, *table, ws, size)
    pa.pa_compact_kv(s["k"], s["v"], s["w"], s["bt"], s["ctx"], s["keep"], s["n_keep"], 3, s["now"],
                     hkv, d, P, *table)
    assert 0 < pa.pa_prefill_weights_workspace_size(B, n, *heads, mb) <= size
    pa.pa_prefill_weights(s["qs"], s["k"], s["w"], s["bt"], s["ctx"], n, 0.1, n, n * hq * d, hq * d,
                          *heads, *table, ws, size)
    assert 0 < pa.pa_evict_kv_workspace_size(B, hkv, d, P, mb, 600) <= size
    pa.pa_evict_kv(s["k"], s["v"], s["w"], s["bt"], s["now"], s["bt"], s["less"], 600, 4, 100, hkv,
                   d, P, B, mb, mb, pages, pa.BF16, ws, size)
    assert pa.pa_last_device_error() == 0
    for x, y, name in zip(_results(s), want, WRITTEN):
        assert torch.equal(x, y), name


def test_the_append_at_other_positions():
    d, n, hq, hkv = 64, 5, 4, 2
    gen = torch.Generator(device="cuda").manual_seed(1)
    w = torch.randn((n, hq + 2 * hkv, d), generator=gen, device="cuda").bfloat16()
    bt = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    seq = torch.zeros(n, dtype=torch.int32, device="cuda")
    pos = torch.arange(14, 14 + n, dtype=torch.int32, device="cuda")
    at = torch.tensor([3, 4, 4, 5, 9], dtype=torch.int32, device="cuda")
    cs = pa.rope_table(16, d)
    k, v = w[:, hq:hq + hkv], w[:, hq + hkv:]
    caches = [torch.zeros((2, hkv, 16, d), dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    want = pa.append_kv_rope(k, v, *caches[:2], bt, seq, pos, cs, q=w[:, :hq], rope_pos=at)
    q = torch.empty((n, hq, d), dtype=torch.bfloat16, device="cuda")
    row = (hq + 2 * hkv) * d
    pa.pa_append_kv_rope_at(k, v, w, *caches[2:], q, bt, seq, pos, at, cs, n, row, row, row, hq,
                            hkv, d, 16, 1, 2, 2, 16, d, False, pa.BF16)
    assert pa.pa_last_device_error() == 0
    assert torch.equal(q, want)
    assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
