"""Calls of the rotated appends and of the 4-bit cache with nothing to do: they return
empty results and write nothing, and their other arguments are still checked."""
import pytest
import torch

import paged_kv_cache_171_gb300 as pa

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_171_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert pa.pa_last_device_error() == 0


def _args(dtype=torch.bfloat16):
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    qkv = torch.empty((0, 12, 128), dtype=dtype, device="cuda")
    bt = torch.zeros((1, 2), dtype=torch.int32, device="cuda")
    return none, qkv[:, :8], qkv[:, 8:10], qkv[:, 10:], bt


def test_appends_of_no_token():
    none, q, k, v, bt = _args()
    kv = torch.full((2, 2, 2176), 7, dtype=torch.uint8, device="cuda")
    kc = torch.full((2, 2, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    cs = pa.rope_table(8, 64)
    assert pa.append_kv4(k, v, kv, bt, none, none) is None
    assert pa.append_kv4(k, v, kv, bt, none, none, cos_sin=cs, q=q).shape == (0, 8, 128)
    out = torch.empty((0, 8, 128), dtype=torch.bfloat16, device="cuda")
    assert pa.append_kv4(k, v, kv, bt, none, none, q=q, q_out=out) is out
    assert pa.append_kv_rope(k, v, kc, vc, bt, none, none, cs) is None
    assert pa.append_kv_rope(k, v, kc, vc, bt, none, none, cs, q=q).shape == (0, 8, 128)
    assert (kv == 7).all() and (kc == 7).all() and (vc == 7).all()
    with pytest.raises(pa.PAError) as e:
        pa.append_kv4(k, v, kv, bt, none, none, cos_sin=cs[:, :24].contiguous())
    assert "PA_ERR_ROPE" in str(e.value)
    assert pa.pa_last_device_error() == 0


def test_a_table_of_no_position_is_refused():
    """Not taken for a call without rotation."""
    _, _, _, _, bt = _args()
    x = torch.ones((1, 2, 128), dtype=torch.bfloat16, device="cuda")
    at = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv = pa.kv4_cache(2, 2, 128)
    kc = torch.zeros((2, 2, 16, 128), dtype=torch.bfloat16, device="cuda")
    none = torch.empty((0, 128), device="cuda")
    for call in (lambda: pa.append_kv4(x, x, kv, bt, at, at, cos_sin=none),
                 lambda: pa.append_kv_rope(x, x, kc, kc.clone(), bt, at, at, none)):
        with pytest.raises(pa.PAError) as e:
            call()
        assert "PA_ERR_ROPE" in str(e.value)
    assert (kv == 0).all() and (kc == 0).all()


def test_read_and_copy_of_nothing():
    none, _, _, _, bt = _args()
    kv = torch.full((2, 2, 2176), 7, dtype=torch.uint8, device="cuda")
    k, v = pa.read_kv4(kv, bt, none, none, dtype=torch.float16)
    assert k.shape == v.shape == (0, 2, 128) and k.dtype == torch.float16
    assert pa.copy_pages_kv4(kv, none, none) is None
    assert (kv == 7).all() and pa.pa_last_device_error() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_chunk_of_no_query(dtype):
    _, _, _, _, bt = _args()
    kv = pa.kv4_cache(2, 2, 128)
    ctx = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    q = torch.empty((1, 0, 8, 128), dtype=dtype, device="cuda")
    out = pa.prefill_kv4(q, kv, bt, ctx, 0.1)
    assert out.shape == (1, 0, 8, 128) and out.dtype == dtype
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    assert pa.prefill_kv4(q, kv, bt, ctx, 0.1, out=out, workspace=ws) is out
    with pytest.raises(pa.PAError):
        pa.prefill_kv4(q[:, :, :7].contiguous(), kv, bt, ctx, 0.1)  # 7 heads over 2
    assert pa.pa_last_device_error() == 0


def test_empty_calls_on_a_stream_and_in_a_graph():
    none, q, k, v, bt = _args()
    kv = pa.kv4_cache(2, 2, 128)
    side = torch.cuda.Stream()
    assert pa.append_kv4(k, v, kv, bt, none, none, q=q, stream=side).shape == (0, 8, 128)
    x = torch.randn((1, 2, 128), device="cuda").bfloat16()
    at = torch.zeros(1, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        pa.append_kv4(k, v, kv, bt, none, none)
        pa.append_kv4(x, x, kv, bt, at, at)
        pa.copy_pages_kv4(kv, none, none)
    graph.replay()
    torch.cuda.synchronize()
    want = pa.kv4_cache(2, 2, 128)
    pa.append_kv4(x, x, want, bt, at, at)
    assert torch.equal(kv, want) and pa.pa_last_device_error() == 0
