"""Arguments that the rotated appends and the 4-bit cache refuse, on the host before
any CUDA call, and the sizes they report."""
import ctypes

import pytest
import torch

import paged_kv_cache_171_gb300 as pa
from paged_kv_cache_171_gb300 import build as pa_build
from tests import kv4_reference as ref

FAKE = 0x1000  # 16-byte aligned, never dereferenced on these paths


@pytest.fixture(scope="module")
def L():
    pa_build.build()
    return pa.lib()


def _rope(L, **kw):
    a = dict(k=FAKE, v=FAKE, q=FAKE, kc=FAKE, vc=FAKE, qo=FAKE, bt=FAKE, seq=FAKE, pos=FAKE,
             cs=FAKE, n=0, ks=1024, vs=1024, qs=4096, hq=32, hkv=8, d=128, p=16, b=2, mb=8,
             pages=16, mp=100, rot=128, it=0, dt=0)
    a.update(kw)
    return L.pa_append_kv_rope(*a.values(), None)


def _kv4(L, **kw):
    a = dict(k=FAKE, v=FAKE, q=FAKE, kc=FAKE, qo=FAKE, bt=FAKE, seq=FAKE, pos=FAKE,
             cs=FAKE, n=0, ks=1024, vs=1024, qs=4096, hq=32, hkv=8, d=128, p=16, b=2, mb=8,
             pages=16, mp=100, rot=128, it=0, dt=0)
    a.update(kw)
    return L.pa_append_kv4(*a.values(), None)


COMMON = [
    (dict(k=None), -1), (dict(v=None), -1), (dict(kc=None), -1), (dict(bt=None), -1),
    (dict(seq=None), -1), (dict(pos=None), -1), (dict(qo=None), -1), (dict(q=None), -1),
    (dict(hq=30), -2), (dict(hkv=0), -2), (dict(d=96), -3), (dict(d=256), -3), (dict(p=32), -4),
    (dict(n=-1), -5), (dict(b=0), -5), (dict(mb=0), -5), (dict(pages=0), -5), (dict(b=70000), -5),
    (dict(ks=1000), -5), (dict(vs=0), -5), (dict(qs=-4096), -5), (dict(qs=4088), -5),
    (dict(dt=2), -6), (dict(ks=1025), -8), (dict(vs=1028), -8), (dict(qs=4100), -8),
    (dict(k=FAKE + 8), -8), (dict(q=FAKE + 2), -8), (dict(qo=FAKE + 4), -8),
    (dict(kc=FAKE + 8), -8), (dict(cs=FAKE + 4), -8),
    (dict(rot=0), -18), (dict(rot=24), -18), (dict(rot=144), -18), (dict(rot=-16), -18),
    (dict(mp=0), -18),
    (dict(), 0), (dict(rot=16), 0), (dict(rot=48), 0), (dict(it=1), 0),
    (dict(q=None, qo=None, hq=0, qs=0), 0), (dict(ks=6144, vs=6144, qs=6144), 0),
]


@pytest.mark.parametrize("kw,code", COMMON)
def test_appends_refuse(L, kw, code):
    assert _rope(L, **kw) == code
    assert _kv4(L, **kw) == code


def test_rotation_is_required_or_optional(L):
    assert _rope(L, cs=None) == -1
    assert _rope(L, vc=None) == -1
    assert _kv4(L, cs=None) == 0
    assert _kv4(L, cs=None, rot=7, mp=-3) == 0  # not used


def test_read_and_copy_refuse(L):
    P = FAKE
    ok = [P, P, P, P, P, P, 0, 8, 128, 16, 2, 8, 16, 0, None]
    assert L.pa_read_kv4(*ok) == 0
    for at, value, code in [(0, None, -1), (3, None, -1), (5, None, -1), (6, -1, -5), (7, 0, -2),
                            (8, 80, -3), (9, 8, -4), (10, 0, -5), (13, 5, -6), (4, P + 4, -8),
                            (0, P + 8, -8)]:
        bad = list(ok)
        bad[at] = value
        assert L.pa_read_kv4(*bad) == code, (at, value)
    ok = [P, P, P, 0, 8, 128, 16, 16, None]
    assert L.pa_copy_pages_kv4(*ok) == 0
    for at, value, code in [(0, None, -1), (1, None, -1), (3, -1, -5), (4, 0, -2), (5, 80, -3),
                            (6, 8, -4), (7, 0, -5), (0, P + 8, -8)]:
        bad = list(ok)
        bad[at] = value
        assert L.pa_copy_pages_kv4(*bad) == code, (at, value)


def test_attention_refuses(L):
    P, f = FAKE, ctypes.c_float(0.1)
    need = L.pa_decode_kv4_workspace_size(128)
    ok = [P, P, P, P, P, f, 32, 8, 128, 16, 2, 8, 16, 0, P, need, None]
    cases = [(0, None, -1), (1, None, -1), (4, None, -1), (6, 30, -2), (8, 96, -3), (9, 8, -4),
             (10, 0, -5), (11, 0, -5), (12, 0, -5), (13, 2, -6), (0, P + 8, -8), (1, P + 2, -8),
             (4, P + 4, -8), (14, None, -7), (15, need - 1, -7), (14, P + 8, -8)]
    for at, value, code in cases:
        bad = list(ok)
        bad[at] = value
        assert L.pa_decode_kv4(*bad) == code, (at, value)
    need = L.pa_prefill_kv4_workspace_size(2, 4, 32, 8, 128, 16, 8)
    ok = [P, P, P, P, 4, P, f, 32, 8, 128, 16, 2, 8, 16, 0, P, need, None]
    cases = [(0, None, -1), (5, None, -1), (4, -1, -5), (4, 129, -5), (7, 30, -2), (9, 96, -3),
             (10, 8, -4), (11, 0, -5), (14, 2, -6), (0, P + 8, -8), (5, P + 4, -8),
             (15, None, -7), (16, need - 1, -7)]
    for at, value, code in cases:
        bad = list(ok)
        bad[at] = value
        assert L.pa_prefill_kv4(*bad) == code, (at, value)
    ok[4] = 0  # an empty chunk: nothing to do, the rest still checked
    assert L.pa_prefill_kv4(*ok) == 0
    ok[9] = 96
    assert L.pa_prefill_kv4(*ok) == -3


def test_sizes_past_32_bits_are_refused(L):
    P, f, big = FAKE, ctypes.c_float(0.1), 1 << 40
    chunk = lambda n, hq, hkv, blocks: L.pa_prefill_kv4(
        P, P, P, P, n, P, f, hq, hkv, 128, 16, 2, blocks, 16, 0, P, big, None)
    assert chunk(1, 65536, 65536, 8) == -2 and chunk(1, 131072, 8, 8) == -2
    assert chunk(1 << 20, 32768, 1, 1 << 20) == -5    # 2^35 rows
    assert chunk(1 << 24, 32, 8, 1 << 22) == -5       # 2^18 x 2^19 tiles
    assert L.pa_prefill_kv4_workspace_size(2, 1 << 24, 32, 8, 128, 16, 1 << 22) == 0
    assert L.pa_prefill_kv4_workspace_size(2, 1 << 17, 64, 8, 128, 16, 1 << 13) > 0
    assert L.pa_decode_kv4(P, P, P, P, P, f, 65536, 8, 128, 16, 2, 8, 16, 0, P, big, None) == -2
    assert L.pa_read_kv4(P, P, P, P, P, P, 4, 65536, 128, 16, 2, 8, 16, 0, None) == -2
    assert L.pa_copy_pages_kv4(P, P, P, 4, 65536, 128, 16, 16, None) == -2


def test_sizes(L):
    assert [L.pa_kv4_block_bytes(d) for d in (64, 128, 96, 0)] == [1152, 2176, 0, 0]
    assert ref.block_bytes(64) == 1152 and ref.block_bytes(128) == 2176
    assert L.pa_decode_kv4_workspace_size(96) == 0
    assert L.pa_decode_kv4_workspace_size(128) > L.pa_decode_kv4_workspace_size(64) > 0
    assert L.pa_prefill_kv4_workspace_size(2, 0, 32, 8, 128, 16, 8) == 0
    assert L.pa_prefill_kv4_workspace_size(2, 129, 32, 8, 128, 16, 8) == 0
    assert L.pa_prefill_kv4_workspace_size(2, 4, 32, 7, 128, 16, 8) == 0


def test_status_has_a_name(L):
    assert "PA_ERR_ROPE" in pa.pa_strerror(-18)


def test_tensor_forms_refuse_what_they_cannot_pass_on():
    """Types, shapes, strides and devices, before the library is called."""
    bf, i32 = torch.bfloat16, torch.int32
    k = torch.zeros((4, 2, 128), dtype=bf)
    pool = torch.zeros((3, 2, 2176), dtype=torch.uint8)
    bt, idx = torch.zeros((1, 2), dtype=i32), torch.zeros(4, dtype=i32)
    cs = torch.zeros((8, 128))

    def bad(call):
        with pytest.raises((ValueError, TypeError)):
            call()

    bad(lambda: pa.append_kv4(k, k, pool, bt, idx, idx))                      # not on a GPU
    bad(lambda: pa.append_kv4(k, k.half(), pool, bt, idx, idx))               # types differ
    bad(lambda: pa.append_kv4(k, k[:3], pool, bt, idx, idx))                  # token counts differ
    bad(lambda: pa.append_kv4(k.transpose(1, 2).contiguous().transpose(1, 2), k, pool, bt, idx, idx))
    bad(lambda: pa.append_kv4(k, k, pool, bt.long(), idx, idx))
    bad(lambda: pa.append_kv4(k, k, pool, bt, idx[:3], idx))
    bad(lambda: pa.append_kv4(k, k, pool[:, :1], bt, idx, idx))
    bad(lambda: pa.append_kv4(k, k, pool[..., :1152].contiguous(), bt, idx, idx))  # head_dim 64
    bad(lambda: pa.append_kv4(k, k, pool, bt, idx, idx, q_out=k))             # q_out without q
    bad(lambda: pa.append_kv4(k, k, pool, bt, idx, idx, cos_sin=cs.double()))
    kc = torch.zeros((3, 2, 16, 128), dtype=bf)
    bad(lambda: pa.append_kv_rope(k, k, kc, kc.half(), bt, idx, idx, cs))
    bad(lambda: pa.append_kv_rope(k, k, kc, kc, bt, idx, idx, cs))            # not on a GPU
    bad(lambda: pa.read_kv4(pool, bt, idx, idx))                              # no type given
    bad(lambda: pa.read_kv4(pool, bt, idx, idx, dtype=torch.float32, k_out=torch.zeros(4, 2, 128)))
    q, ctx = torch.zeros((1, 4, 128), dtype=bf), torch.zeros(1, dtype=i32)
    bad(lambda: pa.decode_kv4(q, pool, bt, ctx, 0.1))                         # not on a GPU
    bad(lambda: pa.decode_kv4(q[..., :64].contiguous(), pool, bt, ctx, 0.1))  # head_dim
    bad(lambda: pa.decode_kv4(q, pool, bt, ctx.long(), 0.1))
    bad(lambda: pa.decode_kv4(q, pool.to(torch.int8), bt, ctx, 0.1))
    bad(lambda: pa.prefill_kv4(q[:, None], pool, bt, torch.zeros(2, dtype=i32), 0.1))


def test_rope_table_is_the_formula():
    t = pa.rope_table(5, 32, base=500.0, device="cpu")
    assert t.shape == (5, 32) and t.dtype == torch.float32
    for p in range(5):
        for i in range(16):
            a = torch.tensor(p * 500.0 ** (-2 * i / 32), dtype=torch.float64)
            assert abs(t[p, i] - a.cos()) <= ref.EPS32 and abs(t[p, 16 + i] - a.sin()) <= ref.EPS32
