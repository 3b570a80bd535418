"""Arguments that weighted decode, prompt weights, eviction, compaction and tree attention
refuse, on the host before any CUDA call, and the sizes they report."""
import ctypes

import pytest
import torch

import paged_kv_cache_171_gb300 as pa
from paged_kv_cache_171_gb300 import build as pa_build

P = 0x1000  # 16-byte aligned, never dereferenced on these paths
f = ctypes.c_float(0.1)


@pytest.fixture(scope="module")
def L():
    pa_build.build()
    return pa.lib()


def _each(call, ok, good, cases):
    if good is not None:
        assert call(*ok) == good
    for at, value, code in cases:
        bad = list(ok)
        bad[at] = value
        assert call(*bad) == code, (at, value)


HEADS = [(30, -2), (0, -2)]


def test_decode_weighted_refuses(L):
    need = L.pa_decode_weighted_workspace_size(2, 32, 8, 128, 16, 8)
    assert need >= 4 * 2 * 32 * 8 * 16
    ok = [P, P, P, P, P, P, P, f, 1, 32, 8, 128, 16, 2, 8, 16, 0, P, need, None]
    _each(L.pa_decode_weighted, ok, None,
          [(i, None, -1) for i in range(7)] +
          [(8, -1, -5), (9, 30, -2), (9, 8 * 1025, -2), (10, 0, -2), (11, 96, -3), (12, 8, -4),
           (13, 0, -5), (13, 70000, -5), (14, 0, -5), (15, 0, -5), (16, 2, -6), (17, None, -7),
           (18, need - 1, -7), (17, P + 8, -8), (0, P + 2, -8), (1, P + 8, -8), (3, P + 4, -8),
           (6, P + 4, -8)])
    assert L.pa_decode_weighted_workspace_size(2, 30, 8, 128, 16, 8) == 0
    assert L.pa_decode_weighted_workspace_size(0, 32, 8, 128, 16, 8) == 0


def test_prefill_weights_refuses(L):
    need = L.pa_prefill_weights_workspace_size(2, 4, 32, 8, 128, 16, 8)
    assert need > 0
    ok = [P, P, P, P, P, 4, f, 4, 16384, 4096, 32, 8, 128, 16, 2, 8, 16, 0, P, need, None]
    _each(L.pa_prefill_weights, ok, None,
          [(i, None, -1) for i in range(5)] +
          [(5, -1, -5), (5, 129, -5), (7, -1, -5), (8, 4095, -5), (9, 4088, -5), (8, 16388, -8),
           (9, 4100, -8), (10, 30, -2), (12, 96, -3), (13, 8, -4), (14, 0, -5), (17, 2, -6),
           (18, None, -7), (19, need - 1, -7), (18, P + 8, -8), (0, P + 8, -8), (2, P + 4, -8)])
    none = list(ok)
    none[5] = 0
    none[18] = None
    assert L.pa_prefill_weights(*none) == 0
    assert L.pa_prefill_weights_workspace_size(2, 0, 32, 8, 128, 16, 8) == 0


def test_evict_refuses(L):
    need = L.pa_evict_kv_workspace_size(2, 8, 128, 16, 8, 64)
    assert need == 4 * (2 * 8 * 64 + 2)
    assert L.pa_evict_kv_workspace_size(2, 8, 128, 16, 8, 128) == 8  # every token stays
    ok = [P, P, P, P, P, P, P + 64, 64, 4, 16, 8, 128, 16, 2, 8, 8, 16, 0, P, need, None]
    _each(L.pa_evict_kv, ok, None,
          [(i, None, -1) for i in range(7)] +
          [(6, P, -5), (7, -1, -5), (8, -1, -5), (9, -1, -5), (9, 61, -5), (8, 2 ** 31 - 1, -5),
           (10, 0, -2), (11, 96, -3), (12, 8, -4), (13, 0, -5), (14, 0, -5), (15, 0, -5),
           (16, 0, -5), (17, 2, -6), (18, None, -7), (19, need - 1, -7), (18, P + 8, -8),
           (0, P + 8, -8), (2, P + 4, -8)])


def test_compact_refuses(L):
    ok = [P, P, P, P, P, P, P, 10, P + 64, 8, 128, 16, 2, 8, 16, 0, None]
    _each(L.pa_compact_kv, ok, None,
          [(0, None, -1), (1, None, -1), (3, None, -1), (4, None, -1), (5, None, -1),
           (6, None, -1), (8, None, -1), (7, -1, -5), (7, 129, -5), (8, P, -5), (9, 0, -2),
           (10, 96, -3), (11, 8, -4), (12, 0, -5), (14, 0, -5), (15, 2, -6), (0, P + 8, -8),
           (2, P + 4, -8)])


def test_new_lengths_lie_apart_from_what_the_calls_read(L):
    A = [0x1000 * (i + 1) for i in range(8)]
    evict = [A[0], A[1], A[2], A[3], A[4], A[5], 0, 64, 4, 16, 8, 128, 16, 2, 8, 8, 16, 0, A[6],
             1 << 20, None]
    for near in (A[4], A[4] + 4, A[4] - 4, A[3] + 60, A[5] + 60):
        evict[6] = near
        assert L.pa_evict_kv(*evict) == -5, near
    compact = [A[0], A[1], None, A[3], A[4], A[5], A[6], 10, 0, 8, 128, 16, 2, 8, 16, 0, None]
    for near in (A[4] + 4, A[4] - 4, A[5] + 76, A[6], A[6] + 4, A[6] - 4, A[3] + 60):
        compact[8] = near
        assert L.pa_compact_kv(*compact) == -5, near


def test_tree_refuses(L):
    need = L.pa_prefill_tree_workspace_size(1, 8, 32, 8, 128, 16, 4096)
    assert need > 0
    ok = [P, P, P, P, P, P, 8, P, f, 32, 8, 128, 16, 1, 4096, 16, 0, P, need, None]
    _each(L.pa_prefill_tree, ok, None,
          [(0, None, -1), (1, None, -1), (5, None, -1), (7, None, -1), (6, -1, -5),
           (6, 65537, -5), (9, 30, -2), (11, 96, -3), (12, 8, -4), (13, 0, -5), (16, 2, -6),
           (17, None, -7), (18, need - 1, -7), (17, P + 8, -8), (0, P + 8, -8), (7, P + 4, -8)])
    none = list(ok)
    none[6] = 0
    none[17] = None
    assert L.pa_prefill_tree(*none) == 0
    assert L.pa_prefill_tree_workspace_size(200, 8, 32, 8, 128, 16, 64) == 0  # one range
    _each(L.pa_tree_mask, [P, P, P, 2, 0, None], 0,
          [(0, None, -1), (1, None, -1), (3, 0, -5), (4, -1, -5), (3, 70000, -5)])


def test_append_at_other_positions_refuses(L):
    ok = [P, P, P, P, P, P, P, P, P, P, P, 0, 1024, 1024, 4096, 32, 8, 128, 16, 2, 8, 16, 100,
          128, 0, 0, None]
    _each(L.pa_append_kv_rope_at, ok, 0,
          [(9, None, -1), (10, None, -1), (8, None, -1), (11, -1, -5), (22, 0, -18)])


def test_bindings_refuse_tensors_that_are_not_theirs():
    t = torch.zeros((1, 8, 128), dtype=torch.bfloat16)
    kc = torch.zeros((4, 2, 16, 128), dtype=torch.bfloat16)
    bt = torch.zeros((1, 4), dtype=torch.int32)
    one = torch.ones(1, dtype=torch.int32)
    w = torch.zeros((4, 2, 16))
    for call in (lambda: pa.decode_weighted(t, kc, kc, w, bt, one, 0.1),
                 lambda: pa.prefill_weights(t[None], kc, w, bt, one, 0.1),
                 lambda: pa.evict_kv(kc, kc, w, bt, one, 3),
                 lambda: pa.compact_kv(kc, kc, bt, one, bt, one),
                 lambda: pa.prefill_tree(t[None], kc, kc, bt, one, bt[None], 0.1),
                 lambda: pa.tree_mask(bt)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
