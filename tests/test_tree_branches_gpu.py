"""A drafted tree, rotated, appended and attended to, against each branch in 64 bits from caches
that it was appended to alone."""
import pytest
import torch

import paged_kv_cache_171_gb300 as pa
from tests import evict_reference as ref
from tests.test_evict_flow_gpu import _built, _i32  # noqa: F401

pytestmark = pytest.mark.gpu
PARENTS = [[-1, 0, 0, 1, 2, 2, 4, 0, -1, 8, 3, 9], [-1, -1, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10]]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("hq,hkv,d", [(4, 2, 64), (24, 2, 128)])
def test_every_branch_by_itself(hq, hkv, d, inter, dt):
    lens, n, scale = [50, 17], 12, d ** -0.5
    parents = _i32(PARENTS)
    mask, depth = pa.tree_mask(parents)
    gen = torch.Generator(device="cuda").manual_seed(2)
    bt = torch.randperm(16, generator=gen, device="cuda").to(torch.int32).view(2, 8)
    cs = pa.rope_table(128, d)
    rows = torch.randn((2, 64, hq + 2 * hkv, d), generator=gen, device="cuda").to(dt)
    drafts = torch.randn((2, n, hq + 2 * hkv, d), generator=gen, device="cuda").to(dt)
    kc = torch.zeros((16, hkv, 16, d), dtype=dt, device="cuda")
    vc = torch.zeros_like(kc)

    def append(b, first, w, caches, rope_pos=None):
        pos = first + torch.arange(len(w), device="cuda", dtype=torch.int32)
        return pa.append_kv_rope(w[:, hq:hq + hkv], w[:, hq + hkv:], *caches, bt,
                                 torch.full_like(pos, b), pos, cs, q=w[:, :hq], interleaved=inter,
                                 rope_pos=rope_pos)

    for b, t in enumerate(lens):
        append(b, 0, rows[b, :t], (kc, vc))
    alone = (kc.clone(), vc.clone())
    q = torch.stack([append(b, t, drafts[b], (kc, vc), (t + depth[b]).to(torch.int32))
                     for b, t in enumerate(lens)])
    out = pa.prefill_tree(q, kc, vc, bt, _i32(lens), mask, scale).cpu()
    half, G, table = torch.finfo(dt).eps / 2, hq // hkv, bt.cpu()
    for b, t in enumerate(lens):
        for i in range(n):
            path, j = [], i
            while j >= 0:
                path.insert(0, j)
                j = PARENTS[b][j]
            caches = (alone[0].clone(), alone[1].clone())
            qs = append(b, t, drafts[b, path], caches)
            assert torch.equal(qs[-1], q[b, i])
            k, v = (ref.rows(x.cpu(), table, b, t + len(path)) for x in caches)
            at = t + torch.tensor(path)
            page, slot = ref.places(table, b, at)
            assert torch.equal(kc.cpu()[page, :, slot].double(), k[:, t:].transpose(0, 1))
            seen = torch.ones((1, t + len(path)), dtype=torch.bool)
            for g in range(hkv):
                qq = qs[-1:, g * G:(g + 1) * G].cpu().double()
                p, _, err = ref.attention(qq, k[g], seen, scale)
                want, size = p[0] @ v[g], p[0] @ v[g].abs()
                # the roundings of the result and of the weights, half a step each, and fp32's:
                # the scores', the exponential's, sums of a tile and its 32 partial sums
                bound = half * want.abs() + (half * 1.01 + err[0] + 2 * ref.H32 * 33) * size
                got = out[b, i, g * G:(g + 1) * G].double()
                assert ((got - want).abs() <= bound).all(), (b, i, g)
    assert pa.pa_last_device_error() == 0
