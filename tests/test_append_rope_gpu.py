"""GPU parity of the rotated append into the 16-bit cache against the rotation in
64 bits: both pairings, partial rotations, views of a fused projection, queries in
place, rows that are not written, refused tokens."""
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


def assert_rounded(got, want, x, dt):
    """A pair's two products and their sum are rounded to fp32 (3 half steps 2^-24
    of at most 2 max |x|) and the result once to dtype: half a step, or half of the
    smallest subnormal."""
    size = 2 * x.double().abs().amax(-1, keepdim=True)
    slack = 3 * 2.0 ** -24 * size
    half = torch.finfo(dt).eps / 2
    tol = (want.abs() + slack) * half + slack + torch.finfo(dt).smallest_normal * half
    assert ((got.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("d,rot,inter", [(128, 128, False), (128, 128, True), (128, 64, False),
                                         (128, 48, False), (128, 16, True), (64, 64, False),
                                         (64, 32, True), (64, 16, False), (64, 48, True)])
@pytest.mark.parametrize("hq,hkv,lens", [(8, 2, [1, 0, 33]), (0, 1, [17]), (5, 5, [3, 4]),
                                         (32, 8, [900, 1700])])
def test_rotation_and_placement(hq, hkv, lens, d, rot, inter, dtype):
    dt, gen = DT[dtype], torch.Generator().manual_seed(d + rot + hkv)
    blocks = [-(-t // 16) for t in lens]
    pages = sum(blocks) + 1
    perm = torch.randperm(pages, generator=gen).to(torch.int32)
    bt = torch.full((len(lens), max(blocks)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(blocks):
        bt[b, :n] = perm[at:at + n]
        at += n
    seq = torch.cat([torch.full((t,), b, dtype=torch.int32) for b, t in enumerate(lens)])
    pos = torch.cat([torch.arange(t, dtype=torch.int32) for t in lens])
    order = torch.randperm(seq.numel(), generator=gen)
    seq, pos = seq[order], pos[order]
    n = seq.numel()
    w = torch.randn((n, hq + 2 * hkv + 2, d), generator=gen).to(dt).cuda()
    cs = pa.rope_table(max(lens), rot)
    kc = torch.full((pages, hkv, 16, d), 7.0, dtype=dt, device="cuda")
    vc = torch.full_like(kc, 8.0)
    q, k, v = w[:, :hq], w[:, hq:hq + hkv], w[:, hq + hkv:hq + 2 * hkv]
    q_out = pa.append_kv_rope(k, v, kc, vc, bt.cuda(), seq.cuda(), pos.cuda(), cs,
                              q=q if hq else None, interleaved=inter)
    torch.cuda.synchronize()
    assert pa.pa_last_device_error() == 0
    page, slot = bt[seq.long(), (pos // 16).long()].long().cuda(), (pos % 16).long().cuda()
    want_k = ref.rotate(k, pos.cuda(), cs, inter)
    got_k = kc[page, :, slot]
    assert_rounded(got_k, want_k, k, dt)
    assert torch.equal(got_k[..., rot:], k[..., rot:])
    assert torch.equal(vc[page, :, slot], v)
    if hq:
        assert_rounded(q_out, ref.rotate(q, pos.cuda(), cs, inter), q, dt)
    else:
        assert q_out is None
    kc[page, :, slot] = 7.0
    vc[page, :, slot] = 8.0
    assert (kc == 7).all() and (vc == 8).all()  # nothing else was written


def test_position_zero_and_inverse():
    """Position 0 leaves the bits alone; turning back by the opposite angle gives the
    row again, to two roundings."""
    dt = torch.float16
    bt = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    seq = torch.zeros(20, dtype=torch.int32, device="cuda")
    pos = torch.arange(20, dtype=torch.int32, device="cuda")
    k = torch.randn((20, 3, 64), device="cuda").to(dt)
    kc = torch.zeros((2, 3, 16, 64), dtype=dt, device="cuda")
    vc = torch.zeros_like(kc)
    cs = pa.rope_table(20, 64)
    q = pa.append_kv_rope(k, k, kc, vc, bt, seq, pos, cs, q=k)
    assert torch.equal(kc[0, :, 0], k[0]) and torch.equal(q[0], k[0])
    back = torch.cat((cs[:, :32], -cs[:, 32:]), -1)
    again = pa.append_kv_rope(q, q, kc, vc, bt, seq, pos, back, q=q)
    # a turned element is at most sqrt(2) max |x|; the first rounding's error turns
    # too (sqrt(2)), the second adds its own
    assert (again.double() - k.double()).abs().max() <= 4 * 2.0 ** -11 * k.abs().max() * 2


def test_queries_in_place():
    dt = torch.bfloat16
    bt = torch.arange(4, dtype=torch.int32, device="cuda")[:, None].contiguous()
    seq = torch.arange(4, dtype=torch.int32, device="cuda")
    pos = torch.tensor([3, 15, 0, 7], dtype=torch.int32, device="cuda")
    k = torch.randn((4, 2, 128), device="cuda").to(dt)
    q = torch.randn((4, 8, 128), device="cuda").to(dt)
    kc = torch.zeros((4, 2, 16, 128), dtype=dt, device="cuda")
    vc = torch.zeros_like(kc)
    cs = pa.rope_table(16, 128)
    for inter in (False, True):
        want = pa.append_kv_rope(k, k, kc, vc, bt, seq, pos, cs, q=q, interleaved=inter)
        mine = q.clone()
        got = pa.append_kv_rope(k, k, kc, vc, bt, seq, pos, cs, q=mine, q_out=mine,
                                interleaved=inter)
        assert got is mine and torch.equal(mine, want)


def test_bad_tokens_are_skipped_and_reported():
    dt, d = torch.bfloat16, 128
    kc = torch.full((3, 2, 16, d), 7.0, dtype=dt, device="cuda")
    vc = kc.clone()
    bt = torch.tensor([[0, 99], [1, -1]], dtype=torch.int32, device="cuda")
    x = torch.randn((7, 2, d), device="cuda").to(dt)
    q = torch.randn((7, 4, d), device="cuda").to(dt)
    out = torch.full((7, 4, d), 5.0, dtype=dt, device="cuda")
    # good, past the table, no such sequence, negative, bad page, unmapped, no angle
    seq = torch.tensor([0, 0, 2, 0, 0, 1, 1], dtype=torch.int32, device="cuda")
    pos = torch.tensor([3, 32, 0, -1, 16, 17, 5], dtype=torch.int32, device="cuda")
    for k in range(7):
        cs = pa.rope_table(5 if k == 6 else 40, d)
        pa.append_kv_rope(x[k:k + 1], x[k:k + 1], kc, vc, bt, seq[k:k + 1], pos[k:k + 1], cs,
                          q=q[k:k + 1], q_out=out[k:k + 1])
        want = (0, -14, -14, -14, -11, -11, -14)[k]
        assert pa.pa_last_device_error() == want, k
    assert (out[1:] == 5).all() and not (out[0] == 5).all()
    assert (kc[1:] == 7).all() and (kc[0, :, 3] != 7).any() and (kc[0, :, 4:] == 7).all()


def test_append_then_decode_and_graph():
    """The rotated append feeds the 16-bit decode; captured and replayed on new data."""
    dt, hq, hkv, d = torch.float16, 8, 2, 128
    bt = torch.arange(6, dtype=torch.int32, device="cuda").view(2, 3)
    kc = torch.randn((6, hkv, 16, d), device="cuda").to(dt)
    vc = torch.randn((6, hkv, 16, d), device="cuda").to(dt)
    k0, v0 = kc.clone(), vc.clone()
    seq = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    pos = torch.tensor([40, 17], dtype=torch.int32, device="cuda")
    lens = pos + 1
    cs = pa.rope_table(48, d)
    qkv = torch.randn((2, hq + 2 * hkv, d), device="cuda").to(dt)
    q_out = torch.empty((2, hq, d), dtype=dt, device="cuda")
    out = torch.empty((2, hq, d), device="cuda")

    def step(q_to, o_to):
        q = pa.append_kv_rope(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], kc, vc, bt, seq, pos, cs,
                              q=qkv[:, :hq], q_out=q_to)
        return pa.decode(q, kc, vc, bt, lens, 0.09, out=o_to)

    step(None, None)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        step(q_out, out)
    for k in range(2):
        qkv.copy_(torch.randn(qkv.shape, device="cuda"))
        kc.copy_(k0), vc.copy_(v0)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        kc.copy_(k0), vc.copy_(v0)
        assert torch.equal(step(None, None), got)
    rot = ref.rotate(qkv[:, hq:hq + hkv], pos, cs, False)
    assert_rounded(kc[bt[seq.long(), (pos // 16).long()].long(), :, (pos % 16).long()], rot,
                   qkv[:, hq:hq + hkv], dt)
    assert pa.pa_last_device_error() == 0
