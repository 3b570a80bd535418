"""Weighted decode, eviction, trees and compaction as a serving loop makes them: one behind the
other, in graphs, on another stream, without a wait in between."""
import math

import pytest
import torch

import paged_kv_cache_171_gb300 as pa
from tests import evict_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_kv_cache_171_gb300 import build
    build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    assert pa.pa_last_device_error() == 0


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("inter", [False, True])
def test_a_drafted_tree_is_verified_and_a_branch_accepted(dt, inter):
    hq, hkv, d, lens = 4, 2, 64, [50, 17]
    parents = _i32([[-1, 0, 0, 1, 2, 2, 4, 0, -1, 8, 3, 9], [-1, -1, 1, 2, 3, 4, 5, 6, 7, 8, 9, 10]])
    n = parents.shape[1]
    mask, depth = pa.tree_mask(parents)
    gen = torch.Generator(device="cuda").manual_seed(1)
    bt = torch.randperm(16, generator=gen, device="cuda").to(torch.int32).view(2, 8)
    ctx = _i32(lens)
    cs = pa.rope_table(128, d)
    rows = torch.randn((2, 64, hq + 2 * hkv, d), generator=gen, device="cuda").to(dt)
    kc = torch.zeros((16, hkv, 16, d), dtype=dt, device="cuda")
    vc = torch.zeros_like(kc)

    def append(b, at, w, caches, rope_pos=None):
        pos = at.to(torch.int32)
        return pa.append_kv_rope(w[:, hq:hq + hkv], w[:, hq + hkv:], *caches, bt,
                                 torch.full_like(pos, b), pos, cs, q=w[:, :hq], interleaved=inter,
                                 rope_pos=rope_pos)

    for b, t in enumerate(lens):
        append(b, torch.arange(t, device="cuda"), rows[b, :t], (kc, vc))
    prompt = (kc.clone(), vc.clone())
    drafts = torch.randn((2, n, hq + 2 * hkv, d), generator=gen, device="cuda").to(dt)
    q = torch.stack([append(b, t + torch.arange(n, device="cuda"), drafts[b], (kc, vc),
                            (t + depth[b]).to(torch.int32)) for b, t in enumerate(lens)])
    out = pa.prefill_tree(q, kc, vc, bt, ctx, mask, 0.125)

    # every drafted token by itself: its branch appended token by token, and decoded
    def branch(b, i):
        path = []
        while i >= 0:
            path.append(i)
            i = int(parents[b, i])
        return path[::-1]

    for b, t in enumerate(lens):
        for i in range(n):
            path = branch(b, i)
            caches = (prompt[0].clone(), prompt[1].clone())
            qs = append(b, t + torch.arange(len(path), device="cuda"), drafts[b, path], caches)
            assert torch.equal(qs[-1], q[b, i])  # rotated by its depth
            want = pa.decode(qs[-1:], *caches, bt[b:b + 1], _i32([t + len(path)]), 0.125)
            # both are within a few half steps of the values: the 16-bit weights' and result's
            # four roundings of values up to 4: the rotated q and k, the weights, the output
            tol = 4 * torch.finfo(dt).eps / 2 * 4.0
            assert (out[b, i].float() - want[0]).abs().max() < tol

    # one branch each is accepted: the caches hold it as if it had been appended alone
    paths = [branch(0, 10), branch(1, 3)]
    keep = torch.full((2, max(map(len, paths))), -1, dtype=torch.int32, device="cuda")
    for b, p in enumerate(paths):
        keep[b, :len(p)] = _i32(p)
    now = pa.compact_kv(kc, vc, bt, ctx, keep, _i32([len(p) for p in paths]))
    assert now.tolist() == [t + len(p) for t, p in zip(lens, paths)]
    for b, t in enumerate(lens):
        append(b, t + torch.arange(len(paths[b]), device="cuda"), drafts[b, paths[b]], prompt)
        pos = torch.arange(int(now[b]), device="cuda")
        page, slot = bt[b, pos // 16].long(), pos % 16
        assert torch.equal(kc[page, :, slot], prompt[0][page, :, slot])
        assert torch.equal(vc[page, :, slot], prompt[1][page, :, slot])
    assert pa.pa_last_device_error() == 0


def test_positions_to_rotate_by_are_checked():
    kc = torch.zeros((2, 1, 16, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.randn((3, 2, 64), device="cuda").bfloat16()
    cs = pa.rope_table(10, 64)
    pa.append_kv_rope(w[:, :1], w[:, 1:], kc, kc.clone(), _i32([[0, 1]]), _i32([0, 0, 0]),
                      _i32([20, 21, 22]), cs, rope_pos=_i32([9, 10, -1]))
    assert pa.pa_last_device_error() == -14
    assert kc[1, 0, 4].abs().sum() > 0 and kc[1, 0, 5:].abs().sum() == 0
    with pytest.raises(ValueError, match="rope_pos"):
        pa.append_kv_rope(w[:, :1], w[:, 1:], kc, kc.clone(), _i32([[0, 1]]), _i32([0, 0, 0]),
                          _i32([20, 21, 22]), cs, rope_pos=_i32([9, 10]))


def test_weights_gathered_over_a_prompt_and_steps_decide_what_stays():
    """A prompt's weights, decode steps, an eviction, more steps: each call against the
    definition on what the ones before it left."""
    hq, hkv, d, dt, lens, n = 8, 2, 64, torch.bfloat16, [180, 9], 9
    gen = torch.Generator().manual_seed(3)
    bt = torch.randperm(30, generator=gen).to(torch.int32).view(2, 15)
    k, v = torch.randn((2, 30, hkv, 16, d), generator=gen).to(dt)
    w = torch.full((30, hkv, 16), math.nan)  # never cleared: every token is fresh once
    gk, gv, gw, gbt = k.cuda(), v.cuda(), w.cuda(), bt.cuda()
    # the prompt: its first part not looked at, its last n queries' weights over all of it
    first = torch.tensor([t - n for t in lens], dtype=torch.int32)
    q = torch.randn((2, n, hq, d), generator=gen).to(dt)
    pa.prefill_weights(q.cuda(), gk, gw, gbt, first.cuda(), 0.125, fresh=200)
    want, bound = ref.chunk_weights(q, k, w, bt, first, 0.125, 200)
    seen = torch.zeros_like(w, dtype=torch.bool)
    for b, t in enumerate(lens):
        page, slot = ref.places(bt, b, torch.arange(t))
        seen[page, :, slot] = True
    assert ((gw.cpu().double() - want).abs() <= bound)[seen].all() and gw.cpu()[~seen].isnan().all()
    ctx = torch.tensor(lens, dtype=torch.int32)
    for step in range(6):
        if step == 3:  # the first sequence has outgrown its budget
            before = (gk.cpu(), gv.cpu(), gw.cpu())
            got = pa.evict_kv(gk, gv, gw, gbt, ctx.cuda(), 64, 4, 16)
            k2, v2, w2, ctx = ref.evict(*before, bt, bt, ctx, 64, 4, 16)
            assert torch.equal(got.cpu(), ctx) and torch.equal(gk.cpu(), k2)
            assert torch.equal(gw.cpu().nan_to_num(-1), w2.nan_to_num(-1))
        ctx = ctx + 1
        new = torch.randn((2, 2, hkv, d), generator=gen).to(dt)
        pa.append_kv(new[0].cuda(), new[1].cuda(), gk, gv, gbt, _i32([0, 1]), (ctx - 1).cuda())
        before = (gk.cpu(), gv.cpu(), gw.cpu())
        q = torch.randn((2, hq, d), generator=gen).to(dt)
        out = pa.decode_weighted(q.cuda(), gk, gv, gw, gbt, ctx.cuda(), 0.125)
        o, ob, want, bound = ref.weighted_decode(q, *before, bt, ctx, 0.125, 1)
        assert ((out.cpu().double() - o).abs() <= ob).all()
        fine = want.isfinite()
        assert ((gw.cpu().double() - want).abs() <= bound)[fine].all()
        for b, t in enumerate(ctx.tolist()):
            page, slot = ref.places(bt, b, torch.arange(t))
            assert gw.cpu()[page, :, slot].isfinite().all()
    assert pa.pa_last_device_error() == 0


def _loop(seed, dt=torch.bfloat16):
    """State of a small serving loop, and its step: everything of this file once."""
    hq, hkv, d, n = 8, 2, 128, 20
    lens = [700, 3, 1500]
    k, v, w, bt, ctx = (x.cuda() for x in ref.pool([t + n for t in lens], hkv, d, dt, seed))
    ctx = _i32(lens)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    parents = (torch.arange(n, device="cuda") - 1 -
               torch.arange(n, device="cuda") % 3).clamp(min=-1).to(torch.int32).repeat(3, 1)
    s = dict(k=k, v=v, w=w, bt=bt, ctx=ctx,
             q=torch.randn((3, hq, d), generator=gen, device="cuda").to(dt),
             qs=torch.randn((3, n, hq, d), generator=gen, device="cuda").to(dt), parents=parents,
             keep=_i32([[0, 2, 5]] * 3), n_keep=_i32([3, 0, 2]),
             mask=torch.empty((3, n, 1), dtype=torch.int32, device="cuda"),
             depth=torch.empty((3, n), dtype=torch.int32, device="cuda"),
             out=torch.empty((3, hq, d), device="cuda"), tree=torch.empty((3, n, hq, d), dtype=dt, device="cuda"),
             now=_i32([0] * 3), less=_i32([0] * 3),
             ws=torch.empty(64 << 20, dtype=torch.uint8, device="cuda"))

    def step():
        pa.decode_weighted(s["q"], s["k"], s["v"], s["w"], s["bt"], s["ctx"], 0.1, out=s["out"],
                           workspace=s["ws"])
        pa.tree_mask(s["parents"], s["mask"], s["depth"])
        pa.prefill_tree(s["qs"], s["k"], s["v"], s["bt"], s["ctx"], s["mask"], 0.1, out=s["tree"],
                        workspace=s["ws"])
        pa.compact_kv(s["k"], s["v"], s["bt"], s["ctx"], s["keep"], s["n_keep"], weights=s["w"],
                      new_lens=s["now"])
        pa.prefill_weights(s["qs"], s["k"], s["w"], s["bt"], s["ctx"], 0.1, workspace=s["ws"])
        pa.evict_kv(s["k"], s["v"], s["w"], s["bt"], s["now"], 600, 4, 100, new_lens=s["less"],
                    workspace=s["ws"])

    return s, step


WRITTEN = ("k", "v", "w", "mask", "depth", "out", "tree", "now", "less")


def _results(s):
    return [s[x].clone() for x in WRITTEN]


def test_graphs_that_share_a_workspace():
    s, step = _loop(1)
    start = {x: s[x].clone() for x in WRITTEN}

    def reset():
        for x, y in start.items():
            s[x].copy_(y)

    step()
    want = _results(s)
    reset()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(side):
        for _ in range(2):
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                step()
            graphs.append(g)
    torch.cuda.synchronize()
    for i in range(4):
        reset()
        s["ws"].fill_(17 * i)
        graphs[i % 2].replay()
        for a, b in zip(_results(s), want):
            assert torch.equal(a, b)
    assert pa.pa_last_device_error() == 0


def test_calls_without_a_wait_see_what_was_written_before():
    """Inputs rewritten right before each step, 30 steps without a wait: each gives what it gives
    alone."""
    s, step = _loop(2)
    start = {x: s[x].clone() for x in WRITTEN}
    perm = torch.randperm(3, device="cuda")
    variants = [(s["q"].clone(), s["bt"].clone(), s["ctx"].clone()),
                (s["q"].clone().flip(2), s["bt"][perm].clone(), s["ctx"][perm].clone())]

    def one(i):
        for x, y in start.items():
            s[x].copy_(y)
        q, bt, ctx = variants[i % 2]
        s["q"].copy_(q), s["bt"].copy_(bt), s["ctx"].copy_(ctx)
        step()
        return _results(s)

    want = []
    for i in range(2):
        want.append(one(i))
        torch.cuda.synchronize()
    got = [one(i) for i in range(30)]
    torch.cuda.synchronize()
    assert pa.pa_last_device_error() == 0
    for i, g in enumerate(got):
        for a, b, name in zip(g, want[i % 2], WRITTEN):
            assert torch.equal(a, b), (i, name)


def test_another_stream():
    s, step = _loop(3)
    t, _ = _loop(3)
    step()
    want = _results(s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    # allocations and launches of the calls belong to the stream they are given
    out = pa.decode_weighted(t["q"], t["k"], t["v"], t["w"], t["bt"], t["ctx"], 0.1, stream=side)
    mask, _ = pa.tree_mask(t["parents"], stream=side)
    tree = pa.prefill_tree(t["qs"], t["k"], t["v"], t["bt"], t["ctx"], mask, 0.1, stream=side)
    now = pa.compact_kv(t["k"], t["v"], t["bt"], t["ctx"], t["keep"], t["n_keep"], weights=t["w"],
                        stream=side)
    pa.prefill_weights(t["qs"], t["k"], t["w"], t["bt"], t["ctx"], 0.1, stream=side.cuda_stream)
    less = pa.evict_kv(t["k"], t["v"], t["w"], t["bt"], now, 600, 4, 100, stream=side)
    side.synchronize()
    got = [t["k"], t["v"], t["w"], mask, want[4], out, tree, now, less]
    for a, b, name in zip(got, want, WRITTEN):
        assert torch.equal(a, b), name


def test_tensors_that_do_not_fit_are_refused():
    s, _ = _loop(4)
    a = (s["k"], s["v"])
    for call in (
            lambda: pa.decode_weighted(s["q"][:, ::2], *a, s["w"], s["bt"], s["ctx"], 0.1),
            lambda: pa.decode_weighted(s["q"], *a, s["w"][:, :1], s["bt"], s["ctx"], 0.1),
            lambda: pa.decode_weighted(s["q"], *a, s["w"].double(), s["bt"], s["ctx"], 0.1),
            lambda: pa.decode_weighted(s["q"].half(), *a, s["w"], s["bt"], s["ctx"], 0.1),
            lambda: pa.decode_weighted(s["q"][..., :64].contiguous(), *a, s["w"], s["bt"], s["ctx"], 0.1),
            lambda: pa.prefill_weights(s["qs"].transpose(1, 2), s["k"], s["w"], s["bt"], s["ctx"], 0.1),
            lambda: pa.prefill_weights(s["qs"][..., ::2], s["k"], s["w"], s["bt"], s["ctx"], 0.1),
            lambda: pa.evict_kv(*a, s["w"], s["bt"], s["ctx"].long(), 5),
            lambda: pa.evict_kv(*a, s["w"], s["bt"], s["ctx"], 5, dst_table=s["bt"][:2]),
            lambda: pa.compact_kv(*a, s["bt"], s["ctx"], s["keep"][:2], s["n_keep"]),
            lambda: pa.compact_kv(s["k"], s["v"][:1], s["bt"], s["ctx"], s["keep"], s["n_keep"]),
            lambda: pa.prefill_tree(s["qs"], *a, s["bt"], s["ctx"], s["mask"][:, :5], 0.1),
            lambda: pa.prefill_tree(s["qs"][:, ::2], *a, s["bt"], s["ctx"], s["mask"], 0.1),
            lambda: pa.tree_mask(s["parents"].long())):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: pa.decode_weighted(s["q"], *a, s["w"], s["bt"], s["ctx"], 0.1, fresh=-1),
                 lambda: pa.decode_weighted(s["q"], *a, s["w"], s["bt"], s["ctx"], 0.1,
                                            workspace=s["ws"][:1024]),
                 lambda: pa.evict_kv(*a, s["w"], s["bt"], s["ctx"], 5, sink=3, recent=3),
                 lambda: pa.compact_kv(*a, s["bt"], s["ctx"], s["keep"], s["n_keep"],
                                       new_lens=s["ctx"])):
        with pytest.raises(pa.PAError):
            call()
    assert pa.pa_last_device_error() == 0
