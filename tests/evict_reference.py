"""Gathered attention weight, eviction by it and tree attention from their definitions, in
64 bits, with the bounds of the kernels' roundings.  Shares no code with the package."""
import torch

PAGE = 16
H32 = 2.0 ** -24  # half a step of fp32


def pool(lens, hkv, d, dt, seed, spare=2, fill=None, blocks=None):
    """(k, v, weights, block table, ctx) with N(0, 1) rows in shuffled pages; rows past a
    sequence's end, and the spare pages, hold `fill` (None: rows like the others)."""
    gen = torch.Generator().manual_seed(seed)
    need = [-(-t // PAGE) for t in lens]
    pages = sum(need) + spare
    perm = torch.randperm(pages, generator=gen).to(torch.int32)
    bt = torch.full((len(lens), blocks or max(1, max(need))), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        bt[b, :n] = perm[at:at + n]
        at += n
    k, v = torch.randn((2, pages, hkv, PAGE, d), generator=gen).to(dt)
    w = torch.rand((pages, hkv, PAGE), generator=gen)
    if fill is not None:
        used = torch.zeros((pages, PAGE), dtype=torch.bool)
        for b, t in enumerate(lens):
            pos = torch.arange(t)
            used[bt[b, pos // PAGE].long(), pos % PAGE] = True
        for x in (k, v):
            x.masked_fill_(~used[:, None, :, None], fill)
    return k, v, w, bt, torch.tensor(lens, dtype=torch.int32)


def places(bt, b, pos):
    return bt[b, pos // PAGE].long(), pos % PAGE


def rows(x, bt, b, t):
    """The first t rows of sequence b, float64 [Hkv, t, ...]."""
    page, slot = places(bt, b, torch.arange(t))
    return x[page, :, slot].transpose(0, 1).double()


def attention(q, k, seen, scale):
    """q [n, heads, D], k [t, D] of their kv head, seen [n, t] -> probabilities
    [n, heads, t] (rows that see nothing: zeros), l relative to the largest, and a bound of
    a weight's relative error in fp32: the scores' (D / 16 steps of the tensor cores, each
    off by at most 2^-22 of the sum of absolute products, and the scaling's roundings),
    twice, the exponential's and the sums' (2^-20)."""
    s = torch.einsum("nhd,td->nht", q, k) * scale
    size = torch.einsum("nhd,td->nht", q.abs(), k.abs()) * abs(scale)
    s = s.masked_fill(~seen[:, None, :], float("-inf"))
    size = size.masked_fill(~seen[:, None, :], 0.0).amax(-1, keepdim=True) if s.shape[-1] else size
    top = s.amax(-1, keepdim=True) if s.shape[-1] else torch.zeros(s.shape[:2] + (1,))
    e = torch.where(seen[:, None, :], (s - torch.where(torch.isinf(top), 0.0, top)).exp(), 0.0)
    l = e.sum(-1, keepdim=True)
    p = e / torch.where(l > 0, l, 1.0)
    err = 2 * (q.shape[-1] / 16 * 2.0 ** -22 + 2.0 ** -23) * size + 2.0 ** -20
    return p, l, err


def weighted_decode(q, k, v, w, bt, ctx, scale, fresh):
    """(out, its bound, weights, their bound); bounds are infinite where nothing is written
    (weights there keep their bits)."""
    B, hq, d = q.shape
    hkv = k.shape[1]
    G = hq // hkv
    out, bound = torch.zeros(q.shape).double(), torch.zeros(q.shape).double()
    new, wb = w.double().clone(), torch.zeros(w.shape).double()
    for b, t in enumerate(ctx.tolist()):
        if t == 0:
            continue
        kk, vv = rows(k, bt, b, t), rows(v, bt, b, t)
        page, slot = places(bt, b, torch.arange(t))
        keep = torch.arange(t) < t - fresh
        adds = 2 * H32 * (t / PAGE + 16)   # of the sums over pages, partial states, heads
        for g in range(hkv):
            p, _, err = attention(q[b, g * G:(g + 1) * G].double()[None], kk[g],
                                  torch.ones((1, t), dtype=torch.bool), scale)
            out[b, g * G:(g + 1) * G] = p[0] @ vv[g]
            bound[b, g * G:(g + 1) * G] = (err[0] + adds) * (p[0] @ vv[g].abs())
            old = torch.where(keep, w[page, g, slot].double(), 0.0)
            add = p[0].sum(0)
            new[page, g, slot] = old + add
            wb[page, g, slot] = ((err[0] + adds) * p[0]).sum(0) + 2 * H32 * (old.abs() + add)
    return out, bound + 1e-30, new, wb


def chunk_weights(q, k, w, bt, ctx, scale, fresh):
    """(weights, bound) after a chunk's queries q [B, n, hq, D]."""
    B, n, hq, d = q.shape
    hkv = k.shape[1]
    G = hq // hkv
    new, wb = w.double().clone(), torch.zeros(w.shape).double()
    for b, c in enumerate(ctx.tolist()):
        t = c + n
        kk = rows(k, bt, b, t)
        page, slot = places(bt, b, torch.arange(t))
        keep = torch.arange(t) < t - fresh
        seen = torch.arange(t)[None, :] <= c + torch.arange(n)[:, None]
        for g in range(hkv):
            qq = q[b, :, g * G:(g + 1) * G].double()
            p, l, err = attention(qq, kk[g], seen, scale)
            # -(m + log2 l) in one fp32 number, and s - that: half a step of each
            s = torch.einsum("nhd,td->nht", qq, kk[g]) * scale
            lse = (s.masked_fill(~seen[:, None, :], 0.0).abs().amax(-1, keepdim=True) + l.log().abs())
            err = err + 4 * H32 * lse + 2 * H32 * (n * G / 4 + 16)
            old = torch.where(keep, w[page, g, slot].double(), 0.0)
            add = p.sum((0, 1))
            new[page, g, slot] = old + add
            wb[page, g, slot] = (err * p).sum((0, 1)) + 2 * H32 * (old.abs() + add)
    return new, wb


def tree(q, k, v, bt, ctx, seen, scale):
    """(out, bound) of drafted tokens; seen [B, n, n] bool.  The bound: the result's rounding
    and the weights', half a step of q's type each, fp16's subnormal weights, fp32's part."""
    B, n, hq, d = q.shape
    hkv = k.shape[1]
    G = hq // hkv
    half = torch.finfo(q.dtype).eps / 2
    out, bound = torch.zeros(q.shape).double(), torch.zeros(q.shape).double()
    for b, c in enumerate(ctx.tolist()):
        t = c + n
        kk, vv = rows(k, bt, b, t), rows(v, bt, b, t)
        vis = torch.cat((torch.ones((n, c), dtype=torch.bool), seen[b]), 1)
        for g in range(hkv):
            # (what a query does not see takes no part, whatever it holds)
            kg = torch.nan_to_num(kk[g], 0.0, 0.0, 0.0)
            p, l, err = attention(q[b, :, g * G:(g + 1) * G].double(), kg, vis, scale)
            vg = torch.nan_to_num(vv[g], 0.0, 0.0, 0.0)
            o = torch.einsum("nht,td->nhd", p, vg)
            size = torch.einsum("nht,td->nhd", p, vg.abs())
            out[b, :, g * G:(g + 1) * G] = o
            sub = 2.0 ** -25 * torch.einsum("nt,td->nd", vis.double(), vg.abs())[:, None]
            bound[b, :, g * G:(g + 1) * G] = (half * o.abs() + (half * 1.01 + err + 2 * H32 * (t / 128 + 32)) * size
                                              + sub / torch.where(l > 0, l, 1.0))
    return out, bound + torch.finfo(q.dtype).smallest_normal * half


def bits(seen):
    """[B, n, n] bool -> the masks' words, int32 [B, n, ceil(n / 32)]."""
    B, n, _ = seen.shape
    words = -(-n // 32)
    full = torch.zeros((B, n, words * 32), dtype=torch.int64)
    full[..., :n] = seen
    word = (full.view(B, n, words, 32) << torch.arange(32)).sum(-1)
    return torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)


def keep_list(w, t, budget, sink, recent):
    """Positions that a row w of weights [t] keeps: heaviest first, ties to the lowest, NaN
    behind every number."""
    if t <= budget:
        return torch.arange(t)
    lo, hi, need = sink, t - recent, budget - sink - recent
    c = w[lo:hi].double() + 0.0
    key = torch.where(torch.isnan(c), float("-inf"), c)
    order = sorted(range(hi - lo), key=lambda i: (bool(torch.isnan(c[i])), -key[i].item(), i)) \
        if hi - lo < 3000 else _order(c)
    chosen = torch.tensor(sorted(order[:need]), dtype=torch.int64) + lo
    return torch.cat((torch.arange(lo), chosen, torch.arange(hi, t)))


def _order(c):
    nan = torch.isnan(c)
    return torch.where(nan, float("-inf"), c).sort(dim=0, descending=True, stable=True).indices.tolist()


def evict(k, v, w, bt, dst, ctx, budget, sink, recent):
    """(k, v, weights, lengths) after the eviction: copies, moved bit for bit."""
    k2, v2, w2 = k.clone(), v.clone(), w.clone()
    lens = []
    for b, t in enumerate(ctx.tolist()):
        lens.append(min(t, budget))
        page, slot = places(bt, b, torch.arange(t))
        for h in range(k.shape[1]):
            src = keep_list(w[page, h, slot], t, budget, sink, recent)
            sp, sl = places(bt, b, src)
            dp, dl = places(dst, b, torch.arange(len(src)))
            k2[dp, h, dl], v2[dp, h, dl], w2[dp, h, dl] = k[sp, h, sl], v[sp, h, sl], w[sp, h, sl]
    return k2, v2, w2, torch.tensor(lens, dtype=torch.int32)
