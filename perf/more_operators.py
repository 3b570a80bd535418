"""Cases of two things a serving loop does around the paged cache's attention:
evicting tokens by the attention weight they have gathered, and verifying a tree
of drafted tokens.

    decode_weighted   one decode step that also adds, for every cached token and kv
                      head, the attention weight the step's queries gave it
    prefill_weights   the same sums over the queries of a chunk (or of the last part
                      of a prompt)
    evict_kv          of every sequence and kv head the first tokens, the most recent
                      ones and the heaviest others stay; their rows move together
    prefill_tree      attention of a tree of drafted tokens over the cache and over
                      each one's ancestors in the tree
    compact_kv        the rows of the accepted branch move behind the cached tokens

The plain forms below say what each computes, in elementary torch operations.

Caches are [pages][kv heads][16 tokens][head_dim]; a token's gathered weight lies at
the same place of a float32 pool [pages][kv heads][16].  Query head h reads kv head
h / (query heads / kv heads).
"""
import math
import random

import torch

own = False

PAGE = 16
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
SCRATCH = 64 << 20  # bytes a serving program sets aside for split attention


# --------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step, the latency case: one short multi-head sequence
        {"name": "decode_weighted_b1_ctx512", "op": "decode_weighted", "batch": 1, "lo": 512,
         "hi": 512, "hq": 16, "hkv": 16, "d": 128, "q_mul": 1.0, "dtype": "bf16"},
        # the ragged grouped-query batch: 64 sequences of 128 to 8192 tokens
        {"name": "decode_weighted_b64_ragged", "op": "decode_weighted", "batch": 64, "lo": 128,
         "hi": 8192, "hq": 32, "hkv": 8, "d": 128, "q_mul": 2.0, "dtype": "bf16"},
        # few long contexts, eight query heads a kv head
        {"name": "decode_weighted_b4_ctx32k", "op": "decode_weighted", "batch": 4, "lo": 32768,
         "hi": 32768, "hq": 64, "hkv": 8, "d": 128, "q_mul": 1.0, "dtype": "fp16"},
        # a prompt's chunk: 512 queries over 8192 cached tokens
        {"name": "prefill_weights_512over8192", "op": "prefill_weights", "batch": 4, "new": 512,
         "lo": 8192, "hi": 8192, "hq": 32, "hkv": 8, "d": 128, "q_mul": 1.0, "dtype": "bf16"},
        # the last 33 queries of long prompts, which say what the answer will look at
        {"name": "prefill_weights_33over32k", "op": "prefill_weights", "batch": 2, "new": 33,
         "lo": 32000, "hi": 32735, "hq": 64, "hkv": 8, "d": 128, "q_mul": 2.0, "dtype": "fp16"},
        # a batch that has outgrown its budget, into pages of its own
        {"name": "evict_b32_to2048", "op": "evict", "batch": 32, "lo": 2000, "hi": 4096,
         "budget": 2048, "sink": 4, "recent": 512, "hkv": 8, "d": 128, "dtype": "bf16"},
        # one long context cut to an eighth
        {"name": "evict_b1_32k_to4096", "op": "evict", "batch": 1, "lo": 32768, "hi": 32768,
         "budget": 4096, "sink": 4, "recent": 256, "hkv": 8, "d": 128, "dtype": "fp16"},
        # a small tree over one short sequence: the latency case of a verify step
        {"name": "tree_b1_26over1000", "op": "tree", "batch": 1, "new": 26, "lo": 1000,
         "hi": 1000, "hq": 32, "hkv": 8, "d": 128, "q_mul": 1.0, "dtype": "bf16"},
        # 60 drafted tokens for each of 16 sequences of 500 to 8000 tokens
        {"name": "tree_b16_60_ragged", "op": "tree", "batch": 16, "new": 60, "lo": 500,
         "hi": 8000, "hq": 32, "hkv": 8, "d": 128, "q_mul": 2.0, "dtype": "fp16"},
        # 64 drafted tokens over long contexts, eight query heads a kv head
        {"name": "tree_b4_64over32k", "op": "tree", "batch": 4, "new": 64, "lo": 32768,
         "hi": 32768, "hq": 64, "hkv": 8, "d": 128, "q_mul": 1.0, "dtype": "bf16"},
        # the accepted branches of a batch's trees
        {"name": "compact_b64_branch", "op": "compact", "batch": 64, "new": 60, "lo": 128,
         "hi": 2048, "keep": 0, "hkv": 8, "d": 128, "weights": False, "dtype": "bf16"},
        # prompts cut to the same half of their tokens for every head, weights too
        {"name": "compact_b4_half_of_8192", "op": "compact", "batch": 4, "new": 8192, "lo": 0,
         "hi": 0, "keep": 4096, "hkv": 8, "d": 128, "weights": True, "dtype": "fp16"},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    hq, hkv = rng.choice([(16, 16), (32, 32), (32, 8), (64, 8), (8, 1), (12, 4), (10, 2),
                          (28, 4), (20, 4), (24, 2), (7, 1), (33, 11)])
    c = {"op": rng.choice(["decode_weighted", "prefill_weights", "evict", "tree", "compact"]),
         "hq": hq, "hkv": hkv, "d": rng.choice([64, 128]), "dtype": rng.choice(["bf16", "fp16"])}
    rows = 4 * 32768 * 8 * 128 // (hkv * c["d"])   # cached tokens of the largest listed case
    if c["op"] == "decode_weighted":
        c["batch"] = _log(rng, 1, 64)
        c["hi"] = _log(rng, 1, min(32768, max(1, rows // c["batch"])))
        c["lo"] = rng.choice([0, c["hi"] // 3, c["hi"]])
        c["q_mul"] = rng.choice([1.0, 2.0])
    elif c["op"] in ("prefill_weights", "tree"):
        c["new"] = _log(rng, 1, 1024 if c["op"] == "prefill_weights" else 256)
        c["batch"] = _log(rng, 1, 16)
        pairs = 4 * 64 * 32832 * 64 * 128 // (c["batch"] * c["new"] * hq * c["d"])
        most = min(32768, pairs - c["new"], rows // c["batch"])
        if most < 1:
            c["batch"], most = 1, 1024
        c["hi"] = rng.choice([0, _log(rng, 1, most)])
        c["lo"] = rng.choice([0, c["hi"] // 2, c["hi"]])
        c["q_mul"] = rng.choice([1.0, 2.0])
    elif c["op"] == "evict":
        c["batch"] = _log(rng, 1, 64)
        c["hi"] = _log(rng, 1, min(32768, max(1, rows // c["batch"])))
        c["lo"] = rng.choice([0, c["hi"] // 2, c["hi"]])
        c["budget"] = _log(rng, 1, c["hi"])
        c["sink"] = min(c["budget"], rng.choice([0, 1, 4]))
        c["recent"] = rng.choice([0, (c["budget"] - c["sink"]) // 3, c["budget"] - c["sink"]])
    else:
        c["batch"] = _log(rng, 1, 64)
        c["new"] = _log(rng, 1, min(8192, max(1, rows // c["batch"])))
        c["hi"] = _log(rng, 1, 2048)
        c["lo"] = rng.choice([0, c["hi"]])
        c["keep"] = rng.choice([0, c["new"] // 2, c["new"]])
        c["weights"] = rng.random() < 0.5
    return c


def _lengths(case):
    """Cached tokens of each sequence: a property of the case."""
    r = random.Random(case["batch"] * 1000003 + case["lo"] * 1009 + case["hi"])
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    n[-1] = case["hi"]
    return n


def _trees(case):
    """Parent of every drafted token (-1: the last cached token): a property of the
    case.  A parent comes before its children."""
    r = random.Random(case["batch"] * 7919 + case["new"] * 31 + case["hi"])
    return [[-1 if i == 0 else r.randint(max(-1, i - 9), i - 1) for i in range(case["new"])]
            for _ in range(case["batch"])]


def _kept(case):
    """Ascending positions, counted from the first of the case's `new` tokens, that
    each sequence keeps: `keep` of them, or one branch of its tree."""
    if case["keep"]:
        r = random.Random(case["new"] * 131 + case["keep"])
        return [sorted(r.sample(range(case["new"]), case["keep"])) for _ in range(case["batch"])]
    kept = []
    r = random.Random(case["batch"] * 17 + case["new"])
    for parents in _trees(case):
        at, branch = r.randrange(-1, case["new"]), []
        while at >= 0:
            branch.append(at)
            at = parents[at]
        kept.append(branch[::-1])
    return kept


# -------------------------------------------------------------------- inputs

def _table(lengths, gen, dev, spare=3, first=0):
    """Block table over a shuffled pool; unmapped entries are -1."""
    blocks = [max(0, -(-t // PAGE)) for t in lengths]
    pages = sum(blocks) + spare
    perm = first + torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    width = max(1, max(blocks))
    bt = torch.full((len(lengths), width), -1, dtype=torch.int32, device=dev)
    n = torch.tensor(blocks, device=dev)
    mask = torch.arange(width, device=dev)[None, :] < n[:, None]
    bt[mask] = perm[:sum(blocks)]
    return bt, pages


def _normal(shape, dt, gen, dev):
    """N(0, 1), drawn a part at a time."""
    x = torch.empty(shape, dtype=dt, device=dev)
    flat = x.view(-1)
    for at in range(0, flat.numel(), 1 << 26):
        part = flat[at:at + (1 << 26)]
        part.copy_(torch.randn(part.shape, generator=gen, device=dev))
    return x


def _gathered(pages, hkv, gen, dev):
    """Weights as attention leaves them: most small, a few large; an eighth zero."""
    w = torch.randn((pages, hkv, PAGE), generator=gen, device=dev).mul_(2).exp_().mul_(0.01)
    return w * (torch.rand(w.shape, generator=gen, device=dev) > 0.125)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt, d, hkv, op = DTYPES[case["dtype"]], case["d"], case["hkv"], case["op"]
    lens, batch, new = _lengths(case), case["batch"], case.get("new", 0)
    held = [t + new for t in lens]
    s = {"op": op, "d": d, "dt": dt, "hkv": hkv, "hq": case["hq"] if "hq" in case else hkv}
    s["bt"], pages = _table(held, gen, dev)
    s["ctx"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    if op == "evict":
        s.update(budget=case["budget"], sink=case["sink"], recent=case["recent"])
        s["dst"], more = _table([min(t, case["budget"]) for t in lens], gen, dev, first=pages)
        pages += more
    s["kc"] = _normal((pages, hkv, PAGE, d), dt, gen, dev)
    if op != "prefill_weights":
        s["vc"] = _normal((pages, hkv, PAGE, d), dt, gen, dev)
    if op != "tree" and (op != "compact" or case["weights"]):
        s["weights"] = _gathered(pages, hkv, gen, dev)
    if op == "evict" or op == "compact":
        s["lens"] = torch.empty(batch, dtype=torch.int32, device=dev)
        s["scratch"] = torch.empty(SCRATCH, dtype=torch.uint8, device=dev)
    if op == "compact":
        kept = _kept(case)
        s["n_keep"] = torch.tensor([len(k) for k in kept], dtype=torch.int32, device=dev)
        width = max(1, max(len(k) for k in kept))
        s["keep"] = torch.tensor([k + [-1] * (width - len(k)) for k in kept], dtype=torch.int32,
                                 device=dev)
        return s
    if op == "evict":
        return s
    s["scale"] = 1.0 / math.sqrt(d)
    rows = (batch, case["hq"], d) if op == "decode_weighted" else (batch, new, case["hq"], d)
    s["q"] = (torch.randn(rows, generator=gen, device=dev) * case["q_mul"]).to(dt)
    # a decode result stays fp32 as the library's other decodes give it; a chunk's
    # rows come in q's type
    s["out"] = torch.empty(rows, dtype=dt if op == "tree" else torch.float32, device=dev)
    scores = 4 * batch * case["hq"] * s["bt"].shape[1] * PAGE if op == "decode_weighted" else 0
    s["scratch"] = torch.empty(SCRATCH + scores, dtype=torch.uint8, device=dev)
    if op == "tree":
        parents = torch.tensor(_trees(case), device=dev)
        seen = torch.eye(new, dtype=torch.bool, device=dev).repeat(batch, 1, 1)
        for i in range(1, new):  # a token sees what its parent sees, and itself
            p = parents[:, i]
            up = seen[torch.arange(batch, device=dev), p.clamp(min=0)]
            seen[:, i] |= up & (p >= 0)[:, None]
        words = -(-new // 32)
        bits = torch.zeros((batch, new, words * 32), dtype=torch.int64, device=dev)
        bits[..., :new] = seen
        word = (bits.view(batch, new, words, 32) << torch.arange(32, device=dev)).sum(-1)
        s["mask"] = torch.where(word >= 1 << 31, word - (1 << 32), word).to(torch.int32)
    return s


# --------------------------------------------------------------- plain forms

def _rows(pool, bt):
    """[pages, Hkv, 16, ...] through a block table -> [B, Hkv, tokens, ...]."""
    x = pool[bt.clamp(min=0).long()].movedim(2, 1)   # [B, Hkv, blocks, 16, ...]
    return x.flatten(2, 3)


def _probabilities(s, seen):
    """softmax(q K^T scale) over the keys that `seen` [B, queries, keys] allows:
    [B, Hkv, queries, group, keys], and the sums' rows without a key as zeros."""
    hkv, d = s["hkv"], s["d"]
    q = s["q"] if s["q"].dim() == 4 else s["q"][:, None]
    b, nq, hq = q.shape[:3]
    k = _rows(s["kc"], s["bt"]).float()
    qg = q.float().view(b, nq, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
    score = (qg @ k.transpose(-1, -2)).mul_(s["scale"]).view(b, hkv, nq, hq // hkv, -1)
    score.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    top = score.amax(-1, keepdim=True)
    w = score.sub_(torch.where(torch.isinf(top), 0.0, top)).exp_()
    total = w.sum(-1, keepdim=True)
    return w.div_(torch.where(total > 0, total, 1.0))


def _times_v(s, p):
    v = _rows(s["vc"], s["bt"]).float()
    v = v.masked_fill_(~(p > 0).any(3).any(2)[..., None], 0.0)
    b, hkv, nq, group, keys = p.shape
    o = (p.view(b, hkv, -1, keys) @ v).view(b, hkv, nq, group, s["d"])
    return o.permute(0, 2, 1, 3, 4).reshape(b, nq, -1, s["d"])


def _gather_weights(s, p, tokens, fresh):
    """Adds the sums of p over queries and heads to the pool: the last `fresh` of a
    sequence's tokens start from nothing."""
    add = p.sum((2, 3))                                          # [B, Hkv, keys]
    at = torch.arange(add.shape[-1], device=add.device)
    b, t = (at[None, :] < tokens[:, None]).nonzero(as_tuple=True)
    page, slot = s["bt"][b, t // PAGE].long(), t % PAGE
    old = torch.where((t < tokens[b] - fresh)[:, None], s["weights"][page, :, slot], 0.0)
    s["weights"][page, :, slot] = old + add[b, :, t]


def _move(s, b, src, dst, heads, table):
    """Rows of sequence b at positions src to positions dst of `table`: one head each,
    or all heads where `heads` is None."""
    sp, sl = s["bt"][b, src // PAGE].long(), src % PAGE
    dp, dl = table[b, dst // PAGE].long(), dst % PAGE
    for name in ("kc", "vc", "weights"):
        pool = s.get(name)
        if pool is None:
            continue
        if heads is None:
            pool[dp, :, dl] = pool[sp, :, sl].clone()
        else:
            pool[dp, heads, dl] = pool[sp, heads, sl].clone()


def _plain_evict(s):
    w = _rows(s["weights"], s["bt"])                             # [B, Hkv, keys]
    length = s["ctx"].long()[:, None, None]
    t = torch.arange(w.shape[-1], device=w.device)
    stays = (t < s["sink"]) | (t >= length - s["recent"])
    rank = torch.where(stays, float("inf"), w).masked_fill(t >= length, -1.0)
    order = rank.sort(dim=-1, descending=True, stable=True).indices
    n = s["ctx"].clamp(max=s["budget"])
    j = torch.arange(min(s["budget"], w.shape[-1]), device=w.device)
    kept = torch.where(j < n[:, None, None], order[..., :j.numel()], 1 << 40).sort(-1).values
    b, h, to = (kept < 1 << 40).nonzero(as_tuple=True)
    _move(s, b, kept[b, h, to], to, h, s["dst"])
    s["lens"].copy_(n)


def _plain_compact(s):
    j = torch.arange(s["keep"].shape[1], device=s["keep"].device)
    b, to = (j[None, :] < s["n_keep"][:, None]).nonzero(as_tuple=True)
    first = s["ctx"].long()[b]
    _move(s, b, first + s["keep"].long()[b, to], first + to, None, s["bt"])
    torch.add(s["ctx"], s["n_keep"], out=s["lens"])


def _tree_seen(s, keys):
    """[B, queries, keys]: the cached tokens, and the drafted ones whose bit is set."""
    b, n = s["q"].shape[:2]
    at = torch.arange(keys, device=s["q"].device)[None, :] - s["ctx"].long()[:, None]
    bit = at.clamp(0, n - 1)[:, None, :].expand(b, n, keys)
    word = s["mask"].long().gather(2, bit // 32)
    drafted = (word >> (bit % 32)) & 1 == 1
    return (at < 0)[:, None, :] | (drafted & (at < n)[:, None, :])


def _moved(s):
    out = {"k_cache": s["kc"], "v_cache": s["vc"], "lens": s["lens"]}
    if "weights" in s:
        out["weights"] = s["weights"]
    return out


def run(state):
    s = state
    op = s["op"]
    if own:
        import paged_kv_cache_171_gb300 as pa
        if op == "decode_weighted":
            pa.decode_weighted(s["q"], s["kc"], s["vc"], s["weights"], s["bt"], s["ctx"],
                               s["scale"], out=s["out"], workspace=s["scratch"])
            return {"out": s["out"], "weights": s["weights"]}
        if op == "prefill_weights":
            pa.prefill_weights(s["q"], s["kc"], s["weights"], s["bt"], s["ctx"], s["scale"],
                               workspace=s["scratch"])
            return {"weights": s["weights"]}
        if op == "evict":
            pa.evict_kv(s["kc"], s["vc"], s["weights"], s["bt"], s["ctx"], s["budget"],
                        sink=s["sink"], recent=s["recent"], dst_table=s["dst"],
                        new_lens=s["lens"], workspace=s["scratch"])
            return _moved(s)
        if op == "tree":
            return pa.prefill_tree(s["q"], s["kc"], s["vc"], s["bt"], s["ctx"], s["mask"],
                                   s["scale"], out=s["out"], workspace=s["scratch"])
        pa.compact_kv(s["kc"], s["vc"], s["bt"], s["ctx"], s["keep"], s["n_keep"],
                      weights=s.get("weights"), new_lens=s["lens"])
        return _moved(s)
    keys = s["bt"].shape[1] * PAGE
    at = torch.arange(keys, device=s["bt"].device)
    if op == "decode_weighted":
        tokens = s["ctx"].long()
        p = _probabilities(s, at < tokens[:, None, None])
        _gather_weights(s, p, tokens, 1)
        return {"out": _times_v(s, p)[:, 0].contiguous(), "weights": s["weights"]}
    if op == "prefill_weights":
        n = s["q"].shape[1]
        last = s["ctx"].long()[:, None] + torch.arange(n, device=at.device)
        p = _probabilities(s, at <= last[:, :, None])
        _gather_weights(s, p, s["ctx"].long() + n, n)
        return {"weights": s["weights"]}
    if op == "tree":
        return _times_v(s, _probabilities(s, _tree_seen(s, keys))).to(s["dt"])
    if op == "evict":
        _plain_evict(s)
    else:
        _plain_compact(s)
    return _moved(s)


def work(case):
    d, hkv, op = case["d"], case["hkv"], case["op"]
    lens, new = _lengths(case), case.get("new", 0)
    row = 2 * d                      # bytes of one 16-bit row
    if op == "decode_weighted":
        q = case["batch"] * case["hq"] * d * 6
        return {"bytes": sum(lens) * hkv * (2 * row + 8) + q, "flops": 4 * sum(lens) * case["hq"] * d}
    if op == "prefill_weights":
        pairs = sum(new * t + new * (new + 1) // 2 for t in lens)
        q = case["batch"] * new * case["hq"] * row
        return {"bytes": sum(t + new for t in lens) * hkv * (row + 8) + q,
                "flops": 2 * pairs * case["hq"] * d}
    if op == "tree":
        pairs = 0
        for t, parents in zip(lens, _trees(case)):
            depth = []
            for p in parents:
                depth.append(1 if p < 0 else depth[p] + 1)
            pairs += new * t + sum(depth)
        q = case["batch"] * new * case["hq"] * row
        return {"bytes": sum(t + new for t in lens) * hkv * 2 * row + 2 * q,
                "flops": 4 * pairs * case["hq"] * d}
    if op == "evict":
        n = sum(min(t, case["budget"]) for t in lens)
        return {"bytes": hkv * (4 * sum(lens) + n * (4 * row + 8)), "flops": hkv * sum(lens)}
    n = sum(len(k) for k in _kept(case))
    return {"bytes": n * (hkv * (4 * row + (8 if case["weights"] else 0)) + 4) + 12 * case["batch"],
            "flops": 0}


# ------------------------------------------------- the definition in 64 bits

def _sequence(pool, bt, b, tokens):
    """The first `tokens` rows of sequence b in 64 bits: [Hkv, tokens, ...]."""
    pages = bt[b, :-(-tokens // PAGE)].long()
    x = pool[pages].transpose(0, 1).double()
    return x.reshape(x.shape[0], -1, *x.shape[3:])[:, :tokens]


def _exact_attention(s, case):
    """out (or None) and weights (or None) by one sequence and kv head at a time."""
    op, hkv, d = s["op"], s["hkv"], s["d"]
    q = s["q"] if s["q"].dim() == 4 else s["q"][:, None]
    n, group, new = q.shape[1], s["hq"] // hkv, case.get("new", 0)
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    weights = s["weights"].double() if "weights" in s else None
    for b, ctx in enumerate(s["ctx"].tolist()):
        held = ctx + new
        if held == 0:
            continue
        hidden = None
        if op != "decode_weighted":
            hidden = torch.zeros((n, held), dtype=torch.bool, device=q.device)
            if op == "tree":
                row = torch.arange(new, device=q.device)
                hidden[:, ctx:] = (s["mask"][b].long()[:, row // 32] // 2 ** (row % 32)) % 2 == 0
            else:
                hidden[:, ctx:] = torch.ones((n, new), device=q.device).triu(1) > 0
        k = _sequence(s["kc"], s["bt"], b, held)
        v = _sequence(s["vc"], s["bt"], b, held) if "vc" in s else None
        t = torch.arange(held, device=q.device)
        page, slot = s["bt"][b, t // PAGE].long(), t % PAGE
        fresh = t >= held - max(1, new)
        for g in range(hkv):
            heads = slice(g * group, (g + 1) * group)
            score = torch.einsum("nhd,td->nht", q[b, :, heads].double(), k[g]) * s["scale"]
            if hidden is not None:
                score.masked_fill_(hidden[:, None, :], float("-inf"))
            p = score.softmax(-1)
            if v is not None:
                out[b, :, heads] = torch.einsum("nht,td->nhd", p, v[g])
            if weights is not None:
                kept = weights[page, g, slot]
                kept[fresh] = 0.0
                weights[page, g, slot] = kept + p.sum((0, 1))
    return out, weights


def _exact_evict(s):
    k, v, w = s["kc"].double(), s["vc"].double(), s["weights"].double()
    old = [k.clone(), v.clone(), w.clone()]
    lens = []
    for b, ctx in enumerate(s["ctx"].tolist()):
        n = min(ctx, s["budget"])
        lens.append(n)
        if n == 0:
            continue
        t = torch.arange(ctx, device=k.device)
        held = _sequence(s["weights"], s["bt"], b, ctx)
        j = torch.arange(n, device=k.device)
        to, slot = s["dst"][b, j // PAGE].long(), j % PAGE
        lo, hi = s["sink"], ctx - s["recent"]
        for h in range(s["hkv"]):
            stays = torch.ones(ctx, dtype=torch.bool, device=k.device)
            if n < ctx:
                others, more = held[h, lo:hi], n - s["sink"] - s["recent"]
                chosen = torch.zeros_like(others, dtype=torch.bool)
                if more > 0:
                    least = others.topk(more).values[-1]
                    chosen = others > least
                    ties = (others == least).nonzero()[:, 0]
                    chosen[ties[:more - int(chosen.sum())]] = True
                stays[lo:hi] = chosen
            src = t[stays]
            page = s["bt"][b, src // PAGE].long()
            for new, was in zip((k, v, w), old):
                new[to, h, slot] = was[page, h, src % PAGE]
    lens = torch.tensor(lens, dtype=torch.int32, device=k.device)
    return {"k_cache": k, "v_cache": v, "weights": w, "lens": lens}


def _exact_compact(s):
    pools = {"k_cache": s["kc"].double(), "v_cache": s["vc"].double()}
    if "weights" in s:
        pools["weights"] = s["weights"].double()
    was = {name: pool.clone() for name, pool in pools.items()}
    lens = []
    for b, (ctx, n) in enumerate(zip(s["ctx"].tolist(), s["n_keep"].tolist())):
        src = ctx + s["keep"][b, :n].long()
        dst = torch.arange(ctx, ctx + n, device=src.device)
        lens.append(ctx + n)
        for name, pool in pools.items():
            pool[s["bt"][b, dst // PAGE].long(), :, dst % PAGE] = \
                was[name][s["bt"][b, src // PAGE].long(), :, src % PAGE]
    return {**pools, "lens": torch.tensor(lens, dtype=torch.int32, device=s["ctx"].device)}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "evict":
        return _exact_evict(s)
    if s["op"] == "compact":
        return _exact_compact(s)
    out, weights = _exact_attention(s, case)
    if s["op"] == "tree":
        return out
    if s["op"] == "prefill_weights":
        return {"weights": weights}
    return {"out": out[:, 0], "weights": weights}
