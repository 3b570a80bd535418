"""Cases of the paged cache's rotated append and of the 4-bit paged cache: the
append that rotates (into the 16-bit cache, and quantising into the 4-bit
one), the read that turns stored rows back into values, and the decode and
prefill attention over the 4-bit cache.

The plain forms below say what each computes, in elementary torch operations.

A 4-bit block holds one (page, kv head): 16 tokens of K and of V.
    bytes [0, 16 D)        codes, [K, V][16 tokens][D / 2]; dimension 2i in the
                           low four bits of byte i, 2i + 1 in the high four
    bytes [16 D, 16 D+128) [K, V][16 tokens][scale, zero], 16-bit floats
and stands for x = zero + scale * (code - 8).
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
        # one decode step of a 64-sequence batch: every sequence's new token,
        # K and V as views of one fused projection's output, q rotated too
        {"name": "rope_step_b64", "op": "rope", "batch": 64, "new": 1, "lo": 128, "hi": 2048,
         "hq": 32, "hkv": 8, "d": 128, "rot": 128, "inter": False, "dtype": "bf16"},
        # the rows of a chunked prefill: 4 sequences x 512 tokens
        {"name": "rope_chunk_4x512", "op": "rope", "batch": 4, "new": 512, "lo": 1000, "hi": 8192,
         "hq": 32, "hkv": 8, "d": 128, "rot": 128, "inter": False, "dtype": "bf16"},
        # a long prompt at head_dim 64, adjacent pairs, half of the dimensions
        # rotated, multi-head
        {"name": "rope_prompt_8191_part", "op": "rope", "batch": 1, "new": 8191, "lo": 0, "hi": 0,
         "hq": 16, "hkv": 16, "d": 64, "rot": 32, "inter": True, "dtype": "fp16"},
        # a decode step into the 4-bit cache, and the rows read back
        {"name": "store4_step_b64", "op": "store4", "batch": 64, "new": 1, "lo": 128, "hi": 2048,
         "hq": 32, "hkv": 8, "d": 128, "rot": 128, "inter": False, "dtype": "bf16"},
        # a prompt stored in 4 bits: 4 sequences x 2048 tokens
        {"name": "store4_prompt_4x2048", "op": "store4", "batch": 4, "new": 2048, "lo": 0, "hi": 77,
         "hq": 32, "hkv": 8, "d": 128, "rot": 128, "inter": False, "dtype": "fp16"},
        # the contexts of 16 sequences turned back into 16-bit rows (to move
        # them into a 16-bit cache)
        {"name": "read4_16x1000", "op": "read4", "batch": 16, "lo": 500, "hi": 1500,
         "hq": 32, "hkv": 8, "d": 128, "dtype": "bf16"},
        # decode attention: the latency case, one short sequence
        {"name": "decode4_b1_ctx512", "op": "decode4", "batch": 1, "lo": 512, "hi": 512,
         "hq": 16, "hkv": 16, "d": 128, "q_mul": 1.0, "dtype": "bf16"},
        # multi-head decode, 8 x 4096
        {"name": "decode4_mha_b8_ctx4096", "op": "decode4", "batch": 8, "lo": 4096, "hi": 4096,
         "hq": 32, "hkv": 32, "d": 128, "q_mul": 1.0, "dtype": "fp16"},
        # the ragged grouped-query batch (64 sequences of 128 to 8192 tokens)
        {"name": "decode4_gqa4_b64_ragged", "op": "decode4", "batch": 64, "lo": 128, "hi": 8192,
         "hq": 32, "hkv": 8, "d": 128, "q_mul": 2.0, "dtype": "bf16"},
        # few long contexts, eight query heads a kv head
        {"name": "decode4_gqa8_b4_ctx32k", "op": "decode4", "batch": 4, "lo": 32768, "hi": 32768,
         "hq": 64, "hkv": 8, "d": 128, "q_mul": 1.0, "dtype": "bf16"},
        # speculative verify: 4 drafted tokens over 32k cached ones
        {"name": "prefill4_verify_4over32k", "op": "prefill4", "batch": 4, "new": 4,
         "lo": 32768, "hi": 32768, "hq": 64, "hkv": 8, "d": 128, "q_mul": 1.0, "dtype": "bf16"},
        # chunked prefill: 512 new tokens over 8192 cached ones
        {"name": "prefill4_chunk_512over8192", "op": "prefill4", "batch": 4, "new": 512,
         "lo": 8192, "hi": 8192, "hq": 32, "hkv": 8, "d": 128, "q_mul": 1.0, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    hq, hkv = rng.choice([(16, 16), (32, 32), (32, 8), (64, 8), (8, 1), (12, 4), (10, 2),
                          (28, 4), (20, 4), (24, 2), (7, 1), (33, 11)])
    c = {"op": rng.choice(["rope", "store4", "read4", "decode4", "decode4", "prefill4"]),
         "hq": hq, "hkv": hkv, "d": rng.choice([64, 128]), "dtype": rng.choice(["bf16", "fp16"])}
    width = hkv * c["d"]
    if c["op"] in ("rope", "store4"):
        tokens = _log(rng, 1, min(8192, (8192 * 48 * 128) // ((hq + 2 * hkv) * c["d"])))
        c["batch"] = min(tokens, _log(rng, 1, 64))
        c["new"] = max(1, tokens // c["batch"])
        c["lo"] = rng.choice([0, rng.randrange(2000)])
        c["hi"] = c["lo"] + rng.choice([0, rng.randrange(2000)])
        c["rot"] = rng.choice([c["d"], c["d"], c["d"] // 2, 16, 48])
        c["inter"] = rng.random() < 0.4
    elif c["op"] == "read4":
        c["batch"] = _log(rng, 1, 64)
        most = max(1, 16 * 1000 * 8 * 128 // (width * c["batch"]))
        c["hi"] = _log(rng, 1, min(8192, most))
        c["lo"] = rng.choice([0, c["hi"] // 2, c["hi"]])
    elif c["op"] == "decode4":
        c["batch"] = _log(rng, 1, 64)
        most = max(1, 64 * 4160 * 8 * 128 // (width * c["batch"]))
        c["hi"] = _log(rng, 1, min(32768, most))
        c["lo"] = rng.choice([0, c["hi"] // 3, c["hi"]])
        c["q_mul"] = rng.choice([1.0, 2.0])
    else:
        c["new"] = _log(rng, 1, 1024)
        c["batch"] = _log(rng, 1, 8)
        pairs = 4 * 512 * 8704 * 32 * 128 // (c["batch"] * c["new"] * hq * c["d"])
        keys = 4 * 32768 * 8 * 128 // (c["batch"] * width)
        most = min(32768, pairs - c["new"], keys)
        if most < 1:
            c["batch"], most = 1, 2048
        c["hi"] = rng.choice([0, _log(rng, 1, most)])
        c["lo"] = rng.choice([0, c["hi"] // 2, c["hi"]])
        c["q_mul"] = rng.choice([1.0, 2.0])
    return c


def _lengths(case):
    """Cached tokens of each sequence: a property of the case."""
    r = random.Random(case["batch"] * 1000003 + case["lo"] * 1009 + case["hi"])
    n = [r.randint(case["lo"], case["hi"]) for _ in range(case["batch"])]
    n[-1] = case["hi"]
    return n


# --------------------------------------------------------------- the layout

def _block(d):
    return 16 * d + 128


def _quantise(x, dt):
    """Rows of x (fp32, last axis head_dim) -> codes (uint8), scale, zero (dt)."""
    mn, mx = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    scale = ((mx - mn) * (1.0 / 15.0)).to(dt)
    zero = (mn + 8.0 * scale.float()).to(dt)
    fine = torch.isfinite(scale) & torch.isfinite(zero) & torch.isfinite(mx - mn)
    s, z = scale.float(), zero.float()
    code = torch.where(fine & (s > 0), torch.round((x - z) / s) + 8.0, 8.0).clamp(0, 15)
    nan = torch.full_like(scale, float("nan"))
    return code.to(torch.uint8), torch.where(fine, scale, nan), torch.where(fine, zero, nan)


def _packed(code):
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _blocks_of(k, v, dt):
    """[..., 16, D] K and V values -> [..., block] bytes."""
    lead, d = k.shape[:-2], k.shape[-1]
    kc, ks, kz = _quantise(k, dt)
    vc, vs, vz = _quantise(v, dt)
    codes = torch.stack((_packed(kc), _packed(vc)), -3).reshape(*lead, 16 * d)
    meta = torch.stack((torch.cat((ks, kz), -1), torch.cat((vs, vz), -1)), -3).contiguous()
    return torch.cat((codes, meta.view(torch.uint8).reshape(*lead, 128)), -1)


def _values(blocks, d, dt, wide):
    """[..., block] bytes -> [..., 2 (K, V), 16, D] values in the type `wide`."""
    lead = blocks.shape[:-1]
    byte = blocks[..., :16 * d].reshape(*lead, 2, PAGE, d // 2)
    code = torch.stack((byte & 15, byte >> 4), -1).reshape(*lead, 2, PAGE, d)
    meta = blocks[..., 16 * d:].contiguous().view(dt).reshape(*lead, 2, PAGE, 2).to(wide)
    return meta[..., 1:2] + meta[..., 0:1] * (code.to(wide) - 8)


# -------------------------------------------------------------------- inputs

def _table(lengths, gen, dev):
    """Block table over a shuffled pool; unmapped entries are -1."""
    blocks = [max(0, -(-t // PAGE)) for t in lengths]
    pages = sum(blocks) + 3
    perm = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)
    width = max(1, max(blocks))
    bt = torch.full((len(lengths), width), -1, dtype=torch.int32, device=dev)
    n = torch.tensor(blocks, device=dev)
    mask = torch.arange(width, device=dev)[None, :] < n[:, None]
    bt[mask] = perm[:sum(blocks)]
    return bt, pages


def _rope_table(positions, rot, dev):
    """fp32 [positions][rot]: cos of the rot / 2 angles, then their sin."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    ang = torch.arange(positions, dtype=torch.float64, device=dev)[:, None] * inv[None, :]
    return torch.cat((ang.cos(), ang.sin()), -1).float()


def _random_pool(pages, hkv, d, dt, gen, dev):
    """A 4-bit pool that holds quantised N(0, 1) rows."""
    pool = torch.empty((pages, hkv, _block(d)), dtype=torch.uint8, device=dev)
    step = max(1, (1 << 24) // (hkv * PAGE * d))
    for at in range(0, pages, step):
        n = min(step, pages - at)
        kv = torch.randn((2, n, hkv, PAGE, d), generator=gen, device=dev)
        pool[at:at + n] = _blocks_of(kv[0], kv[1], dt)
    return pool


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    dt, d, hq, hkv = DTYPES[case["dtype"]], case["d"], case["hq"], case["hkv"]
    lens = _lengths(case)
    new = case.get("new", 0)
    s = {"op": case["op"], "d": d, "dt": dt, "hq": hq, "hkv": hkv}
    if case["op"] in ("rope", "store4"):
        held = [t + new for t in lens]
        s["bt"], pages = _table(held, gen, dev)
        n_tok = case["batch"] * new
        qkv = torch.randn((n_tok, hq + 2 * hkv, d), generator=gen, device=dev).to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        first = torch.tensor(lens, device=dev)
        s["seq"] = torch.arange(case["batch"], device=dev).repeat_interleave(new).to(torch.int32)
        s["pos"] = (first[:, None] + torch.arange(new, device=dev)[None, :]).reshape(-1).to(torch.int32)
        s["cos_sin"] = _rope_table(max(held), case["rot"], dev)
        s["rot"], s["inter"] = case["rot"], case["inter"]
        s["q_out"] = torch.empty((n_tok, hq, d), dtype=dt, device=dev)
        if case["op"] == "rope":
            s["kc"] = torch.zeros((pages, hkv, PAGE, d), dtype=dt, device=dev)
            s["vc"] = torch.zeros_like(s["kc"])
        else:
            s["pool"] = torch.zeros((pages, hkv, _block(d)), dtype=torch.uint8, device=dev)
            s["k_out"] = torch.empty((n_tok, hkv, d), dtype=dt, device=dev)
            s["v_out"] = torch.empty_like(s["k_out"])
        return s
    s["bt"], pages = _table([t + new for t in lens], gen, dev)
    s["pool"] = _random_pool(pages, hkv, d, dt, gen, dev)
    if case["op"] == "read4":
        n = torch.tensor(lens, device=dev)
        mask = torch.arange(max(1, max(lens)), device=dev)[None, :] < n[:, None]
        at = mask.nonzero()
        s["seq"], s["pos"] = at[:, 0].to(torch.int32), at[:, 1].to(torch.int32)
        s["k_out"] = torch.empty((at.shape[0], hkv, d), dtype=dt, device=dev)
        s["v_out"] = torch.empty_like(s["k_out"])
        return s
    s["ctx"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    s["scale"] = 1.0 / math.sqrt(d)
    rows = (case["batch"], new, hq, d) if case["op"] == "prefill4" else (case["batch"], hq, d)
    s["q"] = (torch.randn(rows, generator=gen, device=dev) * case["q_mul"]).to(dt)
    # decode results stay fp32 as the library's other decodes give them; a
    # chunk's rows come in q's type
    s["out"] = torch.empty(rows, dtype=dt if case["op"] == "prefill4" else torch.float32, device=dev)
    s["scratch"] = torch.empty(SCRATCH, dtype=torch.uint8, device=dev)
    return s


# --------------------------------------------------------------- plain forms

def _rotated(x, pos, s, wide):
    """x [tokens, heads, D] rotated at each token's position, in the type `wide`."""
    rot = s["rot"]
    cs = s["cos_sin"][pos.long()].to(wide)[:, None, :]
    c, sn = cs[..., :rot // 2], cs[..., rot // 2:]
    x = x.to(wide)
    if s["inter"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    ra, rb = a * c - b * sn, b * c + a * sn
    if s["inter"]:
        return torch.cat((torch.stack((ra, rb), -1).flatten(-2), x[..., rot:]), -1)
    return torch.cat((ra, rb, x[..., rot:]), -1)


def _places(s):
    """(page, slot) of every listed token."""
    page = s["bt"][s["seq"].long(), (s["pos"] // PAGE).long()].long()
    return page, (s["pos"] % PAGE).long()


def _plain_rope(s):
    page, slot = _places(s)
    s["kc"][page, :, slot] = _rotated(s["k"], s["pos"], s, torch.float32).to(s["dt"])
    s["vc"][page, :, slot] = s["v"]
    return {"q": _rotated(s["q"], s["pos"], s, torch.float32).to(s["dt"]),
            "k_cache": s["kc"], "v_cache": s["vc"]}


def _plain_read(s):
    page, slot = _places(s)
    d, dt = s["d"], s["dt"]
    rows = s["pool"].view(-1, s["hkv"], _block(d))
    byte = rows[..., :16 * d].unflatten(-1, (2, PAGE, d // 2))[page, :, :, slot]
    code = torch.stack((byte & 15, byte >> 4), -1).flatten(-2).float()
    meta = rows[..., 16 * d:].contiguous().view(dt).unflatten(-1, (2, PAGE, 2))[page, :, :, slot].float()
    x = (meta[..., 1:2] + meta[..., 0:1] * (code - 8.0)).to(dt)
    return {"k": x[:, :, 0].contiguous(), "v": x[:, :, 1].contiguous()}


def _plain_store(s):
    page, slot = _places(s)
    d, dt = s["d"], s["dt"]
    codes = s["pool"][..., :16 * d].unflatten(-1, (2, PAGE, d // 2))
    metas = s["pool"][..., 16 * d:].unflatten(-1, (2, PAGE, 4))
    k = _rotated(s["k"], s["pos"], s, torch.float32)
    kc, ks, kz = _quantise(k, dt)
    vc, vs, vz = _quantise(s["v"].float(), dt)
    codes[page, :, :, slot] = torch.stack((_packed(kc), _packed(vc)), 2)
    meta = torch.stack((torch.cat((ks, kz), -1), torch.cat((vs, vz), -1)), 2).contiguous()
    metas[page, :, :, slot] = meta.view(torch.uint8).flatten(3)
    return {"q": _rotated(s["q"], s["pos"], s, torch.float32).to(dt), **_plain_read(s)}


def _attention(s, wide, tokens):
    """softmax(q K^T scale) V of every query over its sequence's first `tokens`
    [batch, queries] keys; q [batch, queries, heads, D]."""
    d, dt, hkv = s["d"], s["dt"], s["hkv"]
    q = s["q"] if s["q"].dim() == 4 else s["q"][:, None]
    b, nq, hq = q.shape[:3]
    kv = s["pool"][s["bt"].clamp(min=0).long()]             # [B, blocks, Hkv, block]
    kv = _values(kv, d, dt, wide).permute(3, 0, 2, 1, 4, 5).reshape(2, b, hkv, -1, d)
    qg = q.to(wide).view(b, nq, hkv, hq // hkv, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, -1, d)
    score = (qg @ kv[0].transpose(-1, -2)).mul_(s["scale"]).view(b, hkv, nq, hq // hkv, -1)
    seen = torch.arange(score.shape[-1], device=q.device) < tokens[:, :, None]  # [B, nq, keys]
    score.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    top = score.amax(-1, keepdim=True)
    w = score.sub_(torch.where(torch.isinf(top), 0.0, top)).exp_()
    total = w.sum(-1, keepdim=True)
    o = (w.view(b, hkv, -1, w.shape[-1]) @ kv[1]).view(b, hkv, nq, hq // hkv, d)
    o = torch.where(total > 0, o / total, 0.0)
    return o.permute(0, 2, 1, 3, 4).reshape(b, nq, hq, d)


def _seen(s):
    """Keys each query sees: its sequence's tokens; in a chunk, the cached ones
    and the chunk's up to itself."""
    if s["q"].dim() == 3:
        return s["ctx"][:, None]
    return s["ctx"][:, None] + 1 + torch.arange(s["q"].shape[1], device=s["q"].device)


def run(state):
    s = state
    op = s["op"]
    if own:
        import paged_kv_cache_171_gb300 as pa
        if op == "rope":
            pa.append_kv_rope(s["k"], s["v"], s["kc"], s["vc"], s["bt"], s["seq"], s["pos"],
                              s["cos_sin"], q=s["q"], q_out=s["q_out"], interleaved=s["inter"])
            return {"q": s["q_out"], "k_cache": s["kc"], "v_cache": s["vc"]}
        if op == "store4":
            pa.append_kv4(s["k"], s["v"], s["pool"], s["bt"], s["seq"], s["pos"],
                          cos_sin=s["cos_sin"], q=s["q"], q_out=s["q_out"],
                          interleaved=s["inter"])
            pa.read_kv4(s["pool"], s["bt"], s["seq"], s["pos"], k_out=s["k_out"],
                        v_out=s["v_out"])
            return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
        if op == "read4":
            pa.read_kv4(s["pool"], s["bt"], s["seq"], s["pos"], k_out=s["k_out"],
                        v_out=s["v_out"])
            return {"k": s["k_out"], "v": s["v_out"]}
        if op == "decode4":
            return pa.decode_kv4(s["q"], s["pool"], s["bt"], s["ctx"], s["scale"], out=s["out"],
                                 workspace=s["scratch"])
        return pa.prefill_kv4(s["q"], s["pool"], s["bt"], s["ctx"], s["scale"], out=s["out"],
                              workspace=s["scratch"])
    if op == "rope":
        return _plain_rope(s)
    if op == "store4":
        return _plain_store(s)
    if op == "read4":
        return _plain_read(s)
    o = _attention(s, torch.float32, _seen(s))
    return o[:, 0].contiguous() if op == "decode4" else o.to(s["dt"])


def work(case):
    d, hq, hkv = case["d"], case["hq"], case["hkv"]
    lens = _lengths(case)
    row4 = hkv * 2 * (d // 2 + 4)   # one token's K and V in 4 bits
    row16 = hkv * 2 * d * 2         # in 16
    if case["op"] in ("rope", "store4"):
        n = case["batch"] * case["new"]
        table = n * case["rot"] * 4
        both = 2 * hq * d * 2       # q read and written
        if case["op"] == "rope":
            return {"bytes": n * (both + 2 * row16 + 8) + table, "flops": n * 3 * case["rot"] * (hq + hkv)}
        # rows in, codes out; codes in, rows out
        return {"bytes": n * (both + 2 * row16 + 2 * row4 + 16) + table,
                "flops": n * (3 * case["rot"] * (hq + hkv) + 10 * hkv * d)}
    if case["op"] == "read4":
        return {"bytes": sum(lens) * (row4 + row16 + 8), "flops": sum(lens) * 4 * hkv * d}
    if case["op"] == "decode4":
        return {"bytes": sum(lens) * row4 + case["batch"] * hq * d * 6, "flops": 4 * sum(lens) * hq * d}
    new = case["new"]
    pairs = sum(new * t + new * (new + 1) // 2 for t in lens)
    return {"bytes": sum(t + new for t in lens) * row4 + case["batch"] * new * hq * d * 4,
            "flops": 4 * pairs * hq * d}


# ------------------------------------------------- the definition in 64 bits

def _turn64(x, pos, s):
    """Each pair (a, b) times e^(i angle) as a complex number."""
    rot, x = s["rot"], x.double()
    cs = s["cos_sin"][pos.long()].double()
    turn = torch.complex(cs[:, :rot // 2], cs[:, rot // 2:])[:, None, :]
    out = x.clone()
    ia = torch.arange(rot // 2, device=x.device)
    ia, ib = (2 * ia, 2 * ia + 1) if s["inter"] else (ia, ia + rot // 2)
    z = torch.complex(x[..., ia], x[..., ib]) * turn
    out[..., ia], out[..., ib] = z.real, z.imag
    return out


def _held64(x, dt):
    """What 4 bits, a scale and a zero of type dt keep of the rows x."""
    lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
    scale = ((hi - lo) / 15).to(dt).double()
    zero = (lo + 8 * scale).to(dt).double()
    step = torch.where(scale > 0, scale, 1.0)
    return zero + scale * ((x - zero) / step).round().clamp(-8, 7)


def exact(case, seed):
    s = prepare(case, seed)
    op, dt = s["op"], s["dt"]
    if op == "rope":
        page, slot = _places(s)
        k, v = s["kc"].double(), s["vc"].double()
        k[page, :, slot] = _turn64(s["k"], s["pos"], s)
        v[page, :, slot] = s["v"].double()
        return {"q": _turn64(s["q"], s["pos"], s), "k_cache": k, "v_cache": v}
    if op == "store4":
        return {"q": _turn64(s["q"], s["pos"], s), "k": _held64(_turn64(s["k"], s["pos"], s), dt),
                "v": _held64(s["v"].double(), dt)}
    d, hkv = s["d"], s["hkv"]
    raw = s["pool"].to(torch.int64)
    codes = raw[..., :16 * d]
    meta = s["pool"][..., 16 * d:].contiguous().view(dt).double().view(-1, hkv, 2, PAGE, 2)
    value = torch.empty((raw.shape[0], hkv, 2, PAGE, d), dtype=torch.float64, device=raw.device)
    halves = codes.view(-1, hkv, 2, PAGE, d // 2)
    value[..., 0::2] = (halves % 16 - 8) * meta[..., :1] + meta[..., 1:]
    value[..., 1::2] = (halves // 16 - 8) * meta[..., :1] + meta[..., 1:]
    del raw, codes, halves
    if op == "read4":
        page, slot = _places(s)
        rows = value[page, :, :, slot]
        return {"k": rows[:, :, 0], "v": rows[:, :, 1]}
    chunk = op == "prefill4"
    q = s["q"] if chunk else s["q"][:, None]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    for b, ctx in enumerate(s["ctx"].tolist()):
        held = ctx + (q.shape[1] if chunk else 0)
        if held == 0:
            continue
        pages = s["bt"][b, :-(-held // PAGE)].long()
        kv = value[pages].permute(2, 1, 0, 3, 4).reshape(2, hkv, -1, d)[:, :, :held]
        for g in range(hkv):
            rows = q[b, :, g * (s["hq"] // hkv):(g + 1) * (s["hq"] // hkv)].double()
            score = torch.einsum("nhd,td->nht", rows, kv[0, g]) * s["scale"]
            if chunk:
                late = torch.arange(held, device=q.device)[None, :] > ctx + torch.arange(q.shape[1], device=q.device)[:, None]
                score.masked_fill_(late[:, None, :], float("-inf"))
            out[b, :, g * (s["hq"] // hkv):(g + 1) * (s["hq"] // hkv)] = torch.einsum(
                "nht,td->nhd", score.softmax(-1), kv[1, g])
    return out if chunk else out[:, 0]
