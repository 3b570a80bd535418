"""The rotated append and the 4-bit cache from their definitions, in plain torch:
the codes in fp32 step by step, attention in 64 bits.  Shares no code with the
package."""
import math

import torch

PAGE = 16
EPS32 = 2.0 ** -24


def block_bytes(d):
    return 2 * PAGE * (d // 2 + 4)


def rotate(x, pos, cos_sin, interleaved, wide=torch.float64):
    """x [n, heads, D] turned by cos_sin [positions, rot] at pos [n]."""
    rot = cos_sin.shape[1]
    out = x.to(wide).clone()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        c = cos_sin[pos.long(), i].to(wide)[:, None]
        s = cos_sin[pos.long(), rot // 2 + i].to(wide)[:, None]
        xa, xb = x[..., a].to(wide), x[..., b].to(wide)
        out[..., a] = xa * c - xb * s
        out[..., b] = xb * c + xa * s
    return out


def quantise(x, dt):
    """fp32 rows -> codes (int), scale, zero (dt), by the documented steps."""
    mn, mx = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    rng = mx - mn
    scale = (rng * torch.tensor(1.0 / 15.0, dtype=torch.float32)).to(dt)
    zero = (mn + 8.0 * scale.float()).to(dt)
    ok = torch.isfinite(rng) & torch.isfinite(scale) & torch.isfinite(zero)
    s, z = scale.float(), zero.float()
    code = torch.full_like(x, 8.0)
    use = (ok & (s > 0)).expand_as(x)
    code[use] = (torch.round((x - z) / s) + 8.0).clamp(0, 15)[use]
    nan = torch.full_like(scale, math.nan)
    return code.to(torch.int64), torch.where(ok, scale, nan), torch.where(ok, zero, nan)


def store(pool, block_table, seq, pos, k, v, dt):
    """Writes fp32 rows k, v [n, Hkv, D] into pool (uint8 [pages, Hkv, block], CPU)."""
    d = k.shape[-1]
    page = block_table[seq.long(), (pos // PAGE).long()].long()
    slot = (pos % PAGE).long()
    codes = pool[..., :16 * d].unflatten(-1, (2, PAGE, d // 2))
    metas = pool[..., 16 * d:].unflatten(-1, (2, PAGE, 4))
    for which, x in enumerate((k, v)):
        code, scale, zero = quantise(x, dt)
        codes[page, :, which, slot] = (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8)
        metas[page, :, which, slot] = torch.cat((scale, zero), -1).contiguous().view(torch.uint8)


def values(pool, dt):
    """What a pool stands for: K and V float64 [pages, Hkv, 16, D], and the
    (scale, zero) pairs [pages, Hkv, 2, 16, 2]."""
    d = (pool.shape[-1] - 128) // 16
    codes = pool[..., :16 * d].reshape(*pool.shape[:2], 2, PAGE, d // 2).to(torch.int64)
    meta = pool[..., 16 * d:].contiguous().view(dt).double().reshape(*pool.shape[:2], 2, PAGE, 2)
    x = torch.empty((*pool.shape[:2], 2, PAGE, d), dtype=torch.float64, device=pool.device)
    x[..., 0::2] = meta[..., 1:] + meta[..., :1] * (codes % 16 - 8)
    x[..., 1::2] = meta[..., 1:] + meta[..., :1] * (codes // 16 - 8)
    return x[:, :, 0], x[:, :, 1], meta


def attention(q, pool, block_table, tokens, scale, dt):
    """softmax(q K^T scale) V in 64 bits.  q [B, queries, Hq, D]; tokens
    [B][queries]: the keys each query sees.  Returns the result and, per row, a
    bound on an fp32 kernel's error:

    A score (log2 units) is a sum whose terms are at most A = log2 e |scale|
    sum |q| max(16 |scale_k| + |zero_k|) in total; 8 tensor-core steps of at most one
    unit 2^-23 of it each and 4 fp32 roundings make |ds| <= 12 A 2^-23.  A weight is
    then off by ds ln 2 + 2^-22 (ex2) + 2^-21 (its two 16-bit terms) relatively, in
    the numerator and in the sum l; each page adds one tensor-core step a term
    (2 2^-23 in the numerator, one rounding in l), merges some 16 roundings.  With
    values of at most vmax the result is off by
      vmax 2^-23 (24 A + 3 pages + 64).
    """
    B, nq, hq, d = q.shape
    hkv = pool.shape[1]
    G = hq // hkv
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    bound = torch.zeros(q.shape[:3], dtype=torch.float64, device=q.device)
    for b in range(B):
        most = max(tokens[b])
        if most == 0:
            continue
        pages = block_table[b, :-(-most // PAGE)].long()
        k, v, meta = values(pool[pages.to(pool.device)], dt)
        k = k.transpose(0, 1).reshape(hkv, -1, d)
        v = v.transpose(0, 1).reshape(hkv, -1, d)
        meta = meta.permute(1, 2, 0, 3, 4).reshape(hkv, 2, -1, 2)
        size = 16 * meta[..., 0].abs() + meta[..., 1].abs()  # [hkv, 2, keys]
        for i in range(nq):
            T = tokens[b][i]
            if T == 0:
                continue
            rows = q[b, i].double().view(hkv, G, d)
            s = rows @ k[:, :T].transpose(-1, -2) * scale
            out[b, i] = (torch.softmax(s, -1) @ v[:, :T]).view(hq, d)
            top = size[..., :T].amax(-1)  # [hkv, 2]
            A = 1.4427 * abs(scale) * rows.abs().sum(-1) * top[:, :1]
            bound[b, i] = (top[:, 1:] * 2.0 ** -23 *
                           (24 * A + 3 * (-(-T // PAGE)) + 64)).view(hq)
    return out, bound
