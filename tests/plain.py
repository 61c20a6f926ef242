"""Plain definitions, in 64 bits on the CPU, of the operators beside the two passes, and the
tolerances their tests use.  Shares no code with the library; loops over rows and tokens."""
from __future__ import annotations

import math

import torch

F64 = torch.float64


def half(dtype):
    """The largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


def token_row(cache, table, max_pages, page, s, h, t):
    """Row of logical token t of sequence s, head h in a paged array [n_phys, Hkv, page, x]."""
    lp = t // page
    phys = s * max_pages + lp if table is None else int(table[s, lp])
    return cache[phys, h, t % page]


# ------------------------------------------------------------------ norm + rotation ----
def norm_rope(x, w, pos, inv_freq, rot, interleaved, scale, eps):
    """x [S, B, H, d] -> (y, size): the result and, per element, the length of its rotated pair
    (what rounding errors of the rotation are relative to)."""
    y = x.to(F64)
    d = y.shape[-1]
    if w is not None:
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / d + eps) * w.to(F64)
    out, size = y.clone(), y.abs()
    for i in range(rot // 2):
        p, q = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        ang = pos.to(F64) * float(inv_freq[i])
        c, s = torch.cos(ang)[..., None], torch.sin(ang)[..., None]
        a, b = y[..., p], y[..., q]
        out[..., p], out[..., q] = (a * c - b * s) * scale, (b * c + a * s) * scale
        size[..., p] = size[..., q] = torch.sqrt(a * a + b * b) * abs(scale)
    return out, size


# ------------------------------------------------------------------------ attention ----
def attend(q, k, v):
    """One query row over keys [m, d]: (o, lse, spread) with spread = sum p |v|."""
    if k.shape[0] == 0:
        z = torch.zeros(q.shape[-1], dtype=F64)
        return z, -math.inf, z
    x = k.to(F64) @ q.to(F64) / math.sqrt(q.shape[-1])
    top = x.max()
    p = torch.exp(x - top)
    l = p.sum()
    p = p / l
    return p @ v.to(F64), float(top + torch.log(l)), p @ v.to(F64).abs()


def window_attn(q, k_cache, v_cache, table, max_pages, n_ctx, blk_k, blk_v, window, sinks, causal,
                n_new=None):
    """(o, lse, spread, reach) of dsa_window_attn; reach [S, B, Hq] = the largest sum |q_i k_i| /
    sqrt(d) over a row's keys.  Rows of tokens that do not exist are NaN."""
    S, B, Hq, d = q.shape
    Hkv, page = k_cache.shape[1], k_cache.shape[2]

    def keys(s, b, h):
        n, m = int(n_ctx[s]), B if n_new is None else int(n_new[s])
        p, ks, vs = n + b, [], []
        for j in range(n + (m if blk_k is not None else 0)):
            if not (j < sinks or abs(p - j) < window) or (causal and j > p):
                continue
            if j < n:
                ks.append(token_row(k_cache, table, max_pages, page, s, h, j))
                vs.append(token_row(v_cache, table, max_pages, page, s, h, j))
            else:
                ks.append(blk_k[s, j - n, h])
                vs.append(blk_v[s, j - n, h])
        return ks, vs

    return _rows(q, Hkv, keys, n_new)


def _rows(q, Hkv, keys, n_new):
    S, B, Hq, d = q.shape
    G = Hq // Hkv
    o = torch.full((S, B, Hq, d), math.nan, dtype=F64)
    lse = torch.full((S, B, Hq), math.nan, dtype=F64)
    spread, reach = torch.zeros_like(o), torch.zeros_like(lse)
    for s in range(S):
        for b in range(B if n_new is None else int(n_new[s])):
            for h in range(Hkv):
                ks, vs = keys(s, b, h)
                k = torch.stack(ks).to(F64) if ks else torch.zeros((0, d), dtype=F64)
                v = torch.stack(vs).to(F64) if vs else torch.zeros((0, d), dtype=F64)
                for g in range(G):
                    x = q[s, b, h * G + g].to(F64)
                    o[s, b, h * G + g], lse[s, b, h * G + g], spread[s, b, h * G + g] = attend(x, k, v)
                    if ks:
                        reach[s, b, h * G + g] = (k.abs() @ x.abs()).max() / math.sqrt(d)
    return o, lse, spread, reach


def check_attention(o, lse, want, what):
    """The kernel's o (bf16) and lse (fp32) against (o, lse, spread, reach).

    A score is a sum of d products in fp32, off by at most d 2^-23 reach (each of d additions half a
    step of a partial sum that is at most reach; a factor two for the accumulator's truncation), so
    a probability is off by that share, doubled for the sum it is divided by; rounding a
    probability to bf16 adds half a step of it, and the exponentials and sums 2^-16.  Each of these
    errors of p weighs |v|: spread.  The output is rounded once more.  The log-sum-exp is off by
    the score's error, the exponentials' 2^-18, and its own rounding."""
    ro, rl, spread, reach = want
    d = o.shape[-1]
    live = ~torch.isnan(rl)
    o, lse = o.detach().cpu().to(F64), lse.detach().cpu().to(F64)
    ds = d * 2.0 ** -23 * reach
    assert torch.equal(torch.isinf(lse[live]), torch.isinf(rl[live])), what
    fin = live & torch.isfinite(rl)
    tol = ds + 2.0 ** -18 + half(torch.float32) * rl.abs()
    worst = ((lse - rl).abs() - tol)[fin]
    assert fin.sum() == 0 or worst.max() <= 0, (what, "lse", float(worst.max()))
    b = half(torch.bfloat16)
    tol = b * ro.abs() + (b + 2 * ds[..., None] + 2.0 ** -16) * (1 + b) * spread
    bad = ((o - ro).abs() > tol)[live]
    assert not torch.isnan(o[live]).any(), (what, "NaN")
    assert not bad.any(), (what, "o", float(((o - ro).abs() - tol)[live].max()), int(bad.sum()))


# ---------------------------------------------------------------------- 4-bit cache ----
GROUP = 32


def kv4_scale(amax: float) -> float:
    if not amax < 2.0 ** 120:
        return math.nan
    if amax < 2.0 ** -100:
        return 0.0
    m, e = math.frexp(amax / 7)
    return math.ldexp(math.ceil(m * 32) / 32, e)


def kv4_codes(row):
    """(codes 0..15 [d], scales [d/32]) of one row, in Python numbers."""
    codes, scales = [], []
    xs = [float(x) for x in row]
    for g in range(0, len(xs), GROUP):
        part = xs[g:g + GROUP]
        bad = any(not math.isfinite(x) for x in part)
        s = math.nan if bad else kv4_scale(max(abs(x) for x in part))
        scales.append(s)
        codes += [int(min(7, max(-7, round(x / s)))) + 8 if s > 0 else 8 for x in part]  # round: ties to even
    return codes, scales


def kv4_pack_row(row):
    """(bytes [d/2] as a list, scales)."""
    codes, scales = kv4_codes(row)
    out = []
    for w in range(0, len(codes), 8):
        word = 0
        for e in range(8):
            word |= codes[w + e] << (4 * (e // 2) + 16 * (e % 2))
        out += list(word.to_bytes(4, "little"))
    return out, scales


def kv4_pack(x):
    """x [..., d] -> (uint8 [..., d/2], bf16 [..., d/32])."""
    flat = x.reshape(-1, x.shape[-1])
    rows = [kv4_pack_row(r) for r in flat.tolist()]
    codes = torch.tensor([r[0] for r in rows], dtype=torch.uint8).view(*x.shape[:-1], x.shape[-1] // 2)
    scales = torch.tensor([r[1] for r in rows], dtype=F64).to(torch.bfloat16).view(*x.shape[:-1], x.shape[-1] // GROUP)
    return codes, scales


def kv4_values(codes, scales):
    """The values held: uint8 [..., d/2], bf16 [..., d/32] -> fp64 [..., d]."""
    b = codes.to(torch.int64).reshape(*codes.shape[:-1], -1, 4)
    word = b[..., 0] + (b[..., 1] << 8) + (b[..., 2] << 16) + (b[..., 3] << 24)
    cols = [((word >> (4 * (e // 2) + 16 * (e % 2))) & 15) - 8 for e in range(8)]
    c = torch.stack(cols, -1).reshape(*codes.shape[:-1], -1).to(F64)
    return c * scales.to(F64).repeat_interleave(GROUP, -1)


def kv4_attn(q, kv, table, max_pages, n_ctx, idx, cnt, blk_k, blk_v, n_new=None):
    """(o, lse, spread, reach) of dsa_kv4_attn; kv = (k, v) already as values [n_phys, Hkv, page, d]."""
    S, B, Hq, d = q.shape
    kval, vval = kv
    Hkv, page = kval.shape[1], kval.shape[2]

    def keys(s, b, h):
        n, m = int(n_ctx[s]), B if n_new is None else int(n_new[s])
        pages = range(-(-n // page)) if idx is None else [int(x) for x in idx[s, h, : int(cnt[s, h])]]
        toks = [t for lp in pages for t in range(lp * page, min(n, (lp + 1) * page))]
        ks = [token_row(kval, table, max_pages, page, s, h, t) for t in toks]
        vs = [token_row(vval, table, max_pages, page, s, h, t) for t in toks]
        if blk_k is not None:
            ks += [blk_k[s, u, h].to(F64) for u in range(m)]
            vs += [blk_v[s, u, h].to(F64) for u in range(m)]
        return ks, vs

    return _rows(q, Hkv, keys, n_new)
