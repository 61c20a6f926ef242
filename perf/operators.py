"""Measured cases of the operators around the paged cache: the queries' and keys' norm with the position rotation,
windowed attention, and the 4-bit cache (storing into it, loading from it, attention over it).

`run` makes the library's calls where `own` is true and computes the same in elementary torch operations, in 32 bits,
where it is false.  `exact` computes the definitions in 64 bits.  Layouts are those of include/dsa.h."""
import math

import torch

own = False

DEV = "cuda"
GROUP = 32  # elements of a head's row that share one scale in the 4-bit cache


# ---------------------------------------------------------------- cases ----
def listed():
    return [
        # a denoising step of one block behind a 128K prefix: the latency of one call counts
        dict(name="rope step", op="rope", S=1, B=32, Hq=32, Hkv=8, d=128, page=16, lo=131072, hi=131072, rot=128, interleaved=False,
             norm=True, append=False, ragged=False),
        # prompts of different lengths written into the paged cache, half of each head rotated, far positions
        dict(name="rope prompts", op="rope", S=4, B=8192, Hq=28, Hkv=4, d=128, page=64, lo=0, hi=1000, rot=64, interleaved=True,
             norm=True, append=True, ragged=True),
        # a denoising step of a windowed layer: 32 tokens, both directions inside the window
        dict(name="window step", op="window", S=1, B=32, Hq=32, Hkv=8, d=128, page=16, lo=131072, hi=131072, window=1024, sinks=16,
             causal=False, table=False, ragged=False),
        # one token of many sequences of different lengths
        dict(name="window decode", op="window", S=64, B=1, Hq=32, Hkv=8, d=128, page=16, lo=701, hi=32768, window=4096, sinks=4,
             causal=True, table=True, ragged=False),
        # a whole prompt at once
        dict(name="window prompt", op="window", S=1, B=8192, Hq=32, Hkv=8, d=128, page=16, lo=0, hi=0, window=2048, sinks=64,
             causal=True, table=False, ragged=False),
        # the finished blocks of a batch go into the 4-bit cache, and are read back
        dict(name="kv4 store blocks", op="store", S=8, B=32, Hq=32, Hkv=8, d=128, page=16, lo=16384, hi=65536, table=True, ragged=False),
        # prompts of odd lengths
        dict(name="kv4 store prompts", op="store", S=2, B=16383, Hq=32, Hkv=8, d=128, page=64, lo=0, hi=77, table=True, ragged=True),
        # one block's worth of a 4-bit prefix back in bf16
        dict(name="kv4 load block", op="load", S=1, B=64, Hq=32, Hkv=8, d=128, page=16, lo=8192, hi=8192, table=False, ragged=False),
        # whole prefixes back in bf16
        dict(name="kv4 load prefixes", op="load", S=4, B=16384, Hq=28, Hkv=4, d=128, page=64, lo=0, hi=130, table=True, ragged=True),
        # a denoising step over 1024 selected tokens of a 128K prefix
        dict(name="kv4 sparse step", op="kv4", S=1, B=32, Hq=32, Hkv=8, d=128, page=16, lo=131072, hi=131072, topk=1024, table=False, ragged=False),
        # one token of each sequence over its whole prefix
        dict(name="kv4 decode", op="kv4", S=8, B=1, Hq=32, Hkv=8, d=128, page=16, lo=16384, hi=65536, topk=0, table=True, ragged=False),
        # a block over a whole 128K prefix
        dict(name="kv4 block 128k", op="kv4", S=1, B=32, Hq=32, Hkv=8, d=128, page=16, lo=131072, hi=131072, topk=0, table=False, ragged=False),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "window", "window", "store", "load", "kv4", "kv4"])
    d = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    G = rng.choice([1, 2, 4, 4, 7, 8])
    c = dict(op=op, d=d, page=rng.choice([16, 32, 64]), Hq=Hkv * G, Hkv=Hkv)
    if op == "rope":
        tokens = log(1, 30000)
        c["S"] = rng.randint(1, max(1, min(16, tokens)))
        c["B"] = max(1, tokens // c["S"])
        c["lo"] = rng.randint(0, 300)
        c["hi"] = c["lo"] + rng.randint(0, 900)
        c["rot"] = 8 * rng.randint(1, d // 8)
        c["interleaved"], c["norm"], c["append"], c["ragged"] = (rng.random() < 0.5 for _ in range(4))
    elif op == "window":
        c["window"], c["sinks"] = log(1, 8192), rng.choice([0, 1, 4, 16, 64, 100])
        c["causal"], c["table"], c["ragged"] = (rng.random() < 0.5 for _ in range(3))
        if rng.random() < 0.3:  # a prompt, or a part of one
            c["S"], c["B"] = rng.randint(1, 2), log(64, 4000)
            c["lo"], c["hi"] = 0, rng.choice([0, rng.randint(1, 2000)])
        else:
            c["S"], c["B"] = log(1, 48), rng.choice([1, 1, rng.randint(2, 48), 32])
            c["lo"] = log(1, 2000)
            c["hi"] = c["lo"] + log(1, 30000)
    elif op in ("store", "load"):
        tokens = log(1, 30000)
        c["S"] = rng.randint(1, max(1, min(16, tokens)))
        c["B"] = max(1, tokens // c["S"])
        c["lo"] = rng.randint(0, 3000)
        c["hi"] = c["lo"] + rng.randint(0, 9000)
        c["table"], c["ragged"] = (rng.random() < 0.5 for _ in range(2))
    else:
        c["S"], c["B"] = log(1, 8), rng.choice([1, 1, rng.randint(2, 256 // G), 256 // G if G > 4 else 32])
        c["lo"] = log(1, 4000)
        c["hi"] = c["lo"] + log(1, 60000)
        c["topk"] = rng.choice([0, 0, 16 * rng.randint(4, 64) // c["page"] * c["page"]])
        c["table"], c["ragged"] = (rng.random() < 0.5 for _ in range(2))
    return c


def _lengths(c):
    """Prefix lengths: spread evenly over [lo, hi], in a mixed order."""
    S = c["S"]
    return [c["hi"] if S == 1 else c["lo"] + (c["hi"] - c["lo"]) * ((s * 37 + 5) % S) // (S - 1) for s in range(S)]


def _news(c):
    """Tokens of each sequence's block that exist: all B, or from B / 3 to B where the batch is padded."""
    S, B = c["S"], c["B"]
    return [B - (s * (2 * B // 3)) // S if c["ragged"] else B for s in range(S)]


# ------------------------------------------------------- what a program holds ----
def _normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _pages(c, g, n, more):
    """(max_pages, table or None): a random permutation of the physical pages where the case has a table."""
    P = c["page"]
    max_pages = max(1, max(-(-(x + more) // P) for x in n))
    if not c.get("table", True):
        return max_pages, None
    perm = torch.randperm(c["S"] * max_pages, generator=g, device=DEV)
    return max_pages, perm.view(c["S"], max_pages).to(torch.int32)


def _keys(g, *shape):
    """Cached keys: normal, some channels several times larger, as rotated keys have."""
    k = _normal(g, *shape)
    k[..., ::17] *= 4
    return k


def prepare(case, seed):
    c = case
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    S, B, Hq, Hkv, d, P = (c[x] for x in ("S", "B", "Hq", "Hkv", "d", "page"))
    n, new = _lengths(c), _news(c)
    bf = torch.bfloat16
    st = dict(c=c, n=torch.tensor(n, dtype=torch.int32, device=DEV), new=torch.tensor(new, dtype=torch.int32, device=DEV) if c["ragged"] else None)
    grows = c["op"] in ("rope", "store", "load")
    st["max_pages"], st["table"] = _pages(c, g, n, B if grows else 0)
    n_phys, kmax = S * st["max_pages"], 1
    if c["op"] == "rope":
        st["qkv"] = _normal(g, S, B, (Hq + 2 * Hkv) * d).to(bf)
        st["q_norm"] = (1 + 0.1 * _normal(g, d)).to(bf) if c["norm"] else None
        st["k_norm"] = (1 + 0.1 * _normal(g, d)).to(bf) if c["norm"] else None
        # frequencies of a base of 1e6, stretched eightfold for the long context, and far positions
        st["inv_freq"] = (1e6 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"]) / 8).float()
        st["pos"] = st["n"][:, None] + 900000 + torch.arange(B, device=DEV, dtype=torch.int32)
        st["q_out"] = torch.zeros(S, B, Hq, d, dtype=bf, device=DEV)
        if c["append"]:
            st["k_cache"], st["v_cache"] = (torch.zeros(n_phys, Hkv, P, d, dtype=bf, device=DEV) for _ in range(2))
        else:
            st["k_out"], st["v_out"] = (torch.zeros(S, B, Hkv, d, dtype=bf, device=DEV) for _ in range(2))
    else:
        st["blk_k"], st["blk_v"] = _keys(g, S, B, Hkv, d).to(bf), _normal(g, S, B, Hkv, d).to(bf)
    if c["op"] in ("window", "kv4"):
        st["q"] = _normal(g, S, B, Hq, d).to(bf)
        st["o"] = torch.zeros(S, B, Hq, d, dtype=bf, device=DEV)
        st["lse"] = torch.zeros(S, B, Hq, dtype=torch.float32, device=DEV)
    if c["op"] == "window":
        st["k_cache"], st["v_cache"] = _keys(g, n_phys, Hkv, P, d).to(bf), _normal(g, n_phys, Hkv, P, d).to(bf)
    if c["op"] in ("store", "load", "kv4"):
        st["cache"] = _cache_of(g, n_phys, Hkv, P, d, empty=c["op"] == "store")
    if c["op"] in ("store", "load"):
        st["k_out"], st["v_out"] = (torch.zeros(S, B, Hkv, d, dtype=bf, device=DEV) for _ in range(2))
    if c["op"] == "kv4" and c["topk"]:
        kmax = c["topk"] // P
        order = torch.rand(S, Hkv, st["max_pages"], generator=g, device=DEV)
        np_ = (st["n"] + P - 1) // P
        order.masked_fill_(torch.arange(st["max_pages"], device=DEV) >= np_[:, None, None], 2.0)
        take = min(kmax, st["max_pages"])
        cnt = torch.clamp(np_, max=kmax)[:, None].expand(S, Hkv).contiguous()
        idx = torch.full((S, Hkv, kmax), -1, dtype=torch.int64, device=DEV)
        best = order.topk(take, dim=-1, largest=False).indices
        far = 1 << 40
        best = best.masked_fill(torch.arange(take, device=DEV) >= cnt[..., None], far).sort(-1).values
        idx[..., :take] = best.masked_fill(best == far, -1)
        st["idx"], st["cnt"] = idx.to(torch.int32), cnt.to(torch.int32)
    if own:
        _plan(st, n_phys, kmax)
    return st


def _plan(st, n_phys, kmax):
    """The library's handles that a program keeps: shapes, rotation, 4-bit cache, workspace."""
    from block_sparse_attention_27_b200 import dsa

    c = st["c"]
    st["dims"] = dsa.make_dims(c["S"], c["B"], c["Hq"], c["Hkv"], c["d"], c["page"], st["max_pages"], kmax, n_phys, st["table"])
    nbytes = dsa.WORKSPACE_HEADER_BYTES
    if c["op"] == "rope":
        st["rope"] = dsa.Rope(st["inv_freq"], c["rot"], interleaved=c["interleaved"], scale=_mscale(), eps=1e-6, q_norm=st["q_norm"], k_norm=st["k_norm"])
    if c["op"] == "window":
        nbytes = dsa.window_workspace_size(st["dims"])
    if c["op"] == "kv4":
        nbytes = dsa.kv4_workspace_size(st["dims"])
    if "cache" in st:
        st["kv4"] = dsa.Kv4Cache(*st["cache"])
    st["ws"] = dsa.Workspace(nbytes)


def _mscale():
    return 0.1 * math.log(8.0) + 1.0  # the factor on cos and sin that goes with an eightfold stretch


# -------------------------------------------------------------- one pass ----
def run(state):
    st = state
    return {"rope": _rope, "window": _window, "store": _store, "load": _load, "kv4": _kv4}[st["c"]["op"]](st)


def _split(st):
    """q, k and v as views of the packed projection."""
    c, x = st["c"], st["qkv"]
    S, B, Hq, Hkv, d = (c[k] for k in ("S", "B", "Hq", "Hkv", "d"))
    at = Hq * d, (Hq + Hkv) * d
    return x[..., :at[0]].view(S, B, Hq, d), x[..., at[0]:at[1]].view(S, B, Hkv, d), x[..., at[1]:].view(S, B, Hkv, d)


def _rope(st):
    c = st["c"]
    q, k, v = _split(st)
    names = ("k_cache", "v_cache") if c["append"] else ("k_out", "v_out")
    if own:
        from block_sparse_attention_27_b200 import dsa

        dsa.dsa_qk_norm_rope(q, k, v, st["q_out"], st.get("k_out"), st.get("v_out"), dims=st["dims"], rope=st["rope"], n_ctx=st["n"],
                             workspace=st["ws"], positions=st["pos"], n_new=st["new"], k_cache=st.get("k_cache"), v_cache=st.get("v_cache"))
        return [st["q_out"], st[names[0]], st[names[1]]]
    live = _live(st)
    angle = st["pos"].double()[..., None] * st["inv_freq"].double()
    cos, sin = (angle.cos() * _mscale()).float()[:, :, None], (angle.sin() * _mscale()).float()[:, :, None]
    q2 = _turn(_scaled(q.float(), st["q_norm"]), cos, sin, c).to(q.dtype)
    k2 = _turn(_scaled(k.float(), st["k_norm"]), cos, sin, c).to(q.dtype)
    st["q_out"][live] = q2[live]
    if c["append"]:
        phys, slot = _places(st)
        st["k_cache"][phys, :, slot] = k2[live]
        st["v_cache"][phys, :, slot] = v[live]
    else:
        st["k_out"][live] = k2[live]
        st["v_out"][live] = v[live]
    return [st["q_out"], st[names[0]], st[names[1]]]


def _live(st):
    """[S, B]: the block's tokens that exist."""
    c = st["c"]
    new = st["new"] if st["new"] is not None else torch.full((c["S"],), c["B"], device=DEV)
    return torch.arange(c["B"], device=DEV) < new[:, None]


def _places(st):
    """Physical page and slot of every token of the block that exists."""
    c = st["c"]
    at = st["n"].long()[:, None] + torch.arange(c["B"], device=DEV)
    table = st["table"].long() if st["table"] is not None else torch.arange(c["S"] * st["max_pages"], device=DEV).view(c["S"], -1)
    page = at // c["page"]
    phys = table.gather(1, page.clamp(max=st["max_pages"] - 1))
    live = _live(st)
    return phys[live], (at % c["page"])[live]


def _scaled(x, w):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()


def _turn(x, cos, sin, c):
    r = c["rot"]
    head, tail = x[..., :r], x[..., r:]
    if c["interleaved"]:
        a, b = head[..., 0::2], head[..., 1::2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = head[..., : r // 2], head[..., r // 2:]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, tail), -1)


def _seen(c, pos, p, end):
    """Whether a key at position pos (below end) takes part for the query at position p."""
    near = (pos > p - c["window"]) & (pos < p + c["window"])
    ok = (pos < end) & (near | (pos < c["sinks"]))
    return ok & (pos <= p) if c["causal"] else ok


def _softmax(q, k, v, ok, c):
    """q [S,B,Hq,d], k and v [S,K,Hkv,d] or [S,Hkv,K,d] folded by the caller, ok broadcast to [S,Hkv,G,B,K]: (o, lse)."""
    S, B, Hq, d = q.shape
    Hkv = k.shape[1]
    qs = q.float().view(S, B, Hkv, Hq // Hkv, d).permute(0, 2, 3, 1, 4).reshape(S, Hkv, -1, d)
    x = (qs @ k.transpose(-1, -2)).view(S, Hkv, Hq // Hkv, B, -1) * (1 / math.sqrt(d))
    x = x.masked_fill_(~ok, -math.inf)
    m = x.amax(-1, keepdim=True)
    m0 = m.masked_fill(m == -math.inf, 0.0)
    p = x.sub_(m0).exp_()
    z = p.sum(-1, keepdim=True)
    o = (p.view(S, Hkv, -1, p.shape[-1]) @ v).view(S, Hkv, Hq // Hkv, B, d) / torch.where(z > 0, z, 1.0)
    lse = (m0 + z.log()).squeeze(-1)
    return o.permute(0, 3, 1, 2, 4).reshape(S, B, Hq, d), lse.permute(0, 3, 1, 2).reshape(S, B, Hq)


def _window(st):
    c = st["c"]
    if own:
        from block_sparse_attention_27_b200 import dsa

        dsa.dsa_window_attn(st["q"], st["k_cache"], st["v_cache"], st["blk_k"], st["blk_v"], st["o"], dims=st["dims"], window=c["window"],
                            sinks=c["sinks"], causal=c["causal"], n_ctx=st["n"], workspace=st["ws"], n_new=st["new"], lse_out=st["lse"])
        return [st["o"], st["lse"]]
    S, B, Hkv, d, P = (c[x] for x in ("S", "B", "Hkv", "d", "page"))
    n = st["n"].long()[:, None]
    new = st["new"].long()[:, None] if st["new"] is not None else B
    # the positions that any of the block's queries can see: the first tokens, the window's, the block's
    low = (n - c["window"] + 1).clamp(min=0)
    sink = torch.arange(min(c["sinks"], c["hi"]), device=DEV).expand(S, -1)
    sink = sink.masked_fill((sink >= low) | (sink >= n), 1 << 40)
    near = low + torch.arange(min(c["window"] - 1, c["hi"]), device=DEV)
    old = torch.cat((sink, near.masked_fill(near >= n, 1 << 40)), 1)
    table = st["table"].long() if st["table"] is not None else torch.arange(S * st["max_pages"], device=DEV).view(S, -1)
    at = torch.where(old < n, old, 0)
    phys = table.gather(1, at // P)
    k = torch.cat((st["k_cache"][phys, :, at % P], st["blk_k"]), 1).float().permute(0, 2, 1, 3)
    v = torch.cat((st["v_cache"][phys, :, at % P], st["blk_v"]), 1).float().permute(0, 2, 1, 3)
    b = torch.arange(B, device=DEV)
    pos, p = torch.cat((old, n + b), 1), n + b
    ok = _seen(c, pos[:, None], p[..., None], (n + new)[..., None] if st["new"] is not None else 1 << 39)[:, None, None]
    o, lse = _softmax(st["q"], k, v, ok, c)
    live = _live(st)
    st["o"][live] = o.to(st["o"].dtype)[live]
    st["lse"][live] = lse[live]
    return [st["o"], st["lse"]]


# ---------------------------------------------------------- the 4-bit cache ----
# A row of d elements is d / 32 groups.  A group's scale s is the smallest number of five significant bits that is at
# least max|x| / 7, in bf16; an element is kept as x / s rounded to the nearest whole number, plus 8.  Four bytes hold
# eight elements: the even ones in the first two bytes, the odd ones in the other two, low bits first.
def _scales(x):
    t = x.abs().amax(-1, keepdim=True)
    t = t / torch.full_like(t, 7)  # a division, not a product with 1/7: a whole multiple of 7 stays on its border
    up = ((t.view(torch.int32) + 0x7FFFF) & ~0x7FFFF).view(torch.float32)
    return up.masked_fill(t * 7 < 2.0 ** -100, 0.0)


def _pack(x):
    """x fp32 [..., d] -> (bytes [..., d / 2], scales bf16 [..., d / 32])."""
    y = x.unflatten(-1, (-1, GROUP))
    s = _scales(y)
    w = torch.where(s > 0, torch.round(y / s), 0.0).clamp_(-7, 7).add_(8).to(torch.uint8).flatten(-2).unflatten(-1, (-1, 8))
    low = w[..., [0, 4, 1, 5]]
    return (low | w[..., [2, 6, 3, 7]] << 4).flatten(-2), s.squeeze(-1).to(torch.bfloat16)


def _unpack(b, s):
    y = b.unflatten(-1, (-1, 4))
    w = torch.stack((y & 15, y >> 4), -1).flatten(-2)[..., [0, 4, 1, 5, 2, 6, 3, 7]]
    return ((w.flatten(-2).float() - 8).unflatten(-1, (-1, GROUP)) * s.float()[..., None]).flatten(-2)


def _cache_of(g, n_phys, Hkv, P, d, empty):
    if empty:
        k, v = (torch.zeros(n_phys, Hkv, P, d // 2, dtype=torch.uint8, device=DEV) for _ in range(2))
        ks, vs = (torch.zeros(n_phys, Hkv, P, d // GROUP, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        return k, v, ks, vs
    k, ks = _pack(_keys(g, n_phys, Hkv, P, d))
    v, vs = _pack(_normal(g, n_phys, Hkv, P, d))
    return k, v, ks, vs


def _fetch(st):
    """The block's tokens out of the 4-bit cache, into the state's outputs."""
    phys, slot = _places(st)
    live = _live(st)
    k, v, ks, vs = st["cache"]
    st["k_out"][live] = _unpack(k[phys, :, slot], ks[phys, :, slot]).to(torch.bfloat16)
    st["v_out"][live] = _unpack(v[phys, :, slot], vs[phys, :, slot]).to(torch.bfloat16)
    return [st["k_out"], st["v_out"]]


def _store(st):
    """The block's tokens into the cache, and back as the values that it holds."""
    if own:
        from block_sparse_attention_27_b200 import dsa

        dsa.dsa_kv4_store(st["blk_k"], st["blk_v"], st["kv4"], dims=st["dims"], n_ctx=st["n"], workspace=st["ws"], n_new=st["new"])
        dsa.dsa_kv4_load(st["kv4"], st["k_out"], st["v_out"], dims=st["dims"], start=st["n"], workspace=st["ws"], n_new=st["new"])
        return [st["k_out"], st["v_out"]]
    phys, slot = _places(st)
    live = _live(st)
    k, v, ks, vs = st["cache"]
    k[phys, :, slot], ks[phys, :, slot] = _pack(st["blk_k"].float()[live])
    v[phys, :, slot], vs[phys, :, slot] = _pack(st["blk_v"].float()[live])
    return _fetch(st)


def _load(st):
    if own:
        from block_sparse_attention_27_b200 import dsa

        dsa.dsa_kv4_load(st["kv4"], st["k_out"], st["v_out"], dims=st["dims"], start=st["n"], workspace=st["ws"], n_new=st["new"])
        return [st["k_out"], st["v_out"]]
    return _fetch(st)


def _kv4(st):
    c = st["c"]
    if own:
        from block_sparse_attention_27_b200 import dsa

        dsa.dsa_kv4_attn(st["q"], st["kv4"], st.get("idx"), st["blk_k"], st["blk_v"], st["o"], dims=st["dims"], n_ctx=st["n"],
                         idx_cnt=st.get("cnt"), workspace=st["ws"], n_new=st["new"], lse_out=st["lse"])
        return [st["o"], st["lse"]]
    S, B, Hkv, d, P = (c[x] for x in ("S", "B", "Hkv", "d", "page"))
    table = st["table"].long() if st["table"] is not None else torch.arange(S * st["max_pages"], device=DEV).view(S, -1)
    if "idx" in st:
        lp = st["idx"].long()
        held = torch.arange(lp.shape[-1], device=DEV) < st["cnt"][..., None]
    else:
        lp = torch.arange(st["max_pages"], device=DEV).expand(S, Hkv, -1)
        held = torch.ones_like(lp, dtype=torch.bool)
    phys = table[:, None].expand(S, Hkv, -1).gather(2, lp.clamp(min=0))
    head = torch.arange(Hkv, device=DEV)[None, :, None]
    kc, vc, ks, vs = st["cache"]
    k = _unpack(kc[phys, head], ks[phys, head]).flatten(2, 3)
    v = _unpack(vc[phys, head], vs[phys, head]).flatten(2, 3)
    pos = (lp[..., None] * P + torch.arange(P, device=DEV)).flatten(2)
    ok = held.repeat_interleave(P, 2) & (pos < st["n"].long()[:, None, None])
    k = torch.cat((k, st["blk_k"].float().transpose(1, 2)), 2)
    v = torch.cat((v, st["blk_v"].float().transpose(1, 2)), 2)
    live = _live(st)
    ok = torch.cat((ok, live[:, None].expand(S, Hkv, B)), 2)[:, :, None, None]
    o, lse = _softmax(st["q"], k, v, ok, c)
    st["o"][live] = o.to(st["o"].dtype)[live]
    st["lse"][live] = lse[live]
    return [st["o"], st["lse"]]


# ------------------------------------------------------------- the least work ----
def work(case):
    c = case
    S, B, Hq, Hkv, d, P = (c[x] for x in ("S", "B", "Hq", "Hkv", "d", "page"))
    n, new = _lengths(c), _news(c)
    tokens = sum(new)
    row4 = d // 2 + 2 * (d // GROUP)  # bytes of one head's row in the 4-bit cache
    if c["op"] == "rope":
        return {"bytes": tokens * (Hq + 2 * Hkv) * d * 2 * 2 + 8 * tokens, "flops": tokens * (Hq + Hkv) * d * 8}
    if c["op"] == "store":
        return {"bytes": tokens * 2 * Hkv * 2 * (2 * d + row4), "flops": tokens * 2 * Hkv * d * 6}
    if c["op"] == "load":
        return {"bytes": tokens * 2 * Hkv * (2 * d + row4), "flops": tokens * 2 * Hkv * d * 2}
    rows = tokens * Hq * (2 * d * 2 + 4)  # queries, outputs and their log-sum-exps
    if c["op"] == "kv4":
        old = [x if not c["topk"] else min(x, c["topk"]) for x in n]
        pairs = sum(m * (x + m) for x, m in zip(old, new))
        return {"bytes": rows + sum(old) * Hkv * 2 * row4 + tokens * Hkv * 2 * 2 * d, "flops": pairs * Hq * d * 4}
    keys = pairs = 0
    for x, m in zip(n, new):
        keys += m + min(x, c["window"] - 1) + min(c["sinks"], max(0, x - c["window"] + 1))
        for b in range(m):
            p = x + b
            low = max(0, p - c["window"] + 1)
            top = p if c["causal"] else min(x + m - 1, p + c["window"] - 1)
            more = 0 if c["causal"] else max(0, min(c["sinks"], x + m) - top - 1)
            pairs += top - low + 1 + min(c["sinks"], low) + more
    return {"bytes": rows + keys * Hkv * 2 * 2 * d, "flops": pairs * Hq * d * 4}


# ----------------------------------------------------------- the definitions ----
def exact(case, seed):
    c, st = case, prepare(case, seed)
    return {"rope": _exact_rope, "window": _exact_attention, "kv4": _exact_attention, "store": _exact_store, "load": _exact_load}[c["op"]](c, st)


def _where(c, st, s, t):
    """(physical pages, slots) of the logical tokens t of sequence s."""
    lp = torch.div(t, c["page"], rounding_mode="floor")
    phys = lp + s * st["max_pages"] if st["table"] is None else st["table"][s].long()[lp]
    return phys, t - lp * c["page"]


def _exact_rope(c, st):
    q, k, v = (t.double() for t in _split(st))
    turn = torch.polar(torch.full((), _mscale(), dtype=torch.float64, device=DEV),
                       st["pos"].double()[:, :, None, None] * st["inv_freq"].double())
    r, new = c["rot"], _news(c)

    def full(x, w):
        if w is not None:
            x = x / torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / c["d"] + 1e-6) * w.double()
        y = x.clone()
        pick = (slice(0, r, 2), slice(1, r, 2)) if c["interleaved"] else (slice(0, r // 2), slice(r // 2, r))
        z = torch.complex(x[..., pick[0]], x[..., pick[1]]) * turn
        y[..., pick[0]], y[..., pick[1]] = z.real, z.imag
        return y

    q, k = full(q, st["q_norm"]), full(k, st["k_norm"])
    for s in range(c["S"]):
        q[s, new[s]:], k[s, new[s]:], v[s, new[s]:] = 0, 0, 0
    if not c["append"]:
        return [q, k, v]
    kc, vc = (torch.zeros(st["k_cache"].shape, dtype=torch.float64, device=DEV) for _ in range(2))
    for s in range(c["S"]):
        phys, slot = _where(c, st, s, int(st["n"][s]) + torch.arange(new[s], device=DEV))
        kc[phys, :, slot], vc[phys, :, slot] = k[s, :new[s]], v[s, :new[s]]
    return [q, kc, vc]


def _exact_values(x):
    """What the 4-bit cache holds of x [..., d], in 64 bits."""
    y = x.double().unflatten(-1, (-1, GROUP))
    top = y.abs().amax(-1, keepdim=True)
    m, e = torch.frexp(top / torch.full_like(top, 7))
    s = torch.ldexp(torch.ceil(m * 32) / 32, e)
    code = torch.where(top > 0, torch.round(y / torch.where(top > 0, s, 1.0)), 0.0)
    return (code * s).flatten(-2)


def _exact_store(c, st):
    out = []
    for x in (st["blk_k"], st["blk_v"]):
        y = _exact_values(x)
        for s, m in enumerate(_news(c)):
            y[s, m:] = 0
        out.append(y)
    return out


def _exact_nibbles(b, s):
    """The values of packed rows b [..., d / 2] with scales s, by words of 32 bits."""
    word = b.long().unflatten(-1, (-1, 4))
    word = word[..., 0] | word[..., 1] << 8 | word[..., 2] << 16 | word[..., 3] << 24
    shift = torch.tensor([4 * (e // 2) + 16 * (e % 2) for e in range(8)], device=DEV)
    code = (word[..., None] >> shift) & 15
    return ((code.flatten(-2) - 8).double().unflatten(-1, (-1, GROUP)) * s.double().unsqueeze(-1)).flatten(-2)


def _exact_load(c, st):
    k, v, ks, vs = st["cache"]
    ko, vo = (torch.zeros(c["S"], c["B"], c["Hkv"], c["d"], dtype=torch.float64, device=DEV) for _ in range(2))
    for s, m in enumerate(_news(c)):
        phys, slot = _where(c, st, s, int(st["n"][s]) + torch.arange(m, device=DEV))
        ko[s, :m], vo[s, :m] = _exact_nibbles(k[phys, :, slot], ks[phys, :, slot]), _exact_nibbles(v[phys, :, slot], vs[phys, :, slot])
    return [ko, vo]


def _exact_attention(c, st):
    S, B, Hq, Hkv, d, P = (c[x] for x in ("S", "B", "Hq", "Hkv", "d", "page"))
    o = torch.zeros(S, B, Hq, d, dtype=torch.float64, device=DEV)
    lse = torch.zeros(S, B, Hq, dtype=torch.float64, device=DEV)
    G = Hq // Hkv
    for s, (n, m) in enumerate(zip(_lengths(c), _news(c))):
        p = n + torch.arange(m, device=DEV)
        for h in range(Hkv):
            if c["op"] == "window":
                # every key that the first query's window, the sinks or the block reach, in their order
                low = max(0, n - c["window"] + 1)
                t = torch.arange(n, device=DEV)
                t = t[(t >= low) | (t < c["sinks"])]
                phys, slot = _where(c, st, s, t)
                k, v = st["k_cache"][phys, h, slot].double(), st["v_cache"][phys, h, slot].double()
            else:
                if "idx" in st:
                    lp = st["idx"][s, h, : int(st["cnt"][s, h])].long()
                    t = (lp[:, None] * P + torch.arange(P, device=DEV)).flatten()
                    t = t[t < n]
                else:
                    t = torch.arange(n, device=DEV)
                phys, slot = _where(c, st, s, t)
                kc, vc, ks, vs = st["cache"]
                k, v = _exact_nibbles(kc[phys, h, slot], ks[phys, h, slot]), _exact_nibbles(vc[phys, h, slot], vs[phys, h, slot])
            k = torch.cat((k, st["blk_k"][s, :m, h].double()))
            v = torch.cat((v, st["blk_v"][s, :m, h].double()))
            pos = torch.cat((t, p))
            gap = pos[None] - p[:, None]
            away = torch.zeros_like(gap, dtype=torch.bool)
            if c["op"] == "window":
                away = (gap.abs() >= c["window"]) & (pos[None] >= c["sinks"])
                if c["causal"]:
                    away |= gap > 0
            for g in range(G):
                x = st["q"][s, :m, h * G + g].double() @ k.T / math.sqrt(d)
                x[away] = -math.inf
                z = torch.logsumexp(x, -1)
                o[s, :m, h * G + g] = torch.exp(x - z[:, None]) @ v
                lse[s, :m, h * G + g] = z
    return [o, lse]
