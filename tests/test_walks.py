"""Attention calls whose CTAs walk through many stops: mixed batches with fresh sequences, the prefix
alone, many short units, units that shares cut, in bf16 and in 4 bits, against the definitions in 64 bits."""
import math

import pytest
import torch

import plain
import walk_model as wm
from block_sparse_attention_27_b200 import build, dsa

BF, F64 = torch.bfloat16, torch.float64


@pytest.fixture(scope="module")
def lib():
    build.build()
    return dsa.load()


def dense(q, keys, seen, Hkv, new):
    """(o, lse, spread, reach) as tests/plain.py has them, a sequence and KV head at a time:
    keys(s, h) = (k, v) [m, d] in 64 bits, seen(s) = bool [B, m]."""
    S, B, Hq, d = q.shape
    G = Hq // Hkv
    o, lse = torch.full((S, B, Hq, d), math.nan, dtype=F64), torch.full((S, B, Hq), math.nan, dtype=F64)
    spread, reach = torch.zeros_like(o), torch.zeros_like(lse)
    for s in range(S):
        m = new[s]
        ok = seen(s)[:m, None]
        for h in range(Hkv):
            k, v = keys(s, h)
            at = s, slice(0, m), slice(h * G, (h + 1) * G)
            if k.shape[0] == 0:
                o[at], lse[at] = 0.0, -math.inf
                continue
            x = q[at].to(F64)
            sc = (x @ k.T / math.sqrt(d)).masked_fill(~ok, -math.inf)
            top = sc.amax(-1, keepdim=True)
            p = torch.exp(sc - top.masked_fill(top == -math.inf, 0.0))
            l = p.sum(-1, keepdim=True)
            p = p / torch.where(l > 0, l, 1.0)
            o[at], spread[at] = p @ v, p @ v.abs()
            lse[at] = (top + torch.log(l)).squeeze(-1)
            reach[at] = (x.abs() @ k.abs().T / math.sqrt(d)).masked_fill(~ok, 0.0).amax(-1)
    return o, lse, spread, reach


class Window:
    """Inputs of a dsa_window_attn call of walk_model.WALKS."""

    def __init__(self, c, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.c, S, B, d, page = c, len(c["n"]), c["B"], c["d"], c["page"]
        self.n, self.new = c["n"], c.get("new") or [B] * S
        self.max_pages = max(1, max(-(-x // page) for x in self.n))
        self.n_phys = S * self.max_pages
        self.table = torch.arange(self.n_phys) if not c.get("table", True) else torch.randperm(self.n_phys, generator=g)
        self.table = self.table.view(S, -1).to(torch.int32)

        def rnd(*shape):
            return torch.randn(shape, generator=g).to(BF)

        Hkv = c["Hkv"]
        self.q = rnd(S, B, Hkv * c["G"], d)
        self.k, self.v = rnd(self.n_phys, Hkv, page, d), rnd(self.n_phys, Hkv, page, d)
        self.bk, self.bv = (rnd(S, B, Hkv, d), rnd(S, B, Hkv, d)) if c.get("block", True) else (None, None)

    def want(self):
        c, page = self.c, self.c["page"]

        def keys(s, h):
            t = torch.arange(self.n[s])
            phys = self.table[s].long()[t // page]
            k, v = self.k[phys, h, t % page], self.v[phys, h, t % page]
            if self.bk is not None:
                k, v = torch.cat((k, self.bk[s, : self.new[s], h])), torch.cat((v, self.bv[s, : self.new[s], h]))
            return k.to(F64), v.to(F64)

        def seen(s):
            p = (self.n[s] + torch.arange(c["B"]))[:, None]
            j = torch.arange(self.n[s] + (self.new[s] if self.bk is not None else 0))[None]
            ok = (j < c["sinks"]) | ((p - j).abs() < c["window"])
            return ok & (j <= p) if c["causal"] else ok

        return dense(self.q, keys, seen, c["Hkv"], self.new)

    def run(self):
        c, up = self.c, lambda t: None if t is None else t.cuda()  # noqa: E731
        S, B, Hq, d = self.q.shape
        tab = up(self.table) if c.get("table", True) else None
        dims = dsa.make_dims(S, B, Hq, c["Hkv"], d, c["page"], self.max_pages, 1, self.n_phys, tab)
        ws = dsa.Workspace(dsa.window_workspace_size(dims))
        o, lse = torch.full((S, B, Hq, d), 5.0, dtype=BF, device="cuda"), torch.full((S, B, Hq), 5.0, device="cuda")
        new = None if "new" not in c else torch.tensor(self.new, dtype=torch.int32, device="cuda")
        dsa.dsa_window_attn(*map(up, (self.q, self.k, self.v, self.bk, self.bv)), o, dims=dims, window=c["window"], sinks=c["sinks"],
                            causal=c["causal"], n_ctx=torch.tensor(self.n, dtype=torch.int32, device="cuda"), workspace=ws, n_new=new,
                            lse_out=lse)
        assert ws.status() == dsa.DSA_OK
        return o, lse


@pytest.mark.parametrize("causal,block", [(True, True), (False, True), (False, False)])
def test_dense_is_the_plain_definition(causal, block):
    c = dict(n=[0, 37, 5], new=[6, 4, 0], B=6, G=2, Hkv=2, d=64, page=16, window=11, sinks=3, causal=causal, block=block)
    w = Window(c)
    want = plain.window_attn(w.q, w.k, w.v, w.table, w.max_pages, w.n, w.bk, w.bv, 11, 3, causal, w.new)
    for a, b in zip(w.want(), want):
        assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.isinf(a), torch.isinf(b))
        assert torch.allclose(torch.nan_to_num(a, neginf=0.0), torch.nan_to_num(b, neginf=0.0), rtol=1e-12, atol=1e-12)


@pytest.mark.gpu
@pytest.mark.parametrize("name", sorted(wm.WALKS))
def test_window(lib, name):
    w = Window(wm.WALKS[name])
    o, lse = w.run()
    plain.check_attention(o, lse, w.want(), name)
    for s, m in enumerate(w.new):
        assert (o[s, m:] == 5.0).all() and (lse[s, m:] == 5.0).all()


KV4 = {
    # more than 16 rows per KV head: shares that cut units, several stops a CTA; whole units; selected pages
    "short_and_long": dict(n=[[0, 40, 130, 1500][s % 4] for s in range(40)], B=20, G=1, Hkv=8, d=128, page=16),
    "prefix_alone": dict(n=[10 + 3 * s for s in range(64)], B=17, G=1, Hkv=8, d=64, page=32, block=False),
    "whole_units": dict(n=[(13 * s) % 150 for s in range(160)], B=17, G=1, Hkv=8, d=64, page=16),
    "whole_units_alone": dict(n=[(13 * s) % 150 for s in range(160)], B=17, G=1, Hkv=8, d=128, page=64, block=False),
    "selected": dict(n=[200 + s for s in range(48)], B=20, G=2, Hkv=8, d=128, page=16, kp=6),
    "fresh_padded": dict(n=[0 if s % 3 else 300 for s in range(48)], new=[(5 * s) % 21 for s in range(48)], B=20, G=2, Hkv=8, d=64,
                         page=64),
    # long units that end inside a page, beside short ones and fresh ones: V of a tile may be late where the
    # scores of two tiles on are there
    "late_values_g128": dict(n=[2500, 2500, 1079, 0, 452, 1862, 0, 2500, 0, 2389], B=2, G=128, Hkv=8, d=128, page=32),
    "late_values_alone": dict(n=[1739, 57, 0, 0, 596, 1739, 1739, 0, 574, 199, 1739, 785, 1095, 1323, 370, 1739, 989, 1739], B=33, G=1,
                              Hkv=8, d=128, page=64, block=False),
    "late_values_selected": dict(n=[816, 0, 378, 0, 685, 270, 65, 198, 816, 592, 295, 749, 0, 302, 816, 816, 559, 0, 617, 816] * 2, B=1,
                                 G=33, Hkv=8, d=64, page=64, kp=17),
    "late_values_padded": dict(n=[1, 595, 568, 217, 600, 0, 274, 0, 288, 200, 570, 600, 0, 0, 92], B=7, G=33, Hkv=8, d=128, page=64,
                               new=[7, 7, 7, 0, 6, 7, 3, 7, 6, 7, 5, 7, 7, 7, 7]),
    # at most 16 rows
    "few_rows": dict(n=[0 if s % 4 == 0 else 500 + s for s in range(60)], B=2, G=4, Hkv=8, d=128, page=16),
}


class FourBits:
    """Inputs of a dsa_kv4_attn call of KV4."""

    def __init__(self, c):
        g = torch.Generator().manual_seed(1)
        self.c, S, B, Hkv, d, page, n = c, len(c["n"]), c["B"], c["Hkv"], c["d"], c["page"], c["n"]
        self.new, kp = c.get("new") or [B] * S, c.get("kp", 0)
        self.max_pages = max(-(-x // page) for x in n)
        self.n_phys = S * self.max_pages
        self.table = torch.randperm(self.n_phys, generator=g).view(S, -1).to(torch.int32)
        self.codes = [torch.randint(0, 256, (self.n_phys, Hkv, page, d // 2), generator=g, dtype=torch.uint8) for _ in range(2)]
        self.scales = [(torch.randint(16, 32, (self.n_phys, Hkv, page, d // 32), generator=g).float() / 128).to(BF) for _ in range(2)]
        self.q = torch.randn(S, B, Hkv * c["G"], d, generator=g).to(BF)
        self.bk = self.bv = self.idx = self.cnt = None
        if c.get("block", True):
            self.bk, self.bv = (torch.randn(S, B, Hkv, d, generator=g).to(BF) for _ in range(2))
        if kp:
            self.idx, self.cnt = torch.full((S, Hkv, kp), -1, dtype=torch.int32), torch.zeros(S, Hkv, dtype=torch.int32)
            for s in range(S):
                for h in range(Hkv):
                    take = torch.randperm(-(-n[s] // page), generator=g)[: kp - h % 3].sort().values
                    self.idx[s, h, : len(take)], self.cnt[s, h] = take.to(torch.int32), len(take)

    def want(self):
        c, page = self.c, self.c["page"]
        values = [plain.kv4_values(a, b) for a, b in zip(self.codes, self.scales)]

        def keys(s, h):
            t = torch.arange(c["n"][s])
            if self.idx is not None:
                t = (self.idx[s, h, : int(self.cnt[s, h])].long()[:, None] * page + torch.arange(page)).flatten()
                t = t[t < c["n"][s]]
            phys = self.table[s].long()[t // page]
            k, v = values[0][phys, h, t % page], values[1][phys, h, t % page]
            if self.bk is not None:
                m = self.new[s]
                k, v = torch.cat((k, self.bk[s, :m, h].to(F64))), torch.cat((v, self.bv[s, :m, h].to(F64)))
            return k, v

        return dense(self.q, keys, lambda s: torch.ones(c["B"], 1, dtype=torch.bool), c["Hkv"], self.new)

    def run(self, times=1):
        c, up = self.c, lambda t: None if t is None else t.cuda()  # noqa: E731
        S, B, Hq, d = self.q.shape
        tab = up(self.table)
        dims = dsa.make_dims(S, B, Hq, c["Hkv"], d, c["page"], self.max_pages, max(1, c.get("kp", 0)), self.n_phys, tab)
        ws = dsa.Workspace(dsa.kv4_workspace_size(dims))
        o, lse = torch.full((S, B, Hq, d), 5.0, dtype=BF, device="cuda"), torch.full((S, B, Hq), 5.0, device="cuda")
        n = torch.tensor(c["n"], dtype=torch.int32, device="cuda")
        new = None if "new" not in c else torch.tensor(self.new, dtype=torch.int32, device="cuda")
        cache = dsa.Kv4Cache(up(self.codes[0]), up(self.codes[1]), up(self.scales[0]), up(self.scales[1]))
        q, idx, cnt, bk, bv = map(up, (self.q, self.idx, self.cnt, self.bk, self.bv))
        first = None
        for _ in range(times):
            dsa.dsa_kv4_attn(q, cache, idx, bk, bv, o, dims=dims, n_ctx=n, idx_cnt=cnt, workspace=ws, n_new=new, lse_out=lse)
            if first is None:
                first = o.clone(), lse.clone()
            assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
        assert ws.status() == dsa.DSA_OK
        return o, lse


@pytest.mark.gpu
@pytest.mark.parametrize("name", sorted(KV4))
def test_four_bits(lib, name):
    """Thirty calls with the same bits, which are the definition's."""
    f = FourBits(KV4[name])
    o, lse = f.run(30)
    plain.check_attention(o, lse, f.want(), name)
    for s, m in enumerate(f.new):
        assert (o[s, m:] == 5.0).all() and (lse[s, m:] == 5.0).all()
