"""The 4-bit cache: stored codes bit for bit, loads, attention over it, refusals."""
import ctypes

import pytest
import torch

import plain
from block_sparse_attention_27_b200 import build, dsa

BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    build.build()
    return dsa.load()


def same(a, b):
    """Equal bit for bit, NaN where the other is NaN."""
    a, b = a.cpu(), b.cpu()
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a), torch.nan_to_num(b))


def awkward(S, B, Hkv, d, seed):
    """Rows that meet the format's borders among ordinary ones."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(S, B, Hkv, d, generator=g)
    x = x * torch.exp2(torch.randint(-20, 20, (S, B, Hkv, 1), generator=g).float())
    x = x.to(BF)
    flat = x.view(-1, d)
    rows = [torch.zeros(d), torch.full((d,), 7 * 1.0625), torch.arange(d) % 15 - 7.0, (torch.arange(d) % 15 - 7.0) / 2 + 0.25,
            torch.full((d,), 2.0 ** -101), torch.full((d,), 2.0 ** -100), torch.full((d,), -2.0 ** 119), torch.full((d,), 2.0 ** 120),
            torch.full((d,), -0.0), torch.full((d,), float("inf"))]
    for i, r in enumerate(rows[: flat.shape[0]]):
        flat[i] = r.to(BF)
    if flat.shape[0] > len(rows):
        flat[len(rows), d // 2] = float("nan")
    return x


def test_plain_format():
    """The definition itself: scales of five significant bits, nothing clipped, ties to even."""
    assert plain.kv4_scale(7.0) == 1.0 and plain.kv4_scale(7 * 1.0625) == 1.0625
    assert plain.kv4_scale(7.03125) == 1.0625 and plain.kv4_scale(0.0) == 0.0
    codes, s = plain.kv4_codes([7.0, 2.5, 3.5, -0.5, -6.5] + [0.0] * 27)
    assert s == [1.0] and codes[:5] == [15, 10, 12, 8, 2]
    x = torch.randn(4, 64, dtype=torch.float64, generator=torch.Generator().manual_seed(0)).to(BF)
    v = plain.kv4_values(*plain.kv4_pack(x))
    step = plain.kv4_pack(x)[1].double().repeat_interleave(32, -1)
    assert ((v - x.double()).abs() <= step / 2).all()
    assert torch.equal(v.to(BF).double(), v)  # every value held is a bf16 number


@pytest.mark.gpu
@pytest.mark.parametrize("S,B,Hkv,d,page,n,new", [
    (1, 1, 1, 64, 16, [0], None),
    (2, 33, 2, 128, 16, [5, 90], None),
    (3, 20, 3, 64, 64, [60, 0, 7], [20, 0, 9]),
    (1, 70, 8, 128, 32, [31], None),
])
def test_store_and_load(lib, S, B, Hkv, d, page, n, new):
    k, v = awkward(S, B, Hkv, d, 1), awkward(S, B, Hkv, d, 2).flip(1)
    max_pages = -(-(max(n) + B) // page)
    n_phys = S * max_pages + 1
    table = torch.randperm(n_phys, generator=torch.Generator().manual_seed(3))[: S * max_pages].view(S, -1).to(torch.int32)
    tab = table.cuda()
    dims = dsa.make_dims(S, B, Hkv, Hkv, d, page, max_pages, 1, n_phys, tab)
    cache = dsa.Kv4Cache.zeros(n_phys, Hkv, page, d)
    for t, fill in ((cache.k, 0xA5), (cache.v, 0x5A), (cache.k_scale, 3.0), (cache.v_scale, 3.0)):
        t.fill_(fill)
    ws = dsa.Workspace(dsa.WORKSPACE_HEADER_BYTES)
    dn = torch.tensor(n, dtype=torch.int32, device="cuda")
    dnew = None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda")
    dsa.dsa_kv4_store(k.cuda(), v.cuda(), cache, dims=dims, n_ctx=dn, workspace=ws, n_new=dnew)
    ko, vo = (torch.full((S, B, Hkv, d), 5.0, dtype=BF, device="cuda") for _ in range(2))
    dsa.dsa_kv4_load(cache, ko, vo, dims=dims, start=dn, workspace=ws, n_new=dnew)
    assert ws.status() == dsa.DSA_OK
    want = [torch.full((n_phys, Hkv, page, d // 2), f, dtype=torch.uint8) for f in (0xA5, 0x5A)]
    want += [torch.full((n_phys, Hkv, page, d // 32), 3.0, dtype=BF) for _ in range(2)]
    for side, x in enumerate((k, v)):
        codes, scales = plain.kv4_pack(x)
        values = plain.kv4_values(codes, scales)
        got = (ko, vo)[side].cpu()
        for s in range(S):
            m = B if new is None else new[s]
            assert same(got[s, :m].double(), values[s, :m]) and (got[s, m:] == 5.0).all()
            for b in range(m):
                t = n[s] + b
                at = (int(table[s, t // page]), slice(None), t % page)
                want[side][at], want[2 + side][at] = codes[s, b], scales[s, b]
    assert torch.equal(cache.k.cpu(), want[0]) and torch.equal(cache.v.cpu(), want[1])
    assert same(cache.k_scale, want[2]) and same(cache.v_scale, want[3])


@pytest.mark.gpu
def test_all_significands(lib):
    """Every significand of a value under every significand of its group's largest, six exponents
    down, against the definition in integers."""
    g = torch.Generator().manual_seed(4)
    a = torch.arange(128, 256).double()
    x = (a[:, None] * torch.exp2(-torch.arange(6).double())).reshape(-1)  # 768 values
    x = torch.cat([x, x[:7]]).view(25, 31).expand(128, 25, 31)
    x = torch.where(x > a[:, None, None], x / 2, x) * torch.where(torch.rand(128, 25, 31, generator=g) < 0.5, -1, 1)
    x = torch.cat([a[:, None, None].expand(128, 25, 1), x], -1) * torch.exp2(torch.randint(-60, 60, (128, 25, 1), generator=g).double())
    x = x.reshape(1, 800, 2, 64).to(BF)
    dims = dsa.make_dims(1, 800, 2, 2, 64, 16, 50, 1, 50)
    cache = dsa.Kv4Cache.zeros(50, 2, 16, 64)
    ws = dsa.Workspace(dsa.WORKSPACE_HEADER_BYTES)
    dsa.dsa_kv4_store(x.cuda(), -x.cuda(), cache, dims=dims, n_ctx=torch.zeros(1, dtype=torch.int32, device="cuda"), workspace=ws)
    assert ws.status() == dsa.DSA_OK
    for y, codes, scales in ((x, cache.k, cache.k_scale), (-x, cache.v, cache.v_scale)):
        c, s = plain.kv4_pack(y)
        assert torch.equal(codes.cpu().transpose(1, 2).reshape(1, 800, 2, 32), c)
        assert torch.equal(scales.cpu().transpose(1, 2).reshape(1, 800, 2, 2), s)


@pytest.mark.gpu
@pytest.mark.parametrize("Hkv,d", [(1, 128), (3, 64)])
def test_many_tokens_as_in_small_calls(lib, Hkv, d):
    """A long padded batch, which takes several tokens a block of threads, leaves what calls of a
    few hundred tokens leave, in the cache and on the way out."""
    S, B, page, part = 3, 4001, 16, 667
    x = torch.randn(S, B, Hkv, d, generator=torch.Generator().manual_seed(5)).to(BF).cuda()
    n, new = [5, 0, 99], [B, 1, 3990]
    max_pages = -(-(max(n) + B) // page)
    table = torch.randperm(S * max_pages, generator=torch.Generator().manual_seed(6)).view(S, -1).to(torch.int32).cuda()
    caches, outs = [], []
    for step in (B, part):
        cache = dsa.Kv4Cache.zeros(S * max_pages, Hkv, page, d)
        out = torch.full((2, S, B, Hkv, d), 5.0, dtype=BF, device="cuda")
        ws = dsa.Workspace(dsa.WORKSPACE_HEADER_BYTES)
        for b in range(0, B, step):
            m = min(step, B - b)
            dims = dsa.make_dims(S, m, Hkv, Hkv, d, page, max_pages, 1, S * max_pages, table)
            at = torch.tensor([i + b for i in n], dtype=torch.int32, device="cuda")
            live = torch.tensor([min(max(i - b, 0), m) for i in new], dtype=torch.int32, device="cuda")
            y = x[:, b:b + m].contiguous()
            dsa.dsa_kv4_store(y, -y, cache, dims=dims, n_ctx=at, workspace=ws, n_new=live)
            o = torch.full((2, S, m, Hkv, d), 5.0, dtype=BF, device="cuda")
            dsa.dsa_kv4_load(cache, o[0], o[1], dims=dims, start=at, workspace=ws, n_new=live)
            out[:, :, b:b + m] = o
        assert ws.status() == dsa.DSA_OK
        caches.append(cache)
        outs.append(out)
    a, b = caches
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v) and torch.equal(a.k_scale, b.k_scale) and torch.equal(a.v_scale, b.v_scale)
    assert torch.equal(*outs) and (outs[0][:, 1, 1:] == 5.0).all() and (outs[0][:, 2, 3990:] == 5.0).all()


@pytest.mark.gpu
def test_bad_pages_are_skipped_and_reported(lib):
    S, B, Hkv, d, page = 1, 8, 2, 64, 16
    x = torch.randn(S, B, Hkv, d, generator=torch.Generator().manual_seed(0)).to(BF).cuda()
    for n, table in ((28, [0, 2]), (28, [0, -7]), (30, [0, 1]), (-1, [0, 1]), (2_147_483_645, [0, 1])):
        tab = torch.tensor([table], dtype=torch.int32, device="cuda")
        dims = dsa.make_dims(S, B, Hkv, Hkv, d, page, 2, 1, 2, tab)
        dn = torch.tensor([n], dtype=torch.int32, device="cuda")
        cache, ws = dsa.Kv4Cache.zeros(2, Hkv, page, d), dsa.Workspace(dsa.WORKSPACE_HEADER_BYTES)
        dsa.dsa_kv4_store(x, x, cache, dims=dims, n_ctx=dn, workspace=ws)
        assert ws.status() == dsa.DSA_ERR_BAD_INDEX, (n, table)
        good = {(table[t // page], t % page) for t in range(n, n + B) if 0 <= n and t // page < 2 and 0 <= table[t // page] < 2}
        assert {(p, i) for p in range(2) for i in range(page) if cache.k[p, 0, i].any()} == good
        ko, vo = (torch.full((S, B, Hkv, d), 5.0, dtype=BF, device="cuda") for _ in range(2))
        ws = dsa.Workspace(dsa.WORKSPACE_HEADER_BYTES)
        dsa.dsa_kv4_load(cache, ko, vo, dims=dims, start=dn, workspace=ws)
        assert ws.status() == dsa.DSA_ERR_BAD_INDEX
        assert int((ko[0, :, 0, 0] == 5.0).sum()) == B - len(good)


class Case:
    def __init__(self, S, B, Hq, Hkv, d, page, n, kp=None, table=True, new=None, block=True, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.shape = S, B, Hq, Hkv, d, page
        self.n = torch.tensor(n, dtype=torch.int32)
        self.new = None if new is None else torch.tensor(new, dtype=torch.int32)
        self.max_pages = max(1, max(-(-x // page) for x in n)) + 1
        self.n_phys = S * self.max_pages + 2
        self.table = None
        if table:
            self.table = torch.randperm(self.n_phys, generator=g)[: S * self.max_pages].view(S, -1).to(torch.int32)
        self.q = torch.randn(S, B, Hq, d, generator=g).to(BF)
        self.codes, self.scales = [], []
        for _ in range(2):  # any codes are legal, 0 (value -8 s) among them
            self.codes.append(torch.randint(0, 256, (self.n_phys, Hkv, page, d // 2), generator=g, dtype=torch.uint8))
            s = torch.randint(16, 32, (self.n_phys, Hkv, page, d // 32), generator=g).float() / 128
            self.scales.append(s.to(BF))
        self.bk, self.bv = ((torch.randn(S, B, Hkv, d, generator=g).to(BF) for _ in range(2)) if block else (None, None))
        self.idx = self.cnt = None
        self.kmax = 1
        if kp is not None:
            self.kmax = kp
            self.idx = torch.full((S, Hkv, kp), -1, dtype=torch.int32)
            self.cnt = torch.zeros((S, Hkv), dtype=torch.int32)
            for s in range(S):
                np_ = -(-int(n[s]) // page)
                for h in range(Hkv):
                    c = min(kp, np_) if h % 2 == 0 else min(kp, np_) // 2  # a different count per head
                    self.idx[s, h, :c] = torch.randperm(np_, generator=g)[:c].sort().values.to(torch.int32) if np_ else 0
                    self.cnt[s, h] = c

    def want(self):
        values = [plain.kv4_values(c, s) for c, s in zip(self.codes, self.scales)]
        return plain.kv4_attn(self.q, values, self.table, self.max_pages, self.n, self.idx, self.cnt, self.bk, self.bv, self.new)

    def device(self):
        S, B, Hq, Hkv, d, page = self.shape
        up = lambda t: None if t is None else t.cuda()  # noqa: E731
        self.tab = up(self.table)
        self.dims = dsa.make_dims(S, B, Hq, Hkv, d, page, self.max_pages, self.kmax, self.n_phys, self.tab)
        self.ws = dsa.Workspace(dsa.kv4_workspace_size(self.dims))
        self.cache = dsa.Kv4Cache(up(self.codes[0]), up(self.codes[1]), up(self.scales[0]), up(self.scales[1]))
        self.dev = dict(q=up(self.q), idx=up(self.idx), bk=up(self.bk), bv=up(self.bv))
        self.kw = dict(n_ctx=up(self.n), idx_cnt=up(self.cnt), n_new=up(self.new))
        self.o = torch.full((S, B, Hq, d), 5.0, dtype=BF, device="cuda")
        self.lse = torch.full((S, B, Hq), 5.0, device="cuda")
        return self

    def call(self, stream=None, **kw):
        d = self.dev
        a = dict(dims=self.dims, workspace=self.ws, lse_out=self.lse, **self.kw)
        a.update(kw)
        dsa.dsa_kv4_attn(d["q"], self.cache, d["idx"], d["bk"], d["bv"], self.o, stream, **a)
        return self

    def check(self, what):
        assert self.ws.status() == dsa.DSA_OK
        plain.check_attention(self.o, self.lse, self.want(), what)
        if self.new is not None:
            for s, m in enumerate(self.new.tolist()):
                assert (self.o[s, m:] == 5.0).all() and (self.lse[s, m:] == 5.0).all()


CASES = {
    "one_token_alone": dict(S=1, B=1, Hq=1, Hkv=1, d=64, page=16, n=[0]),
    "one_key": dict(S=1, B=1, Hq=4, Hkv=1, d=128, page=16, n=[1], block=False),
    "no_key": dict(S=2, B=3, Hq=4, Hkv=1, d=128, page=16, n=[0, 20], block=False),
    "decode": dict(S=4, B=1, Hq=8, Hkv=2, d=128, page=16, n=[1, 100, 1000, 517]),
    "decode_g7": dict(S=2, B=1, Hq=14, Hkv=2, d=128, page=64, n=[400, 65]),
    "decode_g16": dict(S=1, B=1, Hq=16, Hkv=1, d=64, page=32, n=[300]),
    "rows_17": dict(S=1, B=17, Hq=2, Hkv=2, d=128, page=16, n=[140]),
    "block_dense": dict(S=2, B=32, Hq=8, Hkv=2, d=128, page=16, n=[700, 33]),
    "block_sparse": dict(S=2, B=32, Hq=8, Hkv=2, d=128, page=16, n=[900, 300], kp=12),
    "sparse_counts_zero": dict(S=2, B=4, Hq=4, Hkv=2, d=64, page=16, n=[5, 0], kp=3),
    "sparse_no_block": dict(S=2, B=4, Hq=4, Hkv=2, d=64, page=16, n=[70, 0], kp=3, block=False),
    "sparse_decode_p64": dict(S=2, B=1, Hq=8, Hkv=2, d=128, page=64, n=[900, 511], kp=6),
    "g7_two_row_tiles": dict(S=1, B=32, Hq=28, Hkv=4, d=128, page=64, n=[333], kp=4),
    "rows_256": dict(S=1, B=64, Hq=4, Hkv=1, d=64, page=32, n=[257]),
    "rows_256_g1": dict(S=1, B=256, Hq=1, Hkv=1, d=128, page=16, n=[31]),
    "padded": dict(S=3, B=20, Hq=4, Hkv=1, d=128, page=16, n=[40, 0, 300], new=[20, 0, 3]),
    "padded_decode": dict(S=3, B=1, Hq=4, Hkv=1, d=128, page=16, n=[40, 10, 300], new=[1, 0, 1]),
    "identity": dict(S=3, B=2, Hq=4, Hkv=2, d=128, page=32, n=[64, 200, 31], table=False),
    "rows_12": dict(S=2, B=3, Hq=8, Hkv=2, d=128, page=32, n=[500, 129]),
    "rows_16_sparse": dict(S=2, B=4, Hq=8, Hkv=2, d=128, page=16, n=[500, 129], kp=7),
    "few_rows_padded": dict(S=4, B=2, Hq=4, Hkv=2, d=64, page=16, n=[500, 0, 1, 257], new=[2, 2, 0, 1]),
    "many_units": dict(S=200, B=1, Hq=8, Hkv=8, d=64, page=16, n=[(7 * i) % 100 for i in range(200)]),
    "long_block": dict(S=1, B=20, Hq=1, Hkv=1, d=64, page=16, n=[6001]),
    "long": dict(S=1, B=2, Hq=2, Hkv=1, d=128, page=16, n=[6001]),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_attention_against_definition(lib, name):
    Case(**CASES[name]).device().call().check(name)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["decode", "block_sparse", "rows_17", "long"])
def test_repeats_bit_for_bit(lib, name):
    c = Case(**CASES[name]).device().call()
    o, lse = c.o.clone(), c.lse.clone()
    c.ws.buf[dsa.WORKSPACE_HEADER_BYTES:].fill_(0xFF)
    c.call()
    assert torch.equal(c.o, o) and torch.equal(c.lse, lse)
    c.o.fill_(5.0)
    c.call(lse_out=None)
    assert torch.equal(c.o, o) and c.ws.status() == dsa.DSA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["decode", "block_dense", "padded"])
def test_hidden_tokens_never_reach_the_output(lib, name):
    """NaN scales in every token past n_ctx and in pages nobody holds; NaN in missing tokens' rows."""
    c = Case(**CASES[name])
    S, B, Hq, Hkv, d, page = c.shape
    want = c.want()
    keep = torch.zeros(c.n_phys, page, dtype=torch.bool)
    for s in range(S):
        for t in range(int(c.n[s])):
            keep[int(c.table[s, t // page]), t % page] = True
        for lp in range(-(-int(c.n[s]) // page), c.max_pages):
            c.table[s, lp] = -1
        if c.new is not None:
            c.bk[s, int(c.new[s]):] = float("nan")
            c.bv[s, int(c.new[s]):] = float("nan")
    for x in c.scales:
        x[(~keep)[:, None].expand(-1, Hkv, -1)] = float("nan")
    c.device().call()
    assert c.ws.status() == dsa.DSA_OK
    plain.check_attention(c.o, c.lse, want, name)


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 32])
def test_bad_indices_are_skipped_and_reported(lib, B):
    c = Case(S=1, B=B, Hq=4, Hkv=2, d=128, page=16, n=[200], kp=8)
    good = c.idx.clone()
    c.idx[0, 0, 2], c.idx[0, 1, 1] = 13, -4  # a page past the prefix, a negative one
    c.table[0, int(good[0, 0, 5])] = c.n_phys + 5
    drop = {(0, 2), (1, 1), (0, 5)}
    for h in range(2):  # head 1 may hold the page whose entry is bad, too
        for i in range(int(c.cnt[0, h])):
            if int(c.idx[0, h, i]) == int(good[0, 0, 5]):
                drop.add((h, i))
    ref = Case(S=1, B=B, Hq=4, Hkv=2, d=128, page=16, n=[200], kp=8)
    for h in range(2):
        left = [int(good[0, h, i]) for i in range(int(ref.cnt[0, h])) if (h, i) not in drop]
        ref.idx[0, h, : len(left)], ref.cnt[0, h] = torch.tensor(left, dtype=torch.int32), len(left)
    c.device().call()
    assert c.ws.status() == dsa.DSA_ERR_BAD_INDEX
    plain.check_attention(c.o, c.lse, ref.want(), "bad indices")
    for change in (dict(idx_cnt=torch.full((1, 2), 9, dtype=torch.int32, device="cuda")),
                   dict(n_ctx=torch.tensor([100_000], dtype=torch.int32, device="cuda")),
                   dict(n_new=torch.tensor([B + 1], dtype=torch.int32, device="cuda"))):
        c = Case(S=1, B=B, Hq=4, Hkv=2, d=128, page=16, n=[200], kp=8).device().call(**change)
        assert c.ws.status() == dsa.DSA_ERR_BAD_INDEX, change


@pytest.mark.gpu
@pytest.mark.parametrize("B", [1, 20])
def test_far_pages_of_a_large_cache(lib, B):
    """Rows whose byte offsets pass 32 bits, in both kernels' ways to read them."""
    c = Case(S=1, B=B, Hq=4, Hkv=1, d=128, page=64, n=[150])
    want = c.want()
    n_phys = 1_200_000  # 4.9e9 bytes of codes a side
    far = torch.tensor([[n_phys - 1, 7, n_phys - 3, 1_100_000]], dtype=torch.int32)
    big = [torch.empty(n_phys, 1, 64, 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
    big += [torch.empty(n_phys, 1, 64, 4, dtype=BF, device="cuda") for _ in range(2)]
    for t, src in zip(big, (*c.codes, *c.scales)):
        for lp in range(3):
            t[int(far[0, lp])] = src[int(c.table[0, lp])].cuda()
    c.device()
    tab = far.cuda()
    c.dims = dsa.make_dims(1, B, 4, 1, 128, 64, 4, 1, n_phys, tab)
    c.ws = dsa.Workspace(dsa.kv4_workspace_size(c.dims))
    c.cache = dsa.Kv4Cache(*big)
    c.call()
    assert c.ws.status() == dsa.DSA_OK
    plain.check_attention(c.o, c.lse, want, "far pages")


OK, ODD = 1 << 20, (1 << 20) + 2


def test_refusals_on_host(lib):
    base = dict(S=2, B=8, Hq=8, Hkv=2, d=128, page=16, max_pages=64, kmax=4, n_phys=128)
    inv, uns, small = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED, dsa.DSA_ERR_WORKSPACE_TOO_SMALL
    good = dict(k=OK, v=OK, ks=OK, vs=OK, a=OK, b=OK, n=OK, ws=OK, nbytes=1 << 40, q=OK, o=OK, idx=OK, cnt=OK)

    def each(dims=None, **kw):
        x = {**good, **kw}
        dm = dsa.make_dims(**{**base, **(dims or {})})
        c = dsa.dsa_kv4(x["k"], x["v"], x["ks"], x["vs"])
        return {
            "store": lib.dsa_kv4_store(x["a"], x["b"], ctypes.byref(c), None, ctypes.byref(dm), x["n"], None, x["ws"], x["nbytes"]),
            "load": lib.dsa_kv4_load(ctypes.byref(c), x["a"], x["b"], None, ctypes.byref(dm), x["n"], None, x["ws"], x["nbytes"]),
            "attn": lib.dsa_kv4_attn(x["q"], ctypes.byref(c), x["idx"], x["a"], x["b"], x["o"], None, ctypes.byref(dm), x["n"],
                                     x["cnt"], None, x["ws"], x["nbytes"]),
        }

    for name in ("k", "v", "ks", "vs", "a", "b", "ws"):
        for bad in (ODD, None):
            assert set(each(**{name: bad}).values()) == {inv}, (name, bad)
    assert set(each(n=None).values()) == {inv}
    for name in ("q", "o"):
        assert each(**{name: ODD, "nbytes": 0})["attn"] == inv and each(**{name: None, "nbytes": 0})["attn"] == inv
    assert each(idx=None, nbytes=0)["attn"] == inv and each(cnt=None, nbytes=0)["attn"] == inv
    assert set(each(nbytes=4095).values()) == {small}
    assert set(each(dims=dict(d=96)).values()) == {uns}
    assert each(dims=dict(B=128), nbytes=0)["attn"] == uns and each(dims=dict(B=128), nbytes=0)["store"] == small
    assert each(dims=dict(B=1, Hq=258), nbytes=0)["attn"] == uns
    assert dsa.kv4_workspace_size(dsa.make_dims(**{**base, "B": 128})) == 0
    assert dsa.kv4_launches(dsa.make_dims(**base), True) >= 1
    assert dsa.kernels_per_call(4) == dsa.kernels_per_call(5) == 1


@pytest.mark.gpu
def test_binding_refusals(lib):
    c = Case(S=1, B=2, Hq=2, Hkv=1, d=64, page=16, n=[20], kp=2).device()
    with pytest.raises(ValueError):
        dsa.Kv4Cache(c.cache.k, c.cache.v, c.cache.k_scale[..., :1], c.cache.v_scale)
    with pytest.raises(TypeError):
        dsa.Kv4Cache(c.cache.k.to(torch.int8), c.cache.v, c.cache.k_scale, c.cache.v_scale)
    with pytest.raises(ValueError):
        c.call(idx_cnt=c.kw["idx_cnt"][:, :0])
    with pytest.raises(dsa.DsaError):
        c.call(idx_cnt=None)
    other = dsa.make_dims(1, 2, 2, 1, 64, 32, 3, 2, c.n_phys)
    with pytest.raises(ValueError):
        c.call(dims=other)
    k = torch.zeros(1, 2, 1, 64, dtype=BF)
    with pytest.raises(TypeError):
        dsa.dsa_kv4_store(k, k, c.cache, dims=c.dims, n_ctx=c.kw["n_ctx"], workspace=c.ws)
