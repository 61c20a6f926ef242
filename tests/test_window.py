"""dsa_window_attn against its definition in 64 bits, its masks and edges, refusals."""
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


class Case:
    """Inputs of one call on the CPU, and the call on the GPU."""

    def __init__(self, S, B, Hq, Hkv, d, page, n, window, sinks, causal, table=True, new=None, block=True, seed=0,
                 spare=2, scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.shape = S, B, Hq, Hkv, d, page
        self.n = torch.tensor(n, dtype=torch.int32)
        self.new = None if new is None else torch.tensor(new, dtype=torch.int32)
        self.window, self.sinks, self.causal = window, sinks, causal
        self.max_pages = max(1, max(-(-x // page) for x in n)) + 1
        self.n_phys = S * self.max_pages + spare
        self.table = None
        if table:
            self.table = torch.randperm(self.n_phys, generator=g)[: S * self.max_pages].view(S, -1).to(torch.int32)

        def rnd(*shape):
            return (scale * torch.randn(shape, generator=g)).to(BF)

        self.q = rnd(S, B, Hq, d)
        self.k, self.v = rnd(self.n_phys, Hkv, page, d), rnd(self.n_phys, Hkv, page, d)
        self.bk, self.bv = (rnd(S, B, Hkv, d), rnd(S, B, Hkv, d)) if block else (None, None)

    def want(self):
        return plain.window_attn(self.q, self.k, self.v, self.table, self.max_pages, self.n, self.bk, self.bv, self.window,
                                 self.sinks, self.causal, self.new)

    def device(self):
        S, B, Hq, Hkv, d, page = self.shape
        up = lambda t: None if t is None else t.cuda()  # noqa: E731
        self.tab = up(self.table)
        self.dims = dsa.make_dims(S, B, Hq, Hkv, d, page, self.max_pages, 1, self.n_phys, self.tab)
        self.ws = dsa.Workspace(dsa.window_workspace_size(self.dims))
        self.dev = [up(t) for t in (self.q, self.k, self.v, self.bk, self.bv)]
        self.dn, self.dnew = up(self.n), up(self.new)
        self.o = torch.full((S, B, Hq, d), 5.0, dtype=BF, device="cuda")
        self.lse = torch.full((S, B, Hq), 5.0, device="cuda")
        return self

    def call(self, stream=None, **kw):
        a = dict(dims=self.dims, window=self.window, sinks=self.sinks, causal=self.causal, n_ctx=self.dn, workspace=self.ws,
                 n_new=self.dnew, lse_out=self.lse)
        a.update(kw)
        dsa.dsa_window_attn(*self.dev, self.o, stream, **a)
        return self

    def check(self, what="", status=dsa.DSA_OK):
        assert self.ws.status() == status
        plain.check_attention(self.o, self.lse, self.want(), what)
        if self.new is not None:  # rows of tokens that do not exist stay as they were
            for s, m in enumerate(self.new.tolist()):
                assert (self.o[s, m:] == 5.0).all() and (self.lse[s, m:] == 5.0).all()


CASES = {
    "one_token_no_prefix": dict(S=1, B=1, Hq=1, Hkv=1, d=64, page=16, n=[0], window=1, sinks=0, causal=True),
    "one_key_prefix": dict(S=1, B=1, Hq=4, Hkv=1, d=128, page=16, n=[1], window=2, sinks=0, causal=True),
    "decode_ragged": dict(S=5, B=1, Hq=8, Hkv=2, d=128, page=16, n=[0, 1, 130, 777, 1500], window=256, sinks=4, causal=True),
    "window_one": dict(S=2, B=9, Hq=4, Hkv=2, d=64, page=16, n=[33, 50], window=1, sinks=0, causal=False),
    "window_one_sinks": dict(S=2, B=9, Hq=4, Hkv=2, d=64, page=16, n=[33, 50], window=1, sinks=20, causal=True),
    "step_both_ways": dict(S=2, B=32, Hq=8, Hkv=2, d=128, page=16, n=[1000, 613], window=200, sinks=16, causal=False),
    "window_below_block": dict(S=1, B=40, Hq=4, Hkv=1, d=128, page=32, n=[100], window=7, sinks=3, causal=False),
    "window_below_block_causal": dict(S=1, B=40, Hq=4, Hkv=1, d=128, page=32, n=[100], window=7, sinks=3, causal=True),
    "sinks_past_prefix": dict(S=2, B=20, Hq=2, Hkv=2, d=64, page=64, n=[5, 0], window=4, sinks=12, causal=False),
    "sinks_past_prefix_causal": dict(S=2, B=20, Hq=2, Hkv=2, d=64, page=64, n=[5, 0], window=4, sinks=12, causal=True),
    "sinks_meet_window": dict(S=1, B=3, Hq=2, Hkv=1, d=64, page=16, n=[300], window=250, sinks=60, causal=True),
    "everything_visible": dict(S=1, B=17, Hq=14, Hkv=2, d=128, page=64, n=[777], window=1 << 30, sinks=0, causal=False),
    "g7": dict(S=1, B=32, Hq=28, Hkv=4, d=128, page=64, n=[500], window=128, sinks=64, causal=False),
    "g1": dict(S=1, B=130, Hq=2, Hkv=2, d=64, page=16, n=[40], window=90, sinks=1, causal=True),
    "g128": dict(S=1, B=2, Hq=128, Hkv=1, d=64, page=16, n=[200], window=100, sinks=1, causal=True),
    "g96": dict(S=1, B=3, Hq=96, Hkv=1, d=128, page=16, n=[90], window=64, sinks=1, causal=False),
    "prompt": dict(S=1, B=400, Hq=4, Hkv=2, d=128, page=16, n=[0], window=150, sinks=10, causal=True),
    "prompt_second_part": dict(S=2, B=260, Hq=2, Hkv=1, d=64, page=32, n=[131, 5], window=100, sinks=40, causal=True),
    "prompt_padded": dict(S=3, B=150, Hq=4, Hkv=1, d=128, page=16, n=[20, 0, 300], window=60, sinks=2, causal=True,
                          new=[150, 0, 77]),
    "padded_both_ways": dict(S=3, B=33, Hq=4, Hkv=1, d=64, page=16, n=[20, 0, 300], window=1000, sinks=0, causal=False,
                             new=[1, 33, 16]),
    "prefix_alone": dict(S=3, B=8, Hq=4, Hkv=2, d=128, page=16, n=[0, 3, 200], window=5, sinks=0, causal=False, block=False),
    "prefix_alone_long": dict(S=1, B=32, Hq=8, Hkv=2, d=128, page=16, n=[2000], window=1100, sinks=33, causal=True, block=False),
    "identity_table": dict(S=3, B=4, Hq=4, Hkv=2, d=128, page=32, n=[700, 64, 65], window=300, sinks=8, causal=True, table=False),
    # at most 16 rows per KV head and tables of every kind, the other kernel's page sizes
    "few_rows_9_to_16": dict(S=2, B=3, Hq=8, Hkv=2, d=128, page=16, n=[400, 90], window=130, sinks=5, causal=True),
    "few_rows_both_ways": dict(S=2, B=16, Hq=2, Hkv=2, d=64, page=32, n=[200, 33], window=9, sinks=2, causal=False),
    "few_rows_p64": dict(S=3, B=1, Hq=7, Hkv=1, d=64, page=64, n=[1000, 63, 64], window=300, sinks=100, causal=True),
    "few_rows_long": dict(S=1, B=2, Hq=2, Hkv=1, d=128, page=16, n=[6001], window=1 << 20, sinks=0, causal=True),
    "rows_17": dict(S=1, B=17, Hq=1, Hkv=1, d=128, page=64, n=[300], window=200, sinks=7, causal=True),
    "identity_table_wide": dict(S=2, B=20, Hq=4, Hkv=2, d=128, page=16, n=[700, 129], window=400, sinks=20, causal=False, table=False),
    "identity_table_wide_p32": dict(S=2, B=20, Hq=4, Hkv=2, d=64, page=32, n=[700, 129], window=400, sinks=20, causal=True, table=False),
    "identity_table_wide_p64": dict(S=1, B=20, Hq=4, Hkv=2, d=128, page=64, n=[513], window=1000, sinks=0, causal=True, table=False),
    "many_units_few_rows": dict(S=200, B=1, Hq=8, Hkv=8, d=64, page=16, n=[i % 150 for i in range(200)], window=100, sinks=3,
                                causal=True),
    "many_units": dict(S=75, B=20, Hq=16, Hkv=16, d=64, page=16, n=[i % 9 for i in range(75)], window=6, sinks=3, causal=True,
                       new=[20 - i % 21 for i in range(75)]),
    "large_scores": dict(S=1, B=16, Hq=4, Hkv=1, d=128, page=16, n=[600], window=500, sinks=8, causal=True, scale=4.0),
}


@pytest.mark.gpu
@pytest.mark.parametrize("name", list(CASES))
def test_against_definition(lib, name):
    c = Case(**CASES[name]).device().call()
    c.check(name)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["decode_ragged", "step_both_ways", "prompt_padded", "g7"])
def test_repeats_bit_for_bit(lib, name):
    """The same call on a poisoned workspace and without its log-sum-exp: the same bits."""
    c = Case(**CASES[name]).device().call()
    o, lse = c.o.clone(), c.lse.clone()
    c.ws.buf[dsa.WORKSPACE_HEADER_BYTES:].fill_(0xFF)
    c.call()
    assert torch.equal(c.o, o) and torch.equal(c.lse, lse)
    c.o.fill_(5.0)
    c.call(lse_out=None)
    assert torch.equal(c.o, o) and c.ws.status() == dsa.DSA_OK


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
def test_hidden_tokens_never_reach_the_output(lib, causal):
    """NaN and infinities in every token that no query sees, in the pages' tails and in the rows of
    missing tokens; -1 in the table for pages without a visible token."""
    kw = dict(S=2, B=6, Hq=4, Hkv=2, d=128, page=16, n=[500, 331], window=100, sinks=20, causal=causal, new=[6, 4])
    c = Case(**kw)
    S, B, Hq, Hkv, d, page = c.shape
    want = c.want()
    keep = torch.zeros(c.n_phys, page, dtype=torch.bool)
    for s in range(S):
        n = int(c.n[s])
        for t in range(n):
            if t < c.sinks or n - t < c.window:
                keep[int(c.table[s, t // page]), t % page] = True
    for x, bad in ((c.k, float("nan")), (c.v, float("inf"))):
        x[(~keep)[:, None].expand(-1, Hkv, -1)] = bad
    for s in range(S):
        c.bk[s, int(c.new[s]):] = float("nan")
        c.bv[s, int(c.new[s]):] = float("nan")
        for lp in range(c.max_pages):
            if not keep[int(c.table[s, lp])].any():
                c.table[s, lp] = -1
    c.device().call()
    assert c.ws.status() == dsa.DSA_OK
    plain.check_attention(c.o, c.lse, want, "hidden tokens")


@pytest.mark.gpu
def test_masked_keys_of_one_query_do_not_disturb_another(lib):
    """NaN keys that only some queries of the tile see: the others' results are untouched."""
    c = Case(S=1, B=8, Hq=2, Hkv=1, d=64, page=16, n=[64], window=20, sinks=0, causal=True)
    want = c.want()
    t = 64 - 19  # visible to the first query alone
    c.k[int(c.table[0, t // 16]), 0, t % 16] = float("nan")
    c.device().call()
    assert torch.isnan(c.o[0, 0]).all()
    want[0][0, 0], want[1][0, 0] = float("nan"), float("nan")  # not compared
    plain.check_attention(c.o, c.lse, want, "other rows")


@pytest.mark.gpu
def test_bad_pages_and_lengths_are_reported(lib):
    kw = dict(S=1, B=2, Hq=2, Hkv=1, d=64, page=16, n=[100], window=60, sinks=0, causal=True)
    c = Case(**kw)
    c.table[0, 4] = c.n_phys  # tokens 64..79 cannot be read: skipped
    want_pages = c.table.clone()
    c.device().call()
    assert c.ws.status() == dsa.DSA_ERR_BAD_INDEX
    ref = Case(**kw)
    o = torch.zeros_like(c.o, dtype=torch.float64, device="cpu")
    for b in range(2):
        for h in range(2):
            toks = [t for t in range(100) if 100 + b - t < 60 and t // 16 != 4]
            ks = [plain.token_row(ref.k, want_pages, ref.max_pages, 16, 0, 0, t) for t in toks] + [ref.bk[0, u, 0] for u in range(b + 1)]
            vs = [plain.token_row(ref.v, want_pages, ref.max_pages, 16, 0, 0, t) for t in toks] + [ref.bv[0, u, 0] for u in range(b + 1)]
            o[0, b, h] = plain.attend(ref.q[0, b, h].double(), torch.stack(ks), torch.stack(vs))[0]
    assert (c.o.cpu().double() - o).abs().max() < 2e-2  # o is at most 1 in size: a few bf16 steps
    for n, new in (([10_000], None), ([-1], None), ([20], [3]), ([20], [-1])):
        c = Case(**kw)
        c.device()
        c.dn = torch.tensor(n, dtype=torch.int32, device="cuda")
        c.dnew = None if new is None else torch.tensor(new, dtype=torch.int32, device="cuda")
        c.call()
        assert c.ws.status() == dsa.DSA_ERR_BAD_INDEX, (n, new)
        assert torch.isfinite(c.o.float()).all()


@pytest.mark.gpu
def test_far_pages_of_a_large_cache(lib):
    """Rows whose byte and element offsets pass 32 bits."""
    S, B, Hq, Hkv, d, page, n_phys = 1, 2, 4, 1, 128, 64, 300_000  # 2.46e9 elements a side
    c = Case(S=S, B=B, Hq=Hq, Hkv=Hkv, d=d, page=page, n=[150], window=140, sinks=3, causal=True)
    want = c.want()
    far = torch.tensor([[n_phys - 1, 7, n_phys - 3, 290_000]], dtype=torch.int32)
    k, v = (torch.empty(n_phys, Hkv, page, d, dtype=BF, device="cuda") for _ in range(2))
    for lp in range(3):
        k[int(far[0, lp])], v[int(far[0, lp])] = c.k[int(c.table[0, lp])].cuda(), c.v[int(c.table[0, lp])].cuda()
    c.device()
    tab = far.cuda()
    c.dims = dsa.make_dims(S, B, Hq, Hkv, d, page, 4, 1, n_phys, tab)
    c.ws = dsa.Workspace(dsa.window_workspace_size(c.dims))
    c.dev[1], c.dev[2] = k, v
    c.call()
    assert c.ws.status() == dsa.DSA_OK
    plain.check_attention(c.o, c.lse, want, "far pages")


OK, ODD = 1 << 20, (1 << 20) + 2


def test_refusals_on_host(lib):
    base = dict(S=2, B=8, Hq=8, Hkv=2, d=128, page=16, max_pages=64, kmax=1, n_phys=128)

    def rc(dims=None, win=None, **kw):
        a = dict(q=OK, k=OK, v=OK, bk=OK, bv=OK, o=OK, n=OK, ws=OK, nbytes=1 << 40)
        a.update(kw)
        dm = dsa.make_dims(**{**base, **(dims or {})})
        w = dsa.dsa_window(*{**dict(window=64, sinks=4, causal=0, n_new=None), **(win or {})}.values())
        return lib.dsa_window_attn(a["q"], a["k"], a["v"], a["bk"], a["bv"], a["o"], None, ctypes.byref(dm), ctypes.byref(w),
                                   a["n"], a["ws"], a["nbytes"])

    inv, uns = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED
    for name in ("q", "k", "v", "bk", "bv", "o", "ws"):
        assert rc(**{name: ODD}) == inv, name
        assert rc(**{name: None}) == inv, name
    assert rc(n=None) == inv
    for win in (dict(window=0), dict(window=-5), dict(sinks=-1), dict(causal=2)):
        assert rc(win=win) == inv, win
    for dims in (dict(d=96), dict(page=8), dict(Hq=129 * 2), dict(S=1 << 20, B=1 << 12)):
        assert rc(dims=dims) == uns, dims
    assert rc(dims=dict(B=0)) == inv
    need = dsa.window_workspace_size(dsa.make_dims(**base))
    assert need >= dsa.WORKSPACE_HEADER_BYTES and rc(nbytes=dsa.WORKSPACE_HEADER_BYTES - 1) == dsa.DSA_ERR_WORKSPACE_TOO_SMALL
    assert dsa.window_workspace_size(dsa.make_dims(**{**base, "d": 96})) == 0
    assert dsa.window_launches(dsa.make_dims(**base), 64) >= 1
    assert dsa.window_launches(dsa.make_dims(**base), 1 << 40, 1 << 35) >= 1  # past every position, not wrapped
    with pytest.raises(dsa.DsaError):
        dsa.window_launches(dsa.make_dims(**base), 0)


@pytest.mark.gpu
def test_binding_refusals(lib):
    c = Case(S=1, B=2, Hq=2, Hkv=1, d=64, page=16, n=[20], window=8, sinks=0, causal=True).device()
    for name, bad in (("n_ctx", c.dn.long()), ("lse_out", c.lse.half()), ("n_new", c.dn.float())):
        with pytest.raises(TypeError):
            c.call(**{name: bad})
    with pytest.raises(ValueError):
        c.call(lse_out=c.lse[:, :1])
    with pytest.raises(dsa.DsaError):
        c.call(window=0)
    with pytest.raises(dsa.DsaError):
        c.call(workspace=type("W", (), {"buf": c.ws.buf, "nbytes": 16})())
    whole = c.dev
    c.dev = [whole[0].transpose(0, 1), *whole[1:]]
    with pytest.raises(ValueError):
        c.call()
    c.dev = [*whole[:4], None]
    with pytest.raises(dsa.DsaError):
        c.call()
