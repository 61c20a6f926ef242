"""Each call right behind the one that writes its inputs, with nothing between them: kernels launched as
programmatic dependents are resident before the kernel ahead has ended, and must not have read
anything by then.  Compared bit for bit with the same calls one at a time."""
import pytest
import torch

from block_sparse_attention_27_b200 import build, dsa

BF = torch.bfloat16
pytestmark = pytest.mark.gpu

# a long norm + rotation, whose last tokens are the block that the next call takes
TOKENS, B, Hq, Hkv, d, page, N = 20000, 32, 8, 2, 128, 16, 1000


@pytest.fixture(scope="module")
def lib():
    build.build()
    return dsa.load()


class Chain:
    def __init__(self, B=B):
        g = torch.Generator(device="cuda").manual_seed(1)
        self.g, self.B = g, B
        self.max_pages = -(-(N + B) // page)
        self.tab = torch.randperm(self.max_pages, generator=g, device="cuda").to(torch.int32).view(1, -1)
        self.big = dsa.make_dims(1, TOKENS, Hq, Hkv, d, page, TOKENS // page + 1, 1, TOKENS // page + 1)
        self.dims = dsa.make_dims(1, B, Hq, Hkv, d, page, self.max_pages, 12, self.max_pages, self.tab)
        self.tail = dsa.make_dims(1, B, Hq, Hkv, d, page, TOKENS // page + 1, 1, TOKENS // page + 1)
        self.at = torch.tensor([TOKENS - B], dtype=torch.int32, device="cuda")
        inv, scale = dsa.rope_inv_freq(d)
        self.rope = dsa.Rope(inv, d, scale=scale)
        self.n = torch.tensor([N], dtype=torch.int32, device="cuda")
        self.zero = torch.zeros_like(self.n)
        self.topk = torch.tensor([12 * page], dtype=torch.int32, device="cuda")
        self.ws = [dsa.Workspace(max(dsa.window_workspace_size(self.dims), dsa.kv4_workspace_size(self.dims),
                                     dsa.sparse_workspace_size(self.dims), dsa.select_workspace_size(self.dims))) for _ in range(3)]

        def zeros(*shape, dtype=BF):
            return torch.zeros(shape, dtype=dtype, device="cuda")

        self.q, self.k, self.v = zeros(1, TOKENS, Hq, d), zeros(1, TOKENS, Hkv, d), zeros(1, TOKENS, Hkv, d)
        self.qb, self.kb, self.vb = (t[:, TOKENS - B:] for t in (self.q, self.k, self.v))
        self.kc, self.vc = (torch.randn(self.max_pages, Hkv, page, d, generator=g, device="cuda").to(BF) for _ in range(2))
        self.cache4 = dsa.Kv4Cache.zeros(self.max_pages, Hkv, page, d)
        self.kv4big = dsa.Kv4Cache.zeros(TOKENS // page + 1, Hkv, page, d)
        pre = dsa.make_dims(1, N, Hq, Hkv, d, page, self.max_pages, 1, self.max_pages, self.tab)
        old = [torch.randn(1, N, Hkv, d, generator=g, device="cuda").to(BF) for _ in range(2)]
        dsa.dsa_kv4_store(*old, self.cache4, dims=pre, n_ctx=self.zero, workspace=self.ws[0])
        self.o, self.o2 = zeros(1, B, Hq, d), zeros(1, B, Hq, d)
        self.lse, self.lse2 = zeros(1, B, Hq, dtype=torch.float32), zeros(1, B, Hq, dtype=torch.float32)
        self.idx, self.cnt = zeros(1, Hkv, 12, dtype=torch.int32), zeros(1, Hkv, dtype=torch.int32)
        self.ko, self.vo = zeros(1, B, Hkv, d), zeros(1, B, Hkv, d)

    def inputs(self):
        return [torch.randn(1, TOKENS, h, d, generator=self.g, device="cuda").to(BF) for h in (Hq, Hkv, Hkv)]

    # the calls
    def rotate(self, x):
        dsa.dsa_qk_norm_rope(*x, self.q, self.k, self.v, dims=self.big, rope=self.rope, n_ctx=self.zero, workspace=self.ws[0])

    def select(self, x):
        dsa.dsa_select(self.qb, self.kc, self.vc, self.n, page, self.topk, self.idx, self.o, dims=self.dims, cnt_out=self.cnt,
                       workspace=self.ws[1], lse_out=self.lse)

    def sparse(self, x):
        dsa.dsa_sparse_attn(self.qb, self.kc, self.vc, self.idx, self.kb, self.vb, self.o2, dims=self.dims, n_ctx=self.n,
                            idx_cnt=self.cnt, workspace=self.ws[2], lse_out=self.lse2)

    def window(self, x):
        dsa.dsa_window_attn(self.qb, self.kc, self.vc, self.kb, self.vb, self.o, dims=self.dims, window=400, sinks=4, n_ctx=self.n,
                            workspace=self.ws[1], lse_out=self.lse)

    def kv4(self, x):
        dsa.dsa_kv4_attn(self.qb, self.cache4, None, self.kb, self.vb, self.o2, dims=self.dims, n_ctx=self.n, workspace=self.ws[2],
                         lse_out=self.lse2)

    def kv4_selected(self, x):
        dsa.dsa_kv4_attn(self.qb, self.cache4, self.idx, self.kb, self.vb, self.o2, dims=self.dims, n_ctx=self.n, idx_cnt=self.cnt,
                         workspace=self.ws[2], lse_out=self.lse2)

    def merge(self, x):
        dsa.dsa_merge_attn(self.o, self.lse, self.o2, self.lse2, self.o2, self.lse2)

    def store(self, x):
        dsa.dsa_kv4_store(self.k, self.v, self.kv4big, dims=self.big, n_ctx=self.zero, workspace=self.ws[1])

    def load(self, x):
        dsa.dsa_kv4_load(self.kv4big, self.ko, self.vo, dims=self.tail, start=self.at, workspace=self.ws[2])

    def outputs(self):
        return [t.clone() for t in (self.qb, self.kb, self.vb, self.o, self.o2, self.lse, self.lse2, self.idx, self.cnt, self.ko, self.vo)]

    def run(self, calls, x, wait):
        for c in calls:
            getattr(self, c)(x)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        return self.outputs()


CHAINS = ["rotate select", "rotate select sparse", "rotate select kv4_selected", "rotate window", "rotate kv4", "rotate window kv4 merge",
          "rotate select sparse merge", "rotate store load"]


@pytest.mark.parametrize("tokens", [1, 32])
@pytest.mark.parametrize("chain", CHAINS)
def test_chain(lib, chain, tokens):
    c = Chain(tokens)
    calls = chain.split()
    a, b = c.inputs(), c.inputs()
    want = {}
    for name, x in (("a", a), ("b", b)):
        want[name] = c.run(calls, x, wait=True)
    for i in range(10):  # each input behind the other's results
        name, x = (("a", a), ("b", b))[i % 2]
        for got, ref in zip(c.run(calls, x, wait=False), want[name]):
            assert torch.equal(got, ref), (chain, i)
    assert all(w.status() == dsa.DSA_OK for w in c.ws)


class Slow:
    """A selection pass confined to a few SMs, which lets its dependents start at once and writes its
    outputs (o, lse, idx, cnt) at its end, and calls on the free SMs that take those."""

    def __init__(self):
        g = torch.Generator(device="cuda").manual_seed(2)
        self.n1 = 30000
        mp = -(-self.n1 // page)
        self.slow = dsa.make_dims(1, B, Hq, Hkv, d, page, mp, 12, mp, None, sm_limit=8)
        self.max_pages = mp
        self.kc, self.vc = (torch.randn(mp, Hkv, page, d, generator=g, device="cuda").to(BF) for _ in range(2))
        self.n = torch.tensor([self.n1], dtype=torch.int32, device="cuda")
        self.near = torch.tensor([N], dtype=torch.int32, device="cuda")
        self.topk = torch.tensor([12 * page], dtype=torch.int32, device="cuda")
        self.fast = dsa.make_dims(1, B, Hq, Hkv, d, page, mp, 12, mp, None, sm_limit=56)
        self.rows = dsa.make_dims(1, B, Hq, Hq, d, page, mp, 1, mp)  # o as keys and values of Hq heads
        self.cache4 = dsa.Kv4Cache.zeros(mp, Hkv, page, d)
        self.store4 = dsa.Kv4Cache.zeros(mp, Hq, page, d)
        for t in (self.cache4.k, self.cache4.v):
            t.random_(generator=g)
        for t in (self.cache4.k_scale, self.cache4.v_scale):
            t.fill_(0.125)
        inv, scale = dsa.rope_inv_freq(d)
        self.rope = dsa.Rope(inv, d, scale=scale)
        size = max(f(x) for x in (self.slow, self.fast) for f in (dsa.select_workspace_size, dsa.sparse_workspace_size,
                                                                   dsa.window_workspace_size, dsa.kv4_workspace_size))
        self.ws = [dsa.Workspace(size) for _ in range(2)]

        def zeros(*shape, dtype=BF):
            return torch.zeros(shape, dtype=dtype, device="cuda")

        self.q = zeros(1, B, Hq, d)
        self.bk, self.bv = (torch.randn(1, B, Hkv, d, generator=g, device="cuda").to(BF) for _ in range(2))
        self.o, self.o2 = zeros(1, B, Hq, d), zeros(1, B, Hq, d)
        self.other, self.other_lse = zeros(1, B, Hq, d), torch.zeros(1, B, Hq, device="cuda")
        self.lse, self.lse2 = torch.zeros(1, B, Hq, device="cuda"), torch.zeros(1, B, Hq, device="cuda")
        self.idx, self.idx2 = (zeros(1, Hkv, 12, dtype=torch.int32) for _ in range(2))
        self.cnt, self.cnt2 = (zeros(1, Hkv, dtype=torch.int32) for _ in range(2))

    def first(self):
        dsa.dsa_select(self.q, self.kc, self.vc, self.n, page, self.topk, self.idx, self.o, dims=self.slow, cnt_out=self.cnt,
                       workspace=self.ws[0], lse_out=self.lse)

    def select(self):
        dsa.dsa_select(self.o, self.kc, self.vc, self.near, page, self.topk, self.idx2, self.o2, dims=self.fast, cnt_out=self.cnt2,
                       workspace=self.ws[1], lse_out=self.lse2)

    def sparse(self):
        dsa.dsa_sparse_attn(self.o, self.kc, self.vc, self.idx, self.bk, self.bv, self.o2, dims=self.fast, n_ctx=self.n,
                            idx_cnt=self.cnt, workspace=self.ws[1], lse_out=self.lse2)

    def window(self):
        dsa.dsa_window_attn(self.o, self.kc, self.vc, self.bk, self.bv, self.o2, dims=self.fast, window=300, sinks=4,
                            n_ctx=self.near, workspace=self.ws[1], lse_out=self.lse2)

    def kv4(self):
        dsa.dsa_kv4_attn(self.o, self.cache4, self.idx, self.bk, self.bv, self.o2, dims=self.fast, n_ctx=self.n, idx_cnt=self.cnt,
                         workspace=self.ws[1], lse_out=self.lse2)

    def store(self):
        dsa.dsa_kv4_store(self.o, self.o, self.store4, dims=self.rows, n_ctx=self.near, workspace=self.ws[1])

    def store_load(self):
        self.store()
        dsa.dsa_kv4_load(self.store4, self.o2, self.other, dims=self.rows, start=self.near, workspace=self.ws[1])

    def norm_rope(self):
        dsa.dsa_qk_norm_rope(self.o, None, None, self.o2, dims=self.fast, rope=self.rope, n_ctx=self.n, workspace=self.ws[1])

    def merge(self):
        dsa.dsa_merge_attn(self.o, self.lse, self.other, self.other_lse, self.o2, self.lse2)

    def outputs(self):
        return [t.clone() for t in (self.o, self.lse, self.idx, self.cnt, self.o2, self.lse2, self.idx2, self.cnt2, self.store4.k,
                                    self.store4.k_scale)]


@pytest.mark.parametrize("second", ["select", "sparse", "window", "kv4", "store", "store_load", "norm_rope", "merge"])
def test_behind_a_slow_kernel(lib, second):
    c = Slow()
    g = torch.Generator(device="cuda").manual_seed(3)
    inputs = [torch.randn(1, B, Hq, d, generator=g, device="cuda").to(BF) for _ in range(2)]
    want = []
    for x in inputs:
        c.q.copy_(x)
        c.first()
        torch.cuda.synchronize()
        getattr(c, second)()
        torch.cuda.synchronize()
        want.append(c.outputs())
    for i in range(8):
        c.q.copy_(inputs[i % 2])
        torch.cuda.synchronize()
        c.first()
        getattr(c, second)()
        torch.cuda.synchronize()
        for got, ref in zip(c.outputs(), want[i % 2]):
            assert torch.equal(got, ref), (second, i)
    assert all(w.status() == dsa.DSA_OK for w in c.ws)
