"""The operators beside the two passes as a layer uses them: one after the other, with the passes
and the merge, captured into graphs, on two streams at once."""
import pytest
import torch

import plain
from block_sparse_attention_27_b200 import build, dsa

BF = torch.bfloat16
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def lib():
    build.build()
    return dsa.load()


class Layer:
    """A windowed or 4-bit layer: its weights, its paged cache, and one call per block of tokens."""

    def __init__(self, S, B, Hq, Hkv, d, page, capacity, seed=0):
        self.g = torch.Generator().manual_seed(seed)
        self.shape = S, B, Hq, Hkv, d, page
        self.max_pages = -(-capacity // page)
        self.n_phys = S * self.max_pages
        self.table = torch.randperm(self.n_phys, generator=self.g).view(S, -1).to(torch.int32)
        self.tab = self.table.cuda()
        self.dims = dsa.make_dims(S, B, Hq, Hkv, d, page, self.max_pages, self.max_pages, self.n_phys, self.tab)
        self.norms = [(1 + 0.1 * torch.randn(d, generator=self.g)).to(BF) for _ in range(2)]
        inv, scale = dsa.rope_inv_freq(d, 1e4, scaling=("yarn", 4.0, 64))
        self.scale = float(torch.tensor(scale, dtype=torch.float32))
        self.inv = inv
        self.rope = dsa.Rope(inv, d, scale=scale, q_norm=self.norms[0].cuda(), k_norm=self.norms[1].cuda())
        self.kc, self.vc = (torch.zeros(self.n_phys, Hkv, page, d, dtype=BF, device="cuda") for _ in range(2))
        self.kv4 = dsa.Kv4Cache.zeros(self.n_phys, Hkv, page, d)
        self.ws = dsa.Workspace(max(dsa.window_workspace_size(self.dims), dsa.kv4_workspace_size(self.dims),
                                    dsa.sparse_workspace_size(self.dims), dsa.select_workspace_size(self.dims)))
        self.q = torch.zeros(S, B, Hq, d, dtype=BF, device="cuda")
        self.k, self.v = (torch.zeros(S, B, Hkv, d, dtype=BF, device="cuda") for _ in range(2))
        self.o = torch.zeros(S, B, Hq, d, dtype=BF, device="cuda")
        self.lse = torch.zeros(S, B, Hq, device="cuda")

    def projection(self):
        S, B, Hq, Hkv, d, _ = self.shape
        return torch.randn(S, B, (Hq + 2 * Hkv) * d, generator=self.g).to(BF)

    def split(self, qkv):
        S, B, Hq, Hkv, d, _ = self.shape
        a, b = Hq * d, (Hq + Hkv) * d
        return qkv[..., :a].view(S, B, Hq, d), qkv[..., a:b].view(S, B, Hkv, d), qkv[..., b:].view(S, B, Hkv, d)

    def rotate(self, qkv, n, append, stream=None):
        q, k, v = self.split(qkv)
        dsa.dsa_qk_norm_rope(q, k, v, self.q, self.k, self.v, stream, dims=self.dims, rope=self.rope, n_ctx=n, workspace=self.ws,
                             k_cache=self.kc if append else None, v_cache=self.vc if append else None)


@pytest.mark.parametrize("page,d", [(16, 128), (64, 64)])
def test_windowed_layer_over_blocks(lib, page, d):
    """Blocks come one after the other; each is rotated, attends through the window, and is appended."""
    S, B, Hq, Hkv = 2, 24, 4, 2
    L = Layer(S, B, Hq, Hkv, d, page, 4 * B)
    n = torch.tensor([0, 3], dtype=torch.int32)  # the second sequence starts with three tokens of zeros
    for step in range(3):
        qkv = L.projection()
        dn = n.cuda()
        L.rotate(qkv.cuda(), dn, append=True)
        dsa.dsa_window_attn(L.q, L.kc, L.vc, L.k, L.v, L.o, dims=L.dims, window=30, sinks=4, n_ctx=dn, workspace=L.ws, lse_out=L.lse)
        assert L.ws.status() == dsa.DSA_OK
        pos = n[:, None] + torch.arange(B)
        for got, x, w in zip((L.q, L.k), L.split(qkv), L.norms):
            y, size = plain.norm_rope(x, w, pos, L.inv.cpu(), d, False, L.scale, 1e-6)
            tol = plain.half(BF) * y.abs() + 32 * plain.half(torch.float32) * size
            assert ((got.cpu().double() - y).abs() <= tol).all()
        want = plain.window_attn(L.q.cpu(), L.kc.cpu(), L.vc.cpu(), L.table, L.max_pages, n, L.k.cpu(), L.v.cpu(), 30, 4, False)
        plain.check_attention(L.o, L.lse, want, f"block {step}")
        n = n + B


def test_four_bit_layer_beside_the_passes(lib):
    """A prefix goes into the 4-bit cache; its values, read back into a bf16 cache, give the
    selection pass its pages, and the sparse pass over them the 4-bit attention's result."""
    S, B, Hq, Hkv, d, page, n = 2, 32, 8, 2, 128, 16, 600
    L = Layer(S, B, Hq, Hkv, d, page, n + B, seed=3)
    g = torch.Generator().manual_seed(5)
    whole = dsa.make_dims(S, n, Hq, Hkv, d, page, L.max_pages, 1, L.n_phys, L.tab)
    k, v = (torch.randn(S, n, Hkv, d, generator=g).to(BF).cuda() for _ in range(2))
    zero = torch.zeros(S, dtype=torch.int32, device="cuda")
    dsa.dsa_kv4_store(k, v, L.kv4, dims=whole, n_ctx=zero, workspace=L.ws)
    dsa.dsa_kv4_load(L.kv4, k, v, dims=whole, start=zero, workspace=L.ws)  # the values held, in place of the stored ones
    at = torch.arange(n, device="cuda")
    for s in range(S):
        phys = L.tab[s].long()[at // page]
        L.kc[phys, :, at % page], L.vc[phys, :, at % page] = k[s], v[s]
    dn = torch.full((S,), n, dtype=torch.int32, device="cuda")
    L.rotate(L.projection().cuda(), dn, append=False)
    # pages of the selection pass, then both caches over them
    topk = torch.full((S,), 10 * page, dtype=torch.int32, device="cuda")
    idx = torch.full((S, Hkv, L.max_pages), -1, dtype=torch.int32, device="cuda")
    cnt = torch.zeros((S, Hkv), dtype=torch.int32, device="cuda")
    dsa.dsa_select(L.q, L.kc, L.vc, dn, page, topk, idx, torch.empty_like(L.o), dims=L.dims, cnt_out=cnt, workspace=L.ws)
    dsa.dsa_kv4_attn(L.q, L.kv4, idx, L.k, L.v, L.o, dims=L.dims, n_ctx=dn, idx_cnt=cnt, workspace=L.ws, lse_out=L.lse)
    o, lse = torch.empty_like(L.o), torch.empty_like(L.lse)
    dsa.dsa_sparse_attn(L.q, L.kc, L.vc, idx, L.k, L.v, o, dims=L.dims, n_ctx=dn, idx_cnt=cnt, workspace=L.ws, lse_out=lse)
    assert L.ws.status() == dsa.DSA_OK and int(cnt.min()) == 10
    values = [plain.kv4_values(*(t.cpu() for t in x)) for x in ((L.kv4.k, L.kv4.k_scale), (L.kv4.v, L.kv4.v_scale))]
    want = plain.kv4_attn(L.q.cpu(), values, L.table, L.max_pages, dn.cpu(), idx.cpu(), cnt.cpu(), L.k.cpu(), L.v.cpu())
    plain.check_attention(L.o, L.lse, want, "4-bit over the selected pages")
    # the sparse pass holds its row pieces in fp16 (half a step 2^-11) beside bf16 probabilities:
    # within 2e-2 of the same values, its own bound
    assert (o.float() - L.o.float()).abs().max() <= 2e-2 and (lse - L.lse).abs().max() <= 2e-3
    # every page: the same as naming them all
    every = torch.arange(L.max_pages, dtype=torch.int32, device="cuda").expand(S, Hkv, -1).contiguous()
    all_cnt = torch.full((S, Hkv), -(-n // page), dtype=torch.int32, device="cuda")
    a, b = torch.empty_like(L.o), torch.empty_like(L.o)
    dsa.dsa_kv4_attn(L.q, L.kv4, None, L.k, L.v, a, dims=L.dims, n_ctx=dn, workspace=L.ws)
    dsa.dsa_kv4_attn(L.q, L.kv4, every, L.k, L.v, b, dims=L.dims, n_ctx=dn, idx_cnt=all_cnt, workspace=L.ws)
    assert torch.equal(a, b)


@pytest.mark.parametrize("B", [1, 20])
def test_parts_merge_into_the_whole(lib, B):
    """Prefix and block attended apart and joined by dsa_merge_attn: the call over both."""
    S, Hq, Hkv, d, page, n = 2, 4, 2, 128, 16, 200
    L = Layer(S, B, Hq, Hkv, d, page, n + B, seed=7)
    L.kc.normal_()
    L.vc.normal_()
    for t in (L.q, L.k, L.v):
        t.normal_()
    dn = torch.tensor([n, 77], dtype=torch.int32, device="cuda")
    zero = torch.zeros_like(dn)
    kw = dict(dims=L.dims, window=1 << 20, causal=False, workspace=L.ws)
    dsa.dsa_window_attn(L.q, L.kc, L.vc, L.k, L.v, L.o, n_ctx=dn, lse_out=L.lse, **kw)
    parts = []
    for bk, bv, nn in ((None, None, dn), (L.k, L.v, zero)):
        o, lse = torch.empty_like(L.o), torch.empty_like(L.lse)
        dsa.dsa_window_attn(L.q, L.kc, L.vc, bk, bv, o, n_ctx=nn, lse_out=lse, **kw)
        parts += [o, lse]
    o, lse = torch.empty_like(L.o), torch.empty_like(L.lse)
    dsa.dsa_merge_attn(*parts, o, lse)
    assert L.ws.status() == dsa.DSA_OK
    # each part and the whole are rounded to bf16 (and their P): four half steps of values up to max |o|
    top = max(float(x.float().abs().max()) for x in (L.o, parts[0], parts[2]))
    assert (o.float() - L.o.float()).abs().max() <= 4 * plain.half(BF) * top
    assert (lse - L.lse).abs().max() <= 1e-4  # fp32 sums on either side of values around 10


def test_captured_and_replayed(lib):
    """The chain in a graph, replayed on changed inputs and lengths: what eager calls give."""
    S, B, Hq, Hkv, d, page = 2, 20, 4, 2, 128, 16
    L = Layer(S, B, Hq, Hkv, d, page, 6 * B, seed=11)
    L.kc.normal_()
    L.vc.normal_()
    kc0, vc0 = L.kc.clone(), L.vc.clone()
    qkv, dn = L.projection().cuda(), torch.tensor([5, 60], dtype=torch.int32, device="cuda")
    o4, lse4 = torch.zeros_like(L.o), torch.zeros_like(L.lse)
    old_k, old_v = (torch.randn(S, 64, Hkv, d, generator=L.g).to(BF).cuda() for _ in range(2))
    first = dsa.make_dims(S, 64, Hq, Hkv, d, page, L.max_pages, 1, L.n_phys, L.tab)
    dsa.dsa_kv4_store(old_k, old_v, L.kv4, dims=first, n_ctx=torch.zeros_like(dn), workspace=L.ws)

    def chain():
        L.rotate(qkv, dn, append=True)
        dsa.dsa_window_attn(L.q, L.kc, L.vc, L.k, L.v, L.o, dims=L.dims, window=25, sinks=3, causal=True, n_ctx=dn, workspace=L.ws,
                            lse_out=L.lse)
        dsa.dsa_kv4_attn(L.q, L.kv4, None, L.k, L.v, o4, dims=L.dims, n_ctx=dn, workspace=L.ws, lse_out=lse4)
        dsa.dsa_kv4_store(L.k, L.v, L.kv4, dims=L.dims, n_ctx=dn, workspace=L.ws)

    inputs = [(L.projection().cuda(), torch.tensor(n, dtype=torch.int32, device="cuda")) for n in ([5, 60], [64, 64], [0, 31])]
    held = [t.clone() for t in (L.kv4.k, L.kv4.v, L.kv4.k_scale, L.kv4.v_scale)]

    def reset():
        L.kc.copy_(kc0)
        L.vc.copy_(vc0)
        for t, h in zip((L.kv4.k, L.kv4.v, L.kv4.k_scale, L.kv4.v_scale), held):
            t.copy_(h)

    outputs = (L.q, L.k, L.o, L.lse, o4, lse4, L.kc, L.vc, L.kv4.k, L.kv4.k_scale)
    want = []
    for x, n in inputs:
        reset()
        qkv.copy_(x)
        dn.copy_(n)
        chain()
        want.append([t.clone() for t in outputs])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        chain()
    for (x, n), w in zip(inputs, want):
        reset()
        qkv.copy_(x)
        dn.copy_(n)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(outputs, w))
    assert L.ws.status() == dsa.DSA_OK


@pytest.mark.parametrize("B", [1, 24])
def test_two_streams_at_once(lib, B):
    """Calls in flight together on two streams, each with its own workspace: the same bits as alone."""
    S, Hq, Hkv, d, page, n = 4, 8, 2, 128, 16, 700
    layers = [Layer(S, B, Hq, Hkv, d, page, n + B, seed=20 + i) for i in range(2)]
    dn = torch.tensor([n, 1, 333, 512], dtype=torch.int32, device="cuda")
    for L in layers:
        for t in (L.kc, L.vc, L.q, L.k, L.v):
            t.normal_()
        L.kv4.k.random_()
        L.kv4.v.random_()
        L.kv4.k_scale.fill_(0.125)
        L.kv4.v_scale.fill_(0.25)

    def call(L, o4, stream):
        dsa.dsa_window_attn(L.q, L.kc, L.vc, L.k, L.v, L.o, stream, dims=L.dims, window=300, sinks=4, causal=True, n_ctx=dn,
                            workspace=L.ws, lse_out=L.lse)
        dsa.dsa_kv4_attn(L.q, L.kv4, None, L.k, L.v, o4, stream, dims=L.dims, n_ctx=dn, workspace=L.ws)

    o4 = [torch.zeros_like(L.o) for L in layers]
    alone = []
    for L, o in zip(layers, o4):
        call(L, o, None)
        alone.append((L.o.clone(), L.lse.clone(), o.clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in layers]
    for L, o in zip(layers, o4):
        for t in (L.o, L.lse, o):
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for L, o, s in zip(layers, o4, streams):
            call(L, o, s)
    torch.cuda.synchronize()
    for L, o, w in zip(layers, o4, alone):
        assert L.ws.status() == dsa.DSA_OK
        assert all(torch.equal(a, b) for a, b in zip((L.o, L.lse, o), w))
