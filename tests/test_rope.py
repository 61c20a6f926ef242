"""dsa_qk_norm_rope against its definition in 64 bits, the append to the cache, refusals."""
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


def inputs(S, B, Hq, Hkv, d, seed=0):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(S, B, (Hq + 2 * Hkv) * d, generator=g).to(BF)
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(BF) for _ in range(2)]
    return qkv, w


def views(qkv, S, B, Hq, Hkv, d):
    a, b = Hq * d, (Hq + Hkv) * d
    return qkv[..., :a].view(S, B, Hq, d), qkv[..., a:b].view(S, B, Hkv, d), qkv[..., b:].view(S, B, Hkv, d)


def check(got, want, what):
    """One rounding to bf16 of a value whose fp32 errors (norm, cos and sin, two products) are at
    most 32 half steps of the rotated pair's length."""
    y, size = want
    tol = plain.half(BF) * y.abs() + 32 * plain.half(torch.float32) * size
    bad = (got.cpu().double() - y).abs() > tol
    assert not bad.any(), (what, int(bad.sum()), float(((got.cpu().double() - y).abs() - tol).max()))


CASES = [
    # S, B, Hq, Hkv, d, rot, interleaved, norm, start
    (1, 1, 4, 1, 64, 64, False, True, 0),
    (1, 32, 32, 8, 128, 128, False, True, 131072),
    (2, 5, 7, 1, 128, 128, True, True, 900001),
    (3, 7, 6, 3, 64, 8, False, True, 17),
    (1, 9, 5, 5, 128, 40, True, False, 2_000_000_000),
    (2, 33, 28, 4, 128, 104, False, False, 5),
    (1, 3, 64, 2, 64, 56, True, True, 77),
]


@pytest.mark.gpu
@pytest.mark.parametrize("S,B,Hq,Hkv,d,rot,inter,norm,start", CASES)
def test_against_definition(lib, S, B, Hq, Hkv, d, rot, inter, norm, start):
    qkv, w = inputs(S, B, Hq, Hkv, d)
    qkv[0, 0, :d] = 0  # a zero row: the norm's eps
    inv, scale = dsa.rope_inv_freq(rot, 1e5, scaling=("yarn", 4.0, 4096))
    dims = dsa.make_dims(S, B, Hq, Hkv, d, 16, 4, 1, 4 * S)
    dev = qkv.cuda()
    q, k, v = views(dev, S, B, Hq, Hkv, d)
    qo, ko, vo = (torch.full((S, B, H, d), float("nan"), dtype=BF, device="cuda") for H in (Hq, Hkv, Hkv))
    pos = start + torch.arange(B, dtype=torch.int32).repeat(S, 1) + 3 * torch.arange(S, dtype=torch.int32)[:, None]
    wq, wk = (x.cuda() if norm else None for x in w)
    rope = dsa.Rope(inv, rot, interleaved=inter, scale=scale, eps=1e-5, q_norm=wq, k_norm=wk)
    ws = dsa.Workspace(dsa.WORKSPACE_HEADER_BYTES)
    dsa.dsa_qk_norm_rope(q, k, v, qo, ko, vo, dims=dims, rope=rope, workspace=ws, positions=pos.cuda())
    assert ws.status() == dsa.DSA_OK
    cq, ck, cv = views(qkv, S, B, Hq, Hkv, d)
    args = (inv.cpu(), rot, inter, float(torch.tensor(scale, dtype=torch.float32)), 1e-5)
    check(qo, plain.norm_rope(cq, w[0] if norm else None, pos, *args), "q")
    check(ko, plain.norm_rope(ck, w[1] if norm else None, pos, *args), "k")
    assert torch.equal(vo.cpu(), cv)
    # in place: the packed keys rotated where they lie is refused (another stride), a contiguous
    # query tensor may be its own output
    qc = q.contiguous()
    dsa.dsa_qk_norm_rope(qc, None, None, qc, dims=dims, rope=rope, workspace=ws, positions=pos.cuda())
    assert torch.equal(qc, qo)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,d,rot,inter,norm", [
    (3, 1, 128, 64, False, True),
    (6, 2, 64, 64, True, True),
    (2, 1, 128, 24, False, False),
    (6, 3, 64, 16, False, True),
    (1, 1, 64, 56, True, True),
    (8, 2, 128, 128, True, False),
])
def test_many_tokens(lib, Hq, Hkv, d, rot, inter, norm):
    """A long padded batch, which takes several tokens a block of threads: the definition, and the
    rows past n_new left as they were; the cache gets what the outputs get."""
    S, B, page = 2, 1303, 32
    qkv, w = inputs(S, B, Hq, Hkv, d, 3)
    n = torch.tensor([7, 70000], dtype=torch.int32)
    new = [1303, 1290]
    max_pages = 2300
    table = (torch.arange(2 * 42, dtype=torch.int32).view(2, 42)).flip(1)
    tab = torch.full((2, max_pages), -1, dtype=torch.int32)
    tab[0, :42], tab[1, 70000 // page:70000 // page + 42] = table[0], table[1]
    inv, _ = dsa.rope_inv_freq(rot, 1e5)
    dev = qkv.cuda()
    q, k, v = views(dev, S, B, Hq, Hkv, d)
    qo, ko, vo = (torch.full((S, B, H, d), 7.0, dtype=BF, device="cuda") for H in (Hq, Hkv, Hkv))
    kc, vc = (torch.full((84, Hkv, page, d), 9.0, dtype=BF, device="cuda") for _ in range(2))
    gtab = tab.cuda()
    dims = dsa.make_dims(S, B, Hq, Hkv, d, page, max_pages, 1, 84, gtab)
    wq, wk = (x.cuda() if norm else None for x in w)
    rope = dsa.Rope(inv, rot, interleaved=inter, eps=1e-6, q_norm=wq, k_norm=wk)
    ws = dsa.Workspace(dsa.WORKSPACE_HEADER_BYTES)
    dsa.dsa_qk_norm_rope(q, k, v, qo, ko, vo, dims=dims, rope=rope, n_ctx=n.cuda(), workspace=ws,
                         n_new=torch.tensor(new, dtype=torch.int32, device="cuda"), k_cache=kc, v_cache=vc)
    assert ws.status() == dsa.DSA_OK
    cq, ck, cv = views(qkv, S, B, Hq, Hkv, d)
    pos = n[:, None] + torch.arange(B)
    for got, x, wt, what in ((qo, cq, w[0], "q"), (ko, ck, w[1], "k")):
        y, size = plain.norm_rope(x, wt if norm else None, pos, inv.cpu(), rot, inter, 1.0, 1e-6)
        for s in range(S):
            check(got[s, :new[s]], (y[s, :new[s]], size[s, :new[s]]), what)
            assert (got[s, new[s]:] == 7.0).all()
    slots = torch.zeros(84, page, dtype=torch.bool)
    for s in range(S):
        assert torch.equal(vo[s, :new[s]].cpu(), cv[s, :new[s]])
        at = int(n[s]) + torch.arange(new[s])
        pages, inside = tab[s, at // page].long(), at % page
        slots[pages, inside] = True
        assert torch.equal(kc.cpu()[pages, :, inside], ko[s, :new[s]].cpu())
        assert torch.equal(vc.cpu()[pages, :, inside], cv[s, :new[s]])
    assert (kc.cpu().transpose(1, 2)[~slots] == 9.0).all() and (vc.cpu().transpose(1, 2)[~slots] == 9.0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 32, 64])
@pytest.mark.parametrize("both", [False, True])
def test_append_padded_batch(lib, page, both):
    """Tokens land at n_ctx + b through the page table; rows past n_new, every other slot and the
    outputs' rows of missing tokens stay as they were."""
    S, B, Hq, Hkv, d = 4, 37, 4, 2, 128
    qkv, w = inputs(S, B, Hq, Hkv, d, 1)
    n = torch.tensor([0, 5, 63, 40], dtype=torch.int32)
    new = torch.tensor([37, 0, 1, 20], dtype=torch.int32)
    max_pages = -(-(63 + B) // page)
    n_phys = S * max_pages + 2
    table = torch.randperm(n_phys, generator=torch.Generator().manual_seed(2))[: S * max_pages].view(S, -1).to(torch.int32)
    dev = qkv.cuda()
    q, k, v = views(dev, S, B, Hq, Hkv, d)
    tab = table.cuda()
    dims = dsa.make_dims(S, B, Hq, Hkv, d, page, max_pages, 1, n_phys, tab)
    kc, vc = (torch.full((n_phys, Hkv, page, d), 9.0, dtype=BF, device="cuda") for _ in range(2))
    qo = torch.full((S, B, Hq, d), 7.0, dtype=BF, device="cuda")
    ko = torch.full((S, B, Hkv, d), 7.0, dtype=BF, device="cuda") if both else None
    vo = torch.full((S, B, Hkv, d), 7.0, dtype=BF, device="cuda") if both else None
    inv, scale = dsa.rope_inv_freq(d)
    rope = dsa.Rope(inv, d, q_norm=w[0].cuda(), k_norm=w[1].cuda())
    ws = dsa.Workspace(dsa.WORKSPACE_HEADER_BYTES)
    dsa.dsa_qk_norm_rope(q, k, v, qo, ko, vo, dims=dims, rope=rope, n_ctx=n.cuda(), workspace=ws, n_new=new.cuda(),
                         k_cache=kc, v_cache=vc)
    assert ws.status() == dsa.DSA_OK
    cq, ck, cv = views(qkv, S, B, Hq, Hkv, d)
    pos = n[:, None] + torch.arange(B)
    yq = plain.norm_rope(cq, w[0], pos, inv.cpu(), d, False, 1.0, 1e-6)
    yk = plain.norm_rope(ck, w[1], pos, inv.cpu(), d, False, 1.0, 1e-6)
    kh, vh = kc.cpu(), vc.cpu()
    seen = torch.zeros(n_phys, Hkv, page, dtype=torch.bool)
    for s in range(S):
        m = int(new[s])
        check(qo[s, :m], (yq[0][s, :m], yq[1][s, :m]), "q")
        assert (qo[s, m:] == 7.0).all()
        if both:
            check(ko[s, :m], (yk[0][s, :m], yk[1][s, :m]), "k")
            assert torch.equal(vo[s, :m].cpu(), cv[s, :m]) and (ko[s, m:] == 7.0).all() and (vo[s, m:] == 7.0).all()
        for b in range(m):
            t = int(n[s]) + b
            at = (int(table[s, t // page]), slice(None), t % page)
            check(kh[at], (yk[0][s, b], yk[1][s, b]), "cache k")
            assert torch.equal(vh[at], cv[s, b])
            seen[at] = True
    assert (kh[~seen] == 9.0).all() and (vh[~seen] == 9.0).all()


@pytest.mark.gpu
def test_bad_pages_are_skipped_and_reported(lib):
    S, B, Hq, Hkv, d, page = 1, 8, 2, 1, 64, 16
    qkv, _ = inputs(S, B, Hq, Hkv, d)
    dev = qkv.cuda()
    q, k, v = views(dev, S, B, Hq, Hkv, d)
    inv, _ = dsa.rope_inv_freq(d)
    rope = dsa.Rope(inv, d)
    qo = torch.zeros(S, B, Hq, d, dtype=BF, device="cuda")
    for n, table in ((28, [0, 5]), (28, [0, -1]), (12, [9, 0]), (-3, [0, 1]), (2_147_483_640, [0, 1])):
        kc, vc = (torch.zeros(2, Hkv, page, d, dtype=BF, device="cuda") for _ in range(2))
        tab = torch.tensor([table], dtype=torch.int32, device="cuda")
        dims = dsa.make_dims(S, B, Hq, Hkv, d, page, 2, 1, 2, tab)
        ws = dsa.Workspace(dsa.WORKSPACE_HEADER_BYTES)
        dsa.dsa_qk_norm_rope(q, k, v, qo, dims=dims, rope=rope, n_ctx=torch.tensor([n], dtype=torch.int32, device="cuda"),
                             workspace=ws, k_cache=kc, v_cache=vc)
        assert ws.status() == dsa.DSA_ERR_BAD_INDEX, (n, table)
        good = [t for t in range(n, n + B) if 0 <= n and t // page < 2 and 0 <= table[t // page] < 2]
        rows = {(table[t // page], t % page) for t in good}
        filled = {(p, i) for p in range(2) for i in range(page) if vc[p, 0, i].any()}
        assert filled == rows
    ws = dsa.Workspace(dsa.WORKSPACE_HEADER_BYTES)
    dims = dsa.make_dims(S, B, Hq, Hkv, d, page, 2, 1, 2)
    dsa.dsa_qk_norm_rope(q, None, None, qo, dims=dims, rope=rope, n_ctx=torch.zeros(1, dtype=torch.int32, device="cuda"),
                         workspace=ws, n_new=torch.tensor([B + 1], dtype=torch.int32, device="cuda"))
    assert ws.status() == dsa.DSA_ERR_BAD_INDEX


def test_frequencies():
    inv, s = dsa.rope_inv_freq(64, 1e4, device="cpu")
    assert s == 1.0 and inv[0] == 1.0 and abs(float(inv[-1]) - 1e4 ** (-62 / 64)) < 1e-9
    lin, _ = dsa.rope_inv_freq(64, 1e4, scaling=("linear", 4), device="cpu")
    assert torch.equal(lin, inv / 4)
    ntk, _ = dsa.rope_inv_freq(64, 1e4, scaling=("ntk", 4), device="cpu")
    assert ntk[0] == 1.0 and abs(float(inv[-1] / ntk[-1]) - 4) < 1e-5  # the slowest pair stretched fourfold
    yarn, s = dsa.rope_inv_freq(128, 1e4, scaling=("yarn", 8, 4096), device="cpu")
    base, _ = dsa.rope_inv_freq(128, 1e4, device="cpu")
    ratio = base / yarn
    assert abs(s - 1.2079441541679836) < 1e-12
    assert ratio[0] == 1 and abs(float(ratio[-1]) - 8) < 1e-5 and (ratio[1:] >= ratio[:-1] - 1e-6).all()
    for bad in (("linear", 0.5), ("other", 2)):
        with pytest.raises(ValueError):
            dsa.rope_inv_freq(64, scaling=bad, device="cpu")
    with pytest.raises(ValueError):
        dsa.rope_inv_freq(12, device="cpu")


OK, ODD = 1 << 20, (1 << 20) + 2


def refuse(lib, code, *, dims=None, rope=None, **kw):
    a = dict(q=OK, k=OK, v=OK, q_out=OK + 4096, k_out=OK + 8192, v_out=OK + 16384, k_cache=None, v_cache=None, n_ctx=OK,
             ws=OK, nbytes=4096)
    a.update(kw)
    dm = dsa.make_dims(**{**dict(S=1, B=8, Hq=4, Hkv=2, d=128, page=16, max_pages=8, kmax=1, n_phys=8), **(dims or {})})
    r = dict(rot=128, interleaved=0, eps=1e-6, scale=1.0, inv_freq=OK, q_stride=512, k_stride=256, v_stride=256)
    r.update(rope or {})
    rc = lib.dsa_qk_norm_rope(a["q"], a["k"], a["v"], a["q_out"], a["k_out"], a["v_out"], a["k_cache"], a["v_cache"], None,
                              ctypes.byref(dm), ctypes.byref(dsa.dsa_rope(**r)), a["n_ctx"], a["ws"], a["nbytes"])
    assert rc == code, (rc, code, kw, dims, rope)


def test_refusals_on_host(lib):
    inv, uns = dsa.DSA_ERR_INVALID_ARG, dsa.DSA_ERR_UNSUPPORTED
    for name in ("q", "k", "v", "q_out", "k_out", "v_out", "ws"):
        refuse(lib, inv, **{name: ODD})
        refuse(lib, inv, **{name: None})
    refuse(lib, inv, q=None, k=None, v=None, q_out=None, k_out=None, v_out=None)
    refuse(lib, inv, n_ctx=None)
    refuse(lib, inv, k_cache=OK, n_ctx=None, rope=dict(positions=OK))
    refuse(lib, dsa.DSA_ERR_WORKSPACE_TOO_SMALL, nbytes=4095)
    for r in (4, 12, 136, 0, -8):
        refuse(lib, uns, rope=dict(rot=r))
    for bad in (dict(interleaved=2), dict(eps=0.0), dict(eps=float("nan")), dict(scale=float("inf")), dict(inv_freq=None),
                dict(q_norm=ODD), dict(q_stride=504), dict(k_stride=260), dict(v_stride=0)):
        refuse(lib, inv, rope=bad)
    refuse(lib, inv, q_out=OK, rope=dict(q_stride=1024))  # in place needs the same stride
    refuse(lib, uns, dims=dict(d=96))
    refuse(lib, uns, dims=dict(S=1 << 16, B=1 << 14))
    refuse(lib, inv, dims=dict(Hq=5))


def test_binding_refuses_host_tensors():
    t = torch.zeros(64, dtype=torch.float32)
    with pytest.raises(TypeError):
        dsa.Rope(t[:32], 64)


@pytest.mark.gpu
def test_binding_refusals(lib):
    S, B, Hq, Hkv, d = 2, 3, 2, 1, 64
    dims = dsa.make_dims(S, B, Hq, Hkv, d, 16, 2, 1, 4)
    inv, _ = dsa.rope_inv_freq(d)
    rope, ws = dsa.Rope(inv, d), dsa.Workspace(dsa.WORKSPACE_HEADER_BYTES)
    q = torch.zeros(S, B, Hq, d, dtype=BF, device="cuda")
    pos = torch.zeros(S, B, dtype=torch.int32, device="cuda")

    def call(q=q, out=None, rope=rope, pos=pos, **kw):
        dsa.dsa_qk_norm_rope(q, None, None, torch.zeros_like(q) if out is None else out, dims=dims, rope=rope, workspace=ws,
                             positions=pos, **kw)

    call()
    with pytest.raises(TypeError):
        call(q=q.float())
    with pytest.raises(ValueError):
        call(q=torch.zeros(S, B, d, Hq, dtype=BF, device="cuda").transpose(2, 3), out=q)
    with pytest.raises(ValueError):
        call(q=torch.zeros(S, 2 * B, Hq, d, dtype=BF, device="cuda")[:, :B], out=q)  # sequences not evenly spaced
    with pytest.raises(ValueError):
        call(pos=pos[:1])
    with pytest.raises(TypeError):
        call(pos=pos.long())
    with pytest.raises(ValueError):
        call(rope=dsa.Rope(inv, d, q_norm=torch.ones(32, dtype=BF, device="cuda")))
    with pytest.raises(ValueError):
        dsa.Rope(inv[:8], d)
