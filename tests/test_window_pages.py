"""dsa_window_attn reads no page without a visible token, nor its entry in the table."""
import pytest
import torch

import plain
from block_sparse_attention_27_b200 import build, dsa
from test_window import Case


@pytest.fixture(scope="module")
def lib():
    build.build()
    return dsa.load()


@pytest.mark.gpu
@pytest.mark.parametrize("kw", [
    # a window of the query alone behind a prefix that ends inside a page
    dict(S=2, B=1, Hq=4, Hkv=1, d=64, page=16, n=[20, 33], window=1, sinks=0, causal=True),
    dict(S=1, B=1, Hq=8, Hkv=2, d=128, page=64, n=[100], window=1, sinks=3, causal=False),
    dict(S=1, B=24, Hq=1, Hkv=1, d=128, page=16, n=[40], window=1, sinks=0, causal=True),
    dict(S=1, B=24, Hq=1, Hkv=1, d=64, page=64, n=[40], window=1, sinks=0, causal=False),
], ids=["one_token", "one_token_sinks", "wide", "wide_both_ways"])
def test_freed_pages(lib, kw):
    c = Case(**kw)
    want = c.want()
    for s, n in enumerate(c.n.tolist()):
        for lp in range(c.max_pages):
            tokens = range(lp * c.shape[5], min(n, (lp + 1) * c.shape[5]))
            if not any(t < c.sinks or n - t < c.window for t in tokens):
                c.table[s, lp] = -1
    assert (c.table == -1).any()
    c.device().call()
    assert c.ws.status() == dsa.DSA_OK
    plain.check_attention(c.o, c.lse, want, "freed pages")
