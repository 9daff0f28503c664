"""Edges of the decode step's operators on the GPU, against the definitions of
tests/decode_reference.py: bounds that the caller's numbers exceed, weights far apart,
what a row does not see, logits at the ends of their type, buffers that moved."""
import numpy as np
import pytest

import decode_reference as ref
from test_gpu_decode_step import (U16, U32, UBF, check_attention, dev, host, layout, make_cache, run_attention,
                                  run_logprobs)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tw():
    import __graft_entry__ as g
    g.build()
    import activation_sparse_transformer_gb300 as m
    return m


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("fmt,page,heads,group,dim,requests,new", [
    ("e4m3", 64, 8, 4, 128, 2, 64), ("int8", 16, 16, 1, 64, 1, 64), ("int8", 32, 8, 2, 128, 1, 40),
    ("e4m3", 128, 2, 8, 64, 3, 80)])
@pytest.mark.parametrize("length", [513, 600, 1000, 1024])
def test_attention_more_tokens_than_the_bound(tw, fmt, page, heads, group, dim, requests, new, length):
    """max_q_len = 1 where the requests have many tokens (a bound fixed at a graph's
    capture, say): a CTA that was meant for one segment gets its many row blocks."""
    r = np.random.RandomState(length + dim)
    lens = np.array([length - 40 * i for i in range(requests)])
    n_pages = int(sum(-(-lens // page)))
    cache, kc, ks, vc, vs = make_cache(tw, fmt, n_pages, page, heads, dim, 7)
    table = layout(r, lens, page, n_pages, int(max(-(-lens // page))))
    cu = (np.arange(requests + 1) * new).astype(np.int32)
    positions = np.concatenate([np.arange(n - new, n) for n in lens]).astype(np.int32)
    import torch
    q = dev(r.randn(requests * new, heads * group, dim) * 1.3).to(torch.bfloat16)
    for max_q in (0, 1):
        o, lse = run_attention(tw, cache, q, table, cu, positions, lens, max_q=max_q)
        assert tw.twell_kv_read_status(cache) == 0
        check_attention(q, kc, ks, vc, vs, table, cu, positions, lens, group, dim ** -0.5, o, lse)


