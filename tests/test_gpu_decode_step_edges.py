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


def one_dim_cache(tw, fmt, page, dim, logits, values):
    """One request of one head whose token j has the logit q[0] * logits[j] and the value values[j] in
    every dim, all of them codes as they are (scale 1); returns (cache, table)."""
    n = len(logits)
    pages = -(-n // page)
    cache = tw.alloc_kv_cache(pages, page, 1, dim, tw.KV_E4M3 if fmt == "e4m3" else tw.KV_INT8, "cuda")
    k, v = np.zeros((pages * page, dim)), np.zeros((pages * page, dim))
    k[:n, 0], v[:n] = logits, np.asarray(values)[:, None]
    for codes, scale, x in ((cache.k, cache.k_scale, k), (cache.v, cache.v_scale, v)):
        codes.copy_(dev(x.reshape(pages, 1, page, dim)).to(codes.dtype))
        assert np.array_equal(host(codes.float()).reshape(-1, dim), x)
        scale.fill_(1.0)
    return cache, np.arange(pages, dtype=np.int32)[None]


@pytest.mark.parametrize("fmt,dim", [("e4m3", 64), ("int8", 128)])
@pytest.mark.parametrize("rows", [1, 4, 8, 16, 40])
@pytest.mark.parametrize("bound", [300, 1 << 20])
def test_attention_keeps_what_a_larger_logit_follows(tw, fmt, dim, rows, bound):
    """Token 0 outweighs its neighbours by e^96, and a later one outweighs it by e^7: what
    token 0 brought stays in every dim.  o = 64 e^-7 / (1 + e^-7): its terms are exact but for the weight,
    which is rounded to fp16 after an exponential good to 2^-20."""
    import torch
    logits, values = np.full(300, -96.0), np.zeros(300)
    logits[0], values[0], logits[260] = 0.0, 64.0, 7.0
    cache, table = one_dim_cache(tw, fmt, 16, dim, logits, values)
    q = torch.zeros((1, rows, dim), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    o, lse = run_attention(tw, cache, q, table, np.array([0, 1], np.int32), np.array([299], np.int32), [300],
                           max_kv=bound, scale=1.0)
    want = 64 * np.exp(-7.0) / (1 + np.exp(-7.0))
    assert (np.abs(host(o) - want) <= want * (UBF + U16 + 2.0 ** -19)).all()
    assert (np.abs(host(lse) - (7 + np.log1p(np.exp(-7.0)))) <= 2.0 ** -19 + 4 * U32 * 7).all()


@pytest.mark.parametrize("fmt,dim,new", [("e4m3", 128, 70), ("int8", 64, 70), ("e4m3", 64, 1), ("int8", 128, 4)])
@pytest.mark.parametrize("bound", [1, 30000])
def test_attention_of_many_small_weights(tw, fmt, dim, new, bound):
    """One token outweighs each of the others by e^18 and has the value 0, they have the
    value 1: o is their weights' sum, N e^-18 / (1 + N e^-18).  A weight in fp16 is off by 2^-25 of
    fp16's 1 where it is below 2^-14, and the largest weight stands at 2^7 or above: N 2^-32 in all.
    (A short bound keeps the cache in one piece, where they all meet the one large weight.)"""
    import torch
    n = 30000
    logits, values = np.zeros(n), np.ones(n)
    logits[0], values[0] = 18.0, 0.0
    cache, table = one_dim_cache(tw, fmt, 128, dim, logits, values)
    q = torch.zeros((new, 1, dim), dtype=torch.bfloat16, device="cuda")
    q[:, :, 0] = 1.0
    positions = np.arange(n - new, n).astype(np.int32)
    o, _ = run_attention(tw, cache, q, table, np.array([0, new], np.int32), positions, [n], max_q=new, max_kv=bound,
                         scale=1.0)
    tail = positions * np.exp(-18.0)
    want = (tail / (1 + tail))[:, None, None]
    assert (np.abs(host(o) - want) <= want * (UBF + U16 + 2.0 ** -19 + 2 * n * U32) + n * 2.0 ** -32).all()


@pytest.mark.parametrize("fmt,dim", [("e4m3", 64), ("int8", 128)])
@pytest.mark.parametrize("length,new", [(150, 90), (9000, 1), (9000, 12), (20000, 70)])
def test_attention_scales_far_apart_in_chunks_and_parts(tw, fmt, dim, length, new):
    """Value scales from 2^-60 to 2^40 in the chunk kernel and where caches are cut and their parts
    joined: neither weights nor sums nor the parts' references may leave their range.  Bounds as in
    check_attention, and 2^-32 of the row's largest weight for each weight in fp16: it shows where the tokens
    of large weights hold the code 0."""
    import torch
    r = np.random.RandomState(length + new)
    page, lens = 64, np.array([length])
    n_pages = -(-length // page)
    cache, kc, ks, vc, vs = make_cache(tw, fmt, n_pages, page, 1, dim, 2)
    vs = np.exp2(r.randint(-60, 41, vs.shape)).astype(np.float64)
    ks = np.exp2(r.randint(-14, -3, ks.shape)).astype(np.float64)
    cache.v_scale.copy_(dev(vs).float())
    cache.k_scale.copy_(dev(ks).float())
    table = layout(r, lens, page, n_pages, n_pages)
    q = dev(r.randn(new, 4, dim) * np.array([1e-3, 1, 3, 30])[None, :, None]).to(torch.bfloat16)
    cu, positions = np.array([0, new], np.int32), np.arange(length - new, length).astype(np.int32)
    o, lse = run_attention(tw, cache, q, table, cu, positions, lens, max_q=new)
    pages = table[0]
    k = (kc[pages, 0] * ks[pages, 0, None, None]).reshape(-1, dim)[:length]
    v = (vc[pages, 0] * vs[pages, 0, None, None]).reshape(-1, dim)[:length]
    rows, limit = host(q).reshape(-1, dim), np.repeat(positions + 1, 4)
    want, want_lse, spread, most = ref.attention(rows, k, v, dim ** -0.5, limit)
    depth = 2 * 2 * dim * U32 * most + 2.0 ** -20 + 2 * length * U32
    s_v = np.repeat(vs[pages, 0], page)[:length]
    for i, (got, got_lse) in enumerate(zip(host(o).reshape(-1, dim), host(lse).reshape(-1))):
        p = np.exp(dim ** -0.5 * (k[:limit[i]] @ rows[i]) - want_lse[i])
        tiny = length * 2.0 ** -32 * (p * s_v[:limit[i]]).max() * ref.QMAX[fmt]
        tol = UBF * np.abs(want[i]) * (1 + 2.0 ** -6) + (U16 + depth) * spread[i] + tiny + 1e-30
        assert (np.abs(got - want[i]) <= tol).all(), (i, (np.abs(got - want[i]) / tol).max())
        assert abs(got_lse - want_lse[i]) <= depth + 4 * U32 * abs(want_lse[i]), i


HIDDEN = [  # page, group, dim, length, positions: the rows of one request
    (16, 4, 64, 300, [100]),                            # a single token and pages that are to be written yet
    (64, 1, 128, 700, [9]),
    (32, 8, 128, 90, [3, 40, 41, 42]),                  # several tokens that see different parts of a page
    (16, 2, 64, 900, list(range(880, 900))),
    (128, 4, 128, 1500, list(range(700, 760))),         # a chunk
    (16, 1, 64, 300, list(range(180, 260)) + [-1, 5]),
    (128, 1, 128, 20000, list(range(9950, 10050))),     # a chunk whose cache is cut into parts
    (64, 1, 64, 9000, [4000, 4001]),                    # single rows whose cache is cut
]


@pytest.mark.parametrize("page,group,dim,length,positions", HIDDEN)
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("scale", [0.0, float("nan"), float("inf")])
def test_attention_of_hidden_tokens_that_are_no_numbers(tw, page, group, dim, length, positions, fmt, scale):
    """kv_lens beyond the rows' positions: what no row sees (codes of NaN, scales that were never
    written) leaves no trace."""
    import torch
    r = np.random.RandomState(length)
    lens, n_pages = np.array([length]), -(-length // page)
    cache, kc, ks, vc, vs = make_cache(tw, fmt, n_pages, page, 2, dim, 3)
    table = layout(r, lens, page, n_pages, n_pages)
    first = max(positions) + 1   # the first token that nobody sees
    for c in (cache.k, cache.v):
        raw = c.view(torch.uint8)
        for j in range(first // page, n_pages):
            raw[int(table[0, j]), :, max(first - j * page, 0):] = 0x7F if fmt == "e4m3" else 0x80
    for s in (cache.k_scale, cache.v_scale):
        for j in range(-(-first // page), n_pages):
            s[int(table[0, j])] = scale
    positions = np.array(positions, np.int32)
    cu = np.array([0, len(positions)], np.int32)
    q = dev(r.randn(len(positions), 2 * group, dim) * 1.3).to(torch.bfloat16)
    o, lse = run_attention(tw, cache, q, table, cu, positions, lens, max_q=len(positions))
    ks[~np.isin(np.arange(n_pages), table[0, :-(-first // page)])] = 1.0
    vs[~np.isin(np.arange(n_pages), table[0, :-(-first // page)])] = 1.0
    check_attention(q, kc, ks, vc, vs, table, cu, positions, lens, group, dim ** -0.5, o, lse)


@pytest.mark.parametrize("page,group,dim,length,positions", HIDDEN[2:])
@pytest.mark.parametrize("what", ["k", "v"])
def test_attention_of_a_nan_code_that_some_rows_see(tw, page, group, dim, length, positions, what):
    """One NaN among the codes of a token: rows that end before it are as without it, the
    others are no numbers in that dim (a key's: in all dims)."""
    import torch
    r = np.random.RandomState(length + 1)
    lens, n_pages = np.array([length]), -(-length // page)
    cache, kc, ks, vc, vs = make_cache(tw, "e4m3", n_pages, page, 2, dim, 3)
    table = layout(r, lens, page, n_pages, n_pages)
    positions = np.array(positions, np.int32)
    at = int(positions[len(positions) // 2])   # half of the rows see it
    getattr(cache, what).view(torch.uint8)[int(table[0, at // page]), :, at % page, dim - 5] = 0xFF
    cu = np.array([0, len(positions)], np.int32)
    q = dev(r.randn(len(positions), 2 * group, dim) * 1.3).to(torch.bfloat16)
    o, lse = run_attention(tw, cache, q, table, cu, positions, lens, max_q=len(positions))
    sees = positions >= at
    assert sees.any() and not sees.all()
    assert np.isnan(host(o)[sees][..., dim - 5]).all()
    assert what == "v" or np.isnan(host(o)[sees]).all()
    for i in np.flatnonzero(~sees):
        check_attention(q[i:i + 1], kc, ks, vc, vs, table, np.array([0, 1]), positions[i:i + 1], lens, group,
                        dim ** -0.5, o[i:i + 1], lse[i:i + 1])


@pytest.mark.parametrize("fmt,dim,group,lens,new", [
    ("e4m3", 128, 4, [1000] * 16, 1),           # segments with a CTA each
    ("int8", 64, 1, [9000, 20000], 1),          # cut segments
    ("int8", 64, 1, [100 + 3 * i for i in range(120)], 1),   # short segments, one a warp
    ("e4m3", 128, 2, [3000] * 40, 1),           # whole segments, several a CTA
    ("e4m3", 64, 4, [700, 20000], 90),          # chunks, whole and in parts
    ("int8", 128, 4, [100], 40)])               # a chunk of one step
def test_attention_whose_copies_do_not_arrive(tw, fmt, dim, group, lens, new):
    """A barrier that one arrival is missing from: the waits expire (here after 1 ms), every CTA lets
    its copies land and leaves, the status tells, and the next call is right."""
    import torch
    r = np.random.RandomState(dim)
    page, lens, heads = 16, np.array(lens), 4
    n_pages = int(sum(-(-lens // page)))
    cache, kc, ks, vc, vs = make_cache(tw, fmt, n_pages, page, heads, dim, 5)
    table = layout(r, lens, page, n_pages, int(max(-(-lens // page))))
    cu = (np.arange(len(lens) + 1) * new).astype(np.int32)
    positions = np.concatenate([np.arange(n - new, n) for n in lens]).astype(np.int32)
    n, q_heads = len(positions), heads * group
    q = dev(r.randn(n, q_heads, dim)).to(torch.bfloat16)
    o = torch.empty_like(q)
    ws = torch.empty(tw.kv_attention_workspace_bytes(n, len(lens), q_heads, heads, dim), dtype=torch.uint8,
                     device="cuda")
    d = [dev(x) for x in (table, cu, positions, lens.astype(np.int32))]
    ld = q_heads * dim
    args = (q.data_ptr(), ld, cache.struct(), d[0].data_ptr(), table.shape[1], d[1].data_ptr(), d[2].data_ptr(),
            d[3].data_ptr(), n, len(lens), q_heads, int(max(lens)), new, dim ** -0.5, o.data_ptr(), ld, None,
            ws.data_ptr(), ws.numel())
    stall = tw.load_library().twell_selftest_kv_attention_stall
    assert stall(*args, 0, None) == -1 and stall(*args, 2_000_000_000, None) == -1
    assert stall(*args, 1_000_000, torch.cuda.current_stream().cuda_stream) == 0
    assert tw.twell_kv_read_status(cache) == -7
    cache.status.zero_()
    o, lse = run_attention(tw, cache, q, table, cu, positions, lens, max_q=new)
    assert tw.twell_kv_read_status(cache) == 0
    check_attention(q, kc, ks, vc, vs, table, cu, positions, lens, group, dim ** -0.5, o, lse)


# ---------------------------------------------------------------- log probabilities
def far_rows(r, n, vocab, t):
    """Rows of t at the ends of its range: all at its lowest value; all there but for masked ones; one
    at its largest and the rest spread over it all; far from zero with small distances; ordinary ones."""
    import torch
    low, high = torch.finfo(t).min, torch.finfo(t).max
    x = r.randn(n, vocab) * 2
    for i in range(n):
        if i % 6 == 0:
            x[i] = low
        elif i % 6 == 1:
            x[i] = np.where(np.arange(vocab) % 3 == 1, -np.inf, low)
        elif i % 6 == 2:
            x[i] = low + (high / 2 - low / 2) * r.rand(vocab) * 1.9
            x[i, vocab // 2] = high
        elif i % 6 == 3:
            x[i] = np.round(4 * r.randn(vocab)) + 3e6      # a quarter is the distance of fp32 there
        elif i % 6 == 4:
            x[i] = -1e9 - 64 * r.randint(0, 3, vocab)      # 64 is
    return dev(x).to(t)


def far_reference(x, target, k):
    """ref.logprobs for rows without NaN and +inf, by distances from the maximum: lse itself, in 64
    bits too, is too coarse at 1e38."""
    has, order = 0 <= target < len(x), sorted(range(len(x)), key=lambda j: (-x[j], j))[:k]
    m = x.max()
    if m == -np.inf:
        return (-np.inf if has else 0.0), 0.0, -np.inf, np.full(k, -np.inf), np.array(order)
    logp = (x - m) - np.log(np.exp(x - m).sum())
    p = np.exp(logp)
    return (logp[target] if has else 0.0, -(p[p > 0] * logp[p > 0]).sum(), m + np.log(np.exp(x - m).sum()),
            logp[order], np.array(order))


FAR = [(12, 700), (12, 40000), (7, 131072), (400, 30000), (1300, 500), (1300, 40)]


@pytest.mark.parametrize("n,vocab", FAR)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("inv_t", [1.0, 0.5])
@pytest.mark.parametrize("k", [0, 5])
def test_logprobs_at_the_ends_of_the_type(tw, n, vocab, dtype, inv_t, k):
    """x = logits * inv_t is finite there though its product with log2 e is not, or is too coarse.
    Distances from the largest x are exact or one rounding; a result of size S is rounded to 2^-24 S,
    and of distances that are no more than 90 the bounds are the ordinary ones."""
    import torch
    t = getattr(torch, dtype)
    r = np.random.RandomState(vocab)
    x = far_rows(r, n, vocab, t)
    targets = r.randint(-1, vocab + 1, n).astype(np.int32)
    got = [None if v is None else host(v) for v in run_logprobs(tw, x, dev(targets), inv_t, k)]
    xs = host(x.float() * torch.tensor(inv_t, dtype=torch.float32, device="cuda"))
    tol = 2.0 ** -21 + 2 * (vocab / 256 + 40) * U32 + 4 * U32 * 90

    def near(a, b, what):
        if np.abs(b) <= float(torch.finfo(torch.float32).max):
            assert abs(a - b) <= tol + 4 * U32 * abs(b), what
        else:   # no number of the results' type
            assert a == np.copysign(np.inf, b), what

    for i in list(range(min(n, 12))) + list(range(12, n, 61)):
        lp, en, lse, top, index = far_reference(xs[i], int(targets[i]), k)
        near(got[2][i], lse, (i, "lse"))
        near(got[0][i], lp, (i, "logprob"))
        assert abs(got[1][i] - en) <= 4 * (tol + 2 * U32) * (en + 2), (i, "entropy", got[1][i], en)
        if k:
            assert np.array_equal(got[4][i], index), i
            for j in range(k):
                near(got[3][i][j], top[j], (i, "top"))


@pytest.mark.parametrize("n,vocab", [(12, 700), (12, 40000), (6, 131072), (2500, 200)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("inv_t", [1.0, 0.5])
@pytest.mark.parametrize("in_place", [False, True])
def test_logprobs_gradient_at_the_ends_of_the_type(tw, n, vocab, dtype, inv_t, in_place):
    """There lse, in 32 bits, does not tell a row's sum from its maximum: p is still the softmax.  Bounds as for
    ordinary rows: p is off by 2^-20 and the sum's roundings of itself, the result by its type's."""
    import torch
    t = getattr(torch, dtype)
    r = np.random.RandomState(vocab)
    x = far_rows(r, n, vocab, t)
    kept = x.clone()
    targets = r.randint(-1, vocab + 1, n).astype(np.int32)
    _, entropy, lse, *_ = run_logprobs(tw, x, dev(targets), inv_t, 0)
    g, gh = r.randn(n).astype(np.float32), r.randn(n).astype(np.float32)
    out = x if in_place else torch.empty_like(x)
    tw.twell_logprobs_bwd(x, dev(targets), inv_t, lse, entropy, dev(g), dev(gh), out)
    xs, got = host(kept.float() * torch.tensor(inv_t, dtype=torch.float32, device="cuda")), host(out)
    ulp = UBF if dtype == "bfloat16" else U32
    for i in list(range(min(n, 12))) + list(range(12, n, 61)):
        _, en, *_ = far_reference(xs[i], -1, 0)
        m = xs[i].max()
        logp = (xs[i] - m) - np.log(np.exp(xs[i] - m).sum())
        p = np.exp(logp)
        has = 0 <= targets[i] < vocab
        w = -float(gh[i]) * (np.where(p > 0, logp, 0) + en)
        want = p * w - (p * g[i] if has else 0)
        size = p * (np.abs(w) + abs(float(gh[i])) * (np.abs(np.where(p > 0, logp, 0)) + en + 1) + abs(g[i]))
        if has:
            want[targets[i]] += g[i]
        want, size = want * inv_t, size * inv_t
        rel = 2.0 ** -20 + (vocab / 256 + 40) * 2 * U32 + 8 * U32 * 90
        tol = rel * size + 2 * U32 * np.abs(want) + ulp * np.abs(want) * (1 + 2 * rel) + 1e-37
        assert (np.abs(got[i] - want) <= tol + ulp * rel * size).all(), (i, (np.abs(got[i] - want) / tol).max())


# ---------------------------------------------------------------- buffers
def test_buffers_that_moved_are_used_where_they_are(tw):
    """A plan's or a cache's tensor that was given other storage after the first call: the next
    call works on the new one, and checks it."""
    import torch
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    plan = tw.alloc_kv_plan(2, 3)
    ring, pool = tw.alloc_page_ring(4)
    table = torch.zeros((2, 2), dtype=torch.int32, device="cuda")
    args = (i32([0, 0]), i32([1, 2]), table, ring, pool, 16, plan)
    tw.twell_kv_plan(*args)
    old = plan.slots.clone(), plan.slots.view_as(plan.slots)   # the view keeps the old storage
    plan.slots.set_(torch.full((3,), 77, dtype=torch.int64, device="cuda"))
    old[1].fill_(-5)
    tw.twell_kv_plan(*args)
    assert torch.equal(plan.slots, old[0]) and (old[1] == -5).all()
    plan.positions.set_(torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="positions"):
        tw.twell_kv_plan(*args)

    cache = tw.alloc_kv_cache(2, 16, 1, 64, tw.KV_INT8)
    x = torch.ones((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    cu, slots = i32([0, 1]), torch.zeros(1, dtype=torch.int64, device="cuda")
    tw.twell_kv_append(x, x, cu, slots, cache)
    code = cache.k[0, 0, 0].clone()
    before = cache.k.view_as(cache.k)
    cache.k.set_(torch.zeros_like(cache.k))
    before.fill_(3)
    tw.twell_kv_append(x, x, cu, slots, cache)
    assert torch.equal(cache.k[0, 0, 0], code) and (before == 3).all()
    cache.v.set_(torch.zeros((1, 1, 16, 64), dtype=torch.int8, device="cuda"))
    with pytest.raises(ValueError, match="k, v"):
        tw.twell_kv_append(x, x, cu, slots, cache)
    for t in (cache.k, cache.v):
        t.set_(torch.zeros((2, 2, 16, 64), dtype=torch.int8, device="cuda"))
    for t in (cache.k_scale, cache.v_scale):
        t.set_(torch.zeros((2, 2), device="cuda"))
    with pytest.raises(ValueError, match="k, v"):   # K and V have one head
        tw.twell_kv_append(x, x, cu, slots, cache)


def test_alternatives_and_queries_of_the_wrong_shape_are_refused(tw):
    """The k best go to two [rows, k] matrices of the same k; queries have three dimensions."""
    import torch
    x = torch.zeros((4, 100), device="cuda")
    lse = torch.empty(4, device="cuda")
    f = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
    i = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    for top, index in ((f(4, 5), i(4, 6)), (f(4, 5), i(20)), (f(20), i(4, 5)), (f(3, 5), i(3, 5))):
        with pytest.raises(ValueError, match="top_logprob"):
            tw.twell_logprobs(x, None, 1.0, None, None, lse, top, index)
    cache = tw.alloc_kv_cache(1, 16, 1, 64)
    i32 = i(2)
    for q in (torch.empty(64, device="cuda"), torch.empty((1, 64), device="cuda")):
        with pytest.raises(ValueError, match="^Q: shape"):
            tw.twell_kv_attention(q.bfloat16(), cache, i(1, 1), i32, i32, i(1), 1, 1, 0.1, q.bfloat16(), f(256))
