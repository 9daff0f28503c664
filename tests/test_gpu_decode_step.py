"""The decode step's operators on the GPU against plain 64-bit definitions
(tests/decode_reference.py): block tables and slot maps, the append to the
8-bit cache and the log probabilities' indexes exactly; computed numbers within
bounds derived from the formats' rounding."""
import numpy as np
import pytest

import decode_reference as ref

pytestmark = pytest.mark.gpu

U32, U16, UBF = 2.0 ** -24, 2.0 ** -11, 2.0 ** -8   # half a unit of fp32, fp16, bf16 (24, 11, 8 bits)


@pytest.fixture(scope="module")
def tw():
    import __graft_entry__ as g
    g.build()
    import activation_sparse_transformer_gb300 as m
    return m


def dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def host(t):
    import torch
    return t.detach().to(torch.float64 if t.is_floating_point() else t.dtype).cpu().numpy()


# ---------------------------------------------------------------- plan
def run_plan(tw, lens, new, table, ring, pool, page, n_tokens):
    t, g = dev(table), dev(ring)
    plan = tw.alloc_kv_plan(len(lens), n_tokens, "cuda")
    for x in (plan.kv_lens, plan.cu_q, plan.slots, plan.positions, plan.pool, plan.status):
        x.fill_(77)
    args = (dev(lens), dev(new), t, g, dev(np.array(pool, np.int32)), page, plan)
    tw.twell_kv_plan(*args)
    tw.twell_kv_plan(*args)   # nothing that is read was overwritten
    return dict(kv_lens=host(plan.kv_lens), cu_q=host(plan.cu_q), slots=host(plan.slots),
                positions=host(plan.positions), pool=host(plan.pool), table=host(t), ring=host(g),
                status=int(host(plan.status)[0]))


@pytest.mark.parametrize("R,page,n_pages,width,max_new,slack,seed", [
    (1, 64, 8, 4, 1, 0, 0), (1, 16, 40, 40, 500, 3, 1), (16, 64, 600, 70, 1, 0, 2), (33, 16, 900, 40, 40, 7, 3),
    (300, 32, 700, 20, 90, -200, 4), (1000, 16, 20000, 64, 300, 1, 5), (257, 128, 300, 3, 200, 0, 6),
    (16384, 16, 60000, 5, 3, 11, 7)])
def test_plan_matches_definition(tw, R, page, n_pages, width, max_new, slack, seed):
    r = np.random.RandomState(seed)
    lens = (width * page * r.rand(R) * 0.8).astype(np.int32)
    have = -(-lens // page)
    while have.sum() > n_pages * 0.8:   # the pages in use fit
        lens = (lens * 0.7).astype(np.int32)
        have = -(-lens // page)
    new = np.where(r.rand(R) < 0.5, 1, (r.rand(R) * (max_new + 1)).astype(np.int64)).astype(np.int32)
    new[r.rand(R) < 0.15] = -1 - r.randint(3)
    new[r.rand(R) < 0.1] = 0
    order = r.permutation(n_pages).astype(np.int32)
    used = int(have.sum())
    table = np.full((R, width), -5, np.int32)
    at = 0
    for i in range(R):
        table[i, :have[i]] = order[at:at + have[i]]
        at += have[i]
    ring = np.full(n_pages, -9, np.int32)
    head = r.randint(n_pages)
    ring[(head + np.arange(n_pages - used)) % n_pages] = order[used:]
    n_tokens = max(0, int(np.maximum(new, 0).sum()) + slack)
    pool = (head, n_pages - used)
    want = ref.plan(lens, new, table, ring, pool, page, n_tokens)
    got = run_plan(tw, lens, new, table, ring, pool, page, n_tokens)
    for k in want:
        assert np.array_equal(got[k], want[k]), k


def test_plan_steps_never_lose_or_share_a_page(tw):
    """60 steps of a small server that fills up: the pages of the requests and
    the free ones are the whole pool at all times."""
    r = np.random.RandomState(3)
    R, page, n_pages, width = 12, 16, 50, 9
    lens, table = np.zeros(R, np.int32), np.full((R, width), -1, np.int32)
    ring, pool = np.arange(n_pages, dtype=np.int32), np.array([0, n_pages], np.int32)
    refused = 0
    for _ in range(60):
        new = r.randint(0, 30, R).astype(np.int32)
        new[(lens > 60) & (r.rand(R) < 0.5)] = -1
        got = run_plan(tw, lens, new, table, ring, pool, page, int(np.maximum(new, 0).sum()))
        want = ref.plan(lens, new, table, ring, tuple(pool), page, int(np.maximum(new, 0).sum()))
        for k in want:
            assert np.array_equal(got[k], want[k]), k
        refused += got["status"] != 0
        lens, table, ring, pool = got["kv_lens"], got["table"], got["ring"], got["pool"]
        held = [table[i, j] for i in range(R) for j in range(-(-int(lens[i]) // page))]
        free = [ring[(pool[0] + i) % n_pages] for i in range(pool[1])]
        assert sorted(held + free) == list(range(n_pages))
    assert refused > 3


def test_plan_of_no_requests_and_no_tokens(tw):
    import torch
    plan = tw.alloc_kv_plan(0, 3, "cuda")
    ring, pool = tw.alloc_page_ring(4)
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    tw.twell_kv_plan(e, e, torch.empty((0, 4), dtype=torch.int32, device="cuda"), ring, pool, 16, plan)
    assert host(plan.slots).tolist() == [-1] * 3 and host(plan.cu_q).tolist() == [0]
    assert host(plan.pool).tolist() == [0, 4]


# ---------------------------------------------------------------- cache
def make_cache(tw, fmt, n_pages, page, heads, dim, seed, poison=True):
    """A cache of random codes; returns (cache, key codes, key scales, value codes, value scales) in 64 bits."""
    import torch
    r = np.random.RandomState(seed)
    c = tw.alloc_kv_cache(n_pages, page, heads, dim, tw.KV_E4M3 if fmt == "e4m3" else tw.KV_INT8, "cuda")
    out = [c]
    for codes, scale in ((c.k, c.k_scale), (c.v, c.v_scale)):
        x = ref.round_code(np.clip(r.randn(*codes.shape) * (60 if fmt == "int8" else 100),
                                   -ref.QMAX[fmt], ref.QMAX[fmt]), fmt)
        s = np.exp2(r.randint(-9, -4, scale.shape)).astype(np.float64)
        codes.copy_(dev(x).to(codes.dtype))
        scale.copy_(dev(s).float())
        out += [x, s]
    return out


def layout(r, lens, page, n_pages, width):
    """A block table of shuffled pages; entries past a request's pages hold an invalid number."""
    need = [-(-int(n) // page) for n in lens]
    order = r.permutation(n_pages)[:sum(need)]
    table, at = np.full((len(lens), width), -7, np.int32), 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table


APPEND = [  # fmt, page, heads, dim, old lengths, new tokens
    ("e4m3", 64, 8, 128, [0, 63, 64, 65, 1], [1, 1, 1, 1, 1]),
    ("int8", 64, 2, 128, [5, 0, 130], [200, 64, 3]),
    ("e4m3", 16, 3, 64, [15, 16, 0, 40], [1, 33, 0, 7]),
    ("int8", 32, 1, 64, [31, 33], [65, 31]),
    ("int8", 128, 2, 64, [100, 0], [60, 257]),
    ("e4m3", 128, 2, 128, [127, 3], [129, 124]),
    ("int8", 16, 5, 128, [7] * 40, [1] * 40),
]


@pytest.mark.parametrize("fmt,page,heads,dim,old,new", APPEND)
def test_append_is_exact(tw, fmt, page, heads, dim, old, new):
    import torch
    r = np.random.RandomState(len(old) * 31 + page)
    old, new = np.array(old), np.array(new)
    total = old + new
    n_pages = int(sum(-(-total // page))) + 2
    cache, kc, ks, vc, vs = make_cache(tw, fmt, n_pages, page, heads, dim, 9)
    width = int(max(-(-total // page)))
    table = layout(r, total, page, n_pages, width)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    slots = np.concatenate([[table[i, p // page] * page + p % page for p in range(a, a + b)]
                            for i, (a, b) in enumerate(zip(old, new))] + [[]]).astype(np.int64)
    n = int(cu[-1])
    # K and V as slices of one wider matrix; sizes over many powers of two, so that some scales grow and
    # others stay, a token of zeros, and the smallest bf16
    x = r.randn(n, 3 * heads, dim) * np.exp2(r.randint(-14, 8, (n, 1, 1)))
    x[n // 2] = 0
    x[0, heads, 0] = 2.0 ** -133
    both = dev(x).to(torch.bfloat16)
    K, V = both[:, heads:2 * heads], both[:, 2 * heads:]
    tw.twell_kv_append(K, V, dev(cu), dev(slots), cache)
    assert tw.twell_kv_read_status(cache) == 0
    for got_c, got_s, c, s, new_x in ((cache.k, cache.k_scale, kc, ks, host(K)), (cache.v, cache.v_scale, vc, vs, host(V))):
        want_c, want_s = ref.append(c, s, new_x, cu, slots, fmt)
        assert np.array_equal(host(got_s), want_s)
        assert np.array_equal(host(got_c.float()), want_c)


def test_append_token_by_token_equals_the_prompt_for_e4m3(tw):
    """e4m3 codes move to a larger power of two unchanged while they stay above
    2^-6: a sequence written token by token ends with the codes of one call."""
    import torch
    r = np.random.RandomState(0)
    n, heads, dim, page = 50, 2, 64, 16
    # every magnitude within 2^8 of the page's largest
    x = dev(np.sign(r.randn(n, heads, dim)) * np.exp2(r.uniform(-3, 4, (n, heads, dim)))).to(torch.bfloat16)
    caches = [tw.alloc_kv_cache(4, page, heads, dim, tw.KV_E4M3, "cuda") for _ in range(2)]
    slots = torch.arange(n, device="cuda")
    tw.twell_kv_append(x, x, dev(np.array([0, n], np.int32)), slots, caches[0])
    one = dev(np.array([0, 1], np.int32))
    for t in range(n):
        tw.twell_kv_append(x[t:t + 1], x[t:t + 1], one, slots[t:t + 1], caches[1])
    assert torch.equal(caches[0].k_scale, caches[1].k_scale)
    a, b = (c.k.view(torch.uint8).transpose(1, 2).reshape(-1, heads, dim)[:n] for c in caches)
    assert torch.equal(a, b)


def test_append_reports_values_that_are_not_finite_and_slots_outside(tw):
    import torch
    cache, kc, ks, vc, vs = make_cache(tw, "int8", 4, 16, 1, 64, 1)
    x = torch.ones((2, 1, 64), dtype=torch.bfloat16, device="cuda")
    x[0, 0, 3], x[0, 0, 4], x[0, 0, 5] = float("inf"), float("nan"), float("-inf")
    cu = dev(np.array([0, 1, 2], np.int32))
    tw.twell_kv_append(x, x, cu, dev(np.array([0, -1], np.int64)), cache)
    assert tw.twell_kv_read_status(cache) == -11
    row = host(cache.k)[0, 0, 0]
    # the largest bf16 is 255 * 2^120 = 63.75 * 2^122, and 127 * 2^121 is less than it; 1 is far below the step
    assert row[3] == 64 and row[4] == 0 and row[5] == -64 and row[6] == 0
    assert np.array_equal(host(cache.v)[1:], vc[1:])
    cache.status.zero_()
    before = cache.k.clone()
    tw.twell_kv_append(x[1:], x[1:], cu[:2], dev(np.array([64], np.int64)), cache)
    assert tw.twell_kv_read_status(cache) == -9
    assert torch.equal(before, cache.k)


# ---------------------------------------------------------------- attention
def run_attention(tw, cache, q, table, cu, positions, lens, max_q=None, max_kv=None, lse=True, ldo_extra=0,
                  scale=None):
    import torch
    n, heads, dim = q.shape
    o = torch.full((n, heads * dim + ldo_extra), 7.0, dtype=torch.bfloat16, device="cuda")[:, :heads * dim]
    o = o.unflatten(1, (heads, dim))
    out_lse = torch.full((n, heads), 7.0, device="cuda") if lse else None
    ws = torch.empty(tw.kv_attention_workspace_bytes(n, len(lens), heads, cache.n_heads, dim), dtype=torch.uint8,
                     device="cuda")
    ws.fill_(0xFF)   # a workspace's contents do not matter
    tw.twell_kv_attention(q, cache, dev(table), dev(cu), dev(positions), dev(np.array(lens, np.int32)),
                          int(max(lens)) if max_kv is None else max_kv, 1 if max_q is None else max_q,
                          dim ** -0.5 if scale is None else scale, o, ws, lse=out_lse)
    return o, out_lse


def check_attention(q, kc, ks, vc, vs, table, cu, positions, lens, group, scale, o, lse):
    """Every row against the definition.  Bounds: the products are exact and an
    fp32 sum of D of them is off by at most D units of its terms' sum X, so a
    logit by 2 D u X (u = 2^-24, twice for a sum that cuts instead of rounding) and a
    probability by that much of itself, plus 2^-11 of itself for its rounding to fp16 (and
    2^-25 of the largest where it is tiny), 2^-21 for exp2 and the factors; o is rounded once to bf16."""
    heads, page, dim = kc.shape[1], kc.shape[2], kc.shape[3]
    q, o = host(q), host(o)
    lse = None if lse is None else host(lse)
    for r, length in enumerate(lens):
        pages = table[r, :-(-int(length) // page)]
        beg, end = cu[r], cu[r + 1]
        limit = np.repeat(np.minimum(positions[beg:end] + 1, length), group)
        for h in range(heads):
            k = (kc[pages, h] * ks[pages, h, None, None]).reshape(-1, dim)[:length]
            v = (vc[pages, h] * vs[pages, h, None, None]).reshape(-1, dim)[:length]
            rows = q[beg:end, h * group:(h + 1) * group].reshape(-1, dim)
            want, want_lse, spread, most = ref.attention(rows, k, v, scale, limit)
            got = o[beg:end, h * group:(h + 1) * group].reshape(-1, dim)
            rel = U16 + 2 * 2 * dim * U32 * most + 2.0 ** -20 + 2 * max(length, 1) * U32
            tol = UBF * np.abs(want) * (1 + 2.0 ** -6) + rel * spread + 1e-30
            assert np.isfinite(got).all()
            worst = (np.abs(got - want) / tol).max() if got.size else 0
            assert worst <= 1, (r, h, worst)
            if lse is not None:
                got_lse = lse[beg:end, h * group:(h + 1) * group].reshape(-1)
                empty = limit <= 0
                assert (got_lse[empty] == -np.inf).all()
                err = np.abs(got_lse[~empty] - want_lse[~empty])
                tol_lse = (2 * dim * U32 * most + 2.0 ** -20 + 2 * max(length, 1) * U32
                           + 4 * U32 * np.abs(want_lse[~empty]))
                assert (err <= tol_lse).all(), (r, h, (err / tol_lse).max())
    rest = o[cu[len(lens)]:]
    assert (rest == 0).all() and (lse is None or (lse[cu[len(lens)]:] == -np.inf).all())


ATTENTION = [  # fmt, page, kv heads, group, dim, lengths, new tokens
    ("e4m3", 64, 2, 4, 128, [1, 2, 63, 64, 65, 700], [1] * 6),
    ("int8", 64, 2, 4, 128, [1, 17, 300, 0, 129], [1, 1, 1, 0, 1]),
    ("e4m3", 16, 3, 1, 64, [1, 15, 16, 17, 333], [1] * 5),
    ("int8", 16, 1, 8, 64, [5, 100, 31], [1, 4, 2]),
    ("int8", 32, 2, 5, 128, [40, 77], [7, 1]),             # 35 rows: odd groups, several row blocks
    ("e4m3", 128, 1, 16, 128, [129, 250], [1, 3]),
    ("e4m3", 128, 1, 40, 64, [1000], [1]),                 # more rows than a tile for one token
    ("e4m3", 64, 2, 4, 128, [200, 64, 90], [200, 30, 1]),  # prompts and a single token together
    ("int8", 32, 1, 4, 64, [333, 150], [150, 150]),
    ("e4m3", 16, 2, 1, 128, [270], [270]),
    ("e4m3", 64, 8, 4, 128, [9000], [1]),                  # one long cache, split
    ("int8", 16, 1, 1, 64, [5001, 3, 2500], [1, 1, 2]),
    ("int8", 64, 1, 8, 128, [3000, 2900], [130, 40]),      # chunks at the end of longer caches
]


@pytest.mark.parametrize("fmt,page,heads,group,dim,lens,new", ATTENTION)
def test_attention_matches_definition(tw, fmt, page, heads, group, dim, lens, new):
    import torch
    r = np.random.RandomState(page + dim + len(lens))
    lens, new = np.array(lens), np.array(new)
    n_pages = int(sum(-(-lens // page))) + 3
    cache, kc, ks, vc, vs = make_cache(tw, fmt, n_pages, page, heads, dim, 4)
    width = max(1, int(max(-(-lens // page)))) + 1
    table = layout(r, lens, page, n_pages, width)
    # what no request's token occupies holds the worst there is: NaN codes, NaN scales of unused pages
    used = set()
    for i, n in enumerate(lens):
        for j in range(-(-int(n) // page)):
            used.add(int(table[i, j]))
            if fmt == "e4m3" and (j + 1) * page > n:
                for c in (cache.k, cache.v):
                    c.view(torch.uint8)[int(table[i, j]), :, int(n) - j * page:] = 0x7F
    for p in set(range(n_pages)) - used:
        cache.k_scale[p] = cache.v_scale[p] = float("nan")
    pad = 3
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    n = int(cu[-1])
    positions = np.concatenate([np.arange(a - b, a) for a, b in zip(lens, new)] + [np.full(pad, -1)]).astype(np.int32)
    wide = dev(r.randn(n + pad, heads * group + 2, dim) * 1.3).to(torch.bfloat16)
    q = wide[:, 1:-1]
    o, lse = run_attention(tw, cache, q, table, cu, positions, lens, max_q=int(new.max()), ldo_extra=16)
    assert tw.twell_kv_read_status(cache) == 0
    check_attention(q, kc, ks, vc, vs, table, cu, positions, lens, group, dim ** -0.5, o, lse)
    # the bounds choose launch shapes only, lse is optional, and the bits repeat
    for max_q, max_kv in ((0, 0), (5000, 1 << 20)):
        o2, _ = run_attention(tw, cache, q, table, cu, positions, lens, max_q=max_q, max_kv=max_kv, lse=False)
        check_attention(q, kc, ks, vc, vs, table, cu, positions, lens, group, dim ** -0.5, o2, None)
    o3, lse3 = run_attention(tw, cache, q, table, cu, positions, lens, max_q=int(new.max()), ldo_extra=16)
    assert torch.equal(o, o3) and torch.equal(lse, lse3)


def test_attention_rows_that_see_nothing_or_less(tw):
    """Refused requests (positions -1), positions behind the cache's end and in
    its middle, and a request of no cached tokens."""
    import torch
    r = np.random.RandomState(0)
    lens = np.array([100, 50, 0, 30])
    cache, kc, ks, vc, vs = make_cache(tw, "e4m3", 12, 16, 2, 64, 4)
    table = layout(r, lens, 16, 12, 8)
    cu = np.array([0, 4, 6, 8, 9], np.int32)
    positions = np.array([3, 99, 500, 50, -1, -1, 0, 1, 0], np.int32)
    q = dev(r.randn(9, 4, 64)).to(torch.bfloat16)
    o, lse = run_attention(tw, cache, q, table, cu, positions, lens, max_q=4)
    check_attention(q, kc, ks, vc, vs, table, cu, positions, lens, 2, 0.125, o, lse)
    assert (host(o)[4:8] == 0).all() and (host(lse)[4:8] == -np.inf).all()


@pytest.mark.parametrize("fmt,dim", [("e4m3", 128), ("int8", 64)])
def test_attention_chunks_over_cut_caches(tw, fmt, dim):
    """Chunks whose caches are cut into parts: rows that see nothing, that see the
    first part only, that end at parts' borders, and a cache that ends in a part's first page."""
    import torch
    r = np.random.RandomState(dim)
    page, lens, new = 128, np.array([20000, 700, 8193, 129]), np.array([70, 40, 100, 33])
    n_pages = int(sum(-(-lens // page)))
    cache, kc, ks, vc, vs = make_cache(tw, fmt, n_pages, page, 2, dim, 8)
    table = layout(r, lens, page, n_pages, int(max(-(-lens // page))))
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    positions = np.concatenate([np.arange(a - b, a) for a, b in zip(lens, new)]).astype(np.int32)
    positions[:16] = [-1, 0, 1, 127, 128, 255, 511, 639, 640, 5000, 9999, 10000, 14999, 19998, 19999, 30000]
    positions[cu[2]:cu[2] + 40] = -1    # most of a tile sees nothing
    q = dev(r.randn(int(cu[-1]), 8, dim) * 1.3).to(torch.bfloat16)
    o, lse = run_attention(tw, cache, q, table, cu, positions, lens, max_q=100)
    assert tw.twell_kv_read_status(cache) == 0
    check_attention(q, kc, ks, vc, vs, table, cu, positions, lens, 4, dim ** -0.5, o, lse)
    o2, lse2 = run_attention(tw, cache, q, table, cu, positions, lens, max_q=100)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_attention_many_chunks_and_single_tokens(tw):
    """1100 requests: chunks of every length among single tokens and idle requests, each in its place."""
    import torch
    r = np.random.RandomState(5)
    page, n = 16, 1100
    new = np.where(r.rand(n) < 0.3, r.randint(9, 80, n), r.randint(0, 2, n))
    lens = np.where(new > 0, new + r.randint(0, 300, n), 0)
    n_pages = int(sum(-(-lens // page)))
    cache, kc, ks, vc, vs = make_cache(tw, "e4m3", n_pages, page, 1, 64, 6)
    table = layout(r, lens, page, n_pages, int(max(-(-lens // page))))
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    positions = np.concatenate([np.arange(a - b, a) for a, b in zip(lens, new)]).astype(np.int32)
    q = dev(r.randn(int(cu[-1]), 8, 64) * 1.3).to(torch.bfloat16)
    o, lse = run_attention(tw, cache, q, table, cu, positions, lens, max_q=80)
    assert tw.twell_kv_read_status(cache) == 0
    check_attention(q, kc, ks, vc, vs, table, cu, positions, lens, 8, 0.125, o, lse)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_attention_scales_far_apart(tw, fmt):
    """Value scales from 2^-60 to 2^40 and key scales that make some pages' logits
    dominate: neither the weights nor the sums may leave their range.  Each probability's
    share is compared against the largest term of its own output."""
    import torch
    r = np.random.RandomState(1)
    page, lens = 16, np.array([400])
    cache, kc, ks, vc, vs = make_cache(tw, fmt, 25, page, 1, 64, 2)
    vs = np.exp2(r.randint(-60, 41, vs.shape)).astype(np.float64)
    ks = np.exp2(r.randint(-14, -3, ks.shape)).astype(np.float64)
    cache.v_scale.copy_(dev(vs).float())
    cache.k_scale.copy_(dev(ks).float())
    table = layout(r, lens, page, 25, 25)
    q = dev(r.randn(1, 4, 64) * np.array([1e-3, 1, 3, 1e4])[None, :, None]).to(torch.bfloat16)
    cu, positions = np.array([0, 1], np.int32), np.array([399], np.int32)
    o, lse = run_attention(tw, cache, q, table, cu, positions, lens)
    check_attention(q, kc, ks, vc, vs, table, cu, positions, lens, 4, 0.125, o, lse)


@pytest.mark.parametrize("new", [1, 5, 90])
def test_attention_zero_and_tiny_queries_under_a_mask(tw, new):
    """A row of zeros weighs all it sees alike, and what it does not see not at
    all; rows of the smallest numbers, keys of the smallest scales."""
    r = np.random.RandomState(new)
    page, lens = 16, np.array([150])
    cache, kc, ks, vc, vs = make_cache(tw, "e4m3", 12, page, 1, 64, 2)
    import torch
    ks = np.exp2(np.where(r.rand(*ks.shape) < 0.5, -100, -7)).astype(np.float64)
    cache.k_scale.copy_(dev(ks).float())
    table = layout(r, lens, page, 12, 11)
    x = r.randn(new, 4, 64)
    x[:, 0] = 0
    x[:, 1] *= 2.0 ** -120
    x[:, 2, 1:] = 0
    q = dev(x).to(torch.bfloat16)
    cu, positions = np.array([0, new], np.int32), np.arange(150 - new, 150).astype(np.int32)
    o, lse = run_attention(tw, cache, q, table, cu, positions, lens, max_q=new)
    check_attention(q, kc, ks, vc, vs, table, cu, positions, lens, 4, 0.125, o, lse)


def test_attention_page_outside_the_cache_is_reported(tw):
    import torch
    cache, *_ = make_cache(tw, "int8", 3, 16, 1, 64, 4)
    q = torch.ones((1, 1, 64), dtype=torch.bfloat16, device="cuda")
    run_attention(tw, cache, q, np.array([[0, 9]], np.int32), np.array([0, 1], np.int32), np.array([19], np.int32),
                  [20])
    assert tw.twell_kv_read_status(cache) == -9


def test_attention_cache_beyond_32_bit_offsets(tw):
    """A cache of more than 2^31 bytes: the pages in use are its first and last."""
    import torch
    page, heads, dim = 128, 8, 128
    n_pages = (1 << 31) // (page * heads * dim) + 3
    cache = tw.alloc_kv_cache(n_pages, page, heads, dim, tw.KV_INT8, "cuda")
    r = np.random.RandomState(5)
    lens = np.array([300])
    table = np.array([[n_pages - 1, 0, n_pages - 2]], np.int32)
    x = dev(r.randn(300, heads, dim)).to(torch.bfloat16)
    slots = dev(np.array([table[0, p // page] * page + p % page for p in range(300)], np.int64))
    tw.twell_kv_append(x, x, dev(np.array([0, 300], np.int32)), slots, cache)
    small = torch.tensor(table[0], device="cuda").long()
    kc, vc = (host(c[small].float()) for c in (cache.k, cache.v))
    ks, vs = (host(s[small]) for s in (cache.k_scale, cache.v_scale))
    q = dev(r.randn(1, 16, dim)).to(torch.bfloat16)
    cu, positions = np.array([0, 1], np.int32), np.array([299], np.int32)
    o, lse = run_attention(tw, cache, q, table, cu, positions, lens)
    check_attention(q, kc, ks, vc, vs, np.array([[0, 1, 2]]), cu, positions, lens, 2, dim ** -0.5, o, lse)


def test_attention_on_another_stream_and_in_a_graph(tw):
    import torch
    r = np.random.RandomState(2)
    lens = np.array([300, 7000])
    cache, *_ = make_cache(tw, "e4m3", 120, 64, 2, 128, 4)
    table, cu, positions = layout(r, lens, 64, 120, 112), np.array([0, 1, 2], np.int32), (lens - 1).astype(np.int32)
    q = dev(r.randn(2, 8, 128)).to(torch.bfloat16)
    want, want_lse = run_attention(tw, cache, q, table, cu, positions, lens)
    args = [dev(x) for x in (table, cu, positions, lens.astype(np.int32))]
    o, lse = torch.empty_like(want), torch.empty_like(want_lse)
    ws = torch.empty(tw.kv_attention_workspace_bytes(2, 2, 8, 2, 128), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):
        tw.twell_kv_attention(q, cache, *args, 7000, 1, 128 ** -0.5, o, ws, lse=lse, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tw.twell_kv_attention(q, cache, *args, 7000, 1, 128 ** -0.5, o, ws, lse=lse)
    o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, want) and torch.equal(lse, want_lse)


# ---------------------------------------------------------------- log probabilities
def run_logprobs(tw, x, targets, inv_t, k):
    import torch
    n = x.shape[0]
    f = lambda *s: torch.full(s, 7.0, device="cuda")  # noqa: E731
    lp, en, lse = f(n), f(n), f(n)
    top = (f(n, k), torch.full((n, k), 7, dtype=torch.int32, device="cuda")) if k else (None, None)
    tw.twell_logprobs(x, targets, inv_t, lp, en, lse, *top)
    return [lp, en, lse, *top]


def special_rows(r, n, vocab):
    """Logits with ties, masks, a row of one live token, an empty one, and rows with NaN and +inf."""
    x = r.randn(n, vocab) * 3
    x[0] = np.round(x[0])                      # ties everywhere
    if n > 1:
        x[1] = -np.inf
    if n > 2:
        x[2] = -np.inf
        x[2, vocab // 2] = -3.0
    if n > 3:
        x[3, vocab // 3] = np.nan
    if n > 4:
        x[4, vocab - 1] = np.inf
    if n > 5:
        x[5] = 0.0                             # all equal
    if n > 6:
        x[6, r.rand(vocab) < 0.5] = -np.inf
    if n > 7:
        x[7] = np.where(np.arange(vocab) % 2 == 0, 0.0, -0.0)
    if n > 8:
        x[8] -= 1e30                           # far from zero, still a distribution
    return x


@pytest.mark.parametrize("n,vocab,dtype,ld,k,inv_t", [
    (10, 1, "float32", 1, 1, 1.0), (10, 7, "bfloat16", 7, 5, 0.7), (11, 333, "float32", 333, 32, 1.25),
    (11, 1000, "bfloat16", 1003, 20, 1.0), (9, 4099, "float32", 5001, 20, 0.3), (3, 33333, "bfloat16", 33333, 32, 1.0),
    (12, 100003, "float32", 100003, 32, 1.0), (1, 131072, "float32", 131072, 20, 1.0),
    (700, 2048, "bfloat16", 2048, 1, 1.0), (320, 20001, "bfloat16", 20001, 0, 0.9), (2, 400000, "float32", 400000, 8, 1.0)])
def test_logprobs_match_definition(tw, n, vocab, dtype, ld, k, inv_t):
    """Bounds: an exponential is off by 2^-22 plus 2 units of its argument, whose
    size is at most 90 where it counts; sums of the vocabulary in fp32 partial
    sums of at most vocab / 256 + 40 terms; the entropy's terms are of size p |x - m|."""
    import torch
    r = np.random.RandomState(vocab % 1000)
    x = dev(special_rows(r, n, vocab)).to(getattr(torch, dtype))
    buf = torch.full((n, ld), float("nan"), dtype=x.dtype, device="cuda")
    buf[:, :vocab] = x
    x = buf[:, :vocab]
    targets = r.randint(-1, vocab + 1, n).astype(np.int32)   # -1 and vocab: no target
    got = [None if t is None else host(t) for t in run_logprobs(tw, x, dev(targets), inv_t, k)]
    # x * inv_t in fp32, as documented, then 64 bits
    xs = host(x.float() * torch.tensor(inv_t, dtype=torch.float32, device="cuda"))
    depth = vocab / 256 + 40
    for i in list(range(min(n, 12))) + list(range(12, n, 37)):
        lp, en, lse, top, index = ref.logprobs(xs[i], int(targets[i]), k)
        live = xs[i][np.isfinite(xs[i])]
        m = np.abs(live.max()) if live.size else 0.0
        tol = 2.0 ** -21 + 2 * depth * U32 + 4 * U32 * 90 + 6 * U32 * m
        spread = np.abs(en) if np.isfinite(en) else 0.0

        def near(a, b, t, what):
            if np.isnan(b):
                assert np.isnan(a), (i, what)
            elif np.isinf(b):
                assert a == b, (i, what)
            else:
                assert abs(a - b) <= t, (i, what, a, b, t)

        near(got[2][i], lse, tol + 2 * U32 * abs(lse), "lse")
        near(got[0][i], lp, tol + 2 * U32 * (abs(lp) if np.isfinite(lp) else 0), "logprob")
        near(got[1][i], en, (tol + 2 * U32) * (spread + 2) * 2, "entropy")
        if k:
            assert np.array_equal(got[4][i], index), i
            for j in range(k):
                near(got[3][i][j], top[j], tol + 2 * U32 * (abs(top[j]) if np.isfinite(top[j]) else 0), "top")


@pytest.mark.parametrize("n,vocab,dtype,ld,inv_t", [
    (2000, 333, "bfloat16", 335, 0.9), (1300, 4096, "float32", 4099, 1.0), (1217, 8192, "bfloat16", 8192, 1.0),
    (1300, 7, "float32", 7, 1.1), (400, 30011, "bfloat16", 30013, 1.3), (310, 33000, "float32", 33001, 1.0)])
def test_logprobs_of_many_rows_match_definition(tw, n, vocab, dtype, ld, inv_t):
    """Rows that are summed as they are read, by a warp or by a CTA."""
    test_logprobs_match_definition(tw, n, vocab, dtype, ld, 0, inv_t)


@pytest.mark.parametrize("n,vocab,dtype,ld,k", [
    (60, 500, "bfloat16", 503, 20), (60, 170, "bfloat16", 170, 20), (60, 140, "bfloat16", 141, 20),
    (60, 300, "float32", 301, 32), (60, 957, "bfloat16", 957, 20), (60, 40, "float32", 40, 32)])
def test_logprobs_alternatives_of_small_vocabularies(tw, n, vocab, dtype, ld, k):
    """About as many 16-byte pieces as alternatives: with and without a bound of the k largest."""
    test_logprobs_match_definition(tw, n, vocab, dtype, ld, k, 1.0)


@pytest.mark.parametrize("n,vocab", [(3, 5000), (3, 100001), (400, 20000), (1300, 500)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("inv_t", [1.0, 3.0])
def test_logprobs_masked_by_the_lowest_value(tw, n, vocab, dtype, inv_t):
    """Tokens masked by their type's lowest value weigh nothing in sums and gradient, though their
    product with the inverse temperature may be no number's; rows that are all so masked are uniform."""
    import torch
    r = np.random.RandomState(vocab)
    t = getattr(torch, dtype)
    x = dev(r.randn(n, vocab) * 2).to(t)
    masked = dev(r.rand(n, vocab)) < 0.3
    masked[1] = True
    masked[1, 3] = masked[0, 0] = False
    x[masked] = torch.finfo(t).min
    targets = np.full(n, 3, np.int32)
    targets[0] = 0
    lp, en, lse, *_ = [None if v is None else host(v) for v in run_logprobs(tw, x, dev(targets), inv_t, 0)]
    live = x.masked_fill(masked, float("-inf"))
    xs = host(live.float() * torch.tensor(inv_t, dtype=torch.float32, device="cuda"))
    d = torch.empty_like(x)
    ones = torch.ones(n, device="cuda")
    tw.twell_logprobs_bwd(x, dev(targets), inv_t, dev(lse.astype(np.float32)), dev(en.astype(np.float32)), ones, ones, d)
    assert (d[masked & (torch.arange(vocab, device="cuda") != dev(targets)[:, None])] == 0).all()
    assert torch.isfinite(d).all()
    tol = 2.0 ** -21 + 2 * (vocab / 256 + 40) * U32 + 4 * U32 * 90 + 6 * U32 * 10 * inv_t
    for i in list(range(3)) + list(range(3, n, 97)):
        want_lp, want_en, want_lse, *_ = ref.logprobs(xs[i], int(targets[i]), 0)
        assert abs(lse[i] - want_lse) <= tol + 2 * U32 * abs(want_lse), i
        assert abs(en[i] - want_en) <= (tol + 2 * U32) * (want_en + 2) * 2, i
        if np.isfinite(want_lp):
            assert abs(lp[i] - want_lp) <= tol + 2 * U32 * abs(want_lp), i


def test_logprobs_best_values_crowded_in_one_place(tw):
    """The largest values all in the columns of one thread, rising and falling
    rows: more candidates than the quick selection holds."""
    import torch
    vocab = 64 * 1024
    x = np.zeros((4, vocab), np.float32)
    j = np.arange(vocab)
    crowded = (j // 4) % 256 == 5
    x[0] = np.where(crowded, 5 + (j % 977) / 977.0, -1 + (j % 31) / 31.0)
    x[1], x[2] = j / vocab, -j / vocab
    x[3] = np.where(crowded, 3.0, 0.0)
    top, index = torch.empty((4, 32), device="cuda"), torch.empty((4, 32), dtype=torch.int32, device="cuda")
    lse = torch.empty(4, device="cuda")
    tw.twell_logprobs(dev(x), None, 1.0, None, None, lse, top, index)
    for i in range(4):
        _, _, want_lse, _, want = ref.logprobs(x[i].astype(np.float64), -1, 32)
        assert np.array_equal(host(index)[i], want)
        assert abs(host(lse)[i] - want_lse) < 1e-4


@pytest.mark.parametrize("n,vocab,dtype,ld,inv_t,both", [
    (10, 1, "float32", 1, 1.0, True), (10, 7, "bfloat16", 7, 0.7, True), (11, 333, "float32", 336, 1.25, False),
    (12, 8193, "float32", 8193, 1.0, True), (9, 20001, "bfloat16", 20003, 1.0, True),
    (700, 1024, "bfloat16", 1024, 2.0, False)])
def test_logprobs_gradient_matches_formula(tw, n, vocab, dtype, ld, inv_t, both):
    """p is off by 2^-21 plus 2 units of its argument (up to 90, or of lse where
    that is larger); the result is rounded once to its type."""
    import torch
    r = np.random.RandomState(vocab % 97)
    rows = special_rows(r, n, vocab)
    if n > 8:
        rows[8] = r.randn(vocab)
    x = torch.full((n, ld), 3.0, device="cuda").to(getattr(torch, dtype))
    x[:, :vocab] = dev(rows).to(x.dtype)
    view = x[:, :vocab]
    targets = r.randint(-1, vocab + 1, n).astype(np.int32)
    t = dev(targets)
    lse, entropy = run_logprobs(tw, view, t, inv_t, 0)[2:0:-1]
    g, gh = r.randn(n).astype(np.float32), r.randn(n).astype(np.float32)
    out = torch.full((n, ld + 5), 9.0, device="cuda").to(x.dtype)[:, :vocab]
    args = (view, t, inv_t, lse, entropy if both else None, dev(g), dev(gh) if both else None)
    tw.twell_logprobs_bwd(*args, out)
    xs = host(view.float() * torch.tensor(inv_t, dtype=torch.float32, device="cuda"))
    got = host(out)
    ulp = UBF if dtype == "bfloat16" else U32
    for i in range(n):
        if np.isnan(xs[i]).any() or (xs[i] == np.inf).any():
            assert np.isnan(got[i]).all(), i
            continue
        if (xs[i] == -np.inf).all():
            assert (got[i] == 0).all(), i
            continue
        _, en, want_lse, _, _ = ref.logprobs(xs[i], -1, 0)
        logp = xs[i] - want_lse
        p = np.exp(logp)
        has = 0 <= targets[i] < vocab
        w = -float(gh[i]) * (np.where(p > 0, logp, 0) + en) if both else np.zeros(vocab)
        want = p * w - (p * g[i] if has else 0)
        size = p * (np.abs(w) + abs(float(gh[i])) * (np.abs(np.where(p > 0, logp, 0)) + en + 1) * both + abs(g[i]))
        if has:
            want[targets[i]] += g[i]
        want, size = want * inv_t, size * inv_t
        rel = 2.0 ** -20 + (vocab / 256 + 40) * 2 * U32 + 8 * U32 * (90 + np.abs(want_lse))
        tol = rel * size + 2 * U32 * np.abs(want) + ulp * np.abs(want) * (1 + 2 * rel) + 1e-37
        assert (np.abs(got[i] - want) <= tol + ulp * rel * size).all(), (i, (np.abs(got[i] - want) / tol).max())
    # in place: the logits' buffer receives the gradient, what lies between the rows stays
    tw.twell_logprobs_bwd(*args, view)
    assert torch.equal(view.nan_to_num(5.0), out.nan_to_num(5.0))
    if ld > vocab:
        assert (x[:, vocab:] == 3.0).all()


@pytest.mark.parametrize("n,vocab,dtype,ld,inv_t", [
    (2500, 333, "bfloat16", 335, 0.9), (2432, 1024, "float32", 1025, 1.0), (3000, 7, "float32", 7, 1.1)])
def test_logprobs_gradient_of_many_short_rows(tw, n, vocab, dtype, ld, inv_t):
    test_logprobs_gradient_matches_formula(tw, n, vocab, dtype, ld, inv_t, True)


def test_logprobs_gradient_matches_differences(tw):
    """Central differences in 64 bits of g logprob + gh entropy: step 1e-5, so
    their own error is near 1e-10 of the third derivative and 1e-11 of rounding."""
    import torch
    r = np.random.RandomState(8)
    vocab, inv_t, step = 23, 0.8, 1e-5
    x = r.randn(3, vocab).astype(np.float32)
    targets = np.array([4, -1, 22], np.int32)
    g, gh = np.array([1.5, 2.0, -0.7], np.float32), np.array([0.3, -1.0, 0.9], np.float32)
    out = run_logprobs(tw, dev(x), dev(targets), inv_t, 0)
    d = torch.empty((3, vocab), device="cuda")
    tw.twell_logprobs_bwd(dev(x), dev(targets), inv_t, out[2], out[1], dev(g), dev(gh), d)

    def loss(row, i):
        lp, en, *_ = ref.logprobs(row * inv_t, int(targets[i]), 0)
        return float(g[i]) * lp + float(gh[i]) * en

    for i in range(3):
        for j in range(vocab):
            e = np.zeros(vocab)
            e[j] = step
            row = x[i].astype(np.float64)
            diff = (loss(row + e, i) - loss(row - e, i)) / (2 * step)
            assert abs(host(d)[i, j] - diff) <= 5e-6 * (1 + abs(diff)), (i, j)
