"""Log probabilities from hidden rows where one token holds nearly all of the mass, where logits stand far from
zero, and where they stand at the ends of fp32: what a row's sums say is free of the size of its logits.

Logits here are exact.  H [top | offsets], W [ones | unit vectors] makes x_j = top + offset_j, which
needs fewer than 24 bits, so no sum of products loses any.

Error bounds (u = 2^-24): the largest entry's exponential is exactly 1.  The others' exponents, |y| = 32 1.25 log2(e)
at most, are off by 3 u of themselves (log2(e) / T is rounded twice, the product once), so e_j by 120 u + 2^-22 <
2^-17 of itself.  S = 1 + sum e_j: in the accumulator that holds the 1 (a thread's: up to 31 further entries) an
addition loses at most min(e_j, u), and at most 12 additions join it with the others, u each.  So log S is off by the
sum of min(e_j, u) over the 31 largest + 12 u + 2^-17 sum e_j.  S is never below 1, so no log probability is above 0.
lse is rounded once more, by u |lse|, after the product inv_temperature * top in an fma."""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
V = 500


@pytest.fixture(scope="module")
def tw():
    import activation_sparse_transformer_gb300 as m
    m.load_library()
    return m


def forward(tw, h, w, t, inv_t):
    n = h.shape[0]
    out = [torch.full((n,), float("nan"), device="cuda") for _ in range(3)]
    ws = torch.full((tw.linear_logprobs_workspace_bytes(n, h.shape[1], w.shape[0]),), 0xFF, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tw.twell_linear_logprobs(h, w, t, inv_t, *out, ws, st)
    assert int(st) == 0
    return out


def exact_logits(n, d, size, mass, inv_t, seed):
    """(H, W, targets, offsets in 64 bits): the others of a row share about `mass`, the target is the largest."""
    g = torch.Generator().manual_seed(seed)
    # bf16 values between size and 2 size; multiples of 1/32 for the offsets
    top = (size * (1 + torch.rand(n, generator=g))).bfloat16().float()
    gap = torch.log(torch.tensor(V / mass)) / inv_t
    off = -(gap + torch.rand((n, V), generator=g)).clamp(max=31.9)
    off = (off * 8).round().div(8).bfloat16().float()
    t = torch.randint(V, (n,), generator=g)
    off[torch.arange(n), t] = 0.0
    h, w = torch.zeros((n, d)), torch.zeros((V, d))
    h[:, 0], w[:, 0] = top, 1.0
    h[:, 8:8 + V], w[:, 8:8 + V] = off, torch.eye(V)
    return h.bfloat16().cuda(), w.bfloat16().cuda(), t.to(torch.int32).cuda(), top.double().cuda(), off.double().cuda()


# tiles of a CTA and of a pair; d = 512: all of K at once, 2048: in ranges
@pytest.mark.parametrize("n,d", [(40, 512), (300, 512), (40, 2048), (300, 2048)])
@pytest.mark.parametrize("inv_t", [1.0, 1.25])
@pytest.mark.parametrize("size", [10.0, 20.0, 200.0, 10000.0, -200.0])
def test_tokens_that_a_row_is_certain_of(tw, n, d, inv_t, size):
    for k, mass in enumerate((1e-2, 1e-4, 1e-6, 1e-9)):
        h, w, t, top, off = exact_logits(n, d, size, mass, inv_t, 10 * n + k)
        lp, ent, lse = (o.double() for o in forward(tw, h, w, t, inv_t))
        e = torch.exp(inv_t * off)
        e[torch.arange(n), t.long()] = 0.0
        rest = e.sum(1)
        want = -torch.log1p(rest)
        bound = e.topk(31, 1).values.clamp(max=U).sum(1) + 12 * U + 2.0 ** -17 * rest
        assert (lp <= 0).all(), f"{int((lp > 0).sum())} of {n} log probabilities above 0"
        assert ((lp - want).abs() <= bound).all(), f"{mass}: off by {float((lp - want).abs().max()):.2e}"
        assert ((lse - (inv_t * top - want)).abs() <= bound + U * lse.abs()).all()
        # log S and sum e_j |x_j| / S, |x_j| <= 40: its terms are off by 2^-17 as e_j is, and by 3 u more
        entropy = (e * -inv_t * off).sum(1) / (1 + rest) - want
        assert (ent >= 0).all() and ((ent - entropy).abs() <= 2 * bound + 2.0 ** -16 * entropy).all()
        # the same of logits in memory
        logits = (top[:, None] + off).float().contiguous()
        assert torch.equal(logits.double(), top[:, None] + off)
        other = [torch.empty(n, device="cuda") for _ in range(3)]
        tw.twell_logprobs(logits, t, inv_t, *other)
        # whose largest exponential is 2^r, r what rounding left of the maximum: off by 2^-22, as its logarithm is
        assert ((lp - other[0].double()).abs() <= 2 * bound + 2.0 ** -20).all()


@pytest.mark.parametrize("n,d", [(5, 64), (200, 64), (5, 2048), (200, 2048)])
@pytest.mark.parametrize("top", [-3.3e38, -2.5e38, 2.5e38, 3.3e38])
def test_logits_at_the_ends_of_fp32(tw, n, d, top):
    """Finite logits whose products with log2(e) are not: rows masked throughout by their type's lowest value are
    uniform, a token at the highest one has everything."""
    h = torch.zeros((n, d), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((300, d), dtype=torch.bfloat16, device="cuda")
    h[:, 0], w[:, 0] = 1.0, top
    t = torch.arange(n, dtype=torch.int32, device="cuda")
    x = float(w[0, 0])
    lp, ent, lse = forward(tw, h, w, t, 1.0)
    log_v = float(torch.log(torch.tensor(300.0, dtype=torch.float64)))
    assert ((lse.double() - x).abs() <= U * abs(x)).all()
    assert ((lp.double() + log_v).abs() <= 2.0 ** -20 * log_v).all()
    assert ((ent.double() - log_v).abs() <= 2.0 ** -20 * log_v).all()
    # token 7 in the middle, all others at the end
    w[7] = 0
    lp, ent, lse = forward(tw, h, w, t, 1.0)
    few = [i for i in range(n) if i != 7]
    if top < 0:
        assert lse.tolist() == [0.0] * n and ent.tolist() == [0.0] * n
        assert ((lp[few].double() - x).abs() <= U * abs(x)).all()
        assert n <= 7 or float(lp[7]) == 0.0
    else:
        log_v = float(torch.log(torch.tensor(299.0, dtype=torch.float64)))
        assert ((lp[few].double() + log_v).abs() <= 2.0 ** -20 * log_v).all()
        assert n <= 7 or abs(float(lp[7].double()) + x) <= U * x
    # beyond the ends: -inf only, or no number
    lp, ent, lse = forward(tw, h, w[8:].contiguous(), t, 2.0)
    if top < 0:
        inf = float("inf")
        assert lse.tolist() == [-inf] * n and ent.tolist() == [0.0] * n and lp.tolist() == [-inf] * n
    else:
        assert lse.isnan().all() and ent.isnan().all() and lp.isnan().all()


def test_masked_tokens_beside_others(tw):
    """Tokens at the lowest value of bf16 among ordinary ones, in tiles of their own too, take no part."""
    n, d, v = 20, 64, 1500
    g = torch.Generator().manual_seed(3)
    h, w = torch.randn((n, d), generator=g), torch.randn((v, d), generator=g) / 4
    h[:, 0], w[:, 0] = 1.0, 0.0
    keep = torch.rand(v, generator=g) < 0.3
    keep[256:768] = False
    w[~keep] = 0.0
    w[~keep, 0] = torch.finfo(torch.bfloat16).min
    h, w = h.bfloat16().cuda(), w.bfloat16().cuda()
    ids = torch.nonzero(keep)[:, 0].cuda()
    t = ids[torch.randint(len(ids), (n,), generator=g).cuda()].to(torch.int32)
    lp, ent, lse = (o.double() for o in forward(tw, h, w, t, 1.0))
    x = h.double() @ w.double()[ids].T
    logp = torch.log_softmax(x, 1)
    # products of 64 terms of size 1 and S of some 450
    off = 64 * 2.0 ** -23 * (h.double().abs() @ w.double()[ids].abs().T).max() + 2.0 ** -18
    assert ((lse - torch.logsumexp(x, 1)).abs() <= off).all()
    own = logp.gather(1, (ids[None, :] == t[:, None]).long().argmax(1, keepdim=True))[:, 0]
    assert ((lp - own).abs() <= 2 * off).all()
    assert ((ent + (logp.exp() * logp).sum(1)).abs() <= 16 * off).all()
