"""The linear log probabilities and their gradient within what their arithmetic leaves (tests/linear_precision.py has the
bounds and their derivation, tests/test_linear_precision_bounds.py shows what they tell apart): logits added
up in runs, the same ones in the gradient as in the sums, whatever the shape."""
import linear_precision as lp
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def tw():
    import activation_sparse_transformer_gb300 as m
    m.load_library()
    return m


def forward(tw, h, w, t, inv_t=1.0):
    n = h.shape[0]
    out = [torch.full((n,), float("nan"), device="cuda") for _ in range(3)]
    ws = torch.empty(tw.linear_logprobs_workspace_bytes(n, h.shape[1], w.shape[0]), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tw.twell_linear_logprobs(h, w, t, inv_t, *out, ws, st)
    assert int(st) == 0
    return out


def backward(tw, h, w, t, lse, g, inv_t=1.0):
    (n, d), v = h.shape, w.shape[0]
    dh, dw = torch.empty((n, d), dtype=torch.bfloat16, device="cuda"), torch.empty((v, d), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(tw.linear_logprobs_bwd_workspace_bytes(n, d, v), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tw.twell_linear_logprobs_bwd(h, w, t, inv_t, lse, None, g, None, dh, dw, ws, st)
    assert int(st) == 0
    return dh, dw


# tiles of a CTA and of a pair, all of K in one launch (many tiles) and in ranges
@pytest.mark.parametrize("n,v", [(5, 20000), (5, 300), (131, 10000), (131, 300)])
@pytest.mark.parametrize("d", [4096, 4056, 1000])
def test_logits_are_added_up_in_runs(tw, n, v, d):
    """Products of one sign: a sum that loses a step in 16 products over all of d is off by twice the bound."""
    g = torch.Generator().manual_seed(n + v + d)
    h = torch.rand((n, d), generator=g).bfloat16().cuda()
    w = (torch.rand((v, d), generator=g) * 0.05).bfloat16().cuda()
    t = torch.randint(v, (n,), generator=g).to(torch.int32).cuda()
    logprob, entropy, lse = (o.double() for o in forward(tw, h, w, t))
    h, w = h.double(), w.double()
    x = h @ w.T
    off = lp.logit_error(h, w).amax(1)
    want = torch.logsumexp(x, 1)
    rest = 2.0 ** -18 + 2 * U * want.abs()
    assert ((lse - want).abs() <= off + rest).all(), f"{float(((lse - want).abs() / (off + rest)).max()):.2f} of the bound"
    own = x[torch.arange(n), t.long()] - want
    assert ((logprob - own).abs() <= 2 * off + rest).all()
    p = torch.exp(x - want[:, None])
    assert ((entropy + (p * (x - want[:, None])).sum(1)).abs() <= 2 * off * (1 + want.abs()) + 2.0 ** -16).all()


SHAPES = [(40, 4096, 5000), (40, 4096, 50001), (300, 4096, 3000), (300, 2048, 20001), (2100, 1024, 40000)]


@pytest.mark.parametrize("n,d,v", SHAPES)
@pytest.mark.parametrize("size,mass", [(20.0, 1e-3), (20.0, 1e-4), (60.0, 1e-4), (100.0, 1e-2)])
def test_gradient_of_certain_rows(tw, n, d, v, size, mass):
    """Where p is nearly 1 the gradient is what is left of 1 - p: the logits' own error must not be in it."""
    h, w, t = (m.cuda() for m in lp.saturated(n, d, v, size, mass, n + d + v))
    g = torch.randn(n, generator=torch.Generator().manual_seed(4)).cuda()
    dh, dw = backward(tw, h, w, t, forward(tw, h, w, t)[2], g)
    h, w = h.double(), w.double()
    G, off, _, _ = lp.gradient(h, w, t, 1.0, g.double())
    lp.check(dh, G, off, w, "d_hidden")
    lp.check(dw, G.T, off.T, h, "d_weight")


@pytest.mark.parametrize("n,d,v", SHAPES)
def test_rows_of_the_gradient_add_up_to_nothing(tw, n, d, v):
    """A column of ones in W that H does not see makes a column of dH the sum of G over the vocabulary, 0 in exact
    arithmetic: G's roundings to bf16 leave 2^-8 of its magnitudes, and fp32 what lp.gradient says."""
    h, w, t = lp.saturated(n, d, v, 40.0, 1e-4, n + v)
    h[:, 7], w[:, 7] = 0.0, 1.0
    h, w, t = h.cuda(), w.cuda(), t.cuda()
    g = torch.randn(n, generator=torch.Generator().manual_seed(8)).cuda()
    dh, _ = backward(tw, h, w, t, forward(tw, h, w, t)[2], g)
    G, off, _, _ = lp.gradient(h.double(), w.double(), t, 1.0, g.double())
    assert (dh[:, 7].double().abs() <= 2.0 ** -8 * G.abs().sum(1) * 1.01 + off.sum(1) + v / 16 * lp.CUT * G.abs().sum(1)).all()


@pytest.mark.parametrize("n,d,v", [(10, 3640, 500), (129, 4096, 300), (300, 4096, 1001), (413, 1032, 50001), (1500, 512, 33000)])
def test_gradient_within_its_roundings(tw, n, d, v):
    gen = torch.Generator().manual_seed(n + d + v)
    w = torch.randn((v, d), generator=gen) * (2.5 / d ** 0.5)
    h = torch.randn((n, d), generator=gen)
    t = torch.randint(v, (n,), generator=gen)
    h += 4.0 * torch.rand((n, 1), generator=gen) * w[t] / 2.5 ** 2
    t[::9] = -1
    h, w, t = h.bfloat16().cuda(), w.bfloat16().cuda(), t.to(torch.int32).cuda()
    g = torch.randn(n, generator=gen).cuda()
    dh, dw = backward(tw, h, w, t, forward(tw, h, w, t, 1.3)[2], g, 1.3)
    h, w = h.double(), w.double()
    G, off, _, _ = lp.gradient(h, w, t, 1.3, g.double())
    lp.check(dh, G, off, w, "d_hidden")
    lp.check(dw, G.T, off.T, h, "d_weight")
