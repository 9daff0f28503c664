"""Bounds of the linear log probabilities and their gradient that follow what the kernels do, for tests that are
to notice a per mille.

A logit: the tensor cores add 16 products and what is there already and cut off what does not fit, one step of
2^-23 of the result at most; runs of 512 products are added in registers, each to 2^-24.  logit_error adds that up from
the partial sums themselves, logit_bound from the magnitudes alone.

lse comes from the same logits as the gradient's p, bit for bit.  So where one token has nearly all of the mass the
logits' errors e cancel in what is left beside it: p_j = exp(x_j - lse) is off by p_j (1 - p_j) 2 e, by
sums and exponentials (31 + 20 additions of 2^-24 and an exponential's 2^-22: 2^-18 of it) and by lse's own bits
(2^-24 |lse|, and as much again for the fma of x - lse)."""
import torch

CUT = 2.0 ** -23
RUN = 512  # products


def logit_error(h, w):
    """Error of the unscaled logits h w^T (64-bit h [n, d], w [v, d]) by their partial sums: [n, v]."""
    n, d = h.shape
    off = torch.zeros((n, w.shape[0]), dtype=torch.float64, device=h.device)
    total = torch.zeros_like(off)
    for run in range(0, d, RUN):
        part = torch.zeros_like(off)
        for k in range(run, min(run + RUN, d), 16):
            part = part + h[:, k:k + 16] @ w[:, k:k + 16].T
            off += CUT * part.abs()
        total = total + part
        off += CUT / 2 * total.abs()
    return off


def logit_bound(h, w):
    """The same of each row at most, from the magnitudes of the products: [n]."""
    size = (h.abs() @ w.abs().T).amax(1)
    runs = -(-h.shape[1] // RUN)
    return size * (min(RUN, h.shape[1]) / 16 * CUT + runs * CUT / 2)


def gradient(h, w, t, inv_t, g, rounded=False):
    """(G, its error without the rounding to bf16, x, lse), all in 64 bits, of the gradient of sum g logprob with
    respect to the unscaled logits; rounded: G as the nearest bf16 values."""
    x = inv_t * (h @ w.T)
    lse = torch.logsumexp(x, 1)
    p = torch.exp(x - lse[:, None])
    g = torch.where((t >= 0) & (t < w.shape[0]), g, 0.0)
    rows = torch.arange(len(h), device=h.device)
    at = torch.where(g != 0, t, 0).long()
    rest = 1 - p
    # 1 - p of a target from the others' mass
    others = p.clone()
    others[rows, at] = 0.0
    rest[rows, at] = others.sum(1)
    G = -g[:, None] * p
    G[rows, at] = g * rest[rows, at]
    e = inv_t * logit_bound(h, w)[:, None]
    off = inv_t * g.abs()[:, None] * p * (2 * e * rest + 2.0 ** -18 + 2.0 ** -23 * lse.abs()[:, None])
    G = inv_t * G
    return (G.float().bfloat16().double() if rounded else G), off, x, lse


def check(got, G, off, B, name):
    """got (bf16) is G B: off by G's rounding to bf16 (2^-8 of it at most), by `off`, by what the tensor cores cut off
    (a step in 16 terms) and by its own rounding.  As a whole: 2^-8 / sqrt(3) is the root of the mean square of an error
    that is anything up to 2^-8, G's of each term and the result's are independent, and a quarter more is left for
    chance (thousands of results)."""
    want = G @ B
    got = got.double()
    assert torch.isfinite(got).all(), name
    sizes = G.abs() @ B.abs()
    rest = off @ B.abs() + (B.shape[0] // 16 + 1) * CUT * sizes
    bound = 2.0 ** -8 * (sizes + want.abs()) * (1 + 2.0 ** -8) + rest
    over = (got - want).abs() - bound
    assert (over <= 0).all(), f"{name}: {float(over.max()):.3e} past its bound at {int(over.argmax())}"
    mean = 1.25 * 2.0 ** -8 / 3 ** 0.5 * ((G ** 2 @ B ** 2).sum() + (want ** 2).sum()).sqrt()
    # what is off in one direction: the bounds of fp32 themselves
    most = mean + rest.norm()
    norm = (got - want).norm()
    assert norm <= most, f"{name}: off by {float(norm):.3e} as a whole, bound {float(most):.3e} ({float(rest.norm()):.1e} of fp32)"


def saturated(n, d, v, size, mass, seed, pad=0):
    """(H, W, targets): in row i the target's logit is about `size`, added up evenly over all of d, and all other tokens
    together have about `mass`.  W's rows share a direction of signs, along which H's rows give every token the level
    that this takes; what a row of W has beside it lifts its own token."""
    gen = torch.Generator().manual_seed(seed)
    level = size + float(torch.log(torch.tensor(mass / v))) - 0.5  # the others' logits: level + normal
    t = torch.randperm(v, generator=gen)[:n] if n <= v else torch.randint(v, (n,), generator=gen)
    sign = torch.where(torch.rand(d, generator=gen) < 0.5, -1.0, 1.0)
    own = torch.randn((v, d), generator=gen) / d ** 0.5
    own -= (own @ sign)[:, None] * sign / d
    h, w = torch.zeros((n, d + pad)), torch.zeros((v, d + pad))
    w[:, :d] = own + sign * (level / d)
    noise = torch.randn((n, d), generator=gen)
    h[:, :d] = sign + noise - (noise @ sign)[:, None] * sign / d
    lift = size - (h[:, :d] * w[t][:, :d]).sum(1)
    h[:, :d] += own[t] * (lift / (own[t] ** 2).sum(1))[:, None]
    return h.bfloat16(), w.bfloat16(), t.to(torch.int32)
