"""The bounds that tests/test_gpu_linear_precision.py goes by, on the CPU: results that are rounded as the kernels round
pass, and ones with a small mistake planted in the oracle do not."""
import linear_precision as lp
import pytest
import torch

CASES = {
    "few tokens, long rows": lambda: ordinary(10, 3640, 500),
    "a pair's tiles": lambda: ordinary(129, 4096, 300),
    "many tokens": lambda: ordinary(300, 1024, 1001),
    "certain at 20": lambda: lp.saturated(12, 4096, 2000, 20.0, 1e-3, 1),
    "certain at 20, all but 1e-4": lambda: lp.saturated(12, 4096, 2000, 20.0, 1e-4, 1),
    "certain at 60": lambda: lp.saturated(130, 2048, 1000, 60.0, 1e-3, 2),
}


def ordinary(n, d, v):
    g = torch.Generator().manual_seed(n + d + v)
    w = torch.randn((v, d), generator=g) * (2.5 / d ** 0.5)
    h = torch.randn((n, d), generator=g)
    t = torch.randint(v, (n,), generator=g)
    h += 4.0 * torch.rand((n, 1), generator=g) * w[t] / 2.5 ** 2
    return h.bfloat16(), w.bfloat16(), t.to(torch.int32)


def results(h, w, t, g, scale_x=1.0, scale_g=1.0):
    """dH and dW in bf16 of a G that is rounded to bf16, with a mistake."""
    G, _, x, lse = lp.gradient(h, w, t, 1.0, g)
    if scale_x != 1.0:
        p = torch.exp(scale_x * x - lse[:, None])
        G = -g[:, None] * p
        G[torch.arange(len(h)), t.long()] += g
    G = (scale_g * G).float().bfloat16().double()
    return (G @ w).float().bfloat16(), (G.T @ h).float().bfloat16()


@pytest.mark.parametrize("name", CASES)
def test_what_the_bounds_tell_apart(name):
    h, w, t = CASES[name]()
    h, w = h.double(), w.double()
    g = torch.randn(len(h), generator=torch.Generator().manual_seed(5), dtype=torch.float64)
    G, off, x, _ = lp.gradient(h, w, t, 1.0, g)

    def passes(dh, dw):
        found = []
        for got, A, o, B in ((dh, G, off, w), (dw, G.T, off.T, h)):
            try:
                lp.check(got, A, o, B, name)
                found.append(True)
            except AssertionError:
                found.append(False)
        return found

    assert passes(*results(h, w, t, g)) == [True, True]
    if "1e-4" not in name:  # of which fp32 itself leaves 4 % where a row has 1e-4
        assert passes(*results(h, w, t, g, scale_g=1.02)) == [False, False]
        assert passes(*results(h, w, t, g, scale_g=0.98)) == [False, False]
    assert passes(*results(h, w, t, g, scale_x=0.999)) == [False, False]
    if "certain" in name:  # what tensor memory cuts off of a sum over all of d
        assert passes(*results(h, w, t, g, scale_x=1 - 4e-6)) == [False, False]
    else:
        assert passes(*results(h, w, t, g, scale_x=1 - 1e-7)) == [True, True]


def test_the_bound_of_a_logit_tells_one_sum_from_runs():
    """Sums emulated as the tensor cores make them, 16 products at a time and cut off at 24 bits: in runs of 512 they stay
    within logit_error, over all of d they do not."""
    g = torch.Generator().manual_seed(6)
    h, w = torch.rand((4, 4096), generator=g).bfloat16().double(), torch.rand((64, 4096), generator=g).bfloat16().double()

    def cut(x):
        m, e = torch.frexp(x)
        return torch.ldexp(torch.trunc(m * 2 ** 24), e - 24)

    def product(run):
        total = torch.zeros((4, 64), dtype=torch.float64)
        for k0 in range(0, 4096, run):
            part = torch.zeros_like(total)
            for k in range(k0, k0 + run, 16):
                part = cut(part + h[:, k:k + 16] @ w[:, k:k + 16].T)
            total = (total + part).float().double()
        return total

    off = lp.logit_error(h, w)
    assert ((product(512) - h @ w.T).abs() <= off).all()
    assert not ((product(4096) - h @ w.T).abs() <= off).any()
