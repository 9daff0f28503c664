"""The gradient of rows whose lse fp32 tells too coarsely for any p: they give zeros, as rows of -inf do, and the other rows
are as they were."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tw():
    import activation_sparse_transformer_gb300 as m
    m.load_library()
    return m


# one run and several, a CTA's tiles and a pair's, ranges of K, pieces of the vocabulary
@pytest.mark.parametrize("n,d,v", [(40, 64, 1000), (40, 640, 30000), (300, 64, 1000), (300, 640, 20001), (40, 2048, 500), (17000, 64, 8300)])
@pytest.mark.parametrize("size", [-3.3e38, 3.3e38, -2.0e7, 2.0e7])
def test_rows_far_from_zero(tw, n, d, v, size):
    g = torch.Generator().manual_seed(n + d + v)
    h, w = torch.randn((n, d), generator=g), torch.randn((v, d), generator=g) / d ** 0.5
    far = torch.arange(n) % 9 == 4
    h[:, 0] = torch.where(far, size, 0.0)
    h[far, 1:] = 0.0  # every token has the same logit
    w[:, 0] = 1.0
    h, w, far = h.bfloat16().cuda(), w.bfloat16().cuda(), far.cuda()
    t = torch.randint(v, (n,), generator=g).to(torch.int32).cuda()
    up, ge = torch.randn(n, generator=g).cuda(), torch.randn(n, generator=g).cuda()
    lp, ent, lse = (torch.empty(n, device="cuda") for _ in range(3))
    ws = torch.empty(max(tw.linear_logprobs_workspace_bytes(n, d, v), tw.linear_logprobs_bwd_workspace_bytes(n, d, v)),
                     dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tw.twell_linear_logprobs(h, w, t, 1.0, lp, ent, lse, ws, st)
    log_v = float(torch.log(torch.tensor(float(v), dtype=torch.float64)))
    assert ((lse[far].double() - (h[far, 0].double() + log_v)).abs() <= 2.0 ** -23 * abs(size)).all()
    assert ((lp[far].double() + log_v).abs() <= 2.0 ** -19 * log_v).all()

    def backward(lse, h):
        dh, dw = torch.full_like(h, float("nan")), torch.full_like(w, float("nan"))
        tw.twell_linear_logprobs_bwd(h, w, t, 1.0, lse, ent, up, ge, dh, dw, ws, st)
        assert int(st) == 0
        return dh, dw

    dh, dw = backward(lse, h)
    assert not dh[far].any() and dh[~far].any(1).all()
    # as if those rows had nothing at all
    none = torch.where(far[:, None], 0.0, h.float()).bfloat16()
    want = backward(torch.where(far, float("-inf"), lse), none)
    assert torch.equal(dh, want[0]) and torch.equal(dw, want[1])
