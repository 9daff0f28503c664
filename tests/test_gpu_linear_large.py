"""Log probabilities from hidden rows where tokens x vocabulary are too many for a matrix of them (18 GB of bf16 logits and
as much for their gradient), checked on some rows and some tokens in 64 bits."""
import linear_precision as lp
import pytest
import torch

pytestmark = pytest.mark.gpu

N, D, V = 70001, 520, 131075


@pytest.fixture(scope="module")
def tw():
    import activation_sparse_transformer_gb300 as m
    m.load_library()
    return m


@pytest.fixture(scope="module")
def done(tw):
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("24 GB beside what others hold")
    g = torch.Generator(device="cuda").manual_seed(1)
    w = (torch.randn((V, D), generator=g, device="cuda") * (2.5 / D ** 0.5)).bfloat16()
    t = torch.randint(V, (N,), generator=g, device="cuda").to(torch.int32)
    h = torch.randn((N, D), generator=g, device="cuda")
    h += 1.5 * torch.rand((N, 1), generator=g, device="cuda") * w[t.long()].float()
    h = h.bfloat16()
    t[::11] = -1
    up = torch.randn(N, generator=g, device="cuda")
    lps, ent, lse = (torch.empty(N, device="cuda") for _ in range(3))
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    need = tw.linear_logprobs_bwd_workspace_bytes(N, D, V)
    assert need < 2 << 30  # less than a tenth of the logits
    ws = torch.empty(max(need, tw.linear_logprobs_workspace_bytes(N, D, V)), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tw.twell_linear_logprobs(h, w, t, 1.0, lps, ent, lse, ws, st)
    tw.twell_linear_logprobs_bwd(h, w, t, 1.0, lse, None, up, None, dh, dw, ws, st)
    assert int(st) == 0
    return dict(h=h, w=w, t=t, up=up, logprob=lps, entropy=ent, lse=lse, dh=dh, dw=dw, ws=ws, st=st)


ROWS = [0, 1, 127, 255, 256, 4095, 34999, 65535, 65536, 69888, 70000] + list(range(11, 70001, 3500))


def test_rows(done):
    r = torch.tensor(ROWS, device="cuda")
    h, w, t, g = done["h"][r].double(), done["w"].double(), done["t"][r], done["up"][r].double()
    G, off, x, lse = lp.gradient(h, w, t, 1.0, g)
    e = lp.logit_bound(h, w)
    rest = 2.0 ** -18 + 2.0 ** -23 * lse.abs()
    assert ((done["lse"][r].double() - lse).abs() <= e + rest).all()
    logp = x - lse[:, None]
    own = torch.where(t >= 0, logp.gather(1, t.clamp(min=0).long()[:, None])[:, 0], 0.0)
    assert ((done["logprob"][r].double() - own).abs() <= 2 * e + rest).all()
    entropy = -(logp.exp() * logp).sum(1)
    assert ((done["entropy"][r].double() - entropy).abs() <= 2 * e * (1 + lse.abs()) + 2.0 ** -15).all()
    lp.check(done["dh"][r], G, off, w, "d_hidden")


def test_tokens(done):
    cols = torch.tensor([0, 5, 255, 256, 4095, 4096, 65535, 65536, 131071, 131072, 131074] + list(range(3, V, 9001)),
                        device="cuda")
    h, w, t = done["h"].double(), done["w"].double()[cols], done["t"]
    lse, g = done["lse"].double(), torch.where(t >= 0, done["up"].double(), 0.0)
    x = h @ w.T
    p = torch.exp(x - lse[:, None])
    G = -g[:, None] * p + torch.where(t[:, None] == cols[None, :], g[:, None], 0.0)
    # of this lse: the logits' own error does not cancel
    e = (h.abs() @ w.abs().T) * (lp.RUN / 16 * lp.CUT + 2 * lp.CUT)
    off = g.abs()[:, None] * p * (e + 2.0 ** -18 + 2.0 ** -23 * lse.abs()[:, None])
    lp.check(done["dw"][cols], G.T, off.T, h, "d_weight")


@pytest.mark.parametrize("want", ["hidden", "weight"])
def test_one_of_the_gradients(tw, done, want):
    """Pieces of the vocabulary with only one product each give the same bits."""
    dh = torch.empty_like(done["dh"]) if want == "hidden" else None
    dw = torch.empty_like(done["dw"]) if want == "weight" else None
    tw.twell_linear_logprobs_bwd(done["h"], done["w"], done["t"], 1.0, done["lse"], None, done["up"], None, dh, dw,
                                 done["ws"], done["st"])
    assert int(done["st"]) == 0
    for got, before in ((dh, done["dh"]), (dw, done["dw"])):
        assert got is None or torch.equal(got, before)
