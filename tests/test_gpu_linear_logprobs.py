"""Log probabilities from hidden rows and output weights, and their gradient, against the 64-bit
definition.

Error bounds: the products are exact in fp32 and each of a logit's d additions is off by 2^-23 of
the magnitudes at most, so x is off by e = d 2^-23 sum |h w| / T.  Exponentials and sums of a row
(tiles of 32, joined) add less than 2^-20 of S, lse's own bits 2^-22 |lse|.  G is off by 2^-8 of
itself from its rounding to bf16 and by 2 e + 2^-20 + 2^-22 |lse| of its magnitudes; the gradients add
2^-23 a term, and 2^-8 of themselves."""
import pytest
import torch

import training_reference as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tw():
    import activation_sparse_transformer_gb300 as m
    m.load_library()
    return m


def make(n, d, v, seed, pad=0, hot=True):
    g = torch.Generator().manual_seed(seed)
    w = torch.randn((v, d + pad), generator=g) * (2.5 / d ** 0.5)
    h = torch.randn((n, d + pad), generator=g)
    t = torch.randint(v, (n,), generator=g)
    if hot:
        h += 4.0 * torch.rand((n, 1), generator=g) * w[t] / 2.5 ** 2
    t[::5] = -1
    t[1::7] = v + 3
    cut = lambda m: m.bfloat16().cuda()[:, :d]  # noqa: E731
    return cut(h), cut(w), t.to(torch.int32).cuda()


def forward(tw, h, w, t, inv_t, stream=None, status=None):
    n = h.shape[0]
    out = [torch.full((n,), float("nan"), device="cuda") for _ in range(3)]
    ws = torch.full((tw.linear_logprobs_workspace_bytes(n, h.shape[1], w.shape[0]),), 0xFF, dtype=torch.uint8,
                    device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda") if status is None else status
    tw.twell_linear_logprobs(h, w, t, inv_t, *out, ws, st, stream=stream)
    if status is None:
        assert int(st) == 0
    return out


def close(got, want, bound, what):
    got = got.double()
    assert torch.isfinite(got).all(), what
    over = (got - want).abs() - bound
    assert (over <= 0).all(), f"{what}: {float(over.max()):.3e} past its bound at {int(over.argmax())}"


def check_forward(tw, h, w, t, inv_t):
    lp, ent, lse = forward(tw, h, w, t, inv_t)
    x, size = ref.linear_logits(h.double(), w.double(), inv_t)
    want = ref.linear_logprobs(x, t)
    e = size.amax(1) * h.shape[1] * 2.0 ** -23
    row = e + 2.0 ** -20 + 2.0 ** -22 * want[2].abs()
    close(lse, want[2], row, "lse")
    close(lp, want[0], 2 * row, "logprob")
    close(ent, want[1], e * (1 + 2 * want[1]) + 2.0 ** -18 * (1 + want[1]), "entropy")
    assert (lp[(t < 0) | (t >= w.shape[0])] == 0).all()


SHAPES = [(1, 8, 1), (1, 64, 5), (2, 72, 40), (17, 256, 255), (128, 64, 256), (129, 1032, 257), (300, 520, 1000),
          (5, 4096, 5001), (257, 128, 3001), (1, 2048, 40000), (33, 2056, 777)]


@pytest.mark.parametrize("n,d,v", SHAPES)
@pytest.mark.parametrize("inv_t", [1.0, 1.7])
def test_forward(tw, n, d, v, inv_t):
    check_forward(tw, *make(n, d, v, n + d + v), inv_t)


@pytest.mark.parametrize("n,d,v", [(1000, 512, 20000), (700, 200, 50257), (4100, 1024, 8200)])
def test_forward_larger(tw, n, d, v):
    check_forward(tw, *make(n, d, v, 5), 1.0)


def test_forward_of_slices_and_some_outputs(tw):
    h, w, t = make(77, 136, 1111, 6, pad=24)
    assert h.stride(0) == 160
    check_forward(tw, h, w, t, 1.0)
    lp, ent, lse = forward(tw, h, w, t, 1.0)
    n = h.shape[0]
    ws = torch.empty(tw.linear_logprobs_workspace_bytes(n, 136, 1111), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for keep in ((None, None, lse), (None, ent, None), (lp, None, None)):
        out = [None if k is None else torch.empty_like(k) for k in keep]
        tw.twell_linear_logprobs(h, w, t if out[0] is not None else None, 1.0, *out, ws, st)
        for a, b in zip(out, keep):
            assert b is None or torch.equal(a, b)


def test_forward_agrees_with_the_logits_path(tw):
    """The same definition as twell_logprobs on bf16 logits of the same values (weights that pick out entries)."""
    n, v = 64, 512
    g = torch.Generator().manual_seed(7)
    logits = (3 * torch.randn((n, v), generator=g)).bfloat16().cuda()
    eye = torch.eye(v, dtype=torch.bfloat16, device="cuda")
    t = torch.randint(v, (n,), generator=g).to(torch.int32).cuda()
    mine = forward(tw, logits, eye, t, 1.25)
    other = [torch.empty(n, device="cuda") for _ in range(3)]
    tw.twell_logprobs(logits, t, 1.25, *other)
    for a, b in zip(mine, other):
        assert ((a - b).abs() <= 2.0 ** -20 * (1 + b.abs())).all()


def test_rows_with_nan_infinity_or_nothing(tw):
    h, w, t = make(40, 64, 700, 8)
    t = t.clamp(0, 699)
    clean = forward(tw, h, w, t, 1.0)
    h[3, 5], h[9, 0], h[20, 1] = float("nan"), float("inf"), float("-inf")
    got = forward(tw, h, w, t, 1.0)
    bad = [3, 9, 20]
    keep = [i for i in range(40) if i not in bad]
    for a, b in zip(got, clean):
        assert torch.equal(a[keep], b[keep])
        assert a[bad].isnan().all()
    # every logit -inf
    w2 = torch.zeros((300, 64), dtype=torch.bfloat16, device="cuda")
    w2[:, 0] = float("-inf")
    h2 = torch.ones((2, 64), dtype=torch.bfloat16, device="cuda")
    lp, ent, lse = forward(tw, h2, w2, torch.tensor([4, -1], dtype=torch.int32, device="cuda"), 1.0)
    assert lse.tolist() == [float("-inf")] * 2 and ent.tolist() == [0.0, 0.0] and lp.tolist() == [float("-inf"), 0.0]
    # some of them -inf, whole tiles among them
    w2[290] = 0
    lp, ent, lse = forward(tw, h2, w2, torch.tensor([290, 4], dtype=torch.int32, device="cuda"), 1.0)
    assert lse.tolist() == [0.0, 0.0] and ent.tolist() == [0.0, 0.0] and lp.tolist() == [0.0, float("-inf")]


def test_equal_and_very_unequal_logits(tw):
    n, d, v = 4, 64, 1000
    w = torch.zeros((v, d), dtype=torch.bfloat16, device="cuda")
    h = torch.ones((n, d), dtype=torch.bfloat16, device="cuda")
    t = torch.tensor([0, 999, 256, -1], dtype=torch.int32, device="cuda")
    lp, ent, lse = forward(tw, h, w, t, 1.0)
    want = torch.log(torch.tensor(float(v), dtype=torch.float64))
    for got in (lse, ent):
        assert ((got.double().cpu() - want).abs() <= 2.0 ** -20 * 8).all()
    w[700, 0] = 10000.0  # one token far above the others, another far below
    w[5, 0] = -10000.0
    lp, ent, lse = forward(tw, h, w, torch.tensor([700, 0, 5, -1], dtype=torch.int32, device="cuda"), 1.0)
    top = float(w[700, 0])
    # the largest entry's own y = fma(x, log2(e), -m) is what rounding m left, r with |r| <= 2^-24 |m| < 2^-10; S = 2^r
    # to 2^-22 and U = S r, so log2 S - U / S, 0 in exact arithmetic, is off by 1.5 2^-22 + 2^-23 |r| at most
    assert lse.tolist() == [top] * 4 and (ent.abs() <= 2.0 ** -20).all()
    assert lp.tolist() == [0.0, -top, float(w[5, 0]) - top, 0.0]


# ---------------------------------------------------------------- the gradient
def gradient_inputs(n, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(n, generator=g).cuda(), (0.3 * torch.randn(n, generator=g)).cuda()


def backward(tw, h, w, t, inv_t, lse, ent, g, ge, want_h=True, want_w=True, stream=None, pad=0):
    n, d, v = h.shape[0], h.shape[1], w.shape[0]

    def new(rows, on):
        m = torch.full((rows, d + pad), float("nan"), dtype=torch.bfloat16, device="cuda")
        return m[:, :d] if on else None

    dh, dw = new(n, want_h), new(v, want_w)
    ws = torch.full((tw.linear_logprobs_bwd_workspace_bytes(n, d, v),), 0xFF, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(stream=stream):
        tw.twell_linear_logprobs_bwd(h, w, t, inv_t, lse, ent, g, ge, dh, dw, ws, st, stream=stream)
    call()
    assert int(st) == 0
    return dh, dw, call


def check_backward(h, w, t, inv_t, lse, ent, g, ge, dh, dw):
    n, d, v = h.shape[0], h.shape[1], w.shape[0]
    up = lambda a: None if a is None else a.double()  # noqa: E731
    hd, wd = h.double(), w.double()
    x, size = ref.linear_logits(hd, wd, inv_t)
    e = size.amax(1, keepdim=True) * d * 2.0 ** -23
    none = torch.full((n,), -1, device="cuda")
    G, big = ref.linear_grad(x, none if t is None else t, inv_t, up(lse), up(ent), up(g), up(ge))
    fp32 = (2 * e + 2.0 ** -20 + 2.0 ** -22 * lse.double().abs()[:, None]) * big
    off = 2.0 ** -8 * G.abs() + fp32
    for got, A, B, terms, what in ((dh, (G, off, big, fp32), wd, v, "d_hidden"),
                                 (dw, (G.T, off.T, big.T, fp32.T), hd, n, "d_weight")):
        if got is None:
            continue
        want = A[0] @ B
        bound = A[1] @ B.abs() + terms * 2.0 ** -23 * (A[2] @ B.abs()) + 2.0 ** -8 * want.abs()
        close(got, want, bound + 1e-36, what)
        # as a whole: a result of one term is off by its two roundings to bf16, 2^-7 of itself; in a sum of many these
        # add like random numbers, so that the norm of all of them is within that too.  Beside it stands what fp32 leaves
        # where G's own terms cancel (a vocabulary of one token: p = 1, G = 0), the second part of G's bound
        assert (got.double() - want).norm() <= 2.0 ** -7 * want.norm() + (A[3] @ B.abs()).norm(), what


@pytest.mark.parametrize("n,d,v", SHAPES + [(400, 264, 2500), (70, 64, 12345)])
def test_backward(tw, n, d, v):
    h, w, t = make(n, d, v, n + d + v)
    _, ent, lse = forward(tw, h, w, t, 1.3)
    g, ge = gradient_inputs(n, 9)
    dh, dw, _ = backward(tw, h, w, t, 1.3, lse, ent, g, ge)
    check_backward(h, w, t, 1.3, lse, ent, g, ge, dh, dw)


@pytest.mark.parametrize("n,d,v", [(8200, 72, 9001), (17000, 64, 8300), (3000, 512, 30000)])
def test_backward_in_pieces(tw, n, d, v):
    h, w, t = make(n, d, v, 10)
    _, ent, lse = forward(tw, h, w, t, 1.0)
    g, ge = gradient_inputs(n, 11)
    dh, dw, _ = backward(tw, h, w, t, 1.0, lse, ent, g, ge)
    check_backward(h, w, t, 1.0, lse, ent, g, ge, dh, dw)


@pytest.mark.parametrize("want", [dict(), dict(want_h=False), dict(want_w=False), dict(pad=8)])
@pytest.mark.parametrize("n,d,v", [(1100, 264, 130), (2100, 72, 300), (1025, 520, 1000), (9080, 376, 232), (12000, 128, 1),
                                   (4097, 8, 257)])
def test_backward_of_many_rows_and_few_tokens(tw, n, d, v, want):
    """dW's product runs over the rows, cut into ranges where its tiles are few."""
    h, w, t = make(n, d, v, n + v)
    lp, ent, lse = forward(tw, h, w, t, 1.0)
    g, ge = gradient_inputs(n, 44)
    dh, dw, call = backward(tw, h, w, t, 1.0, lse, ent, g, ge, **want)
    check_backward(h, w, t, 1.0, lse, ent, g, ge, dh, dw)
    first = [m.clone() for m in (dh, dw) if m is not None]
    call()
    assert all(torch.equal(a, b) for a, b in zip(first, [m for m in (dh, dw) if m is not None]))


@pytest.mark.parametrize("given", ["logprob", "entropy", "hidden", "weight", "slices"])
def test_backward_of_some(tw, given):
    pad = 40 if given == "slices" else 0
    h, w, t = make(150, 328, 2049, 12, pad=pad)
    _, ent, lse = forward(tw, h, w, t, 1.0)
    g, ge = gradient_inputs(150, 13)
    if given == "logprob":
        ent = ge = None
    if given == "entropy":
        t = g = None
    dh, dw, _ = backward(tw, h, w, t, 1.0, lse, ent, g, ge, want_h=given != "weight", want_w=given != "hidden", pad=pad)
    check_backward(h, w, t, 1.0, lse, ent, g, ge, dh, dw)
    if pad:
        assert dh._base[:, 328:].isnan().all() and dw._base[:, 328:].isnan().all()


def test_rows_that_take_no_part(tw):
    """Without a target and without an entropy gradient a row's gradient is zero, and so is what it adds to the weights."""
    h, w, t = make(130, 64, 900, 14)
    _, ent, lse = forward(tw, h, w, t, 1.0)
    g, ge = gradient_inputs(130, 15)
    t[:], ge[:] = -1, 0
    t[7] = 3
    dh, dw, _ = backward(tw, h, w, t, 1.0, lse, ent, g, ge)
    assert not dh[:7].any() and not dh[8:].any() and dh[7].any()
    one = backward(tw, h[7:8].clone(), w, t[7:8].clone(), 1.0, lse[7:8].clone(), ent[7:8].clone(), g[7:8].clone(),
                   ge[7:8].clone())[1]
    assert torch.equal(dw, one)


def test_rows_of_minus_infinity_and_nan(tw):
    w = torch.zeros((300, 64), dtype=torch.bfloat16, device="cuda")
    w[:, 0] = -3e38
    h = torch.ones((3, 64), dtype=torch.bfloat16, device="cuda")
    h[0, 0] = 100.0  # every logit -inf
    t = torch.tensor([1, 2, 3], dtype=torch.int32, device="cuda")
    lp, ent, lse = forward(tw, h, w, t, 1.0)
    assert lse[0] == float("-inf")
    g = torch.ones(3, device="cuda")
    dh, dw, _ = backward(tw, h, w, t, 1.0, lse, ent, g, g)
    assert not dh[0].any()
    h[1, 3] = float("nan")
    lp, ent, lse = forward(tw, h, w, t, 1.0)
    dh, _, _ = backward(tw, h, w, t, 1.0, lse, ent, g, g)
    assert not dh[0].any() and dh[1].isnan().all() and not dh[2].isnan().any()


def test_repeats_bit_for_bit_on_streams_and_in_graphs(tw):
    h, w, t = make(260, 264, 3000, 16)
    fwd = forward(tw, h, w, t, 1.0)
    g, ge = gradient_inputs(260, 17)
    dh, dw, call = backward(tw, h, w, t, 1.0, fwd[2], fwd[1], g, ge)
    first = (dh.clone(), dw.clone())
    # two streams at once, each with its own workspace and outputs
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for s in streams:
        with torch.cuda.stream(s):
            got.append((forward(tw, h, w, t, 1.0, status=torch.zeros(1, dtype=torch.int32, device="cuda")),
                        backward(tw, h, w, t, 1.0, fwd[2], fwd[1], g, ge)[:2]))
    torch.cuda.synchronize()
    for f, b in got:
        assert all(torch.equal(x, y) for x, y in zip(f, fwd))
        assert torch.equal(b[0], first[0]) and torch.equal(b[1], first[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(stream=None)
    dh.fill_(float("nan"))
    dw.fill_(float("nan"))
    graph.replay()
    graph.replay()
    assert torch.equal(dh, first[0]) and torch.equal(dw, first[1])


def test_no_rows(tw):
    h = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((10, 64), dtype=torch.bfloat16, device="cuda")
    z = torch.empty(0, device="cuda")
    t = torch.empty(0, dtype=torch.int32, device="cuda")
    dw = torch.full((10, 72), float("nan"), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    tw.twell_linear_logprobs(h, w, t, 1.0, z, z, z, ws, st)
    tw.twell_linear_logprobs_bwd(h, w, t, 1.0, z, z, z, z, h, dw[:, :64], ws, st)
    assert not dw[:, :64].any() and dw[:, 64:].isnan().all() and int(st) == 0


def test_rows_far_apart(tw):
    """Offsets past 2^31 elements in every matrix."""
    n, d, v, ld = 3, 64, 5, 1_100_000_000
    h, w, t = make(n, d, v, 18)
    far = lambda m: torch.empty(ld * (m.shape[0] - 1) + d, dtype=m.dtype,  # noqa: E731
                                device="cuda").as_strided((m.shape[0], d), (ld, 1))
    fh, fw = far(h), far(w)
    fh.copy_(h)
    fw.copy_(w)
    near = forward(tw, h, w, t, 1.0)
    assert all(torch.equal(a, b) for a, b in zip(forward(tw, fh, fw, t, 1.0), near))
    g, ge = gradient_inputs(n, 19)
    dh, dw, _ = backward(tw, h, w, t, 1.0, near[2], near[1], g, ge)
    oh, ow = far(h), far(w)
    ws = torch.empty(tw.linear_logprobs_bwd_workspace_bytes(n, d, v), dtype=torch.uint8, device="cuda")
    tw.twell_linear_logprobs_bwd(fh, fw, t, 1.0, near[2], near[1], g, ge, oh, ow, ws,
                                 torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert torch.equal(oh, dh) and torch.equal(ow, dw)


def test_gradient_against_differences(tw):
    """Along random directions against central differences of the 64-bit definition."""
    n, d, v, inv_t = 6, 64, 300, 1.2
    h, w, t = make(n, d, v, 20)
    _, ent, lse = forward(tw, h, w, t, inv_t)
    g, ge = gradient_inputs(n, 21)
    dh, dw, _ = backward(tw, h, w, t, inv_t, lse, ent, g, ge)

    def loss(a, b):
        lp, en, _ = ref.linear_logprobs(ref.linear_logits(a, b, inv_t)[0], t)
        return float((g.double() * lp + ge.double() * en).sum())

    rng = torch.Generator().manual_seed(22)
    for got, k in ((dh, 0), (dw, 1)):
        at = [h.double(), w.double()]
        way = torch.randn(at[k].shape, generator=rng, dtype=torch.float64).cuda()
        ends = []
        for s in (1e-5, -1e-5):
            moved = list(at)
            moved[k] = at[k] + s * way
            ends.append(loss(*moved))
        numeric = (ends[0] - ends[1]) / 2e-5
        scale = float((got.double() * way).abs().sum())
        assert abs(float((got.double() * way).sum()) - numeric) <= 2.0 ** -7 * scale + 1e-6 * abs(numeric)


# few tiles and long rows: the logits are multiplied in ranges of K
RANGES = [(10, 3640, 500), (1, 4016, 1210), (33, 1600, 255), (128, 2048, 513), (129, 4096, 300), (300, 4096, 1001), (1, 16384, 1)]


@pytest.mark.parametrize("pad", [0, 24])
@pytest.mark.parametrize("n,d,v", RANGES)
def test_few_tokens_and_long_rows(tw, n, d, v, pad):
    h, w, t = make(n, d, v, n + v, pad=pad)
    check_forward(tw, h, w, t, 1.3)
    lp, ent, lse = forward(tw, h, w, t, 1.3)
    again = forward(tw, h, w, t, 1.3)
    assert all(torch.equal(a, b) for a, b in zip(again, (lp, ent, lse)))
    g, ge = gradient_inputs(n, 24)
    dh, dw, call = backward(tw, h, w, t, 1.3, lse, ent, g, ge, pad=pad)
    check_backward(h, w, t, 1.3, lse, ent, g, ge, dh, dw)
    first = (dh.clone(), dw.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(stream=None)
    dh.fill_(float("nan"))
    dw.fill_(float("nan"))
    graph.replay()
    assert torch.equal(dh, first[0]) and torch.equal(dw, first[1])


def test_long_rows_with_nan_infinity_or_nothing(tw):
    h, w, t = make(40, 2048, 700, 25)
    clean = forward(tw, h, w, t, 1.0)
    h[3, 5], h[9, 2000], h[20, 1024] = float("nan"), float("inf"), float("-inf")
    got = forward(tw, h, w, t, 1.0)
    bad = [3, 9, 20]
    keep = [i for i in range(40) if i not in bad]
    for a, b in zip(got, clean):
        assert torch.equal(a[keep], b[keep])
    assert got[1][bad].isnan().all() and got[2][bad].isnan().all()
    w2 = torch.zeros((300, 2048), dtype=torch.bfloat16, device="cuda")
    w2[:, 1000] = float("-inf")
    h2 = torch.ones((2, 2048), dtype=torch.bfloat16, device="cuda")
    lp, ent, lse = forward(tw, h2, w2, torch.tensor([4, -1], dtype=torch.int32, device="cuda"), 1.0)
    assert lse.tolist() == [float("-inf")] * 2 and ent.tolist() == [0.0, 0.0] and lp.tolist() == [float("-inf"), 0.0]
    w2[290] = 0
    lp, ent, lse = forward(tw, h2, w2, torch.tensor([290, 4], dtype=torch.int32, device="cuda"), 1.0)
    assert lse.tolist() == [0.0, 0.0] and ent.tolist() == [0.0, 0.0] and lp.tolist() == [0.0, float("-inf")]


@pytest.mark.parametrize("n", [40, 300])
def test_an_expired_wait_of_ranges_is_reported(tw, n):
    d, v = 4096, 500
    h, w, t = make(n, d, v, 26)
    ws = torch.empty(tw.linear_logprobs_workspace_bytes(n, d, v), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    rc = tw.load_library().twell_selftest_linear_stall(h.data_ptr(), d, w.data_ptr(), d, n, d, v, ws.data_ptr(),
                                                       ws.numel(), st.data_ptr(), 1_000_000,
                                                       torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    assert int(st) == -7
    check_forward(tw, h, w, t, 1.0)


@pytest.mark.parametrize("n", [40, 300])  # a CTA to a tile, and a pair
def test_an_expired_wait_is_reported(tw, n):
    """Every stage waits for an arrival that never comes: the call ends, says so, and the next one is sound."""
    h, w, t = make(n, 128, 2000, 23)
    ws = torch.empty(tw.linear_logprobs_workspace_bytes(n, 128, 2000), dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib = tw.load_library()
    rc = lib.twell_selftest_linear_stall(h.data_ptr(), 128, w.data_ptr(), 128, n, 128, 2000, ws.data_ptr(), ws.numel(),
                                         st.data_ptr(), 1_000_000, torch.cuda.current_stream().cuda_stream)
    assert rc == 0
    torch.cuda.synchronize()
    assert int(st) == -7
    check_forward(tw, h, w, t, 1.0)
