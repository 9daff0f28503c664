"""The norms around a block with its gate and residual sum, and their gradient, against the
64-bit definition.

Error bounds: fp32 operations are off by u = 2^-24 of their result.  A thread adds at most 16
squares one after the other and a tree of at most 10 steps follows, so a row's sum is off by 26 u
of the magnitudes in it at most, its root's inverse by 13 u + 4 u; what is built from them takes
fewer than 30 further operations.  Sums over n rows are off by n u of the magnitudes at most, in
any order.  An output rounded to bf16 is off by 2^-8 of itself more."""
import numpy as np
import pytest
import torch

import training_reference as ref

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
EPS = 1e-5


@pytest.fixture(scope="module")
def tw():
    import activation_sparse_transformer_gb300 as m
    m.load_library()
    return m


def step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def make(rows, dim, stream, flags, seed, w_dtype=torch.bfloat16, pad=0):
    """Inputs of a call on the device; flags: letters of y (block), p (post), g (gate), r (row gate), n (next norm)."""
    g = torch.Generator().manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g)  # noqa: E731

    def mat(dtype, scale):
        m = (scale * rand(rows, dim + pad) * torch.exp(0.5 * rand(rows, 1))).to(dtype).cuda()
        return m[:, :dim] if pad else m

    vec = lambda on: (1 + 0.5 * rand(dim)).to(w_dtype).cuda() if on else None  # noqa: E731
    row = None
    if "r" in flags:
        row = torch.rand(rows, generator=g) - 0.3
        row[::3] = 0.0
        row = row.cuda()
    return dict(x=mat(stream, 1.0), y=mat(torch.bfloat16, 0.7) if "y" in flags else None, w_post=vec("p" in flags),
                gate=vec("g" in flags), w_pre=vec("n" in flags), row_gate=row)


def run(tw, i, skip, branch, stream=None, in_place=False, outputs=("x_out", "h", "rstd_post", "rstd_pre")):
    n, d = i["x"].shape
    new = lambda dt: torch.full((n, d), float("nan"), dtype=dt, device="cuda")  # noqa: E731
    o = {"x_out": i["x"] if in_place else new(i["x"].dtype), "h": new(torch.bfloat16) if i["w_pre"] is not None else None,
         "rstd_post": torch.empty(n, device="cuda") if i["w_post"] is not None else None,
         "rstd_pre": torch.empty(n, device="cuda") if i["w_pre"] is not None else None}
    o = {k: (v if k in outputs else None) for k, v in o.items()}
    tw.twell_block_norm(i["x"], i["y"], o["x_out"], o["h"], w_post=i["w_post"], gate=i["gate"], w_pre=i["w_pre"],
                        row_gate=i["row_gate"], skip_scale=skip, branch_scale=branch, eps=EPS, rstd_post=o["rstd_post"],
                        rstd_pre=o["rstd_pre"], stream=stream)
    return o


def within(got, want, bound, what):
    got = f64(got)
    off = np.abs(got - want)
    assert np.isfinite(got).all(), what
    worst = np.unravel_index(np.argmax(off - bound), off.shape)
    assert (off <= bound).all(), f"{what}: off by {off[worst]:.3e}, bound {np.broadcast_to(bound, off.shape)[worst]:.3e} at {worst}"


def check_forward(i, o, skip, branch, x=None):
    args = [f64(i[k]) for k in ("w_post", "gate", "w_pre", "row_gate")]
    x = f64(i["x"]) if x is None else x
    z, h, r1, r2, size = ref.block_norm(x, f64(i["y"]), *args, skip, branch, EPS)
    f32 = 32 * U * size  # of z before its rounding
    if o["x_out"] is not None:
        within(o["x_out"], z, f32 + step(o["x_out"].dtype) * np.abs(z), "x_out")
    if o["rstd_post"] is not None:
        within(o["rstd_post"], r1, 17 * U * r1, "rstd_post")
    if h is not None and o["h"] is not None:
        # a row's sum of squares moves by 2 |z| |error of z| at most
        moved = (f32 * np.abs(z)).mean(1) * r2 ** 2
        if o["rstd_pre"] is not None:
            within(o["rstd_pre"], r2, (17 * U + moved) * r2, "rstd_pre")
        w = np.abs(f64(i["w_pre"]))
        within(o["h"], h, (f32 * r2[:, None] * w + (20 * U + moved[:, None] + step(torch.bfloat16)) * np.abs(h))
               * (1 + 1e-6), "h")


FLAGS = ["ypgrn", "ypn", "yn", "y", "yg", "ypr", "n", "yrn", ""]


@pytest.mark.parametrize("flags", FLAGS)
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,dim", [(1, 8), (3, 264), (33, 1352), (7, 4104)])
def test_forward_parts(tw, rows, dim, stream, flags):
    i = make(rows, dim, stream, flags, 1)
    check_forward(i, run(tw, i, 0.75, -1.25), 0.75, -1.25)


@pytest.mark.parametrize("rows,dim", [(1, 16384), (2, 16376), (1, 64), (5, 72), (2, 248), (9, 256), (17, 512), (300, 520),
                                      (1000, 2048), (4097, 64), (64, 8200), (152, 4096), (2431, 1024), (700, 8), (5001, 24),
                                      (301, 40), (90, 5008), (33, 8192)])
def test_forward_sizes(tw, rows, dim):
    i = make(rows, dim, torch.bfloat16, "ypgrn", 2)
    check_forward(i, run(tw, i, 1.0, 1.0), 1.0, 1.0)


@pytest.mark.parametrize("w_dtype", [torch.bfloat16, torch.float32])
def test_forward_strides_weights_and_in_place(tw, w_dtype):
    i = make(45, 712, torch.bfloat16, "ypgn", 3, w_dtype, pad=24)
    x = f64(i["x"])
    beyond = i["x"]._base[:, 712:].clone()
    check_forward(i, run(tw, i, 0.5, 2.0, in_place=True), 0.5, 2.0, x)
    assert torch.equal(i["x"]._base[:, 712:], beyond)  # what lies between the rows stays


def test_outputs_that_are_not_wanted(tw):
    i = make(20, 320, torch.float32, "ypn", 4)
    full = run(tw, i, 1.0, 0.5)
    for outputs in (("x_out", "h"), ("h",), ("h", "rstd_pre")):
        o = run(tw, i, 1.0, 0.5, outputs=outputs)
        for k in outputs:
            assert torch.equal(o[k], full[k])


def test_rows_of_zeros_and_of_any_size(tw):
    """A row of zeros has the norm 0; magnitudes from 1e-17 to 1e17 square within fp32's range or below eps."""
    i = make(8, 512, torch.float32, "ypn", 5)
    for r, s in enumerate([0.0, 1e17, 1e-17, 1e10, 1e-10, 1e4, 1e-4, 1.0]):
        i["x"][r] *= s
        i["y"][r] *= s
    o = run(tw, i, 1.0, 1.0)
    assert not o["x_out"][0].any() and not o["h"][0].any()
    check_forward(i, o, 1.0, 1.0)


def test_a_row_with_nan_or_infinity_keeps_to_itself(tw):
    i = make(6, 328, torch.bfloat16, "ypgn", 6)
    clean = run(tw, i, 1.0, 1.0)
    i["y"][2, 5], i["x"][4, 0] = float("nan"), float("inf")
    o = run(tw, i, 1.0, 1.0)
    keep = [0, 1, 3, 5]
    for k in ("x_out", "h", "rstd_post", "rstd_pre"):
        assert torch.equal(o[k][keep], clean[k][keep])
    assert o["h"][2].isnan().all() and o["h"][4].isnan().any()


WIDE = [(76, 8200), (77, 16384), (401, 8208), (155, 12296), (229, 10240)]  # several rows side by side, the last round not full


@pytest.mark.parametrize("flags", ["ypgrn", "yn", "ypr", "n"])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,dim", WIDE)
def test_forward_of_wide_rows(tw, rows, dim, stream, flags):
    i = make(rows, dim, stream, flags, 31, pad=16)
    check_forward(i, run(tw, i, 0.75, -1.25), 0.75, -1.25)


# ---------------------------------------------------------------- the gradient
def backward(tw, i, skip, branch, seed, dh=True, d_out=True, dx=True, dy=True, dw=True, stream=None, in_place=False):
    n, d = i["x"].shape
    g = torch.Generator().manual_seed(seed)
    o = run(tw, i, skip, branch)
    r = lambda dt: torch.randn((n, d), generator=g).to(dt).cuda()  # noqa: E731
    b = dict(dh=r(torch.bfloat16) if dh and i["w_pre"] is not None else None, d_out=r(i["x"].dtype) if d_out else None)
    if b["dh"] is None:
        i = dict(i, w_pre=None)
    up = None if b["d_out"] is None else f64(b["d_out"])
    out = dict(dx=None if not dx else b["d_out"] if in_place else torch.full_like(o["x_out"], float("nan")),
               dy=torch.full_like(i["y"], float("nan")) if dy and i["y"] is not None else None)
    vec = lambda k, m: torch.full((m,), float("nan"), device="cuda") if dw and i[k] is not None else None  # noqa: E731
    out.update(dw_post=vec("w_post", d), dgate=vec("gate", d), dw_pre=vec("w_pre", d), drow_gate=vec("row_gate", n))
    ws = torch.empty(tw.block_norm_bwd_workspace_bytes(n, d), dtype=torch.uint8, device="cuda")
    rstd_pre = o["rstd_pre"] if i["w_pre"] is not None else None

    def call():
        tw.twell_block_norm_bwd(b["dh"], b["d_out"], o["x_out"], i["y"], out["dx"], out["dy"], w_post=i["w_post"],
                                gate=i["gate"], w_pre=i["w_pre"], row_gate=i["row_gate"], skip_scale=skip,
                                branch_scale=branch, rstd_post=o["rstd_post"], rstd_pre=rstd_pre,
                                dw_post=out["dw_post"], dgate=out["dgate"], dw_pre=out["dw_pre"],
                                drow_gate=out["drow_gate"], workspace=ws, stream=stream)
    call()
    want, size = ref.block_norm_bwd(f64(b["dh"]), up, f64(o["x_out"]), f64(i["y"]), f64(i["w_post"]), f64(i["gate"]),
                                    f64(i["w_pre"]), f64(i["row_gate"]), skip, branch, f64(o["rstd_post"]),
                                    f64(rstd_pre))
    return out, want, size, call


def check_backward(out, want, size, rows):
    for k, t in out.items():
        if t is None:
            continue
        if k in ("dx", "dy"):
            bound = 128 * U * size[k] + step(t.dtype) * np.abs(want[k])
        elif k == "drow_gate":
            bound = 128 * U * size[k]
        else:
            bound = (rows + 128) * U * size[k]
        within(t, want[k], bound + 1e-38, k)


@pytest.mark.parametrize("flags", [f for f in FLAGS if f])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,dim", [(1, 8), (3, 264), (33, 1352), (7, 4104)])
def test_backward_parts(tw, rows, dim, stream, flags):
    i = make(rows, dim, stream, flags, 11)
    check_backward(*backward(tw, i, 0.75, -1.25, 12)[:3], rows)


@pytest.mark.parametrize("rows,dim", [(1, 16384), (2, 16376), (1, 64), (5, 72), (2, 248), (300, 520), (1000, 2048),
                                      (4097, 64), (400, 8200), (2431, 1024), (20000, 128), (700, 8),
                                      (5001, 24), (301, 40), (200, 5008), (155, 8192)])
def test_backward_sizes(tw, rows, dim):
    i = make(rows, dim, torch.bfloat16, "ypgrn", 13)
    check_backward(*backward(tw, i, 1.0, 1.0, 14)[:3], rows)


@pytest.mark.parametrize("flags", ["ypgrn", "yn", "ypr", "n"])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,dim", WIDE)
def test_backward_of_wide_rows(tw, rows, dim, stream, flags):
    i = make(rows, dim, stream, flags, 32, pad=16)
    out, want, size, call = backward(tw, i, 0.75, -1.25, 33)
    check_backward(out, want, size, rows)
    first = {k: v.clone() for k, v in out.items() if v is not None}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in first:
        out[k].fill_(float("nan"))
    graph.replay()
    for k in first:
        assert torch.equal(out[k], first[k]), k


@pytest.mark.parametrize("given", [dict(dh=False), dict(d_out=False), dict(dx=False), dict(dy=False), dict(dw=False),
                                   dict(dx=False, dy=False), dict(in_place=True)])
def test_backward_of_some(tw, given):
    i = make(37, 648, torch.bfloat16, "ypgrn", 15, torch.float32, pad=16)
    check_backward(*backward(tw, i, 0.5, 1.5, 16, **given)[:3], 37)


def test_backward_repeats_bit_for_bit_and_replays(tw):
    i = make(701, 1032, torch.bfloat16, "ypgrn", 17)
    out, want, size, call = backward(tw, i, 1.0, 1.0, 18)
    first = {k: v.clone() for k, v in out.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    for k, v in out.items():
        assert torch.equal(v, first[k]), k
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for v in out.values():
        v.fill_(float("nan"))
    graph.replay()
    for k, v in out.items():
        assert torch.equal(v, first[k]), k
    check_backward(out, want, size, 701)


def test_no_rows(tw):
    d = 64
    e = torch.empty((0, d), dtype=torch.bfloat16, device="cuda")
    w = torch.ones(d, device="cuda")
    z = torch.empty(0, device="cuda")
    tw.twell_block_norm(e, e, e, e, w_post=w, w_pre=w)
    dw = torch.full((2, d), float("nan"), device="cuda")
    ws = torch.empty(tw.block_norm_bwd_workspace_bytes(0, d), dtype=torch.uint8, device="cuda")
    tw.twell_block_norm_bwd(e, e, e, e, e, e, w_post=w, w_pre=w, rstd_post=z, rstd_pre=z, dw_post=dw[0], dw_pre=dw[1],
                            workspace=ws)
    assert not dw.any()


def test_rows_far_apart(tw):
    """Offsets past 2^31 elements."""
    n, d, ld = 5, 72, 600_000_000
    base = torch.empty(ld * (n - 1) + d, dtype=torch.bfloat16, device="cuda")
    far = base.as_strided((n, d), (ld, 1))
    near = make(n, d, torch.bfloat16, "ypn", 19)
    far.copy_(near["x"])
    want = run(tw, near, 1.0, 1.0)
    got = run(tw, dict(near, x=far), 1.0, 1.0, in_place=True)
    for k in ("x_out", "h", "rstd_post", "rstd_pre"):
        assert torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("flags", ["ypgrn", "yn"])
def test_gradient_against_differences(tw, flags):
    """The gradients along random directions against central differences of the 64-bit definition."""
    n, d, skip, branch = 5, 96, 0.9, 1.3
    i = make(n, d, torch.float32, flags, 21, torch.float32)
    g = torch.Generator().manual_seed(22)
    o = run(tw, i, skip, branch)
    dh, d_out = torch.randn((n, d), generator=g).bfloat16().cuda(), torch.randn((n, d), generator=g).cuda()
    at = {k: f64(v) for k, v in i.items() if v is not None}
    out = {k: torch.empty_like(i[k] if k != "row_gate" else i[k]) for k in at}
    ws = torch.empty(tw.block_norm_bwd_workspace_bytes(n, d), dtype=torch.uint8, device="cuda")
    tw.twell_block_norm_bwd(dh, d_out, o["x_out"], i["y"], out["x"], out["y"], w_post=i["w_post"], gate=i["gate"],
                            w_pre=i["w_pre"], row_gate=i["row_gate"], skip_scale=skip, branch_scale=branch,
                            rstd_post=o["rstd_post"], rstd_pre=o["rstd_pre"], dw_post=out.get("w_post"),
                            dgate=out.get("gate"), dw_pre=out.get("w_pre"), drow_gate=out.get("row_gate"), workspace=ws)

    def loss(v):
        z, h = ref.block_norm(v["x"], v["y"], v.get("w_post"), v.get("gate"), v.get("w_pre"), v.get("row_gate"), skip,
                              branch, EPS)[:2]
        return (f64(dh) * h).sum() + (f64(d_out) * z).sum()

    rng = np.random.default_rng(23)
    for k in at:
        way = rng.standard_normal(at[k].shape)
        e = 1e-5
        up, down = ({**at, k: at[k] + s * e * way} for s in (1, -1))
        numeric = (loss(up) - loss(down)) / (2 * e)
        got = (f64(out[k]) * way).sum()
        # dy is bf16: 2^-8 of each term; the others 2^-16 leaves room for fp32 sums; differences are good to e^2
        scale = (np.abs(f64(out[k]) * way)).sum()
        assert abs(got - numeric) <= (2.0 ** -8 if k == "y" else 2.0 ** -16) * scale + 1e-6 * abs(numeric), k
