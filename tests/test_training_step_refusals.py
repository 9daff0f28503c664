"""The training step's calls refuse bad arguments on the host, before any launch: the C ABI by its
codes (aligned fake pointers, never dereferenced), the binding by type, shape, stride and size."""
import ctypes

import pytest

P = ctypes.c_void_p
A, B, C, D, E, F = (P(0x10000 * i) for i in range(1, 7))


@pytest.fixture(scope="module")
def tw():
    import __graft_entry__ as g
    g.build()
    import activation_sparse_transformer_gb300 as m
    return m


@pytest.fixture(scope="module")
def lib(tw):
    return tw.load_library()


NORM = dict(x=A, dtype=0, ldx=256, y=B, ldy=256, n=5, d=256, w_post=A, gate=A, w_pre=A, w_dtype=0, row_gate=A, skip=1.0,
            branch=1.0, eps=1e-6, x_out=C, ldo=256, h=D, ldh=256, rstd_post=A, rstd_pre=A, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(x=None), -1), (dict(n=-1), -1), (dict(d=0), -1), (dict(d=-8), -1), (dict(dtype=2), -1), (dict(dtype=-1), -1),
    (dict(w_dtype=2), -1), (dict(eps=0.0), -1), (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1),
    (dict(eps=float("inf")), -1), (dict(skip=float("nan")), -1), (dict(branch=float("inf")), -1),
    (dict(y=None), -1), (dict(y=None, w_post=None, gate=None, rstd_post=None), -1),     # a gate without a block
    (dict(h=None), -1), (dict(w_pre=None), -1), (dict(w_pre=None, h=None), -1),         # rstd_pre without a norm
    (dict(w_post=None), -1), (dict(x_out=None, h=None, w_pre=None, rstd_pre=None), -1),
    (dict(ldx=248), -1), (dict(ldy=260), -1), (dict(ldo=255), -1), (dict(ldh=0), -1),
    (dict(h=A), -1), (dict(h=B), -1), (dict(h=C), -1), (dict(x_out=B), -1),             # over what is read, or each other
    (dict(x_out=A, ldo=264), -1),                                                     # in place with another distance
    (dict(d=260, ldx=264, ldy=264, ldo=264, ldh=264), -3),
    (dict(d=16392, ldx=16392, ldy=16392, ldo=16392, ldh=16392), -3),
    (dict(x=P(0x10008)), -2), (dict(y=P(0x10008)), -2), (dict(h=P(0x10004)), -2), (dict(gate=P(0x10002)), -2),
    (dict(row_gate=P(0x10002)), -2), (dict(rstd_pre=P(0x10001)), -2)])
def test_block_norm_refuses(lib, over, code):
    assert lib.twell_block_norm(*{**NORM, **over}.values()) == code


BWD = dict(dh=A, lddh=256, d_out=B, dtype=0, lddo=256, x_out=C, ldo=256, y=D, ldy=256, n=5, d=256, w_post=A, gate=A,
           w_pre=A, w_dtype=0, row_gate=A, skip=1.0, branch=1.0, rstd_post=A, rstd_pre=A, dx=E, lddx=256, dy=F,
           lddy=256, dw_post=A, dgate=A, dw_pre=A, drow_gate=A, ws=A, ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(dh=None), -1), (dict(w_pre=None), -1), (dict(rstd_pre=None), -1), (dict(x_out=None), -1),
    (dict(dh=None, w_pre=None, rstd_pre=None), -1),                                   # dw_pre without a norm
    (dict(dh=None, w_pre=None, rstd_pre=None, dw_pre=None, d_out=None), -1),
    (dict(w_post=None), -1), (dict(rstd_post=None), -1), (dict(gate=None), -1), (dict(row_gate=None), -1),
    (dict(y=None), -1), (dict(n=-1), -1), (dict(d=0), -1), (dict(dtype=5), -1), (dict(w_dtype=-1), -1),
    (dict(skip=float("inf")), -1), (dict(branch=float("nan")), -1), (dict(lddh=248), -1), (dict(lddx=250), -1),
    (dict(dx=B, lddx=264), -1), (dict(dx=A), -1), (dict(dx=C), -1), (dict(dx=F), -1), (dict(dy=A), -1), (dict(dy=B), -1),
    (dict(dy=D), -1), (dict(d=100, lddh=104), -3), (dict(dh=P(0x10008)), -2), (dict(dy=P(0x10008)), -2),
    (dict(dw_pre=P(0x10002)), -2), (dict(w_post=P(0x10008)), -2), (dict(ws=None), -5), (dict(ws_bytes=100), -5),
    (dict(ws=P(0x10010)), -2)])
def test_block_norm_bwd_refuses(lib, over, code):
    assert lib.twell_block_norm_bwd(*{**BWD, **over}.values()) == code


def test_block_norm_workspace_is_host_arithmetic(tw):
    assert tw.block_norm_bwd_workspace_bytes(100, 256) > 0
    for bad in ((-1, 256), (10, 0), (10, 12), (10, 16392)):
        assert tw.block_norm_bwd_workspace_bytes(*bad) == 0


def test_binding_of_the_norms_checks(tw):
    """CPU tensors: everything else is refused before they are."""
    import torch
    bf = torch.bfloat16
    x, w = torch.zeros((4, 64), dtype=bf), torch.ones(64, dtype=bf)
    with pytest.raises(ValueError, match="^x: torch.float16"):
        tw.twell_block_norm(x.half(), x, x)
    with pytest.raises(ValueError, match="^y: torch.float32"):
        tw.twell_block_norm(x, x.float(), x)
    with pytest.raises(ValueError, match="^y: shape"):
        tw.twell_block_norm(x, x[:3], x)
    with pytest.raises(ValueError, match="^x_out: torch.float32"):
        tw.twell_block_norm(x, x, x.float())
    with pytest.raises(ValueError, match="^h: a tensor whose rows"):
        tw.twell_block_norm(x, x, x, torch.zeros((64, 4), dtype=bf).t(), w_pre=w)
    with pytest.raises(ValueError, match="^w_pre: 63"):
        tw.twell_block_norm(x, x, x, x, w_pre=w[:63])
    with pytest.raises(ValueError, match="^w_pre: torch.float32, the other"):
        tw.twell_block_norm(x, x, x, x, w_post=w, w_pre=w.float())
    with pytest.raises(ValueError, match="^row_gate: 3"):
        tw.twell_block_norm(x, x, x, row_gate=torch.zeros(3))
    with pytest.raises(ValueError, match="CUDA"):
        tw.twell_block_norm(x, x, x)
    r = torch.zeros(4)
    with pytest.raises(ValueError, match="^d_out, x_out, dx"):
        tw.twell_block_norm_bwd(x, None, None, x)
    with pytest.raises(ValueError, match="^dx: torch.float32"):
        tw.twell_block_norm_bwd(x, x, x, x, x.float(), x, w_pre=w, rstd_pre=r)
    with pytest.raises(ValueError, match="^dw_pre: torch.bfloat16"):
        tw.twell_block_norm_bwd(x, x, x, x, x, x, w_pre=w, rstd_pre=r, dw_pre=w)
    with pytest.raises(ValueError, match="CUDA"):
        tw.twell_block_norm_bwd(x, x, x, x, x, x, w_pre=w, rstd_pre=r)


LIN = dict(H=A, ldh=256, W=B, ldw=256, n=5, d=256, vocab=1000, targets=C, inv_t=1.0, logprob=D, entropy=E, lse=F, ws=A,
           ws_bytes=1 << 40, status=A, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(H=None), -1), (dict(W=None), -1), (dict(n=-1), -1), (dict(d=0), -1), (dict(vocab=0), -1), (dict(ldh=248), -1),
    (dict(ldw=260), -1), (dict(inv_t=0.0), -1), (dict(inv_t=-1.0), -1), (dict(inv_t=float("nan")), -1),
    (dict(inv_t=float("inf")), -1), (dict(inv_t=2.5e38), -1), (dict(targets=None), -1), (dict(logprob=None), -1),
    (dict(status=None), -1), (dict(d=100, ldh=104), -3), (dict(n=(1 << 30) + 1), -3), (dict(vocab=(1 << 30) + 1), -3), (dict(H=P(0x10008)), -2), (dict(W=P(0x10008)), -2), (dict(lse=P(0x10002)), -2),
    (dict(status=P(0x10002)), -2), (dict(ws=None), -5), (dict(ws_bytes=100), -5), (dict(ws=P(0x10010)), -2)])
def test_linear_logprobs_refuse(lib, over, code):
    assert lib.twell_linear_logprobs(*{**LIN, **over}.values()) == code


LINB = dict(H=A, ldh=256, W=B, ldw=256, n=5, d=256, vocab=1000, targets=C, inv_t=1.0, lse=D, entropy=E, g=F, ge=A,
            dH=C, lddh=256, dW=D, lddw=256, ws=A, ws_bytes=1 << 40, status=A, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(H=None), -1), (dict(W=None), -1), (dict(lse=None), -1), (dict(targets=None), -1), (dict(g=None), -1),
    (dict(entropy=None), -1), (dict(ge=None), -1), (dict(dH=None, dW=None), -1),
    (dict(dH=A), -1), (dict(dW=B), -1), (dict(dH=B), -1), (dict(dW=A), -1), (dict(dW=C), -1),   # over what is read, or each other
 (dict(lddh=248), -1),
    (dict(lddw=257), -1), (dict(n=-1), -1), (dict(inv_t=0.0), -1), (dict(status=None), -1), (dict(d=100), -3),
    (dict(dH=P(0x10008)), -2), (dict(dW=P(0x10008)), -2), (dict(g=P(0x10001)), -2), (dict(ws=None), -5),
    (dict(ws_bytes=1000), -5), (dict(ws=P(0x10010)), -2)])
def test_linear_logprobs_bwd_refuses(lib, over, code):
    assert lib.twell_linear_logprobs_bwd(*{**LINB, **over}.values()) == code


def test_linear_workspaces_are_host_arithmetic(tw):
    assert tw.linear_logprobs_workspace_bytes(0, 64, 10) > 0 and tw.linear_logprobs_bwd_workspace_bytes(0, 64, 10) > 0
    assert tw.linear_logprobs_workspace_bytes(16, 4096, 131072) >= 16 * 4 * 3
    assert tw.linear_logprobs_bwd_workspace_bytes(16, 4096, 131072) >= 16 * 131072 * 2
    # pieces: far less than the logits
    assert tw.linear_logprobs_bwd_workspace_bytes(65536, 4096, 131072) < 65536 * 131072 * 2 // 4
    for f in (tw.linear_logprobs_workspace_bytes, tw.linear_logprobs_bwd_workspace_bytes):
        for bad in ((-1, 64, 10), (1, 0, 10), (1, 12, 10), (1, 64, 0), ((1 << 30) + 1, 64, 10), (1, 64, (1 << 30) + 1)):
            assert f(*bad) == 0


def test_a_linear_workspace_holds_what_fewer_rows_take(tw, lib):
    """With the bytes for n rows, calls of fewer rows get past the workspace's check (to that of the device, here without one)."""
    import random

    import torch
    if torch.cuda.is_available():
        pytest.skip("the calls would go on to the GPU")
    rng = random.Random(5)
    size = lambda a, b: int(2 ** rng.uniform(a, b))  # noqa: E731
    for _ in range(4000):
        n, d, v = size(0, 17), 8 * size(0, 11), size(0, 18)
        fewer = min(n, rng.choice([1, 128, 129, 256, 257, 1024, size(0, 17), n]))
        shape = dict(n=fewer, d=d, vocab=v, ldh=d, ldw=d)
        ws = tw.linear_logprobs_workspace_bytes(n, d, v)
        assert lib.twell_linear_logprobs(*{**LIN, **shape, "ws_bytes": ws}.values()) == -8, (n, d, v, fewer)
        ws = tw.linear_logprobs_bwd_workspace_bytes(n, d, v)
        assert lib.twell_linear_logprobs_bwd(*{**LINB, **shape, "lddh": d, "lddw": d, "ws_bytes": ws}.values()) == -8, (
            n, d, v, fewer)
    # not much more than what n rows take themselves
    assert tw.linear_logprobs_bwd_workspace_bytes(8192, 2048, 32768) < 400 << 20
    assert tw.linear_logprobs_workspace_bytes(16, 4096, 131072) < 1 << 20


def test_binding_of_the_linear_calls_checks(tw):
    import torch
    bf, i32 = torch.bfloat16, torch.int32
    h, w, f, t = torch.zeros((4, 64), dtype=bf), torch.zeros((10, 64), dtype=bf), torch.zeros(4), torch.zeros(4, dtype=i32)
    ws, st = torch.zeros(256, dtype=torch.uint8), torch.zeros(1, dtype=i32)
    with pytest.raises(ValueError, match="^hidden: torch.float32"):
        tw.twell_linear_logprobs(h.float(), w, t, 1.0, f, f, f, ws, st)
    with pytest.raises(ValueError, match="^weight: rows of 56"):
        tw.twell_linear_logprobs(h, w[:, :56], t, 1.0, f, f, f, ws, st)
    with pytest.raises(ValueError, match="^targets: torch.int64"):
        tw.twell_linear_logprobs(h, w, t.long(), 1.0, f, f, f, ws, st)
    with pytest.raises(ValueError, match="^lse: 3"):
        tw.twell_linear_logprobs(h, w, t, 1.0, f, f, f[:3], ws, st)
    with pytest.raises(ValueError, match="CUDA"):
        tw.twell_linear_logprobs(h, w, t, 1.0, f, f, f, ws, st)
    with pytest.raises(ValueError, match="^d_weight: shape"):
        tw.twell_linear_logprobs_bwd(h, w, t, 1.0, f, f, f, f, h, w[:9], ws, st)
    with pytest.raises(ValueError, match="^d_hidden: torch.float32"):
        tw.twell_linear_logprobs_bwd(h, w, t, 1.0, f, f, f, f, h.float(), w, ws, st)
    with pytest.raises(ValueError, match="CUDA"):
        tw.twell_linear_logprobs_bwd(h, w, t, 1.0, f, f, f, f, h, w, ws, st)


@pytest.mark.parametrize("over,code", [(dict(limit=0), -1), (dict(limit=2_000_000_000), -1), (dict(H=None), -1),
                                       (dict(status=None), -1), (dict(ws=None), -5)])
def test_linear_selftest_refuses(lib, over, code):
    a = dict(H=A, ldh=256, W=B, ldw=256, n=5, d=256, vocab=1000, ws=A, ws_bytes=1 << 40, status=A, limit=1_000_000,
             stream=None)
    assert lib.twell_selftest_linear_stall(*{**a, **over}.values()) == code
