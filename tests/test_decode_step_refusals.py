"""The decode step's calls refuse bad arguments on the host, before any launch:
the C ABI by its codes (aligned fake pointers, never dereferenced), the binding by
type, shape, stride and size."""
import ctypes

import pytest

P = ctypes.c_void_p
A = P(0x10000)


@pytest.fixture(scope="module")
def tw():
    import __graft_entry__ as g
    g.build()
    import activation_sparse_transformer_gb300 as m
    return m


@pytest.fixture(scope="module")
def lib(tw):
    return tw.load_library()


def kv(tw, **over):
    f = dict(n_pages=8, page_size=64, n_heads=2, head_dim=128, format=0, reserved=0, k=0x10000, v=0x20000,
             k_scale=0x30000, v_scale=0x40000, status=0x50000)
    f.update(over)
    return ctypes.byref(tw.twell_kv_t(*f.values()))


def test_new_status_strings(tw):
    for code in (-10, -11):
        assert tw.status_string(code) not in ("", "unknown status")


PLAN = dict(kv_lens=A, new=P(0x11000), R=4, page=64, n_pages=8, blocks=3, table=A, ring=A, pool=A, pool_out=P(0x12000),
            lens_out=P(0x13000), cu=A, slots=A, positions=A, n_tokens=5, status=A, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(kv_lens=None), -1), (dict(new=None), -1), (dict(lens_out=None), -1), (dict(table=None), -1),
    (dict(ring=None), -1), (dict(pool=None), -1), (dict(pool_out=None), -1), (dict(cu=None), -1),
    (dict(slots=None), -1), (dict(positions=None), -1), (dict(status=None), -1), (dict(R=-1), -1),
    (dict(n_pages=0), -1), (dict(blocks=-1), -1), (dict(n_tokens=-1), -1),
    (dict(lens_out=A), -1), (dict(pool_out=A), -1),                      # read and written: the same buffer
    (dict(page=48), -3), (dict(page=8), -3), (dict(page=256), -3), (dict(R=16385), -3),
    (dict(slots=P(0x10004)), -2), (dict(kv_lens=P(0x10002)), -2), (dict(status=P(0x10001)), -2)])
def test_plan_refuses(lib, over, code):
    assert lib.twell_kv_plan(*{**PLAN, **over}.values()) == code


@pytest.mark.parametrize("over,code", [
    (dict(n_pages=0), -1), (dict(n_heads=0), -1), (dict(head_dim=0), -1), (dict(format=2), -1), (dict(format=-1), -1),
    (dict(reserved=1), -1), (dict(k=0), -1), (dict(v=0), -1), (dict(k_scale=0), -1), (dict(v_scale=0), -1),
    (dict(status=0), -1), (dict(page_size=24), -3), (dict(page_size=256), -3), (dict(head_dim=96), -3),
    (dict(head_dim=256), -3), (dict(k=0x10008), -2), (dict(v=0x10008), -2), (dict(k_scale=0x10002), -2)])
def test_cache_refused_by_append_and_attention(tw, lib, over, code):
    c = kv(tw, **over)
    assert lib.twell_kv_append(A, 256, A, 256, A, A, 3, 2, c, None) == code
    assert lib.twell_kv_attention(A, 1024, c, A, 4, A, A, A, 3, 2, 8, 100, 1, 0.1, A, 1024, A, A, 1 << 30, None) == code


@pytest.mark.parametrize("over,code", [
    (dict(K=None), -1), (dict(V=None), -1), (dict(cu=None), -1), (dict(slots=None), -1), (dict(ldk=248), -1),
    (dict(ldv=260), -1), (dict(n=-1), -1), (dict(R=-1), -1), (dict(K=P(0x10008)), -2), (dict(slots=P(0x10004)), -2),
    (dict(n=2 ** 31 - 1, R=2 ** 31 - 1), -3)])
def test_append_refuses(tw, lib, over, code):
    a = dict(K=A, ldk=256, V=A, ldv=256, cu=A, slots=A, n=3, R=2, cache=kv(tw), stream=None)
    assert lib.twell_kv_append(*{**a, **over}.values()) == code


@pytest.mark.parametrize("over,code", [
    (dict(Q=None), -1), (dict(O=None), -1), (dict(cu=None), -1), (dict(positions=None), -1), (dict(lens=None), -1),
    (dict(table=None), -1), (dict(heads=0), -1), (dict(heads=7), -1), (dict(ldq=1016), -1), (dict(ldo=1028), -1),
    (dict(n=-1), -1), (dict(R=-1), -1), (dict(blocks=-1), -1), (dict(max_kv=-1), -1), (dict(max_q=-1), -1),
    (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=float("nan")), -1), (dict(scale=float("inf")), -1),
    (dict(R=4097), -3), (dict(n=1 << 29), -3), (dict(Q=P(0x10008)), -2), (dict(lse=P(0x10002)), -2),
    (dict(ws=None), -5), (dict(ws_bytes=0), -5), (dict(ws=P(0x10010)), -2)])
def test_attention_refuses(tw, lib, over, code):
    a = dict(Q=A, ldq=1024, cache=kv(tw), table=A, blocks=4, cu=A, positions=A, lens=A, n=3, R=2, heads=8, max_kv=100,
             max_q=1, scale=0.1, O=A, ldo=1024, lse=A, ws=A, ws_bytes=1 << 32, stream=None)
    assert lib.twell_kv_attention(*{**a, **over}.values()) == code


def test_attention_workspace_is_host_arithmetic(tw):
    small = tw.kv_attention_workspace_bytes(16, 16, 32, 8, 128)
    assert small > 0 and small % 256 == 0
    for bad in ((-1, 1, 8, 2, 128), (1, -1, 8, 2, 128), (1, 1, 7, 2, 128), (1, 1, 8, 0, 128), (1, 1, 8, 2, 96)):
        assert tw.kv_attention_workspace_bytes(*bad) == 0


LP = dict(logits=A, dtype=0, ld=100, n=3, vocab=100, targets=A, inv_t=1.0, logprob=A, entropy=A, lse=A, k=5, top=A,
          index=A, stream=None)


@pytest.mark.parametrize("over,code", [
    (dict(logits=None), -1), (dict(dtype=2), -1), (dict(ld=99), -1), (dict(n=-1), -1), (dict(vocab=0), -1),
    (dict(inv_t=0.0), -1), (dict(inv_t=-2.0), -1), (dict(inv_t=float("nan")), -1), (dict(inv_t=float("inf")), -1),
    (dict(targets=None), -1), (dict(logprob=None), -1), (dict(k=-1), -1), (dict(top=None), -1), (dict(index=None), -1),
    (dict(k=33), -3), (dict(k=5, vocab=4), -3), (dict(vocab=400001, ld=400001), -3), (dict(logits=P(0x10008)), -2),
    (dict(lse=P(0x10002)), -2)])
def test_logprobs_refuse(lib, over, code):
    assert lib.twell_logprobs(*{**LP, **over}.values()) == code


@pytest.mark.parametrize("over,code", [
    (dict(logits=None), -1), (dict(lse=None), -1), (dict(out=None), -1), (dict(targets=None), -1), (dict(g=None), -1),
    (dict(entropy=None), -1), (dict(gh=None), -1), (dict(ldd=99), -1), (dict(dtype=-1), -1),
    (dict(out=A, ldd=104), -1),                                          # in place with another row distance
    (dict(out=P(0x20008)), -2), (dict(g=P(0x10001)), -2)])
def test_logprobs_bwd_refuses(lib, over, code):
    a = dict(logits=A, dtype=1, ld=100, n=3, vocab=100, targets=A, inv_t=1.0, lse=A, entropy=A, g=A, gh=A,
             out=P(0x20000), ldd=100, stream=None)
    assert lib.twell_logprobs_bwd(*{**a, **over}.values()) == code


def test_read_status_refuses(tw, lib):
    assert lib.twell_kv_read_status(None, None) == -1
    assert lib.twell_kv_read_status(kv(tw, status=0), None) == -1


def test_binding_checks_types_shapes_and_sizes(tw):
    """CPU tensors: everything else is refused before they are."""
    import torch
    i32, bf = torch.int32, torch.bfloat16
    with pytest.raises(ValueError, match="k, v"):
        tw.KVCache(*(torch.empty((2, 1, 16, 64), dtype=torch.uint8) for _ in range(2)), torch.empty((2, 1)),
                   torch.empty((2, 1)), torch.empty(1, dtype=i32))
    with pytest.raises(ValueError, match="k_scale"):
        tw.KVCache(*(torch.empty((2, 1, 16, 64), dtype=torch.int8) for _ in range(2)), torch.empty(1),
                   torch.empty((2, 1)), torch.empty(1, dtype=i32))
    cache = tw.alloc_kv_cache(4, 16, 2, 64, tw.KV_INT8, "cpu")
    plan = tw.alloc_kv_plan(3, 5, "cpu")
    ring, pool = tw.alloc_page_ring(4, "cpu")
    lens = torch.zeros(3, dtype=i32)
    with pytest.raises(ValueError, match="^new_tokens"):
        tw.twell_kv_plan(lens, lens.long(), torch.zeros((3, 2), dtype=i32), ring, pool, 16, plan)
    with pytest.raises(ValueError, match="^block_table"):
        tw.twell_kv_plan(lens, lens, torch.zeros((2, 2), dtype=i32), ring, pool, 16, plan)
    with pytest.raises(ValueError, match="CUDA"):
        tw.twell_kv_plan(lens, lens, torch.zeros((3, 2), dtype=i32), ring, pool, 16, plan)
    x = torch.zeros((5, 2, 64), dtype=bf)
    with pytest.raises(ValueError, match="^K: torch.float32"):
        tw.twell_kv_append(x.float(), x, plan.cu_q, plan.slots, cache)
    with pytest.raises(ValueError, match="CUDA"):
        tw.twell_kv_append(x, x, plan.cu_q, plan.slots, cache)
    with pytest.raises(ValueError, match="^Q: torch.float16"):
        tw.twell_kv_attention(x.half(), cache, torch.zeros((3, 2), dtype=i32), plan.cu_q, plan.positions, lens, 16, 1,
                              0.1, x, torch.empty(256, dtype=torch.uint8))
    logits, f = torch.zeros((3, 10), dtype=torch.float16), torch.zeros(3)
    with pytest.raises(ValueError, match="^logits"):
        tw.twell_logprobs(logits, lens, 1.0, f, f, f)
    with pytest.raises(ValueError, match="^logits"):
        tw.twell_logprobs_bwd(logits, lens, 1.0, f, f, f, f, logits)
