"""Python binding of libtwell.so, the TwELL activation-sparse FFN for GB300.

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels (include/twell.h documents each call).  torch supplies device memory
and the current stream; bf16 tensors are passed by pointer.  If the library
has not been built, every call raises -- there is no CPU or eager fallback.

One training step of a layer (X [N, d] bf16; W_inT, W_down [f, d] bf16; b [f]
bf16; T the tile width, C the per-tile capacity, fb_cap the dense fallback
rows):

    import activation_sparse_transformer_gb300 as tw
    H = tw.alloc_packed(N, f, T, C, fb_cap, "cuda")      # the packed activations
    ws = torch.empty(max(tw.fwd_workspace_bytes(N, d, f, T, C, fb_cap),
                         tw.bwd_workspace_bytes(N, d, f, T, C, fb_cap)),
                     dtype=torch.uint8, device="cuda")      # one scratch for both calls
    tw.twell_ffn_fwd(X, W_inT, b, W_down, H, Y, ws)          # Y [N, d] bf16
    tw.twell_ffn_bwd(X, W_inT, W_down, H, dY, l1_lambda,     # dX bf16; dW_inT, dW_down,
                     dX, dW_inT, dW_down, db, ws)           # db fp32
    assert tw.twell_read_status(H) == 0                      # e.g. fallback overflow

The calls are asynchronous on the current stream and can be captured in a CUDA
graph; twell_pack / twell_unpack convert between dense bf16 H and the packed form.

One decode step around the layer (R requests, each with new tokens; examples/decode_step.py
runs it whole):

    cache = tw.alloc_kv_cache(n_pages, 64, kv_heads, 128, tw.KV_E4M3, "cuda")
    plan = tw.alloc_kv_plan(R, n_tokens, "cuda")
    tw.twell_kv_plan(kv_lens, new_tokens, block_table, ring, pool, 64, plan)
    tw.twell_kv_append(K, V, plan.cu_q, plan.slots, cache)       # [n_tokens, kv_heads, 128] bf16
    tw.twell_kv_attention(Q, cache, block_table, plan.cu_q, plan.positions, plan.kv_lens, max_kv_len,
                          max_q_len, 128 ** -0.5, O, workspace)  # [n_tokens, q_heads, 128] bf16
    ...                                                          # the sparse layer, the output projection
    tw.twell_logprobs(logits, targets, 1.0, logprob, entropy, lse, top_logprob, top_index)
    tw.twell_logprobs_bwd(logits, targets, 1.0, lse, entropy, d_logprob, d_entropy, d_logits)
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass
from typing import Optional

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtwell.so")

TWELL_OK = 0
KERNELS = {
    "up_pack": 0, "route": 1, "fb_assemble": 2, "spmm": 4, "fb_down": 5, "pack": 6,
    "check_format": 3, "unpack": 7, "sddmm": 8, "dx": 9, "dw": 10, "dense_gemm": 11, "aux": 12,
    "dw_fallback": 13, "dx_fallback": 14, "kv_plan": 15, "kv_append": 16, "kv_attention": 17,
    "kv_join": 18, "logprobs": 19, "logprobs_bwd": 20,
}
EXPORTED = [
    "twell_pack", "twell_unpack", "twell_ffn_fwd", "twell_fwd_workspace_bytes", "twell_ffn_bwd",
    "twell_bwd_workspace_bytes", "twell_dense_ffn_fwd", "twell_read_status", "twell_status_string",
    "twell_launch_count", "twell_profile_enable", "twell_profile_reset", "twell_profile_read",
    "twell_profile_timeline",
    "twell_ffn_fwd_noalloc", "twell_ffn_fwd_noalloc_max_scratch", "twell_gated_ffn_fwd",
    "twell_selftest_wait_timeout", "twell_check_format", "twell_dense_ffn_bwd", "twell_dense_bwd_workspace_bytes",
    "twell_bwd_tiles_workspace_bytes", "twell_gated_ffn_fwd_train", "twell_gated_ffn_bwd",
    "twell_gated_bwd_workspace_bytes", "twell_gated_bwd_tiles_workspace_bytes",
    "twell_kv_plan", "twell_kv_append", "twell_kv_attention", "twell_kv_attention_workspace_bytes",
    "twell_kv_read_status", "twell_logprobs", "twell_logprobs_bwd", "twell_selftest_kv_attention_stall",
]


class TwellError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} ({code})")


class twell_t(ctypes.Structure):
    _fields_ = [
        ("n_rows", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("tile", ctypes.c_int32),
        ("cap", ctypes.c_int32), ("fb_cap", ctypes.c_int32), ("hybrid", ctypes.c_int32),
        ("values", ctypes.c_void_p), ("idx", ctypes.c_void_p), ("counts", ctypes.c_void_p),
        ("row_fb", ctypes.c_void_p), ("fb_rows", ctypes.c_void_p), ("fb_dense", ctypes.c_void_p),
        ("n_fb", ctypes.c_void_p), ("status", ctypes.c_void_p),
    ]


class twell_kv_t(ctypes.Structure):
    _fields_ = [
        ("n_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("n_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("format", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p),
        ("status", ctypes.c_void_p),
    ]


_lib_handle = None


def load_library() -> ctypes.CDLL:
    """Loads libtwell.so; raises if it is missing (build it with __graft_entry__.build())."""
    global _lib_handle
    if _lib_handle is not None:
        return _lib_handle
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    L = ctypes.POINTER(twell_t)
    KV = ctypes.POINTER(twell_kv_t)
    sig = {
        "twell_pack": (ctypes.c_int, [P, I64, L, P]),
        "twell_unpack": (ctypes.c_int, [L, P, I64, P]),
        "twell_ffn_fwd": (ctypes.c_int, [P, P, P, P, I32, I32, I32, L, P, P, SZ, P]),
        "twell_fwd_workspace_bytes": (SZ, [I32, I32, I32, I32, I32, I32]),
        "twell_ffn_bwd": (ctypes.c_int, [P, P, P, L, I32, P, ctypes.c_float, P, P, P, P, P, SZ, P]),
        "twell_bwd_workspace_bytes": (SZ, [I32, I32, I32, I32, I32, I32]),
        "twell_bwd_tiles_workspace_bytes": (SZ, [I32, I32, I32, I32, I32, I32]),
        "twell_dense_ffn_fwd": (ctypes.c_int, [P, P, P, P, I32, I32, I32, P, P, P]),
        "twell_read_status": (ctypes.c_int, [L, P]),
        "twell_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "twell_launch_count": (I64, []),
        "twell_profile_enable": (ctypes.c_int, [ctypes.c_int]),
        "twell_profile_reset": (ctypes.c_int, []),
        "twell_profile_read": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(I64), ctypes.POINTER(ctypes.c_double)]),
        "twell_profile_timeline": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(ctypes.c_int32),
                                                  ctypes.POINTER(ctypes.c_uint64), ctypes.POINTER(ctypes.c_double),
                                                  ctypes.POINTER(ctypes.c_double)]),
        "twell_ffn_fwd_noalloc": (ctypes.c_int, [P, P, P, P, I32, I32, I32, L, P, P]),
        "twell_ffn_fwd_noalloc_max_scratch": (SZ, []),
        "twell_gated_ffn_fwd": (ctypes.c_int, [P, P, P, P, P, I32, I32, I32, L, P, P, SZ, P]),
        "twell_gated_ffn_fwd_train": (ctypes.c_int, [P, P, P, P, P, I32, I32, I32, L, P, P, P, SZ, P]),
        "twell_gated_ffn_bwd": (ctypes.c_int, [P, P, P, P, P, L, P, I32, P, ctypes.c_float, P, P, P, P, P, P, SZ,
                                               P]),
        "twell_gated_bwd_workspace_bytes": (SZ, [I32, I32, I32, I32, I32, I32]),
        "twell_gated_bwd_tiles_workspace_bytes": (SZ, [I32, I32, I32, I32, I32, I32]),
        "twell_selftest_wait_timeout": (ctypes.c_int, [P, ctypes.c_uint64, P]),
        "twell_check_format": (ctypes.c_int, [L, P, P]),
        "twell_dense_ffn_bwd": (ctypes.c_int, [P, P, P, P, I32, I32, I32, P, ctypes.c_float, P, P, P, P, P, SZ, P]),
        "twell_dense_bwd_workspace_bytes": (SZ, [I32, I32, I32]),
        "twell_kv_plan": (ctypes.c_int, [P, P, I32, I32, I32, I32, P, P, P, P, P, P, P, P, I32, P, P]),
        "twell_kv_append": (ctypes.c_int, [P, I64, P, I64, P, P, I32, I32, KV, P]),
        "twell_kv_attention": (ctypes.c_int, [P, I64, KV, P, I32, P, P, P, I32, I32, I32, I32, I32, ctypes.c_float, P,
                                              I64, P, P, SZ, P]),
        "twell_selftest_kv_attention_stall": (ctypes.c_int, [P, I64, KV, P, I32, P, P, P, I32, I32, I32, I32, I32,
                                                             ctypes.c_float, P, I64, P, P, SZ, ctypes.c_uint64, P]),
        "twell_kv_attention_workspace_bytes": (SZ, [I32, I32, I32, I32, I32]),
        "twell_kv_read_status": (ctypes.c_int, [KV, P]),
        "twell_logprobs": (ctypes.c_int, [P, I32, I64, I32, I32, P, ctypes.c_float, P, P, P, I32, P, P, P]),
        "twell_logprobs_bwd": (ctypes.c_int, [P, I32, I64, I32, I32, P, ctypes.c_float, P, P, P, P, P, I64, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib_handle = lib
    return lib


def status_string(code: int) -> str:
    return load_library().twell_status_string(int(code)).decode()


def _check(code: int, where: str) -> None:
    if code != TWELL_OK:
        raise TwellError(code, where)


def _stream(stream=None) -> int:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _need(t, nbytes: int, name: str) -> None:
    """Rejects a buffer smaller than the bytes the call reads or writes through
    it (the C ABI receives only the pointer)."""
    have = 0 if t is None else t.numel() * t.element_size()
    if have < nbytes:
        raise ValueError(f"{name}: {have} bytes, the call needs {nbytes}")


def _need_dense(t, rows: int, row_elems: int, ld: int, elem_bytes: int, name: str) -> None:
    """A [rows][ld] buffer of which the first row_elems of every row are used."""
    _need(t, ((rows - 1) * ld + row_elems) * elem_bytes if rows > 0 else 0, name)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if not (t.is_cuda and t.is_contiguous()):
        raise ValueError("tensors passed to libtwell must be contiguous CUDA tensors")
    return t.data_ptr()


@dataclass
class Packed:
    """Device buffers of one TwELL hybrid layout and the twell_t that names them."""
    values: "object"
    idx: "object"
    counts: "object"
    row_fb: "object"
    fb_rows: "object"
    fb_dense: "object"
    n_fb: "object"
    status: "object"
    n_rows: int
    d_ff: int
    tile: int
    cap: int
    fb_cap: int
    hybrid: int = 0   # HYBRID_ROWS or HYBRID_TILES

    def struct(self) -> twell_t:
        N, nt = self.n_rows, self.d_ff // self.tile
        cells = N * nt
        _need(self.values, cells * self.cap * 2, "values")
        _need(self.idx, cells * self.cap, "idx")
        _need(self.counts, cells, "counts")
        _need(self.row_fb, N * 4, "row_fb")
        _need(self.fb_rows, self.fb_cap * 4, "fb_rows")
        _need(self.fb_dense, self.fb_cap * self.d_ff * 2, "fb_dense")
        _need(self.n_fb, 4, "n_fb")
        _need(self.status, 4, "status")
        p = lambda t: t.data_ptr() if t is not None and t.numel() else None
        return twell_t(self.n_rows, self.d_ff, self.tile, self.cap, self.fb_cap, self.hybrid,
                       p(self.values), p(self.idx), p(self.counts), p(self.row_fb), p(self.fb_rows),
                       p(self.fb_dense), p(self.n_fb), p(self.status))


HYBRID_ROWS, HYBRID_TILES, DENSE_TILE = 0, 1, 255


def alloc_packed(n_rows: int, d_ff: int, tile: int, cap: int, fb_cap: int, device="cuda",
                 hybrid: int = HYBRID_ROWS) -> Packed:
    """Buffers of a packed layer.  With hybrid=HYBRID_TILES, fb_dense is the pool
    of fb_cap * d_ff / tile dense tiles."""
    import torch
    nt = d_ff // tile
    kw = dict(device=device)
    return Packed(
        values=torch.empty((n_rows, nt, cap), dtype=torch.bfloat16, **kw),
        idx=torch.empty((n_rows, nt, cap), dtype=torch.uint8, **kw),
        counts=torch.empty((n_rows, nt), dtype=torch.uint8, **kw),
        row_fb=torch.empty((max(n_rows, 1),), dtype=torch.int32, **kw),
        fb_rows=torch.empty((max(fb_cap, 1),), dtype=torch.int32, **kw),
        fb_dense=torch.empty((max(fb_cap, 1), d_ff), dtype=torch.bfloat16, **kw),
        n_fb=torch.zeros((4,), dtype=torch.int32, **kw),
        status=torch.zeros((4,), dtype=torch.int32, **kw),
        n_rows=n_rows, d_ff=d_ff, tile=tile, cap=cap, fb_cap=fb_cap, hybrid=hybrid,
    )


def twell_pack(H, packed: Packed, stream=None) -> None:
    """Dense bf16 H [n_rows, >= d_ff] -> TwELL hybrid (asynchronous)."""
    _need_dense(H, packed.n_rows, packed.d_ff, H.stride(0), 2, "H")
    st = packed.struct()
    _check(load_library().twell_pack(_ptr(H), H.stride(0), ctypes.byref(st), _stream(stream)), "twell_pack")


def twell_unpack(packed: Packed, H, stream=None) -> None:
    _need_dense(H, packed.n_rows, packed.d_ff, H.stride(0), 2, "H")
    st = packed.struct()
    _check(load_library().twell_unpack(ctypes.byref(st), _ptr(H), H.stride(0), _stream(stream)), "twell_unpack")


def fwd_workspace_bytes(n_rows, d_model, d_ff, tile, cap, fb_cap) -> int:
    return int(load_library().twell_fwd_workspace_bytes(n_rows, d_model, d_ff, tile, cap, fb_cap))


def bwd_workspace_bytes(n_rows, d_model, d_ff, tile, cap, fb_cap, hybrid=None) -> int:
    """Workspace of twell_ffn_bwd; hybrid=HYBRID_TILES for a tile-granular layout."""
    lib = load_library()
    fn = lib.twell_bwd_tiles_workspace_bytes if hybrid == HYBRID_TILES else lib.twell_bwd_workspace_bytes
    return int(fn(n_rows, d_model, d_ff, tile, cap, fb_cap))


def _need_layer(n, d, f, W_inT, b, W_down, Y) -> None:
    _need(W_inT, f * d * 2, "W_inT")
    _need(b, f * 2, "b")
    _need(W_down, f * d * 2, "W_down")
    _need(Y, n * d * 2, "Y")


def twell_ffn_fwd(X, W_inT, b, W_down, packed: Packed, Y, workspace, stream=None) -> None:
    n, d = X.shape
    f = W_inT.shape[0]
    _need_layer(n, d, f, W_inT, b, W_down, Y)
    st = packed.struct()
    _check(load_library().twell_ffn_fwd(_ptr(X), _ptr(W_inT), _ptr(b), _ptr(W_down), n, d, f, ctypes.byref(st),
                                        _ptr(Y), _ptr(workspace), workspace.numel() * workspace.element_size(),
                                        _stream(stream)), "twell_ffn_fwd")


def twell_gated_ffn_fwd(X, W_gT, W_uT, b, W_down, packed: Packed, Y, workspace, stream=None) -> None:
    """Gated ReLU layer: H = ReLU(X.W_g + b) * (X.W_u) packed in TwELL, Y = H.W_down."""
    n, d = X.shape
    f = W_gT.shape[0]
    _need_layer(n, d, f, W_gT, b, W_down, Y)
    _need(W_uT, f * d * 2, "W_uT")
    st = packed.struct()
    _check(load_library().twell_gated_ffn_fwd(_ptr(X), _ptr(W_gT), _ptr(W_uT), _ptr(b), _ptr(W_down), n, d, f,
                                              ctypes.byref(st), _ptr(Y), _ptr(workspace),
                                              workspace.numel() * workspace.element_size(), _stream(stream)),
           "twell_gated_ffn_fwd")


def twell_gated_ffn_fwd_train(X, W_gT, W_uT, b, W_down, packed: Packed, Y, gu, workspace, stream=None) -> None:
    """twell_gated_ffn_fwd that also keeps (g, u) fp32 at every stored slot in gu
    ([n_rows][d_ff / tile][cap][2] float32), for twell_gated_ffn_bwd."""
    n, d = X.shape
    f = W_gT.shape[0]
    _need_layer(n, d, f, W_gT, b, W_down, Y)
    _need(W_uT, f * d * 2, "W_uT")
    _need(gu, n * (f // packed.tile) * packed.cap * 8, "gu")
    st = packed.struct()
    _check(load_library().twell_gated_ffn_fwd_train(_ptr(X), _ptr(W_gT), _ptr(W_uT), _ptr(b), _ptr(W_down), n, d,
                                                    f, ctypes.byref(st), _ptr(Y), _ptr(gu), _ptr(workspace),
                                                    workspace.numel() * workspace.element_size(), _stream(stream)),
           "twell_gated_ffn_fwd_train")


def twell_ffn_fwd_noalloc(X, W_inT, b, W_down, packed: Packed, Y, stream=None) -> None:
    """twell_ffn_fwd without a workspace argument: the library's fixed scratch
    array is used (for callers that cannot allocate device memory)."""
    n, d = X.shape
    f = W_inT.shape[0]
    _need_layer(n, d, f, W_inT, b, W_down, Y)
    st = packed.struct()
    _check(load_library().twell_ffn_fwd_noalloc(_ptr(X), _ptr(W_inT), _ptr(b), _ptr(W_down), n, d, f,
                                                ctypes.byref(st), _ptr(Y), _stream(stream)),
           "twell_ffn_fwd_noalloc")


def twell_ffn_bwd(X, W_inT, W_down, packed: Packed, dY, l1_lambda: float, dX, dW_inT, dW_down, db, workspace,
                  stream=None) -> None:
    d = X.shape[1]
    n, f = packed.n_rows, packed.d_ff
    for t, nbytes, name in ((X, n * d * 2, "X"), (W_inT, f * d * 2, "W_inT"), (W_down, f * d * 2, "W_down"),
                            (dY, n * d * 2, "dY"), (dX, n * d * 2, "dX"), (dW_inT, f * d * 4, "dW_inT"),
                            (dW_down, f * d * 4, "dW_down"), (db, f * 4, "db")):
        _need(t, nbytes, name)
    st = packed.struct()
    _check(load_library().twell_ffn_bwd(_ptr(X), _ptr(W_inT), _ptr(W_down), ctypes.byref(st), d, _ptr(dY),
                                        float(l1_lambda), _ptr(dX), _ptr(dW_inT), _ptr(dW_down), _ptr(db),
                                        _ptr(workspace), workspace.numel() * workspace.element_size(),
                                        _stream(stream)), "twell_ffn_bwd")


def gated_bwd_workspace_bytes(n_rows, d_model, d_ff, tile, cap, fb_cap, hybrid=None) -> int:
    """Workspace of twell_gated_ffn_bwd; hybrid=HYBRID_TILES for a tile-granular layout."""
    lib = load_library()
    fn = lib.twell_gated_bwd_tiles_workspace_bytes if hybrid == HYBRID_TILES else lib.twell_gated_bwd_workspace_bytes
    return int(fn(n_rows, d_model, d_ff, tile, cap, fb_cap))


def twell_gated_ffn_bwd(X, W_gT, W_uT, b, W_down, packed: Packed, gu, dY, l1_lambda: float, dX, dW_gT, dW_uT,
                        dW_down, db, workspace, stream=None) -> None:
    """Backward of the gated layer; gu is what twell_gated_ffn_fwd_train kept."""
    d = X.shape[1]
    n, f = packed.n_rows, packed.d_ff
    for t, nbytes, name in ((X, n * d * 2, "X"), (W_gT, f * d * 2, "W_gT"), (W_uT, f * d * 2, "W_uT"),
                            (b, f * 2, "b"), (W_down, f * d * 2, "W_down"),
                            (gu, n * (f // packed.tile) * packed.cap * 8, "gu"), (dY, n * d * 2, "dY"),
                            (dX, n * d * 2, "dX"), (dW_gT, f * d * 4, "dW_gT"), (dW_uT, f * d * 4, "dW_uT"),
                            (dW_down, f * d * 4, "dW_down"), (db, f * 4, "db")):
        _need(t, nbytes, name)
    st = packed.struct()
    _check(load_library().twell_gated_ffn_bwd(_ptr(X), _ptr(W_gT), _ptr(W_uT), _ptr(b), _ptr(W_down),
                                              ctypes.byref(st), _ptr(gu), d, _ptr(dY), float(l1_lambda), _ptr(dX),
                                              _ptr(dW_gT), _ptr(dW_uT), _ptr(dW_down), _ptr(db), _ptr(workspace),
                                              workspace.numel() * workspace.element_size(), _stream(stream)),
           "twell_gated_ffn_bwd")


def twell_dense_ffn_fwd(X, W_inT, b, W_down, Hbuf, Y, stream=None) -> None:
    """Dense comparator: Y = ReLU(X.W_in + b).W_down on the same tensor-core GEMM."""
    n, d = X.shape
    f = W_inT.shape[0]
    _need_layer(n, d, f, W_inT, b, W_down, Y)
    _need(Hbuf, n * f * 2, "Hbuf")
    _check(load_library().twell_dense_ffn_fwd(_ptr(X), _ptr(W_inT), _ptr(b), _ptr(W_down), n, d, f, _ptr(Hbuf),
                                              _ptr(Y), _stream(stream)), "twell_dense_ffn_fwd")


def dense_bwd_workspace_bytes(n_rows, d_model, d_ff) -> int:
    return int(load_library().twell_dense_bwd_workspace_bytes(n_rows, d_model, d_ff))


def twell_dense_ffn_bwd(X, W_inT, W_down, Hbuf, dY, l1_lambda: float, dX, dW_inT, dW_down, db, workspace,
                        stream=None) -> None:
    """Dense comparator's backward: the gradients of twell_ffn_bwd for the layer
    run densely (Hbuf = the dense forward's H), with no sparsity used."""
    n, d = X.shape
    f = W_inT.shape[0]
    for t, nbytes, name in ((X, n * d * 2, "X"), (W_inT, f * d * 2, "W_inT"), (W_down, f * d * 2, "W_down"),
                            (Hbuf, n * f * 2, "Hbuf"), (dY, n * d * 2, "dY"), (dX, n * d * 2, "dX"),
                            (dW_inT, f * d * 4, "dW_inT"), (dW_down, f * d * 4, "dW_down"), (db, f * 4, "db"),
                            (workspace, dense_bwd_workspace_bytes(n, d, f), "workspace")):
        _need(t, nbytes, name)
    _check(load_library().twell_dense_ffn_bwd(_ptr(X), _ptr(W_inT), _ptr(W_down), _ptr(Hbuf), n, d, f, _ptr(dY),
                                              float(l1_lambda), _ptr(dX), _ptr(dW_inT), _ptr(dW_down), _ptr(db),
                                              _ptr(workspace), workspace.numel() * workspace.element_size(),
                                              _stream(stream)), "twell_dense_ffn_bwd")


def twell_check_format(packed: Packed, violations, stream=None) -> None:
    """Check the layout's format rules on the device (asynchronous): bit k of
    the device int32 tensor `violations` is set when rule k is broken."""
    _need(violations, 4, "violations")
    st = packed.struct()
    _check(load_library().twell_check_format(ctypes.byref(st), _ptr(violations), _stream(stream)),
           "twell_check_format")


def twell_read_status(packed: Packed, stream=None) -> int:
    st = packed.struct()
    return int(load_library().twell_read_status(ctypes.byref(st), _stream(stream)))


def twell_selftest_wait_timeout(status, limit_ns: int, stream=None) -> None:
    """Run the pipelines' bounded wait on a barrier nothing arrives on; status
    (a device int32 tensor) becomes TWELL_ERR_WAIT_TIMEOUT once limit_ns pass."""
    _check(load_library().twell_selftest_wait_timeout(_ptr(status), int(limit_ns), _stream(stream)),
           "twell_selftest_wait_timeout")


def twell_launch_count() -> int:
    return int(load_library().twell_launch_count())


def twell_profile_enable(on: bool) -> None:
    _check(load_library().twell_profile_enable(1 if on else 0), "twell_profile_enable")


def twell_profile_reset() -> None:
    _check(load_library().twell_profile_reset(), "twell_profile_reset")


def twell_profile_timeline(max_entries: int = 4096) -> list:
    """Recorded launches in order: dicts with kernel (name), stream, start_ms,
    end_ms (device times relative to the first recorded launch)."""
    k = (ctypes.c_int32 * max_entries)()
    st = (ctypes.c_uint64 * max_entries)()
    a = (ctypes.c_double * max_entries)()
    b = (ctypes.c_double * max_entries)()
    n = load_library().twell_profile_timeline(max_entries, k, st, a, b)
    _check(min(n, 0), "twell_profile_timeline")
    names = {v: name for name, v in KERNELS.items()}
    return [{"kernel": names.get(k[i], str(k[i])), "stream": int(st[i]), "start_ms": a[i], "end_ms": b[i]}
            for i in range(n)]


def twell_profile_read(kernel) -> tuple:
    """(launches, total_ms) of one kernel id or name since the last reset."""
    k = KERNELS[kernel] if isinstance(kernel, str) else int(kernel)
    n = ctypes.c_int64(0)
    ms = ctypes.c_double(0.0)
    _check(load_library().twell_profile_read(k, ctypes.byref(n), ctypes.byref(ms)), "twell_profile_read")
    return int(n.value), float(ms.value)


# ---------------------------------------------------------------- decode step
KV_E4M3, KV_INT8 = 0, 1
_torch = None
_raw_stream = None


def _setup():
    """torch, imported at the first call, and the current stream's handle without
    the Stream object around it (these calls are as short as the kernels they start)."""
    global _torch, _raw_stream
    import torch
    get = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _raw_stream = ((lambda: get(torch._C._cuda_getDevice())) if get is not None
                   else (lambda: torch.cuda.current_stream().cuda_stream))
    _torch = torch
    return torch


def _on(stream) -> int:
    return _raw_stream() if stream is None else int(stream.cuda_stream)


def _arg(t, dtype, n: int, name: str) -> int:
    """The address of a contiguous tensor of dtype with at least n elements; that
    it is on the device is looked at last, by _on_device."""
    if t.dtype != dtype:
        raise ValueError(f"{name}: {t.dtype}, the call takes {dtype}")
    if t.numel() < n:
        raise ValueError(f"{name}: {t.numel()} elements, the call needs {n}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor")
    return t.data_ptr()


def _on_device(*tensors) -> None:
    for t in tensors:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors passed to libtwell must be CUDA tensors")


def _maybe(t, dtype, n: int, name: str):
    return None if t is None else _arg(t, dtype, n, name)


def _need_rows(t, dtype, heads: int, dim: int, name: str) -> int:
    """The distance between the tokens of a device tensor [tokens, heads, dim], which
    may be a slice of wider rows but holds each token in one piece."""
    if t.dtype != dtype:
        raise ValueError(f"{name}: {t.dtype}, the call takes {dtype}")
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name}: shape {tuple(shape)}, the call takes [tokens, {heads}, {dim}]")
    if (stride[2] != 1 and dim > 1) or (stride[1] != dim and heads > 1):
        raise ValueError(f"{name}: strides {tuple(stride)}, a token's {heads * dim} elements must lie together")
    return stride[0] if shape[0] > 1 else max(stride[0], heads * dim)


@dataclass(frozen=True)
class KVCache:
    """An 8-bit paged cache: k and v [n_pages, n_heads, page_size, head_dim] of
    torch.float8_e4m3fn or torch.int8, k_scale and v_scale [n_pages, n_heads]
    float32, status int32.  The buffers stay the caller's."""
    k: "object"
    v: "object"
    k_scale: "object"
    v_scale: "object"
    status: "object"

    def __post_init__(self):
        self._check()

    def _check(self):
        torch = _torch or _setup()
        formats = {torch.float8_e4m3fn: KV_E4M3, torch.int8: KV_INT8}
        if self.k.dtype not in formats or self.v.dtype != self.k.dtype:
            raise ValueError(f"k, v: {self.k.dtype}, {self.v.dtype}; a cache holds float8_e4m3fn or int8")
        if self.k.dim() != 4 or self.v.shape != self.k.shape:
            raise ValueError(f"k, v: shapes {tuple(self.k.shape)}, {tuple(self.v.shape)}")
        keep = dict(zip(("n_pages", "n_heads", "page_size", "head_dim"), self.k.shape), format=formats[self.k.dtype],
                    _struct=None, _at=None)
        for t, name in ((self.k_scale, "k_scale"), (self.v_scale, "v_scale")):
            if t.dtype != torch.float32 or t.numel() < keep["n_pages"] * keep["n_heads"]:
                raise ValueError(f"{name}: {t.numel()} elements of {t.dtype}, a cache needs [n_pages, n_heads] float32")
        if self.status.dtype != torch.int32 or self.status.numel() < 1:
            raise ValueError("status: an int32 tensor")
        for name, value in keep.items():
            object.__setattr__(self, name, value)

    def struct(self):
        # looked at anew when a buffer has moved (set_, resize_): the storage is where it is now
        at = (self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr(),
              self.status.data_ptr())
        if at != self._at:
            pages = (self.n_heads, self.page_size, self.head_dim)
            self._check()
            if (self.n_heads, self.page_size, self.head_dim) != pages:
                raise ValueError(f"k, v: pages of {tuple(self.k.shape[1:])}, the cache was made of pages of {pages}")
            object.__setattr__(self, "_struct", ctypes.pointer(twell_kv_t(
                self.n_pages, self.page_size, self.n_heads, self.head_dim, self.format, 0, _ptr(self.k),
                _ptr(self.v), _ptr(self.k_scale), _ptr(self.v_scale), _ptr(self.status))))
            object.__setattr__(self, "_at", at)
        return self._struct


def alloc_kv_cache(n_pages: int, page_size: int, n_heads: int, head_dim: int, fmt: int = KV_E4M3,
                   device="cuda") -> KVCache:
    torch = _torch or _setup()
    shape, dt = (n_pages, n_heads, page_size, head_dim), (torch.float8_e4m3fn if fmt == KV_E4M3 else torch.int8)
    return KVCache(k=torch.empty(shape, dtype=dt, device=device), v=torch.empty(shape, dtype=dt, device=device),
                   k_scale=torch.zeros(shape[:2], dtype=torch.float32, device=device),
                   v_scale=torch.zeros(shape[:2], dtype=torch.float32, device=device),
                   status=torch.zeros((4,), dtype=torch.int32, device=device))


@dataclass(frozen=True)
class KVPlan:
    """What twell_kv_plan writes: kv_lens [R], cu_q [R + 1], slots [n_tokens]
    int64, positions [n_tokens], pool [2] (for the next step's plan), status."""
    kv_lens: "object"
    cu_q: "object"
    slots: "object"
    positions: "object"
    pool: "object"
    status: "object"

    def _outputs(self) -> tuple:
        """(requests, tokens, addresses in the call's order, status), checked when a buffer has moved."""
        at = (self.kv_lens.data_ptr(), self.cu_q.data_ptr(), self.slots.data_ptr(), self.positions.data_ptr(),
              self.pool.data_ptr(), self.status.data_ptr())
        kept = self.__dict__.get("_kept")
        if kept is None or kept[4] != at:
            i32, R, n = _torch.int32, self.kv_lens.numel(), self.slots.numel()
            kept = (R, n, (_arg(self.pool, i32, 2, "plan.pool"), _arg(self.kv_lens, i32, R, "plan.kv_lens"),
                           _arg(self.cu_q, i32, R + 1, "plan.cu_q"),
                           _arg(self.slots, _torch.int64, n, "plan.slots"),
                           _arg(self.positions, i32, n, "plan.positions")), _arg(self.status, i32, 1, "plan.status"),
                    at)
            _on_device(self.pool, self.kv_lens, self.cu_q, self.slots, self.positions, self.status)
            object.__setattr__(self, "_kept", kept)
        return kept


def alloc_kv_plan(n_requests: int, n_tokens: int, device="cuda") -> KVPlan:
    torch = _torch or _setup()
    i32 = lambda n: torch.zeros((n,), dtype=torch.int32, device=device)  # noqa: E731
    return KVPlan(kv_lens=i32(n_requests), cu_q=i32(n_requests + 1),
                  slots=torch.zeros((n_tokens,), dtype=torch.int64, device=device), positions=i32(n_tokens),
                  pool=i32(2), status=i32(4))


def alloc_page_ring(n_pages: int, device="cuda") -> tuple:
    """(ring, pool) of a cache whose pages are all free."""
    torch = _torch or _setup()
    return (torch.arange(n_pages, dtype=torch.int32, device=device),
            torch.tensor([0, n_pages], dtype=torch.int32, device=device))


def _table(block_table, R: int) -> tuple:
    if block_table.dim() != 2:
        raise ValueError("block_table: the call takes [requests, blocks]")
    width = block_table.shape[1]
    return _arg(block_table, _torch.int32, R * width, "block_table"), width


def twell_kv_plan(kv_lens, new_tokens, block_table, ring, pool, page_size: int, plan: KVPlan, stream=None) -> None:
    """Block tables and slot maps of one step; the pages are ring.numel()."""
    i32 = (_torch or _setup()).int32
    R = kv_lens.numel()
    lens_p, new_p = _arg(kv_lens, i32, R, "kv_lens"), _arg(new_tokens, i32, R, "new_tokens")
    table, width = _table(block_table, R)
    ring_p, pool_p = _arg(ring, i32, 1, "ring"), _arg(pool, i32, 2, "pool")
    _on_device(kv_lens, new_tokens, block_table, ring, pool)
    rows, n_tokens, out, status, _ = plan._outputs()
    if rows != R:
        raise ValueError(f"plan: {rows} requests, kv_lens has {R}")
    rc = load_library().twell_kv_plan(lens_p, new_p, R, page_size, ring.numel(), width, table, ring_p,
                                      pool_p, *out, n_tokens, status, _on(stream))
    if rc:
        _check(rc, "twell_kv_plan")


def twell_kv_append(K, V, cu_q, slots, cache: KVCache, stream=None) -> None:
    """Keys and values [n_tokens, n_heads, head_dim] bf16 into the cache's slots."""
    torch = _torch or _setup()
    ldk = _need_rows(K, torch.bfloat16, cache.n_heads, cache.head_dim, "K")
    ldv = _need_rows(V, torch.bfloat16, cache.n_heads, cache.head_dim, "V")
    n = K.shape[0]
    if V.shape[0] != n:
        raise ValueError(f"V: {V.shape[0]} tokens, K has {n}")
    cu, at = _arg(cu_q, torch.int32, 1, "cu_q"), _arg(slots, torch.int64, n, "slots")
    _on_device(K, V, cu_q, slots)
    rc = load_library().twell_kv_append(K.data_ptr(), ldk, V.data_ptr(), ldv, cu, at, n, cu_q.numel() - 1,
                                        cache.struct(), _on(stream))
    if rc:
        _check(rc, "twell_kv_append")


def kv_attention_workspace_bytes(n_tokens, n_requests, n_q_heads, n_kv_heads, head_dim) -> int:
    return int(load_library().twell_kv_attention_workspace_bytes(n_tokens, n_requests, n_q_heads, n_kv_heads,
                                                                 head_dim))


def twell_kv_attention(Q, cache: KVCache, block_table, cu_q, positions, kv_lens, max_kv_len: int, max_q_len: int,
                       softmax_scale: float, O, workspace, lse=None, stream=None) -> None:
    """O [n_tokens, n_q_heads, head_dim] bf16 = attention of Q over the cache;
    lse [n_tokens, n_q_heads] float32 when given."""
    torch = _torch or _setup()
    if Q.dim() != 3:
        raise ValueError(f"Q: shape {tuple(Q.shape)}, the call takes [tokens, heads, {cache.head_dim}]")
    n, heads = Q.shape[0], Q.shape[1]
    ldq = _need_rows(Q, torch.bfloat16, heads, cache.head_dim, "Q")
    ldo = _need_rows(O, torch.bfloat16, heads, cache.head_dim, "O")
    if O.shape[0] != n:
        raise ValueError(f"O: {O.shape[0]} tokens, Q has {n}")
    i32, R = torch.int32, kv_lens.numel()
    table, width = _table(block_table, R)
    args = (_arg(cu_q, i32, R + 1, "cu_q"), _arg(positions, i32, n, "positions"), _arg(kv_lens, i32, R, "kv_lens"))
    lse_p = _maybe(lse, torch.float32, n * heads, "lse")
    if not workspace.is_contiguous():
        raise ValueError("workspace: a contiguous tensor")
    _on_device(Q, O, block_table, cu_q, positions, kv_lens, lse, workspace)
    rc = load_library().twell_kv_attention(
        Q.data_ptr(), ldq, cache.struct(), table, width, *args, n, R, heads, max_kv_len, max_q_len, softmax_scale,
        O.data_ptr(), ldo, lse_p, workspace.data_ptr(), workspace.numel() * workspace.element_size(), _on(stream))
    if rc:
        _check(rc, "twell_kv_attention")


def twell_kv_read_status(cache: KVCache, stream=None) -> int:
    _torch or _setup()
    return int(load_library().twell_kv_read_status(cache.struct(), _on(stream)))


def _logits(t, name: str) -> tuple:
    """(dtype code, rows, vocabulary, distance between rows) of a logits tensor."""
    code = 0 if t.dtype == _torch.bfloat16 else 1 if t.dtype == _torch.float32 else -1
    shape = t.shape
    if code < 0 or len(shape) != 2:
        raise ValueError(f"{name}: {t.dtype} of {len(shape)} dimensions, the call takes [rows, vocab] of bfloat16 or "
                         "float32")
    stride = t.stride()
    if shape[1] > 1 and stride[1] != 1:
        raise ValueError(f"{name}: a tensor whose rows are contiguous")
    return code, shape[0], shape[1], max(stride[0], shape[1]) if shape[0] < 2 else stride[0]


def twell_logprobs(logits, targets, inv_temperature: float, logprob, entropy, lse, top_logprob=None, top_index=None,
                   stream=None) -> None:
    """logprob, entropy, lse [rows] float32 (None: not wanted; targets and logprob
    together) and the top_logprob.shape[1] best alternatives [rows, k]."""
    torch = _torch or _setup()
    f32, i32 = torch.float32, torch.int32
    code, rows, vocab, ld = _logits(logits, "logits")
    k, top, index = 0, None, None
    if top_logprob is not None or top_index is not None:
        if top_logprob is None or top_index is None:
            raise ValueError("top_logprob, top_index: give both or neither")
        if top_logprob.dim() != 2 or top_index.dim() != 2 or top_logprob.shape[1] != top_index.shape[1]:
            raise ValueError(f"top_logprob, top_index: shapes {tuple(top_logprob.shape)}, {tuple(top_index.shape)}, the "
                             f"call takes [{rows}, k] twice")
        k = top_logprob.shape[1]
        top = _arg(top_logprob, f32, rows * k, "top_logprob")
        index = _arg(top_index, i32, rows * k, "top_index")
    _on_device(logits, targets, logprob, entropy, lse, top_logprob, top_index)
    rc = load_library().twell_logprobs(logits.data_ptr(), code, ld, rows, vocab, _maybe(targets, i32, rows, "targets"),
                                       inv_temperature, _maybe(logprob, f32, rows, "logprob"),
                                       _maybe(entropy, f32, rows, "entropy"), _maybe(lse, f32, rows, "lse"), k, top,
                                       index, _on(stream))
    if rc:
        _check(rc, "twell_logprobs")


def twell_logprobs_bwd(logits, targets, inv_temperature: float, lse, entropy, d_logprob, d_entropy, d_logits,
                       stream=None) -> None:
    """d_logits (type of logits; may be logits itself) from the upstream gradients
    of logprob and entropy; targets with d_logprob, or entropy with d_entropy, may be None."""
    torch = _torch or _setup()
    f32 = torch.float32
    code, rows, vocab, ld = _logits(logits, "logits")
    code_d, rows_d, vocab_d, ldd = _logits(d_logits, "d_logits")
    if (code_d, rows_d, vocab_d) != (code, rows, vocab):
        raise ValueError("d_logits: type and shape are those of logits")
    _on_device(logits, targets, lse, entropy, d_logprob, d_entropy, d_logits)
    rc = load_library().twell_logprobs_bwd(
        logits.data_ptr(), code, ld, rows, vocab, _maybe(targets, torch.int32, rows, "targets"), inv_temperature,
        _arg(lse, f32, rows, "lse"), _maybe(entropy, f32, rows, "entropy"), _maybe(d_logprob, f32, rows, "d_logprob"),
        _maybe(d_entropy, f32, rows, "d_entropy"), d_logits.data_ptr(), ldd, _on(stream))
    if rc:
        _check(rc, "twell_logprobs_bwd")
