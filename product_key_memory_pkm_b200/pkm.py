"""Thin Python binding of the C ABI in ``include/pkm.h`` (ctypes).

Argument marshalling only (the feed-forward, checkpoint and 4-bit functions also check
the tensors they get): every step runs in the CUDA kernels of ``libpkm_b200.so``.
PyTorch is used for device memory and streams.  There is no CPU fallback: loading fails
loudly when the library has not been built.

The functions carry the C names (``pkm_forward``, ``pkm_backward``,
``pkm_query``, ``pkm_subkey_scores``, ``pkm_candidate_topk``,
``pkm_gather_bag``, ``pkm_check_status``, ...) and take torch tensors (device
pointers are read with ``data_ptr()``) or raw integer addresses.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

HERE = os.path.dirname(os.path.abspath(__file__))
# PKM_B200_LIB overrides the library path (e.g. to compare two builds)
LIB_PATH = os.environ.get("PKM_B200_LIB") or os.path.join(HERE, "libpkm_b200.so")

PKM_OK = 0
PKM_ERR_INVALID_ARG = 1
PKM_ERR_UNSUPPORTED = 2
PKM_ERR_WORKSPACE = 3
PKM_ERR_CUDA = 4
PKM_ERR_DEVICE_TIMEOUT = 5
PKM_ERR_DEVICE_INDEX = 6

PKM_F_FP32 = 0x1
PKM_F_SIMT = 0x2
PKM_F_VALUES_FP32 = 0x4
PKM_F_BF16_Q = 0x8
PKM_F_BN_TRAIN = 0x10
PKM_F_ALL_K2 = 0x20
PKM_F_IDW = 0x40
PKM_FWD, PKM_BWD, PKM_FWD_FUSED = 0, 1, 2
PKM_FW_LOOKAHEAD = 0x1
PKM_FW_SORT_GLOBAL = 0x2
PKM_FW_PER_CHUNK = 0x4
PKM_ACT_SILU, PKM_ACT_GELU = 0, 1
PKM_FFN_CKPT8 = 0x100
PKM_FFN_GRAD_BF16 = 0x200
PKM_W4_MAX_TOKENS = 64
CKPT8_RUN = 32  # columns that share one scale of an 8-bit checkpoint
FFN_SAVED_FIELDS = ("g", "u", "g_scale", "u_scale")
SAVED_FIELDS = ("q", "qhat", "sub_s", "sub_i", "idx", "w", "bn_batch")
PKM_MAX_SHARDS = 1024
PKM_SHARD_ROUTE, PKM_SHARD_OWNER = 1, 2

# every symbol include/pkm.h declares
EXPORTED = ("pkm_saved_bytes", "pkm_workspace_bytes", "pkm_forward", "pkm_backward", "pkm_query",
            "pkm_subkey_scores", "pkm_candidate_topk", "pkm_gather_bag", "pkm_check_status",
            "pkm_status_string", "pkm_build_info", "pkm_value_grad", "pkm_value_sort",
            "pkm_value_rows", "pkm_query_grad",
            "pkm_launch_count", "pkm_selftest_wait_timeout", "pkm_value_grad_noalloc",
            "pkm_fastweight_workspace_bytes", "pkm_fastweight_chunks", "pkm_value_sgd",
            "pkm_value_grad_rows", "pkm_value_adam", "pkm_hit_counts", "pkm_bn_running_update",
            "pkm_shard_workspace_bytes", "pkm_shard_route", "pkm_shard_bag", "pkm_shard_combine",
            "pkm_shard_gather_dy", "pkm_shard_value_grad", "pkm_shard_scatter_dw",
            "pkm_ffn_saved_bytes", "pkm_ffn_workspace_bytes", "pkm_ffn_forward",
            "pkm_ffn_backward", "pkm_ckpt8_pack", "pkm_ckpt8_unpack", "pkm_w4_pack",
            "pkm_w4_unpack", "pkm_w4_matvec", "pkm_w4_ffn")


class PKMError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} (status {code})")


class pkm_dims(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("d_in", ctypes.c_int32), ("h", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("C1", ctypes.c_int32), ("C2", ctypes.c_int32),
                ("k", ctypes.c_int32), ("d_v", ctypes.c_int32), ("bn_eps", ctypes.c_float),
                ("score_scale", ctypes.c_float), ("flags", ctypes.c_uint32)]


class pkm_saved(ctypes.Structure):
    _fields_ = [(f, ctypes.c_void_p) for f in SAVED_FIELDS]


class pkm_ffn_dims(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int64), ("d_in", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("d_out", ctypes.c_int32), ("act", ctypes.c_int32), ("flags", ctypes.c_uint32)]


class pkm_ffn_saved(ctypes.Structure):
    _fields_ = [(f, ctypes.c_void_p) for f in FFN_SAVED_FIELDS]


class pkm_w4(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p)]


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the shared library (once).  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with "
                          "`python -m product_key_memory_pkm_b200.build`")
    lib = ctypes.CDLL(path)
    P, S, I, U64 = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint64
    D = ctypes.POINTER(pkm_dims)
    SV = ctypes.POINTER(pkm_saved)
    FD, FS, W4 = (ctypes.POINTER(t) for t in (pkm_ffn_dims, pkm_ffn_saved, pkm_w4))
    I64, I32, U32 = ctypes.c_int64, ctypes.c_int32, ctypes.c_uint32
    sig = {
        "pkm_saved_bytes": (S, [D, I]),
        "pkm_workspace_bytes": (S, [D, I]),
        "pkm_forward": (I, [D, P, P, P, P, P, P, SV, P, S, P]),
        "pkm_backward": (I, [D, P, P, P, P, P, SV, P, P, P, P, P, P, P, P, S, P]),
        "pkm_query": (I, [D, P, P, P, SV, P]),
        "pkm_subkey_scores": (I, [D, P, SV, P]),
        "pkm_candidate_topk": (I, [D, SV, P]),
        "pkm_gather_bag": (I, [D, P, P, P, P, P]),
        "pkm_check_status": (I, [P]),
        "pkm_status_string": (ctypes.c_char_p, [I]),
        "pkm_build_info": (ctypes.c_char_p, []),
        "pkm_value_grad": (I, [D, P, SV, P, P, P, P, S, P]),
        "pkm_value_sort": (I, [D, SV, P, S, P]),
        "pkm_value_rows": (I, [D, P, P, P, P, P, S, P]),
        "pkm_query_grad": (I, [D, P, P, P, P, SV, P, P, P, P, P, P, S, P]),
        "pkm_launch_count": (ctypes.c_ulonglong, []),
        "pkm_selftest_wait_timeout": (I, [ctypes.c_uint32, P]),
        "pkm_value_grad_noalloc": (I, [D, P, SV, P, P, P, P]),
        "pkm_value_sgd": (I, [D, ctypes.c_float, P, SV, P, P, S, P]),
        "pkm_value_grad_rows": (I, [D, P, SV, P, P, P, P, P, P, S, P]),
        "pkm_value_adam": (I, [D, ctypes.c_float, ctypes.c_float, ctypes.c_float, ctypes.c_float,
                               ctypes.c_int64, P, P, P, SV, P, P, S, P]),
        "pkm_hit_counts": (I, [D, P, P, P, P]),
        "pkm_bn_running_update": (I, [D, P, P, ctypes.c_float, P]),
        "pkm_fastweight_workspace_bytes": (S, [D, ctypes.c_int64, ctypes.c_uint32]),
        "pkm_fastweight_chunks": (I, [D, ctypes.c_int64, ctypes.c_float, ctypes.c_uint32, P, P, P,
                                      P, P, P, P, P, S, P]),
        "pkm_shard_workspace_bytes": (S, [D, ctypes.c_int32, I, ctypes.c_int64]),
        "pkm_shard_route": (I, [D, ctypes.c_int32, ctypes.c_int64, P, P, P, P, P, P, P, S, P]),
        "pkm_shard_bag": (I, [D, ctypes.c_int32, ctypes.c_int64, P, ctypes.c_int64, ctypes.c_int64,
                              P, P, P, P, S, P]),
        "pkm_shard_combine": (I, [D, ctypes.c_int32, P, P, ctypes.c_int64, P, P]),
        "pkm_shard_gather_dy": (I, [D, ctypes.c_int32, P, P, P, ctypes.c_int64, P]),
        "pkm_shard_value_grad": (I, [D, ctypes.c_int32, ctypes.c_int64, P, ctypes.c_int64,
                                     ctypes.c_int64, P, P, P, P, P, P, S, P]),
        "pkm_shard_scatter_dw": (I, [D, P, P, P, P]),
        "pkm_ffn_saved_bytes": (S, [FD, I]),
        "pkm_ffn_workspace_bytes": (S, [FD, I]),
        "pkm_ffn_forward": (I, [FD, P, P, P, P, P, FS, P, S, P]),
        "pkm_ffn_backward": (I, [FD, P, P, P, P, FS, P, P, P, P, P, P, S, P]),
        "pkm_ckpt8_pack": (I, [I64, I32, U32, P, P, P, P]),
        "pkm_ckpt8_unpack": (I, [I64, I32, U32, P, P, P, P]),
        "pkm_w4_pack": (I, [I32, I32, I32, P, P, P, P]),
        "pkm_w4_unpack": (I, [I32, I32, I32, W4, P, P]),
        "pkm_w4_matvec": (I, [I64, I32, I32, I32, P, W4, P, P]),
        "pkm_w4_ffn": (I, [FD, I32, P, W4, W4, W4, P, P, S, P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    del U64
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load().pkm_status_string(int(code)).decode()


# ----------------------------------------------------------------- marshalling
def _ptr(t) -> int | None:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(code: int, where: str) -> None:
    if code != PKM_OK:
        raise PKMError(code, where)


@dataclass
class Dims:
    """Python mirror of ``pkm_dims``."""
    N: int
    d_in: int
    h: int
    dk: int
    C1: int
    C2: int
    k: int
    d_v: int
    bn_eps: float = 1e-5
    score_scale: float = 1.0
    flags: int = 0

    def c(self) -> pkm_dims:
        return pkm_dims(self.N, self.d_in, self.h, self.dk, self.C1, self.C2, self.k, self.d_v,
                        self.bn_eps, self.score_scale, self.flags)

    @classmethod
    def from_config(cls, cfg, flags: int = 0, N: int | None = None) -> "Dims":
        f = flags | (PKM_F_FP32 if cfg.dtype == "f32" else 0)
        if cfg.dtype != "f32" and cfg.vdtype == "f32":
            f |= PKM_F_VALUES_FP32
        return cls(cfg.N if N is None else N, cfg.d_in, cfg.h, cfg.dk, cfg.C1, cfg.C2, cfg.k,
                   cfg.d_v, cfg.bn_eps, cfg.score_scale, f)


def _saved_c(saved: dict) -> pkm_saved:
    return pkm_saved(*[_ptr(saved.get(f)) for f in SAVED_FIELDS])


def pkm_saved_bytes(dims: Dims, field: str) -> int:
    return int(load().pkm_saved_bytes(ctypes.byref(dims.c()), SAVED_FIELDS.index(field)))


def pkm_workspace_bytes(dims: Dims, which: int) -> int:
    return int(load().pkm_workspace_bytes(ctypes.byref(dims.c()), which))


def pkm_forward(dims: Dims, x, Wq, bn, subkeys, values, y, saved: dict, workspace=None,
                workspace_bytes: int = 0, stream=None) -> None:
    ws_bytes = workspace_bytes or (workspace.numel() * workspace.element_size()
                                   if workspace is not None and not isinstance(workspace, int) else 0)
    s = _saved_c(saved)
    _check(load().pkm_forward(ctypes.byref(dims.c()), _ptr(x), _ptr(Wq), _ptr(bn), _ptr(subkeys),
                              _ptr(values), _ptr(y), ctypes.byref(s), _ptr(workspace), ws_bytes,
                              _stream(stream)), "pkm_forward")


def pkm_backward(dims: Dims, x, Wq, bn, subkeys, values, saved: dict, dy, dx=None, dWq=None,
                 dbn=None, dsubkeys=None, dvalues=None, dw_out=None, workspace=None,
                 workspace_bytes: int = 0, stream=None) -> None:
    ws_bytes = workspace_bytes or (workspace.numel() * workspace.element_size()
                                   if workspace is not None and not isinstance(workspace, int) else 0)
    s = _saved_c(saved)
    _check(load().pkm_backward(ctypes.byref(dims.c()), _ptr(x), _ptr(Wq), _ptr(bn), _ptr(subkeys),
                               _ptr(values), ctypes.byref(s), _ptr(dy), _ptr(dx), _ptr(dWq),
                               _ptr(dbn), _ptr(dsubkeys), _ptr(dvalues), _ptr(dw_out),
                               _ptr(workspace), ws_bytes, _stream(stream)), "pkm_backward")


def _ws(workspace, workspace_bytes):
    if workspace_bytes:
        return workspace_bytes
    if workspace is None or isinstance(workspace, int):
        return 0
    return workspace.numel() * workspace.element_size()


def pkm_value_grad(dims: Dims, values, saved: dict, dy, dw, dvalues=None, workspace=None,
                   workspace_bytes: int = 0, stream=None) -> None:
    s = _saved_c(saved)
    _check(load().pkm_value_grad(ctypes.byref(dims.c()), _ptr(values), ctypes.byref(s), _ptr(dy),
                                 _ptr(dvalues), _ptr(dw), _ptr(workspace),
                                 _ws(workspace, workspace_bytes), _stream(stream)),
           "pkm_value_grad")


def pkm_value_sort(dims: Dims, saved: dict, workspace=None, workspace_bytes: int = 0,
                   stream=None) -> None:
    """First half of pkm_value_grad: the selections sorted by value row, into the workspace."""
    s = _saved_c(saved)
    _check(load().pkm_value_sort(ctypes.byref(dims.c()), ctypes.byref(s), _ptr(workspace),
                                 _ws(workspace, workspace_bytes), _stream(stream)),
           "pkm_value_sort")


def pkm_value_rows(dims: Dims, values, dy, dw, dvalues=None, workspace=None,
                   workspace_bytes: int = 0, stream=None) -> None:
    """Second half of pkm_value_grad: the per-row pass over what pkm_value_sort left in the
    same workspace."""
    _check(load().pkm_value_rows(ctypes.byref(dims.c()), _ptr(values), _ptr(dy), _ptr(dvalues),
                                 _ptr(dw), _ptr(workspace), _ws(workspace, workspace_bytes),
                                 _stream(stream)),
           "pkm_value_rows")


def pkm_value_grad_noalloc(dims: Dims, values, saved: dict, dy, dw, dvalues=None,
                           stream=None) -> None:
    """pkm_value_grad without a workspace argument: the scratch is a fixed device
    array inside the library (for callers that cannot allocate device memory)."""
    s = _saved_c(saved)
    _check(load().pkm_value_grad_noalloc(ctypes.byref(dims.c()), _ptr(values), ctypes.byref(s),
                                         _ptr(dy), _ptr(dvalues), _ptr(dw), _stream(stream)),
           "pkm_value_grad_noalloc")


def pkm_value_sgd(dims: Dims, lr: float, values, saved: dict, dy, workspace=None,
                  workspace_bytes: int = 0, stream=None) -> None:
    """values[r] -= lr * (sum of w * dy over the selections of r), in place (fp32)."""
    s = _saved_c(saved)
    _check(load().pkm_value_sgd(ctypes.byref(dims.c()), float(lr), _ptr(values), ctypes.byref(s),
                                _ptr(dy), _ptr(workspace), _ws(workspace, workspace_bytes),
                                _stream(stream)), "pkm_value_sgd")


def pkm_value_grad_rows(dims: Dims, values, saved: dict, dy, rows_out, dvalues_rows, num_rows,
                        dw=None, workspace=None, workspace_bytes: int = 0, stream=None) -> None:
    """Compact value gradient: num_rows[0] = U, rows_out[:U] (ascending), dvalues_rows[:U]."""
    s = _saved_c(saved)
    _check(load().pkm_value_grad_rows(ctypes.byref(dims.c()), _ptr(values), ctypes.byref(s),
                                      _ptr(dy), _ptr(dw), _ptr(rows_out), _ptr(dvalues_rows),
                                      _ptr(num_rows), _ptr(workspace),
                                      _ws(workspace, workspace_bytes), _stream(stream)),
           "pkm_value_grad_rows")


def pkm_value_adam(dims: Dims, lr: float, beta1: float, beta2: float, eps: float, step: int,
                   values, m, v, saved: dict, dy, workspace=None, workspace_bytes: int = 0,
                   stream=None) -> None:
    """Lazy Adam on the selected value rows (values, m, v fp32, in place)."""
    s = _saved_c(saved)
    _check(load().pkm_value_adam(ctypes.byref(dims.c()), float(lr), float(beta1), float(beta2),
                                 float(eps), int(step), _ptr(values), _ptr(m), _ptr(v),
                                 ctypes.byref(s), _ptr(dy), _ptr(workspace),
                                 _ws(workspace, workspace_bytes), _stream(stream)),
           "pkm_value_adam")


def pkm_hit_counts(dims: Dims, idx, slot_hits=None, subkey_hits=None, stream=None) -> None:
    """slot_hits [C1*C2] int32 and subkey_hits [h][C1+C2] int32 accumulate (+=)."""
    _check(load().pkm_hit_counts(ctypes.byref(dims.c()), _ptr(idx), _ptr(slot_hits),
                                 _ptr(subkey_hits), _stream(stream)), "pkm_hit_counts")


def pkm_bn_running_update(dims: Dims, bn, bn_batch, momentum: float = 0.1, stream=None) -> None:
    """Fold a training-mode batch's statistics into bn's running mean and variance."""
    _check(load().pkm_bn_running_update(ctypes.byref(dims.c()), _ptr(bn), _ptr(bn_batch),
                                        float(momentum), _stream(stream)),
           "pkm_bn_running_update")


def pkm_fastweight_workspace_bytes(dims: Dims, chunk: int, mode: int = 0) -> int:
    return int(load().pkm_fastweight_workspace_bytes(ctypes.byref(dims.c()), int(chunk),
                                                     int(mode)))


def alloc_fastweight_workspace(dims: Dims, chunk: int, mode: int = 0, device="cuda"):
    import torch
    return torch.empty(max(pkm_fastweight_workspace_bytes(dims, chunk, mode), 256),
                       dtype=torch.uint8, device=device)


def pkm_fastweight_chunks(dims: Dims, chunk: int, lr: float, x, Wq, bn, subkeys, values, y,
                          targets=None, lookahead: bool = False, strategy: int = 0,
                          workspace=None, workspace_bytes: int = 0, stream=None) -> None:
    """Chunked read-then-write of the fast-weight memory: ``values`` (fp32) is updated
    in place, ``y`` receives every chunk's read.  ``strategy``: 0, PKM_FW_SORT_GLOBAL or
    PKM_FW_PER_CHUNK (same results)."""
    mode = (PKM_FW_LOOKAHEAD if lookahead else 0) | int(strategy)
    _check(load().pkm_fastweight_chunks(ctypes.byref(dims.c()), int(chunk), float(lr), mode,
                                        _ptr(x), _ptr(Wq), _ptr(bn), _ptr(subkeys),
                                        _ptr(values), _ptr(targets), _ptr(y), _ptr(workspace),
                                        _ws(workspace, workspace_bytes), _stream(stream)),
           "pkm_fastweight_chunks")


def pkm_query_grad(dims: Dims, x, Wq, bn, subkeys, saved: dict, dw, dx=None, dWq=None, dbn=None,
                   dsubkeys=None, workspace=None, workspace_bytes: int = 0, stream=None) -> None:
    s = _saved_c(saved)
    _check(load().pkm_query_grad(ctypes.byref(dims.c()), _ptr(x), _ptr(Wq), _ptr(bn),
                                 _ptr(subkeys), ctypes.byref(s), _ptr(dw), _ptr(dx), _ptr(dWq),
                                 _ptr(dbn), _ptr(dsubkeys), _ptr(workspace),
                                 _ws(workspace, workspace_bytes), _stream(stream)),
           "pkm_query_grad")


def pkm_selftest_wait_timeout(budget_cycles: int = 2_000_000, stream=None) -> None:
    _check(load().pkm_selftest_wait_timeout(int(budget_cycles), _stream(stream)),
           "pkm_selftest_wait_timeout")


def pkm_launch_count() -> int:
    return int(load().pkm_launch_count())


def pkm_query(dims: Dims, x, Wq, bn, saved: dict, stream=None) -> None:
    s = _saved_c(saved)
    _check(load().pkm_query(ctypes.byref(dims.c()), _ptr(x), _ptr(Wq), _ptr(bn), ctypes.byref(s),
                            _stream(stream)), "pkm_query")


def pkm_subkey_scores(dims: Dims, subkeys, saved: dict, stream=None) -> None:
    s = _saved_c(saved)
    _check(load().pkm_subkey_scores(ctypes.byref(dims.c()), _ptr(subkeys), ctypes.byref(s),
                                    _stream(stream)), "pkm_subkey_scores")


def pkm_candidate_topk(dims: Dims, saved: dict, stream=None) -> None:
    s = _saved_c(saved)
    _check(load().pkm_candidate_topk(ctypes.byref(dims.c()), ctypes.byref(s), _stream(stream)),
           "pkm_candidate_topk")


def pkm_gather_bag(dims: Dims, values, idx, w, y, stream=None) -> None:
    _check(load().pkm_gather_bag(ctypes.byref(dims.c()), _ptr(values), _ptr(idx), _ptr(w), _ptr(y),
                                 _stream(stream)), "pkm_gather_bag")


def pkm_check_status(stream=None) -> int:
    """Synchronise the stream and return the device status code (0 = PKM_OK)."""
    return int(load().pkm_check_status(_stream(stream)))


def pkm_build_info() -> str:
    return load().pkm_build_info().decode()


# ----------------------------------------------------------------- allocation helpers
def alloc_saved(dims: Dims, device="cuda", with_qhat: bool = True) -> dict:
    """Caller-owned buffers the forward writes and the backward reads (torch)."""
    import torch
    N, hq = dims.N, dims.h * dims.dk
    ksel = dims.k * dims.k if dims.flags & PKM_F_ALL_K2 else dims.k
    fp32 = bool(dims.flags & PKM_F_FP32)
    q = (torch.empty(N, hq, dtype=torch.float32, device=device) if fp32 else
         torch.empty(2, N, hq, dtype=torch.bfloat16, device=device))
    return dict(
        q=q,
        qhat=torch.empty(N, hq, dtype=torch.float32, device=device) if with_qhat else None,
        sub_s=torch.empty(N, dims.h, 2, dims.k, dtype=torch.float32, device=device),
        sub_i=torch.empty(N, dims.h, 2, dims.k, dtype=torch.int32, device=device),
        idx=torch.empty(N, dims.h, ksel, dtype=torch.int32, device=device),
        w=torch.empty(N, dims.h, ksel, dtype=torch.float32, device=device),
        bn_batch=torch.empty(2, hq, dtype=torch.float32, device=device),
    )


def alloc_workspace(dims: Dims, which: int, device="cuda"):
    import torch
    n = pkm_workspace_bytes(dims, which)
    return torch.empty(max(n, 256), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------- row-sharded table
# Triples travel as int32 tensors of shape [n, 3] (segment, row, bits of the fp32 weight),
# the layout of pkm_triple.

def pkm_shard_workspace_bytes(dims: Dims, G: int, which: int, n_triples: int = 0) -> int:
    return int(load().pkm_shard_workspace_bytes(ctypes.byref(dims.c()), int(G), int(which),
                                                int(n_triples)))


def pkm_shard_route(dims: Dims, G: int, rows_per_shard: int, idx, w, counts, segpos, send, perm,
                    workspace=None, workspace_bytes: int = 0, stream=None) -> None:
    _check(load().pkm_shard_route(ctypes.byref(dims.c()), int(G), int(rows_per_shard), _ptr(idx),
                                  _ptr(w), _ptr(counts), _ptr(segpos), _ptr(send), _ptr(perm),
                                  _ptr(workspace), _ws(workspace, workspace_bytes),
                                  _stream(stream)), "pkm_shard_route")


def pkm_shard_bag(dims: Dims, G: int, shard_rows: int, recv_counts, n_triples: int,
                  n_segments: int, recv, values, partial, workspace=None,
                  workspace_bytes: int = 0, stream=None) -> None:
    _check(load().pkm_shard_bag(ctypes.byref(dims.c()), int(G), int(shard_rows),
                                _ptr(recv_counts), int(n_triples), int(n_segments), _ptr(recv),
                                _ptr(values), _ptr(partial), _ptr(workspace),
                                _ws(workspace, workspace_bytes), _stream(stream)),
           "pkm_shard_bag")


def pkm_shard_combine(dims: Dims, G: int, segpos, partial_recv, n_rows: int, y,
                      stream=None) -> None:
    _check(load().pkm_shard_combine(ctypes.byref(dims.c()), int(G), _ptr(segpos),
                                    _ptr(partial_recv), int(n_rows), _ptr(y), _stream(stream)),
           "pkm_shard_combine")


def pkm_shard_gather_dy(dims: Dims, G: int, segpos, dy, dy_send, n_rows: int,
                        stream=None) -> None:
    _check(load().pkm_shard_gather_dy(ctypes.byref(dims.c()), int(G), _ptr(segpos), _ptr(dy),
                                      _ptr(dy_send), int(n_rows), _stream(stream)),
           "pkm_shard_gather_dy")


def pkm_shard_value_grad(dims: Dims, G: int, shard_rows: int, recv_counts, n_triples: int,
                         n_segments: int, recv, values, dy_recv, dvalues, dw_recv,
                         workspace=None, workspace_bytes: int = 0, stream=None) -> None:
    _check(load().pkm_shard_value_grad(ctypes.byref(dims.c()), int(G), int(shard_rows),
                                       _ptr(recv_counts), int(n_triples), int(n_segments),
                                       _ptr(recv), _ptr(values), _ptr(dy_recv), _ptr(dvalues),
                                       _ptr(dw_recv), _ptr(workspace),
                                       _ws(workspace, workspace_bytes), _stream(stream)),
           "pkm_shard_value_grad")


def pkm_shard_scatter_dw(dims: Dims, perm, dw_ret, dw, stream=None) -> None:
    _check(load().pkm_shard_scatter_dw(ctypes.byref(dims.c()), _ptr(perm), _ptr(dw_ret), _ptr(dw),
                                       _stream(stream)), "pkm_shard_scatter_dw")


# ------------------------------------------------------- gated feed-forward block
# Unlike the raw-address calls above, these check the tensors they are given: type, shape,
# contiguity and device.  (An integer address passes unchecked; not for a tensor that gives the
# call its sizes, as the checkpoints' values and the 4-bit products' x and codes do.)

_torch = None


class _Checked:
    """Checks of one call's tensors and the call's stream.  Few-token calls run for a few
    microseconds on the GPU, so this avoids what costs one on the host: repeated imports, the
    wrapper objects of torch.cuda.current_stream(), and telling apart what is wrong with a
    tensor before anything is."""
    __slots__ = ("torch", "device")

    def __init__(self):
        global _torch
        if _torch is None:
            import torch
            _torch = torch
        self.torch = _torch
        try:
            self.device = _torch._C._cuda_getDevice()
        except (AttributeError, RuntimeError):  # no GPU, or a build without CUDA
            self.device = -2                    # no tensor is there

    def __call__(self, t, name: str, dtype, shape: tuple, optional: bool = False) -> int | None:
        """Address of a contiguous ``shape`` tensor of ``dtype`` on the current device."""
        if t is None or isinstance(t, int):
            if t is None and not optional:
                raise ValueError(f"{name} is missing")
            return t
        if (t.dtype is dtype and t.shape == shape and t.is_contiguous()
                and t.get_device() == self.device):
            return t.data_ptr()
        if t.dtype != dtype:
            raise TypeError(f"{name}: {dtype} wanted, got {t.dtype}")
        if t.shape != shape:
            raise ValueError(f"{name}: shape {tuple(shape)} wanted, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} is not contiguous")
        self.place(t, name)
        return t.data_ptr()

    def place(self, t, name: str) -> None:
        if not t.is_cuda:
            raise ValueError(f"{name} is not on a GPU")
        if t.get_device() != self.device:
            raise ValueError(f"{name} is on {t.device}, the current device is {self.device}")

    def stream(self, stream):
        if stream is None and self.device >= 0:
            return self.torch._C._cuda_getCurrentRawStream(self.device)
        return _stream(stream)

    def workspace(self, workspace, workspace_bytes):
        if workspace_bytes < 0:  # the largest size there is, as size_t
            raise ValueError(f"workspace_bytes: {workspace_bytes}")
        if workspace is None or isinstance(workspace, int):
            return workspace, workspace_bytes
        if not workspace.is_contiguous():
            raise ValueError("workspace is not contiguous")
        self.place(workspace, "workspace")
        if workspace_bytes > workspace.nbytes:
            raise ValueError(f"workspace has {workspace.nbytes} bytes, not {workspace_bytes}")
        return workspace.data_ptr(), workspace_bytes or workspace.nbytes


def _int32(v: int, name: str, side: str = "") -> int:
    """A size the library takes in 32 bits (of more, ctypes would pass the low bits)."""
    if not -0x80000000 <= v <= 0x7fffffff:
        raise ValueError(f"{name}{side}: {v} is beyond the library's integers")
    return v


@dataclass(frozen=True)
class FfnDims:
    """Python mirror of ``pkm_ffn_dims``."""
    N: int
    d_in: int
    d_ff: int
    d_out: int
    act: int = PKM_ACT_SILU
    flags: int = 0

    def __post_init__(self):
        s = pkm_ffn_dims(self.N, self.d_in, self.d_ff, self.d_out, self.act, self.flags)
        for f, _ in s._fields_:  # ctypes cuts what does not fit to its low bits
            if getattr(s, f) != getattr(self, f):
                raise ValueError(f"{f}: {getattr(self, f)} is beyond the library's integers")
        object.__setattr__(self, "_c", s)  # the dims do not change: made once

    def c(self) -> pkm_ffn_dims:
        return self._c

    @property
    def dtype(self):
        t = _Checked().torch if _torch is None else _torch
        return t.float32 if self.flags & PKM_F_FP32 else t.bfloat16

    @property
    def runs(self) -> int:
        """Scales per row of an 8-bit checkpoint of g or u."""
        return -(-self.d_ff // CKPT8_RUN)


def pkm_ffn_saved_bytes(dims: FfnDims, field: str) -> int:
    return int(load().pkm_ffn_saved_bytes(ctypes.byref(dims.c()), FFN_SAVED_FIELDS.index(field)))


def pkm_ffn_workspace_bytes(dims: FfnDims, which: int) -> int:
    return int(load().pkm_ffn_workspace_bytes(ctypes.byref(dims.c()), which))


def alloc_ffn_saved(dims: FfnDims, device="cuda") -> dict:
    """Caller-owned buffers pkm_ffn_forward writes and pkm_ffn_backward reads (torch)."""
    import torch
    if dims.flags & PKM_FFN_CKPT8:
        g, gs = alloc_ckpt8(dims.N, dims.d_ff, device)
        u, us = alloc_ckpt8(dims.N, dims.d_ff, device)
        return dict(g=g, u=u, g_scale=gs, u_scale=us)
    g, u = (torch.empty(dims.N, dims.d_ff, dtype=dims.dtype, device=device) for _ in range(2))
    return dict(g=g, u=u, g_scale=None, u_scale=None)


def alloc_ffn_workspace(dims: FfnDims, which: int, device="cuda"):
    import torch
    return torch.empty(max(pkm_ffn_workspace_bytes(dims, which), 256), dtype=torch.uint8,
                       device=device)


def _ffn_saved_c(ck: _Checked, d: FfnDims, saved: dict) -> pkm_ffn_saved:
    if d.flags & PKM_FFN_CKPT8:
        i8, f32 = ck.torch.int8, ck.torch.float32
        codes, runs = (d.N, d.runs * CKPT8_RUN), (d.N, d.runs)
        return pkm_ffn_saved(ck(saved.get("g"), "saved g", i8, codes),
                             ck(saved.get("u"), "saved u", i8, codes),
                             ck(saved.get("g_scale"), "saved g_scale", f32, runs),
                             ck(saved.get("u_scale"), "saved u_scale", f32, runs))
    dt, shape = d.dtype, (d.N, d.d_ff)
    return pkm_ffn_saved(ck(saved.get("g"), "saved g", dt, shape),
                         ck(saved.get("u"), "saved u", dt, shape), None, None)


def pkm_ffn_forward(dims: FfnDims, x, Wg, Wu, Wd, y, saved: dict | None = None, workspace=None,
                    workspace_bytes: int = 0, stream=None) -> None:
    """y = (act(x Wg^T) * (x Wu^T)) Wd^T; ``saved`` (alloc_ffn_saved) keeps what
    pkm_ffn_backward needs, None keeps nothing."""
    d, ck = dims, _Checked()
    dt = d.dtype
    xp, yp = ck(x, "x", dt, (d.N, d.d_in)), ck(y, "y", dt, (d.N, d.d_out))
    g, u = ck(Wg, "Wg", dt, (d.d_ff, d.d_in)), ck(Wu, "Wu", dt, (d.d_ff, d.d_in))
    o = ck(Wd, "Wd", dt, (d.d_out, d.d_ff))
    s = None if saved is None else ctypes.byref(_ffn_saved_c(ck, d, saved))
    ws, ws_bytes = ck.workspace(workspace, workspace_bytes)
    _check(load().pkm_ffn_forward(ctypes.byref(d._c), xp, g, u, o, yp, s, ws, ws_bytes, ck.stream(stream)),
           "pkm_ffn_forward")


def pkm_ffn_backward(dims: FfnDims, x, Wg, Wu, Wd, saved: dict, dy, dx=None, dWg=None, dWu=None,
                     dWd=None, workspace=None, workspace_bytes: int = 0, stream=None) -> None:
    """Gradients of sum(dy * y).  dx is overwritten; dWg, dWu, dWd are fp32 and accumulate, or
    with PKM_FFN_GRAD_BF16 bf16 and overwritten.  A gradient that is None is skipped."""
    d, ck = dims, _Checked()
    dt = d.dtype
    wt = ck.torch.bfloat16 if d.flags & PKM_FFN_GRAD_BF16 else ck.torch.float32
    xs, ins, outs = (d.N, d.d_in), (d.d_ff, d.d_in), (d.d_out, d.d_ff)
    args = (ck(x, "x", dt, xs), ck(Wg, "Wg", dt, ins), ck(Wu, "Wu", dt, ins),
            ck(Wd, "Wd", dt, outs), ctypes.byref(_ffn_saved_c(ck, d, saved)),
            ck(dy, "dy", dt, (d.N, d.d_out)), ck(dx, "dx", dt, xs, True),
            ck(dWg, "dWg", wt, ins, True), ck(dWu, "dWu", wt, ins, True),
            ck(dWd, "dWd", wt, outs, True))
    ws, ws_bytes = ck.workspace(workspace, workspace_bytes)
    _check(load().pkm_ffn_backward(ctypes.byref(d._c), *args, ws, ws_bytes, ck.stream(stream)),
           "pkm_ffn_backward")


# ------------------------------------------------------- 8-bit activation checkpoints
def alloc_ckpt8(rows: int, cols: int, device="cuda") -> tuple:
    """(codes, scale) of an 8-bit checkpoint of a [rows, cols] activation."""
    import torch
    runs = -(-cols // CKPT8_RUN)
    return (torch.empty(rows, runs * CKPT8_RUN, dtype=torch.int8, device=device),
            torch.empty(rows, runs, dtype=torch.float32, device=device))


def _ckpt8(ck: _Checked, values, name, codes, scale):
    dt, f32 = values.dtype, ck.torch.float32
    if dt != f32 and dt != ck.torch.bfloat16:
        raise TypeError(f"{name}: bfloat16 or float32 wanted, got {dt}")
    if values.dim() != 2:
        raise ValueError(f"{name}: two dimensions wanted, got {values.dim()}")
    rows, cols = values.shape
    runs = -(-_int32(cols, name, " columns") // CKPT8_RUN)
    return (rows, cols, PKM_F_FP32 if dt == f32 else 0, ck(values, name, dt, (rows, cols)),
            ck(codes, "codes", ck.torch.int8, (rows, runs * CKPT8_RUN)),
            ck(scale, "scale", f32, (rows, runs)))


def pkm_ckpt8_pack(src, codes, scale, stream=None) -> None:
    """``src`` [rows, cols] bf16 or fp32 into 8-bit codes and a scale per 32 columns."""
    ck = _Checked()
    rows, cols, flags, v, c, s = _ckpt8(ck, src, "src", codes, scale)
    _check(load().pkm_ckpt8_pack(rows, cols, flags, v, c, s, ck.stream(stream)), "pkm_ckpt8_pack")


def pkm_ckpt8_unpack(codes, scale, dst, stream=None) -> None:
    """The values (codes * scale) into ``dst`` [rows, cols], bf16 or fp32."""
    ck = _Checked()
    rows, cols, flags, v, c, s = _ckpt8(ck, dst, "dst", codes, scale)
    _check(load().pkm_ckpt8_unpack(rows, cols, flags, c, s, v, ck.stream(stream)),
           "pkm_ckpt8_unpack")


# ------------------------------------------------------- products with 4-bit weights
# A 4-bit matrix is the pair (codes, scale): codes uint8 [d_out, d_in / 2], scale bf16
# [d_out, ceil(d_in / group)].

def alloc_w4(d_out: int, d_in: int, group: int, device="cuda") -> tuple:
    import torch
    return (torch.empty(d_out, d_in // 2, dtype=torch.uint8, device=device),
            torch.empty(d_out, -(-d_in // group), dtype=torch.bfloat16, device=device))


def _w4(ck: _Checked, W, name: str, d_out: int, d_in: int, group: int) -> pkm_w4:
    if _int32(group, "group") <= 0:
        raise ValueError(f"group: a positive multiple of 32 wanted, got {group}")
    _int32(d_out, name, " rows")
    _int32(d_in, name, " columns")
    codes, scale = W
    return pkm_w4(ck(codes, name, ck.torch.uint8, (d_out, d_in // 2)),
                  ck(scale, name, ck.torch.bfloat16, (d_out, -(-d_in // group))))


def _matrix(ck: _Checked, t, name: str):
    if t.dim() != 2:
        raise ValueError(f"{name}: two dimensions wanted, got {t.dim()}")
    return ck(t, name, ck.torch.bfloat16, t.shape)


def pkm_w4_pack(W, codes, scale, group: int = 64, stream=None) -> None:
    """A bf16 matrix ``W`` [d_out, d_in] into 4-bit codes and a bf16 scale per group."""
    ck = _Checked()
    w = _matrix(ck, W, "W")
    q = _w4(ck, (codes, scale), "packed", *W.shape, group)
    _check(load().pkm_w4_pack(*W.shape, group, w, q.codes, q.scale, ck.stream(stream)),
           "pkm_w4_pack")


def pkm_w4_unpack(codes, scale, W, group: int = 64, stream=None) -> None:
    """The bf16 matrix the codes stand for."""
    ck = _Checked()
    w = _matrix(ck, W, "W")
    q = _w4(ck, (codes, scale), "packed", *W.shape, group)
    _check(load().pkm_w4_unpack(*W.shape, group, ctypes.byref(q), w, ck.stream(stream)),
           "pkm_w4_unpack")


def pkm_w4_matvec(x, codes, scale, y, group: int = 64, stream=None) -> None:
    """y [N, d_out] fp32 = x W^T for up to PKM_W4_MAX_TOKENS rows of bf16 ``x``."""
    ck = _Checked()
    xp = _matrix(ck, x, "x")
    N, d_in = x.shape
    d_out = codes.shape[0]
    q = _w4(ck, (codes, scale), "W", d_out, d_in, group)
    yp = ck(y, "y", ck.torch.float32, (N, d_out))
    _check(load().pkm_w4_matvec(N, d_in, d_out, group, xp, ctypes.byref(q), yp,
                                ck.stream(stream)), "pkm_w4_matvec")


def pkm_w4_ffn(dims: FfnDims, x, Wg, Wu, Wd, y, group: int = 64, workspace=None,
               workspace_bytes: int = 0, stream=None) -> None:
    """pkm_ffn_forward with 4-bit weights, each a (codes, scale) pair, for up to
    PKM_W4_MAX_TOKENS tokens."""
    d, ck = dims, _Checked()
    b16 = ck.torch.bfloat16
    xp, yp = ck(x, "x", b16, (d.N, d.d_in)), ck(y, "y", b16, (d.N, d.d_out))
    g = _w4(ck, Wg, "Wg", d.d_ff, d.d_in, group)
    u = _w4(ck, Wu, "Wu", d.d_ff, d.d_in, group)
    o = _w4(ck, Wd, "Wd", d.d_out, d.d_ff, group)
    ws, ws_bytes = ck.workspace(workspace, workspace_bytes)
    _check(load().pkm_w4_ffn(ctypes.byref(d._c), group, xp, ctypes.byref(g), ctypes.byref(u), ctypes.byref(o),
                             yp, ws, ws_bytes, ck.stream(stream)), "pkm_w4_ffn")
