"""ctypes binding of ``libspark_bsa.so`` (include/spark_bsa.h).

Argument marshalling only: every step of the forward pass runs in the library's sm_100a
kernels.  PyTorch provides device memory, the current CUDA stream and dtype/shape checks.
There is no fallback: if the library is missing or was built for another GPU the calls raise.
"""

from __future__ import annotations

import ctypes
import os

import torch

from .build import LIB_PATH

__all__ = [
    "SparkError", "SPARK_BF16", "SPARK_F32", "DEVERR", "Layout", "lib",
    "spark_status_string", "spark_bsa_topk_count", "spark_bsa_workspace_layout",
    "spark_bsa_workspace_size", "spark_bsa_forward", "spark_bsa_read_error",
    "spark_bsa_gather_q", "spark_bsa_anchor", "spark_bsa_gather_kv_summarize",
    "spark_bsa_route", "spark_bsa_attend", "workspace_views", "spark_bsa_forward_noalloc",
    "spark_bsa_workspace_size_ctx", "spark_bsa_forward_ctx", "spark_bsa_context_bf16",
    "spark_bsa_attend_ctx", "ReblockLayout", "spark_reblock_workspace_layout",
    "spark_reblock_workspace_size", "spark_reblock_levels", "spark_reblock",
    "spark_reblock_whiten", "spark_reblock_level", "reblock_views",
    "spark_bsa_host_staging_size", "spark_bsa_forward_host", "spark_bsa_quantize_fp8",
    "spark_bsa_attend_fp8", "spark_bsa_workspace_size_fp8", "spark_bsa_forward_fp8",
    "spark_bsa_gather_kv_meanpool", "spark_bsa_route_threshold", "spark_bsa_attend_var",
    "spark_bsa_set_wait_limit_ns", "spark_bsa_get_wait_limit_ns",
    "spark_bsa_host_staging_size_ex", "spark_bsa_fused_supported", "spark_bsa_forward_fused",
    "spark_bsa_attend_fused", "spark_qk_norm_rope", "spark_rope_frequencies",
    "spark_attend_dense", "spark_attend_dense_workspace_size", "spark_attend_ranges",
    "spark_bsa_workspace_size_joint", "spark_bsa_forward_joint",
]

SPARK_BF16, SPARK_F32 = 0, 1
DEVERR = {"perm": 0x1, "offsets": 0x2, "sel": 0x4, "timeout": 0x8}
EXPORTED = [
    "spark_status_string", "spark_bsa_topk_count", "spark_bsa_workspace_layout",
    "spark_bsa_workspace_size", "spark_bsa_forward", "spark_bsa_read_error",
    "spark_bsa_gather_q", "spark_bsa_anchor", "spark_bsa_gather_kv_summarize",
    "spark_bsa_route", "spark_bsa_attend", "spark_bsa_forward_noalloc",
    "spark_bsa_workspace_size_ctx", "spark_bsa_forward_ctx", "spark_bsa_context_bf16",
    "spark_bsa_attend_ctx", "spark_reblock_workspace_layout", "spark_reblock_workspace_size",
    "spark_reblock_levels", "spark_reblock", "spark_reblock_whiten", "spark_reblock_level",
    "spark_bsa_host_staging_size", "spark_bsa_forward_host", "spark_bsa_quantize_fp8",
    "spark_bsa_attend_fp8", "spark_bsa_workspace_size_fp8", "spark_bsa_forward_fp8",
    "spark_bsa_gather_kv_meanpool", "spark_bsa_route_threshold", "spark_bsa_attend_var",
    "spark_bsa_set_wait_limit_ns", "spark_bsa_get_wait_limit_ns",
    "spark_bsa_host_staging_size_ex", "spark_bsa_forward_host_ex", "spark_bsa_fused_supported",
    "spark_bsa_forward_fused", "spark_bsa_attend_fused", "spark_qk_norm_rope",
    "spark_rope_frequencies", "spark_attend_dense", "spark_attend_dense_workspace_size",
    "spark_attend_ranges", "spark_bsa_workspace_size_joint", "spark_bsa_forward_joint",
]
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
REBLOCK_MODES = {"q_reuse_k": 0, "separate": 1}


class SparkError(RuntimeError):
    def __init__(self, fn, status, msg=""):
        super().__init__(f"{fn} failed: {spark_status_string(status)} ({status}) {msg}".strip())
        self.status = status


class Layout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "Qp", "Kp", "Vp", "qbar_blocks", "qbar", "kbar", "k_tilde", "v_tilde", "cbias", "sel",
        "err", "total")] + [("k", ctypes.c_int)]


class ReblockLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("M", "W", "X", "total")] + \
        [("levels", ctypes.c_int), ("nb", ctypes.c_int)]


_LIB = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_D = ctypes.c_double
_SZ = ctypes.c_size_t


def lib():
    """Loads the library once; raises if it has not been built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with `python -m block_sparse_attention_gather_b200.build`"
            " (nvcc, sm_100a). There is no fallback implementation.")
    L = ctypes.CDLL(LIB_PATH)
    sig = {
        "spark_status_string": (ctypes.c_char_p, [_I]),
        "spark_bsa_topk_count": (_I, [_I, _D]),
        "spark_bsa_set_wait_limit_ns": (None, [ctypes.c_uint64]),
        "spark_bsa_get_wait_limit_ns": (ctypes.c_uint64, []),
        "spark_bsa_workspace_layout": (_I, [_I, _I, _I, _I, _I, _D, ctypes.POINTER(Layout)]),
        "spark_bsa_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _D]),
        "spark_bsa_forward": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _I, _P, _I, _D, _P,
                                   _P, _SZ, _P]),
        "spark_bsa_read_error": (_I, [_P, _P, ctypes.POINTER(ctypes.c_uint32)]),
        "spark_bsa_gather_q": (_I, [_P, _I, _I, _I, _I, _P, _P, _I, _P, _P, _P, _P]),
        "spark_bsa_anchor": (_I, [_P, _P, _I, _I, _I, _I, _P, _P]),
        "spark_bsa_gather_kv_summarize": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _I, _P, _P, _P,
                                               _P, _P, _P, _P, _P, _P]),
        "spark_bsa_route": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _P, _P]),
        "spark_bsa_attend": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _I, _P, _I, _I, _I,
                                  _I, _P, _I, _P, _P]),
        "spark_bsa_forward_noalloc": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _I, _P, _I,
                                           _D, _P, _P]),
        "spark_bsa_workspace_size_ctx": (_SZ, [_I, _I, _I, _I, _I, _D, _I]),
        "spark_bsa_forward_ctx": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _I,
                                       _P, _I, _D, _P, _P, _SZ, _P]),
        "spark_bsa_context_bf16": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _P]),
        "spark_bsa_attend_ctx": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _I, _P, _P, _I,
                                      _P, _I, _I, _I, _I, _P, _I, _P, _P]),
        "spark_reblock_workspace_layout": (_I, [_I, _I, _I, _I, ctypes.POINTER(ReblockLayout)]),
        "spark_reblock_workspace_size": (_SZ, [_I, _I, _I, _I]),
        "spark_reblock_levels": (_I, [_I, _I]),
        "spark_reblock": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _SZ, _P]),
        "spark_reblock_whiten": (_I, [_P, _P, _I, _I, _I, _I, _I, _P, _SZ, _P]),
        "spark_reblock_level": (_I, [_I, _I, _I, _I, _I, _P, _P, _P, _SZ, _P]),
        "spark_bsa_host_staging_size": (_SZ, [_I, _I, _I, _I, _I, _I, _I]),
        "spark_bsa_host_staging_size_ex": (_SZ, [_I, _I, _I, _I, _I, _I, _I, _I]),
        "spark_bsa_fused_supported": (_I, [_I, _I, _D]),
        "spark_bsa_forward_fused": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _I, _P, _I, _D,
                                         _P, _P, _SZ, _P]),
        "spark_bsa_attend_fused": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _I, _P, _I,
                                        _I, _I, _I, _P, _I, _P, _P, _P]),
        "spark_bsa_forward_host_ex": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _P, _P,
                                           _P, _I, _P, _I, _D, _P, _I, _P, _SZ, _P, _SZ, _P,
                                           _P, _P]),
        "spark_bsa_forward_host": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _I, _P, _I, _D,
                                        _P, _I, _P, _SZ, _P, _SZ, _P, _P, _P]),
        "spark_bsa_quantize_fp8": (_I, [_P, _I, _I, _I, _P, _I, _P, _P, _P, _P]),
        "spark_bsa_route_threshold": (_I, [_P, _P, _I, _I, _I, _I, _D, _I, _P, _P, _P, _P]),
        "spark_bsa_attend_var": (_I, [_P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _I, _P, _I,
                                      _I, _I, _I, _P, _I, _P, _P]),
        "spark_bsa_gather_kv_meanpool": (_I, [_P, _P, _I, _I, _I, _I, _P, _P, _I, _P, _P, _P,
                                              _P, _P, _P, _P, _P]),
        "spark_bsa_attend_fp8": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _I, _P, _P, _P, _I,
                                      _P, _P, _I, _P, _I, _I, _I, _I, _P, _I, _P, _P]),
        "spark_qk_norm_rope": (_I, [_P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _D, _P, _I, _I, _P,
                                    _I, _P, _I, _D, _P, _P, _P, _P]),
        "spark_rope_frequencies": (_I, [_P, _I, _D, _I, _D, _D, _P, _P]),
        "spark_attend_dense_workspace_size": (_SZ, [_I, _I, _I, _I, _I]),
        "spark_attend_dense": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _I, _P, _P,
                                    _SZ, _P, _P]),
        "spark_attend_ranges": (_I, [_I, _I, _P, _P, _P, _P, _I, _P, _P, _P]),
        "spark_bsa_workspace_size_joint": (_SZ, [_I, _I, _I, _I, _I, _D, _I]),
        "spark_bsa_forward_joint": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P,
                                         _I, _P, _I, _D, _P, _P, _P, _SZ, _P]),
        "spark_bsa_workspace_size_fp8": (_SZ, [_I, _I, _I, _I, _I, _D, _I]),
        "spark_bsa_forward_fp8": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _P, _P, _P, _I,
                                       _P, _I, _D, _P, _P, _SZ, _P]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _LIB = L
    return L


# ---------------------------------------------------------------------------- helpers

def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _need(t, name, dtype=None, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _code(dtype):
    if dtype == torch.bfloat16:
        return SPARK_BF16
    if dtype == torch.float32:
        return SPARK_F32
    raise TypeError(f"unsupported dtype {dtype}")


def _check(fn, status):
    if status != 0:
        raise SparkError(fn, status)


def _empty(shape, dtype, device, stream):
    """torch.empty for a call on `stream`, from that stream's pool: memory of the current stream's
    could still be in use there, or be handed out again, while the call works on it.  The current
    stream is where the caller reads and drops it."""
    current = None if stream is None else torch.cuda.current_stream(device)
    if stream == current:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(current)
    return t


# ------------------------------------------------------------------------- host calls

def spark_status_string(status: int) -> str:
    return lib().spark_status_string(int(status)).decode()


def spark_bsa_topk_count(nkb: int, topk_ratio: float) -> int:
    return int(lib().spark_bsa_topk_count(int(nkb), float(topk_ratio)))


def spark_bsa_set_wait_limit_ns(limit_ns: int) -> None:
    """Process-wide limit of the kernels' bounded waits (nanoseconds; default 4e9)."""
    lib().spark_bsa_set_wait_limit_ns(int(limit_ns))


def spark_bsa_get_wait_limit_ns() -> int:
    return int(lib().spark_bsa_get_wait_limit_ns())


def spark_bsa_workspace_layout(H, N, d, nqb, nkb, topk_ratio) -> Layout:
    L = Layout()
    _check("spark_bsa_workspace_layout",
           lib().spark_bsa_workspace_layout(H, N, d, nqb, nkb, float(topk_ratio), ctypes.byref(L)))
    return L


def spark_bsa_workspace_size(H, N, d, nqb, nkb, topk_ratio) -> int:
    return int(lib().spark_bsa_workspace_size(H, N, d, nqb, nkb, float(topk_ratio)))


def workspace_views(workspace: torch.Tensor, layout: Layout, H, N, d, nqb, nkb) -> dict:
    """Typed views of the intermediates a spark_bsa_forward call left in `workspace`."""
    def view(off, count, dt):
        nbytes = count * torch.empty(0, dtype=dt).element_size()
        return workspace[off:off + nbytes].view(dt)
    k = layout.k
    return {
        "Qp": view(layout.Qp, H * N * d, torch.bfloat16).view(H, N, d),
        "Kp": view(layout.Kp, H * N * d, torch.bfloat16).view(H, N, d),
        "Vp": view(layout.Vp, H * N * d, torch.bfloat16).view(H, N, d),
        "qbar_blocks": view(layout.qbar_blocks, H * nqb * d, torch.float32).view(H, nqb, d),
        "qbar": view(layout.qbar, H * d, torch.float32).view(H, d),
        "kbar": view(layout.kbar, H * nkb * d, torch.float32).view(H, d, nkb),   # d-major
        "k_tilde": view(layout.k_tilde, H * nkb * d, torch.bfloat16).view(H, nkb, d),
        "v_tilde": view(layout.v_tilde, H * nkb * d, torch.bfloat16).view(H, nkb, d),
        "cbias": view(layout.cbias, H * nkb, torch.float32).view(H, nkb),
        "sel": view(layout.sel, H * nqb * k, torch.int32).view(H, nqb, k),
        "err": view(layout.err, 1, torch.int32),
    }


# --------------------------------------------------------------------------- device calls

def spark_bsa_forward(Q, K, V, q_perm, k_perm, q_offsets, k_offsets, topk_ratio, out=None,
                      workspace=None, stream=None):
    """The whole forward pass on the current CUDA stream; returns (out, workspace, layout)."""
    _need(Q, "Q", (torch.bfloat16, torch.float32))
    dev = Q.device
    for n, t in (("K", K), ("V", V)):
        _need(t, n, Q.dtype, dev)
    H, N, d = Q.shape
    if K.shape != Q.shape or V.shape != Q.shape:
        raise ValueError("Q, K, V must share the shape [H, N, d]")
    for n, t in (("q_perm", q_perm), ("k_perm", k_perm)):
        _need(t, n, torch.int32, dev)
        if t.shape != (H, N):
            raise ValueError(f"{n} must have shape [H, N]")
    for n, t in (("q_offsets", q_offsets), ("k_offsets", k_offsets)):
        _need(t, n, torch.int32, dev)
    nqb, nkb = q_offsets.numel() - 1, k_offsets.numel() - 1
    layout = spark_bsa_workspace_layout(H, N, d, nqb, nkb, topk_ratio)
    if out is None:
        out = torch.empty_like(Q)
    _need(out, "out", Q.dtype, dev)
    if workspace is None:
        workspace = torch.empty(layout.total, dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    st = lib().spark_bsa_forward(_ptr(Q), _ptr(K), _ptr(V), _code(Q.dtype), H, N, d,
                                 _ptr(q_perm), _ptr(k_perm), _ptr(q_offsets), nqb,
                                 _ptr(k_offsets), nkb, float(topk_ratio), _ptr(out),
                                 _ptr(workspace), workspace.numel(), _stream(stream))
    _check("spark_bsa_forward", st)
    return out, workspace, layout


def spark_bsa_fused_supported(d: int, nkb: int, topk_ratio: float) -> bool:
    return bool(lib().spark_bsa_fused_supported(int(d), int(nkb), float(topk_ratio)))


def spark_bsa_forward_fused(Q, K, V, q_perm, k_perm, q_offsets, k_offsets, topk_ratio, out=None,
                            workspace=None, stream=None):
    """spark_bsa_forward with the routing inside the attention kernel; returns (out, workspace,
    layout) with the selections copied to the workspace's sel region."""
    _need(Q, "Q", (torch.bfloat16, torch.float32))
    dev = Q.device
    for n, t in (("K", K), ("V", V)):
        _need(t, n, Q.dtype, dev)
    H, N, d = Q.shape
    for n, t in (("q_perm", q_perm), ("k_perm", k_perm), ("q_offsets", q_offsets),
                 ("k_offsets", k_offsets)):
        _need(t, n, torch.int32, dev)
    nqb, nkb = q_offsets.numel() - 1, k_offsets.numel() - 1
    layout = spark_bsa_workspace_layout(H, N, d, nqb, nkb, topk_ratio)
    if out is None:
        out = torch.empty_like(Q)
    _need(out, "out", Q.dtype, dev)
    if workspace is None:
        workspace = torch.empty(layout.total, dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    st = lib().spark_bsa_forward_fused(_ptr(Q), _ptr(K), _ptr(V), _code(Q.dtype), H, N, d,
                                       _ptr(q_perm), _ptr(k_perm), _ptr(q_offsets), nqb,
                                       _ptr(k_offsets), nkb, float(topk_ratio), _ptr(out),
                                       _ptr(workspace), workspace.numel(), _stream(stream))
    _check("spark_bsa_forward_fused", st)
    return out, workspace, layout


def spark_bsa_attend_fused(Qp, Kp, Vp, k_tilde, v_tilde, cbias, qbar_blocks, kbar, k, q_perm,
                           q_offsets, k_offsets, out_dtype=torch.bfloat16, out=None, sel_out=None,
                           err=None, stream=None):
    _need(Qp, "Qp", torch.bfloat16)
    dev = Qp.device
    H, N, d = Qp.shape
    for n, t, dt in (("Kp", Kp, torch.bfloat16), ("Vp", Vp, torch.bfloat16),
                     ("k_tilde", k_tilde, torch.bfloat16), ("v_tilde", v_tilde, torch.bfloat16),
                     ("cbias", cbias, torch.float32), ("qbar_blocks", qbar_blocks, torch.float32),
                     ("kbar", kbar, torch.float32), ("q_perm", q_perm, torch.int32),
                     ("q_offsets", q_offsets, torch.int32), ("k_offsets", k_offsets, torch.int32)):
        _need(t, n, dt, dev)
    nqb, nkb = q_offsets.numel() - 1, k_offsets.numel() - 1
    if out is None:
        out = torch.empty(H, N, d, dtype=out_dtype, device=dev)
    st = lib().spark_bsa_attend_fused(_ptr(Qp), _ptr(Kp), _ptr(Vp), _ptr(k_tilde), _ptr(v_tilde),
                                      _ptr(cbias), _ptr(qbar_blocks), _ptr(kbar), int(k),
                                      _ptr(q_perm), _ptr(q_offsets), nqb, _ptr(k_offsets), nkb,
                                      H, N, d, _ptr(out), _code(out.dtype), _ptr(sel_out),
                                      _ptr(err), _stream(stream))
    _check("spark_bsa_attend_fused", st)
    return out


def spark_bsa_read_error(err_word: torch.Tensor, stream=None) -> int:
    """Synchronises the stream and returns the device error word (0 = no error)."""
    _need(err_word, "err_word")
    flags = ctypes.c_uint32(0)
    st = lib().spark_bsa_read_error(_ptr(err_word), _stream(stream), ctypes.byref(flags))
    if st not in (0, 5):
        raise SparkError("spark_bsa_read_error", st)
    return int(flags.value)


def spark_bsa_gather_q(Q, q_perm, q_offsets, Qp=None, qbar_blocks=None, err=None, stream=None):
    _need(Q, "Q", (torch.bfloat16, torch.float32))
    H, N, d = Q.shape
    nqb = q_offsets.numel() - 1
    Qp = torch.empty(H, N, d, dtype=torch.bfloat16, device=Q.device) if Qp is None else Qp
    qbar_blocks = (torch.empty(H, nqb, d, dtype=torch.float32, device=Q.device)
                   if qbar_blocks is None else qbar_blocks)
    for n, t, dt in (("q_perm", q_perm, torch.int32), ("q_offsets", q_offsets, torch.int32),
                     ("Qp", Qp, torch.bfloat16), ("qbar_blocks", qbar_blocks, torch.float32)):
        _need(t, n, dt, Q.device)
    st = lib().spark_bsa_gather_q(_ptr(Q), _code(Q.dtype), H, N, d, _ptr(q_perm),
                                  _ptr(q_offsets), nqb, _ptr(Qp), _ptr(qbar_blocks), _ptr(err),
                                  _stream(stream))
    _check("spark_bsa_gather_q", st)
    return Qp, qbar_blocks


def spark_bsa_anchor(qbar_blocks, q_offsets, N, qbar=None, stream=None):
    _need(qbar_blocks, "qbar_blocks", torch.float32)
    H, nqb, d = qbar_blocks.shape
    qbar = torch.empty(H, d, dtype=torch.float32, device=qbar_blocks.device) if qbar is None else qbar
    _need(q_offsets, "q_offsets", torch.int32, qbar_blocks.device)
    _need(qbar, "qbar", torch.float32, qbar_blocks.device)
    st = lib().spark_bsa_anchor(_ptr(qbar_blocks), _ptr(q_offsets), H, N, d, nqb, _ptr(qbar),
                                _stream(stream))
    _check("spark_bsa_anchor", st)
    return qbar


def spark_bsa_gather_kv_summarize(K, V, k_perm, k_offsets, qbar, err=None, stream=None):
    _need(K, "K", (torch.bfloat16, torch.float32))
    _need(V, "V", K.dtype, K.device)
    H, N, d = K.shape
    nkb = k_offsets.numel() - 1
    dev = K.device
    _need(k_perm, "k_perm", torch.int32, dev)
    _need(k_offsets, "k_offsets", torch.int32, dev)
    _need(qbar, "qbar", torch.float32, dev)
    Kp = torch.empty(H, N, d, dtype=torch.bfloat16, device=dev)
    Vp = torch.empty_like(Kp)
    kbar = torch.empty(H, d, nkb, dtype=torch.float32, device=dev)          # d-major
    k_tilde = torch.empty(H, nkb, d, dtype=torch.bfloat16, device=dev)
    v_tilde = torch.empty_like(k_tilde)
    cbias = torch.empty(H, nkb, dtype=torch.float32, device=dev)
    st = lib().spark_bsa_gather_kv_summarize(
        _ptr(K), _ptr(V), _code(K.dtype), H, N, d, _ptr(k_perm), _ptr(k_offsets), nkb,
        _ptr(qbar), _ptr(Kp), _ptr(Vp), _ptr(kbar), _ptr(k_tilde), _ptr(v_tilde), _ptr(cbias),
        _ptr(err), _stream(stream))
    _check("spark_bsa_gather_kv_summarize", st)
    return Kp, Vp, kbar, k_tilde, v_tilde, cbias


def spark_bsa_route_threshold(qbar_blocks, kbar, tau, kcap, err=None, stream=None):
    """Threshold routing (mu + tau*sigma per query block, at most kcap blocks); returns
    (sel [H, nqb, kcap] with the first count entries of each row valid, count [H, nqb])."""
    _need(qbar_blocks, "qbar_blocks", torch.float32)
    _need(kbar, "kbar", torch.float32, qbar_blocks.device)
    H, nqb, d = qbar_blocks.shape
    nkb = kbar.shape[2]                                                     # kbar is [H, d, nkb]
    sel = torch.full((H, nqb, kcap), -1, dtype=torch.int32, device=qbar_blocks.device)
    count = torch.empty(H, nqb, dtype=torch.int32, device=qbar_blocks.device)
    st = lib().spark_bsa_route_threshold(_ptr(qbar_blocks), _ptr(kbar), H, nqb, nkb, d,
                                         float(tau), int(kcap), _ptr(sel), _ptr(count),
                                         _ptr(err), _stream(stream))
    _check("spark_bsa_route_threshold", st)
    return sel, count


def spark_bsa_attend_var(Qp, Kp, Vp, k_tilde, v_tilde, cbias, sel, count, q_perm, q_offsets,
                         k_offsets, out_dtype=torch.bfloat16, out=None, err=None, stream=None):
    """spark_bsa_attend with a per-query-block count of selected blocks (sel [H, nqb, kcap])."""
    _need(Qp, "Qp", torch.bfloat16)
    dev = Qp.device
    H, N, d = Qp.shape
    for n, t, dt in (("Kp", Kp, torch.bfloat16), ("Vp", Vp, torch.bfloat16),
                     ("k_tilde", k_tilde, torch.bfloat16), ("v_tilde", v_tilde, torch.bfloat16),
                     ("cbias", cbias, torch.float32), ("sel", sel, torch.int32),
                     ("count", count, torch.int32), ("q_perm", q_perm, torch.int32),
                     ("q_offsets", q_offsets, torch.int32), ("k_offsets", k_offsets, torch.int32)):
        _need(t, n, dt, dev)
    nqb, nkb = q_offsets.numel() - 1, k_offsets.numel() - 1
    kcap = sel.shape[-1]
    if out is None:
        out = torch.empty(H, N, d, dtype=out_dtype, device=dev)
    _need(out, "out", out_dtype, dev)
    st = lib().spark_bsa_attend_var(_ptr(Qp), _ptr(Kp), _ptr(Vp), _ptr(k_tilde), _ptr(v_tilde),
                                    _ptr(cbias), _ptr(sel), kcap, _ptr(count), _ptr(q_perm),
                                    _ptr(q_offsets), nqb, _ptr(k_offsets), nkb, H, N, d,
                                    _ptr(out), _code(out_dtype), _ptr(err), _stream(stream))
    _check("spark_bsa_attend_var", st)
    return out


def spark_bsa_gather_kv_meanpool(K, V, k_perm, k_offsets, err=None, stream=None):
    """The baseline BSA compressed branch (mean key, mean value, offset log|B|) with the same
    gathered Kp, Vp and key-block means as spark_bsa_gather_kv_summarize; returns
    (Kp, Vp, kbar, k_tilde, v_tilde, cbias)."""
    _need(K, "K", (torch.bfloat16, torch.float32))
    dev = K.device
    H, N, d = K.shape
    _need(V, "V", K.dtype, dev)
    _need(k_perm, "k_perm", torch.int32, dev)
    _need(k_offsets, "k_offsets", torch.int32, dev)
    nkb = k_offsets.numel() - 1
    Kp = torch.empty(H, N, d, dtype=torch.bfloat16, device=dev)
    Vp = torch.empty_like(Kp)
    kbar = torch.empty(H, d, nkb, dtype=torch.float32, device=dev)          # d-major
    k_tilde = torch.empty(H, nkb, d, dtype=torch.bfloat16, device=dev)
    v_tilde = torch.empty_like(k_tilde)
    cbias = torch.empty(H, nkb, dtype=torch.float32, device=dev)
    st = lib().spark_bsa_gather_kv_meanpool(
        _ptr(K), _ptr(V), _code(K.dtype), H, N, d, _ptr(k_perm), _ptr(k_offsets), nkb, _ptr(Kp),
        _ptr(Vp), _ptr(kbar), _ptr(k_tilde), _ptr(v_tilde), _ptr(cbias), _ptr(err),
        _stream(stream))
    _check("spark_bsa_gather_kv_meanpool", st)
    return Kp, Vp, kbar, k_tilde, v_tilde, cbias


def spark_bsa_route(qbar_blocks, kbar, k, err=None, stream=None):
    _need(qbar_blocks, "qbar_blocks", torch.float32)
    _need(kbar, "kbar", torch.float32, qbar_blocks.device)
    H, nqb, d = qbar_blocks.shape
    nkb = kbar.shape[2]                                                     # kbar is [H, d, nkb]
    sel = torch.empty(H, nqb, k, dtype=torch.int32, device=qbar_blocks.device)
    st = lib().spark_bsa_route(_ptr(qbar_blocks), _ptr(kbar), H, nqb, nkb, d, int(k), _ptr(sel),
                               _ptr(err), _stream(stream))
    _check("spark_bsa_route", st)
    return sel


def spark_bsa_attend(Qp, Kp, Vp, k_tilde, v_tilde, cbias, sel, q_perm, q_offsets, k_offsets,
                     out_dtype=torch.bfloat16, out=None, err=None, stream=None):
    _need(Qp, "Qp", torch.bfloat16)
    dev = Qp.device
    H, N, d = Qp.shape
    for n, t, dt in (("Kp", Kp, torch.bfloat16), ("Vp", Vp, torch.bfloat16),
                     ("k_tilde", k_tilde, torch.bfloat16), ("v_tilde", v_tilde, torch.bfloat16),
                     ("cbias", cbias, torch.float32), ("sel", sel, torch.int32),
                     ("q_perm", q_perm, torch.int32), ("q_offsets", q_offsets, torch.int32),
                     ("k_offsets", k_offsets, torch.int32)):
        _need(t, n, dt, dev)
    nqb, nkb = q_offsets.numel() - 1, k_offsets.numel() - 1
    k = sel.shape[-1]
    if out is None:
        out = torch.empty(H, N, d, dtype=out_dtype, device=dev)
    _need(out, "out", out_dtype, dev)
    st = lib().spark_bsa_attend(_ptr(Qp), _ptr(Kp), _ptr(Vp), _ptr(k_tilde), _ptr(v_tilde),
                                _ptr(cbias), _ptr(sel), k, _ptr(q_perm), _ptr(q_offsets), nqb,
                                _ptr(k_offsets), nkb, H, N, d, _ptr(out), _code(out_dtype),
                                _ptr(err), _stream(stream))
    _check("spark_bsa_attend", st)
    return out


def spark_bsa_forward_noalloc(Q, K, V, q_perm, k_perm, q_offsets, k_offsets, topk_ratio,
                              out, stream=None):
    """The forward pass with the library's static scratch array as its workspace (for callers
    that cannot allocate device memory while they run); `out` must be preallocated.  Small
    problems only: the workspace must fit SPARK_NOALLOC_SCRATCH_BYTES (16 MiB)."""
    _need(Q, "Q", (torch.bfloat16, torch.float32))
    dev = Q.device
    H, N, d = Q.shape
    for n, t in (("K", K), ("V", V), ("out", out)):
        _need(t, n, Q.dtype, dev)
    for n, t in (("q_perm", q_perm), ("k_perm", k_perm), ("q_offsets", q_offsets),
                 ("k_offsets", k_offsets)):
        _need(t, n, torch.int32, dev)
    nqb, nkb = q_offsets.numel() - 1, k_offsets.numel() - 1
    st = lib().spark_bsa_forward_noalloc(_ptr(Q), _ptr(K), _ptr(V), _code(Q.dtype), H, N, d,
                                         _ptr(q_perm), _ptr(k_perm), _ptr(q_offsets), nqb,
                                         _ptr(k_offsets), nkb, float(topk_ratio), _ptr(out),
                                         _stream(stream))
    _check("spark_bsa_forward_noalloc", st)
    return out


# ------------------------------------------------------------------ context (sink) tokens

def spark_bsa_workspace_size_ctx(H, N, d, nqb, nkb, topk_ratio, nc) -> int:
    return int(lib().spark_bsa_workspace_size_ctx(H, N, d, nqb, nkb, float(topk_ratio), int(nc)))


def _context_args(Kc, Vc, H, d, dtype, dev):
    if Kc is None and Vc is None:
        return None, None, 0
    _need(Kc, "Kc", dtype, dev)
    _need(Vc, "Vc", dtype, dev)
    if Kc.dim() != 3 or Kc.shape[0] != H or Kc.shape[2] != d or Vc.shape != Kc.shape:
        raise ValueError("Kc and Vc must have the shape [H, nc, d]")
    return Kc, Vc, Kc.shape[1]


def spark_bsa_forward_ctx(Q, K, V, Kc, Vc, q_perm, k_perm, q_offsets, k_offsets, topk_ratio,
                          out=None, workspace=None, stream=None):
    """spark_bsa_forward with context (sink) tokens Kc, Vc [H, nc, d] (same dtype as Q);
    returns (out, workspace, layout).  The workspace holds the layout's intermediates followed
    by the bf16 context rows."""
    _need(Q, "Q", (torch.bfloat16, torch.float32))
    dev = Q.device
    H, N, d = Q.shape
    for n, t in (("K", K), ("V", V)):
        _need(t, n, Q.dtype, dev)
    if K.shape != Q.shape or V.shape != Q.shape:
        raise ValueError("Q, K, V must share the shape [H, N, d]")
    Kc, Vc, nc = _context_args(Kc, Vc, H, d, Q.dtype, dev)
    for n, t in (("q_perm", q_perm), ("k_perm", k_perm)):
        _need(t, n, torch.int32, dev)
        if t.shape != (H, N):
            raise ValueError(f"{n} must have shape [H, N]")
    for n, t in (("q_offsets", q_offsets), ("k_offsets", k_offsets)):
        _need(t, n, torch.int32, dev)
    nqb, nkb = q_offsets.numel() - 1, k_offsets.numel() - 1
    layout = spark_bsa_workspace_layout(H, N, d, nqb, nkb, topk_ratio)
    size = spark_bsa_workspace_size_ctx(H, N, d, nqb, nkb, topk_ratio, nc)
    if out is None:
        out = torch.empty_like(Q)
    _need(out, "out", Q.dtype, dev)
    if workspace is None:
        workspace = torch.empty(size, dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    st = lib().spark_bsa_forward_ctx(_ptr(Q), _ptr(K), _ptr(V), _ptr(Kc), _ptr(Vc), nc,
                                     _code(Q.dtype), H, N, d, _ptr(q_perm), _ptr(k_perm),
                                     _ptr(q_offsets), nqb, _ptr(k_offsets), nkb,
                                     float(topk_ratio), _ptr(out), _ptr(workspace),
                                     workspace.numel(), _stream(stream))
    _check("spark_bsa_forward_ctx", st)
    return out, workspace, layout


def spark_bsa_context_bf16(Kc, Vc, Kc_bf16=None, Vc_bf16=None, stream=None):
    """bf16 copies of the context rows ([H, nc, d]); returns (Kc_bf16, Vc_bf16)."""
    _need(Kc, "Kc", (torch.bfloat16, torch.float32))
    H, nc, d = Kc.shape
    Kc, Vc, nc = _context_args(Kc, Vc, H, d, Kc.dtype, Kc.device)
    if Kc_bf16 is None:
        Kc_bf16 = torch.empty(H, nc, d, dtype=torch.bfloat16, device=Kc.device)
    if Vc_bf16 is None:
        Vc_bf16 = torch.empty(H, nc, d, dtype=torch.bfloat16, device=Kc.device)
    _need(Kc_bf16, "Kc_bf16", torch.bfloat16, Kc.device)
    _need(Vc_bf16, "Vc_bf16", torch.bfloat16, Kc.device)
    st = lib().spark_bsa_context_bf16(_ptr(Kc), _ptr(Vc), _code(Kc.dtype), H, nc, d,
                                      _ptr(Kc_bf16), _ptr(Vc_bf16), _stream(stream))
    _check("spark_bsa_context_bf16", st)
    return Kc_bf16, Vc_bf16


def spark_bsa_attend_ctx(Qp, Kp, Vp, k_tilde, v_tilde, cbias, sel, Kc, Vc, q_perm, q_offsets,
                         k_offsets, out_dtype=torch.bfloat16, out=None, err=None, stream=None):
    """spark_bsa_attend with bf16 context rows Kc, Vc [H, nc, d]."""
    _need(Qp, "Qp", torch.bfloat16)
    dev = Qp.device
    H, N, d = Qp.shape
    for n, t, dt in (("Kp", Kp, torch.bfloat16), ("Vp", Vp, torch.bfloat16),
                     ("k_tilde", k_tilde, torch.bfloat16), ("v_tilde", v_tilde, torch.bfloat16),
                     ("cbias", cbias, torch.float32), ("sel", sel, torch.int32),
                     ("q_perm", q_perm, torch.int32), ("q_offsets", q_offsets, torch.int32),
                     ("k_offsets", k_offsets, torch.int32)):
        _need(t, n, dt, dev)
    Kc, Vc, nc = _context_args(Kc, Vc, H, d, torch.bfloat16, dev)
    nqb, nkb = q_offsets.numel() - 1, k_offsets.numel() - 1
    k = sel.shape[-1]
    if out is None:
        out = torch.empty(H, N, d, dtype=out_dtype, device=dev)
    _need(out, "out", out_dtype, dev)
    st = lib().spark_bsa_attend_ctx(_ptr(Qp), _ptr(Kp), _ptr(Vp), _ptr(k_tilde), _ptr(v_tilde),
                                    _ptr(cbias), _ptr(sel), k, _ptr(Kc), _ptr(Vc), nc,
                                    _ptr(q_perm), _ptr(q_offsets), nqb, _ptr(k_offsets), nkb,
                                    H, N, d, _ptr(out), _code(out_dtype), _ptr(err),
                                    _stream(stream))
    _check("spark_bsa_attend_ctx", st)
    return out


# ------------------------------------------------------------------------- FP8 logits

def spark_bsa_quantize_fp8(src, group_offsets=None, dst=None, scales=None, err=None,
                           stream=None):
    """e4m3 codes (torch.uint8 [H, R, d]) and power-of-two group scales (fp32 [H, ngroups]) of
    bf16 rows src [H, R, d]; groups are the blocks of group_offsets (int32 [ngroups+1]) or,
    when it is None, 128-row tiles.  Returns (dst, scales)."""
    _need(src, "src", torch.bfloat16)
    dev = src.device
    H, R, d = src.shape
    if group_offsets is None:
        ngroups = (R + 127) // 128
    else:
        _need(group_offsets, "group_offsets", torch.int32, dev)
        ngroups = group_offsets.numel() - 1
    if dst is None:
        dst = torch.empty(H, R, d, dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty(H, ngroups, dtype=torch.float32, device=dev)
    _need(dst, "dst", torch.uint8, dev)
    _need(scales, "scales", torch.float32, dev)
    st = lib().spark_bsa_quantize_fp8(_ptr(src), H, R, d, _ptr(group_offsets), ngroups,
                                      _ptr(dst), _ptr(scales), _ptr(err), _stream(stream))
    _check("spark_bsa_quantize_fp8", st)
    return dst, scales


def spark_bsa_attend_fp8(Qp8, q_scale, Kp8, k_scale, Vp, kt8, kt_scale, v_tilde, cbias, sel,
                         q_perm, q_offsets, k_offsets, Kc8=None, kc_scale=None, Vc=None,
                         out_dtype=torch.bfloat16, out=None, err=None, stream=None):
    """The attention step with FP8 logits (codes and scales from spark_bsa_quantize_fp8,
    values in bf16; d = 128)."""
    _need(Qp8, "Qp8", torch.uint8)
    dev = Qp8.device
    H, N, d = Qp8.shape
    for n, t, dt in (("q_scale", q_scale, torch.float32), ("Kp8", Kp8, torch.uint8),
                     ("k_scale", k_scale, torch.float32), ("Vp", Vp, torch.bfloat16),
                     ("kt8", kt8, torch.uint8), ("kt_scale", kt_scale, torch.float32),
                     ("v_tilde", v_tilde, torch.bfloat16), ("cbias", cbias, torch.float32),
                     ("sel", sel, torch.int32), ("q_perm", q_perm, torch.int32),
                     ("q_offsets", q_offsets, torch.int32), ("k_offsets", k_offsets, torch.int32)):
        _need(t, n, dt, dev)
    nc = 0
    if Kc8 is not None:
        _need(Kc8, "Kc8", torch.uint8, dev)
        _need(kc_scale, "kc_scale", torch.float32, dev)
        _need(Vc, "Vc", torch.bfloat16, dev)
        nc = Kc8.shape[1]
    nqb, nkb = q_offsets.numel() - 1, k_offsets.numel() - 1
    k = sel.shape[-1]
    if out is None:
        out = torch.empty(H, N, d, dtype=out_dtype, device=dev)
    _need(out, "out", out_dtype, dev)
    st = lib().spark_bsa_attend_fp8(_ptr(Qp8), _ptr(q_scale), _ptr(Kp8), _ptr(k_scale), _ptr(Vp),
                                    _ptr(kt8), _ptr(kt_scale), _ptr(v_tilde), _ptr(cbias),
                                    _ptr(sel), k, _ptr(Kc8), _ptr(kc_scale), _ptr(Vc), nc,
                                    _ptr(q_perm), _ptr(q_offsets), nqb, _ptr(k_offsets), nkb,
                                    H, N, d, _ptr(out), _code(out_dtype), _ptr(err),
                                    _stream(stream))
    _check("spark_bsa_attend_fp8", st)
    return out


def spark_bsa_workspace_size_fp8(H, N, d, nqb, nkb, topk_ratio, nc=0) -> int:
    return int(lib().spark_bsa_workspace_size_fp8(H, N, d, nqb, nkb, float(topk_ratio), int(nc)))


def spark_bsa_forward_fp8(Q, K, V, q_perm, k_perm, q_offsets, k_offsets, topk_ratio, Kc=None,
                          Vc=None, out=None, workspace=None, stream=None):
    """spark_bsa_forward_ctx with FP8 logits (d = 128); returns (out, workspace, layout)."""
    _need(Q, "Q", (torch.bfloat16, torch.float32))
    dev = Q.device
    H, N, d = Q.shape
    for n, t in (("K", K), ("V", V)):
        _need(t, n, Q.dtype, dev)
    if K.shape != Q.shape or V.shape != Q.shape:
        raise ValueError("Q, K, V must share the shape [H, N, d]")
    Kc, Vc, nc = _context_args(Kc, Vc, H, d, Q.dtype, dev)
    for n, t in (("q_perm", q_perm), ("k_perm", k_perm)):
        _need(t, n, torch.int32, dev)
    for n, t in (("q_offsets", q_offsets), ("k_offsets", k_offsets)):
        _need(t, n, torch.int32, dev)
    nqb, nkb = q_offsets.numel() - 1, k_offsets.numel() - 1
    layout = spark_bsa_workspace_layout(H, N, d, nqb, nkb, topk_ratio)
    size = spark_bsa_workspace_size_fp8(H, N, d, nqb, nkb, topk_ratio, nc)
    if size == 0:
        raise SparkError("spark_bsa_workspace_size_fp8", 2)
    if out is None:
        out = torch.empty_like(Q)
    _need(out, "out", Q.dtype, dev)
    if workspace is None:
        workspace = torch.empty(size, dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    st = lib().spark_bsa_forward_fp8(_ptr(Q), _ptr(K), _ptr(V), _ptr(Kc), _ptr(Vc), nc,
                                     _code(Q.dtype), H, N, d, _ptr(q_perm), _ptr(k_perm),
                                     _ptr(q_offsets), nqb, _ptr(k_offsets), nkb,
                                     float(topk_ratio), _ptr(out), _ptr(workspace),
                                     workspace.numel(), _stream(stream))
    _check("spark_bsa_forward_fp8", st)
    return out, workspace, layout


# ------------------------------------------------------------ Spark-Reblock partitioner

def spark_reblock_workspace_layout(H, N, d, block) -> ReblockLayout:
    L = ReblockLayout()
    _check("spark_reblock_workspace_layout",
           lib().spark_reblock_workspace_layout(H, N, d, block, ctypes.byref(L)))
    return L


def spark_reblock_workspace_size(H, N, d, block) -> int:
    return int(lib().spark_reblock_workspace_size(H, N, d, block))


def spark_reblock_levels(N, block) -> int:
    return int(lib().spark_reblock_levels(N, block))


def reblock_views(workspace: torch.Tensor, layout: ReblockLayout, H, N, d) -> dict:
    """Typed views of M, W (fp32 [H,d,d]) and X (bf16 [H,N,d]) in a reblock workspace."""
    def view(off, count, dt):
        nbytes = count * torch.empty(0, dtype=dt).element_size()
        return workspace[off:off + nbytes].view(dt)
    return {"M": view(layout.M, H * d * d, torch.float32).view(H, d, d),
            "W": view(layout.W, H * d * d, torch.float32).view(H, d, d),
            "X": view(layout.X, H * N * d, torch.bfloat16).view(H, N, d)}


def spark_reblock(Q, K, block, mode="q_reuse_k", workspace=None, stream=None):
    """Spark-Reblock partition of Q, K [H, N, d]; returns (q_perm, k_perm, offsets)."""
    _need(Q, "Q", (torch.bfloat16, torch.float32))
    _need(K, "K", Q.dtype, Q.device)
    H, N, d = Q.shape
    if K.shape != Q.shape:
        raise ValueError("Q and K must share the shape [H, N, d]")
    layout = spark_reblock_workspace_layout(H, N, d, block)
    if workspace is None:
        workspace = _empty(layout.total, torch.uint8, Q.device, stream)
    _need(workspace, "workspace", torch.uint8, Q.device)
    q_perm = _empty((H, N), torch.int32, Q.device, stream)
    k_perm = _empty((H, N), torch.int32, Q.device, stream)
    offsets = _empty(layout.nb + 1, torch.int32, Q.device, stream)
    st = lib().spark_reblock(_ptr(Q), _ptr(K), _code(Q.dtype), H, N, d, int(block),
                             REBLOCK_MODES[mode], _ptr(q_perm), _ptr(k_perm), _ptr(offsets),
                             _ptr(workspace), workspace.numel(), _stream(stream))
    _check("spark_reblock", st)
    return q_perm, k_perm, offsets


def spark_reblock_whiten(X, Y, block, workspace=None, stream=None):
    """Step: second moment of Y, its square root W, unit rows of W x into the workspace;
    returns (workspace, layout, views)."""
    _need(X, "X", (torch.bfloat16, torch.float32))
    _need(Y, "Y", X.dtype, X.device)
    H, N, d = X.shape
    layout = spark_reblock_workspace_layout(H, N, d, block)
    if workspace is None:
        workspace = torch.empty(layout.total, dtype=torch.uint8, device=X.device)
    st = lib().spark_reblock_whiten(_ptr(X), _ptr(Y), _code(X.dtype), H, N, d, int(block),
                                    _ptr(workspace), workspace.numel(), _stream(stream))
    _check("spark_reblock_whiten", st)
    return workspace, layout, reblock_views(workspace, layout, H, N, d)


def spark_reblock_level(H, N, d, block, level, perm_in, workspace, perm_out=None, stream=None):
    """Step: the splits of one tree level over the workspace's X rows; returns perm_out."""
    _need(perm_in, "perm_in", torch.int32)
    if perm_out is None:
        perm_out = torch.empty_like(perm_in)
    st = lib().spark_reblock_level(H, N, d, int(block), int(level), _ptr(perm_in),
                                   _ptr(perm_out), _ptr(workspace), workspace.numel(),
                                   _stream(stream))
    _check("spark_reblock_level", st)
    return perm_out


# ------------------------------------------------ host buffers, pipelined by head chunks

def spark_bsa_host_staging_size(H, N, d, dtype, nqb, nkb, heads_per_chunk) -> int:
    return int(lib().spark_bsa_host_staging_size(H, N, d, _code(dtype), nqb, nkb,
                                                  heads_per_chunk))


def _need_host(t, name, dtype=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.is_cuda:
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")


def spark_bsa_host_staging_size_ex(H, N, d, dtype, nqb, nkb, heads_per_chunk, nc) -> int:
    return int(lib().spark_bsa_host_staging_size_ex(H, N, d, _code(dtype), nqb, nkb,
                                                    heads_per_chunk, nc))


def spark_bsa_forward_host(Q, K, V, q_perm, k_perm, q_offsets, k_offsets, topk_ratio, out=None,
                           heads_per_chunk=1, device=None, staging=None, workspace=None,
                           streams=None, Kc=None, Vc=None, fp8=False):
    """The forward pass on HOST tensors (page-locked for overlap), pipelined by head chunks
    over three CUDA streams; returns `out` (host) once the work is enqueued on the compute
    stream (synchronise that stream, or the device, before reading it).  Kc, Vc (host
    [H, nc, d]) add context rows; fp8=True takes the logits in e4m3 (d = 128)."""
    _need_host(Q, "Q", (torch.bfloat16, torch.float32))
    for n, t in (("K", K), ("V", V)):
        _need_host(t, n, Q.dtype)
    for n, t in (("q_perm", q_perm), ("k_perm", k_perm), ("q_offsets", q_offsets),
                 ("k_offsets", k_offsets)):
        _need_host(t, n, torch.int32)
    H, N, d = Q.shape
    nc = 0
    if Kc is not None or Vc is not None:
        for n, t in (("Kc", Kc), ("Vc", Vc)):
            _need_host(t, n, Q.dtype)
        if Kc.shape != Vc.shape or Kc.shape[0] != H or Kc.shape[2] != d:
            raise ValueError("Kc, Vc must have the shape [H, nc, d]")
        nc = Kc.shape[1]
    nqb, nkb = q_offsets.numel() - 1, k_offsets.numel() - 1
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    hpc = max(1, min(int(heads_per_chunk), H))
    if out is None:
        out = torch.empty_like(Q).pin_memory()
    _need_host(out, "out", Q.dtype)
    if streams is None:
        streams = (torch.cuda.current_stream(dev), torch.cuda.Stream(dev), torch.cuda.Stream(dev))
    streams = tuple(streams)
    if staging is None:                  # the copy streams start and end within the compute stream
        staging = _empty(spark_bsa_host_staging_size_ex(H, N, d, Q.dtype, nqb, nkb, hpc, nc),
                         torch.uint8, dev, streams[0])
    if workspace is None:
        size = (spark_bsa_workspace_size_fp8(hpc, N, d, nqb, nkb, topk_ratio, nc) if fp8 else
                spark_bsa_workspace_size_ctx(hpc, N, d, nqb, nkb, topk_ratio, nc))
        workspace = _empty(size, torch.uint8, dev, streams[0])
    sc, sh, sd = (ctypes.c_void_p(s.cuda_stream) for s in streams)
    st = lib().spark_bsa_forward_host_ex(_ptr(Q), _ptr(K), _ptr(V),
                                         _ptr(Kc) if nc else None, _ptr(Vc) if nc else None, nc,
                                         1 if fp8 else 0, _code(Q.dtype), H, N, d,
                                         _ptr(q_perm), _ptr(k_perm), _ptr(q_offsets), nqb,
                                         _ptr(k_offsets), nkb, float(topk_ratio), _ptr(out), hpc,
                                         _ptr(staging), staging.numel(), _ptr(workspace),
                                         workspace.numel(), sc, sh, sd)
    _check("spark_bsa_forward_host", st)
    return out


# ------------------------------------------------ norm and rotation, dense attention

# The calls below can take as long on the host as their kernels do on the GPU, so the usual case of
# a check is one expression, and the messages are made where one fails.

def _launch(index, fn, *args):
    """fn(*args) with device `index` current, whose stream the arguments name."""
    if index == torch.cuda.current_device():
        return fn(*args)
    with torch.cuda.device(index):
        return fn(*args)


def _stream_of(index, stream):
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(index)
    return stream.cuda_stream


def _refuse(t, name, dtype, device, shape):
    """Raises what is wrong with a tensor that failed its check."""
    _need(t, name, dtype, device)
    raise ValueError(f"{name} must have the shape {shape}")


def _type_error(required, **tensors):
    """An attribute was missing: names the argument that is no tensor."""
    for name, t in tensors.items():
        if not isinstance(t, torch.Tensor) and (t is not None or name in required):
            raise TypeError(f"{name} must be a torch.Tensor") from None


def spark_rope_frequencies(axis_pairs, base=10000.0, scaling="none", factor=1.0, original=0.0):
    """Rotation frequencies of the axes (fp32 CPU tensor of sum(axis_pairs)) and the factor for
    rope_scale; scaling is "none", "linear", "ntk" or "yarn"."""
    n = len(axis_pairs)
    counts = (ctypes.c_int32 * max(n, 1))(*(int(p) for p in axis_pairs))
    out = torch.empty(max(sum(max(int(p), 0) for p in axis_pairs), 1), dtype=torch.float32)
    scale = ctypes.c_double(1.0)
    st = lib().spark_rope_frequencies(counts, n, float(base), ROPE_SCALINGS[scaling],
                                      float(factor), float(original), _ptr(out),
                                      ctypes.byref(scale))
    _check("spark_rope_frequencies", st)
    return out[:sum(int(p) for p in axis_pairs)], scale.value


def _refuse_rows(t, name, dtype, device):
    """_refuse for a tensor [H, N, d] whose last dimension alone has to be contiguous."""
    if t.dim() == 3 and t.stride(2) != 1:
        raise ValueError(f"{name}: the last dimension must be contiguous")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    _refuse(t.contiguous(), name, dtype, device, "[H, N, d] of Q")


_Strides = ctypes.c_int64 * 6
_AXES = {}                       # axis counts -> (their sum, the array the library takes)


def _axes(axis_pairs):
    key = tuple(axis_pairs)
    made = _AXES.get(key)
    if made is None:                 # one look: another thread may empty the table at any point
        if len(_AXES) > 256:
            _AXES.clear()
        made = _AXES[key] = (sum(key), (ctypes.c_int32 * len(key))(*key))
    return made


def spark_qk_norm_rope(Q, K=None, V=None, q_weight=None, k_weight=None, eps=1e-6, positions=None,
                       inv_freq=None, axis_pairs=None, interleaved=False, rope_scale=1.0,
                       Q_out=None, K_out=None, V_out=None, stream=None):
    """Per-head RMS norm and position rotation of Q and K [H, N, d] (any head and token strides,
    such as the transposed views of a fused projection's output), laid out contiguous; V is laid
    out along.  Weights fp32 [d] (None: no norm); positions [N, axes] int32 or fp32; inv_freq
    fp32 [pairs], axis_pairs the pairs of each axis (None: one axis).  Returns (Q_out, K_out,
    V_out), None for what is absent."""
    f32 = torch.float32
    try:
        index, dt, shape = Q.get_device(), Q.dtype, Q.shape
        if index < 0 or len(shape) != 3:
            _refuse(Q.contiguous(), "Q", (torch.bfloat16, f32), None, "[H, N, d]")
        code = _code(dt)
        H, N, d = shape
        q, (qh, qt, inner) = Q.data_ptr(), Q.stride()
        if inner != 1:
            _refuse_rows(Q, "Q", dt, Q.device)
        if Q_out is None:
            Q_out = _empty(shape, dt, Q.device, stream)
        if not (Q_out.dtype is dt and Q_out.get_device() == index and Q_out.is_contiguous()
                and Q_out.shape == shape):
            _refuse(Q_out, "Q_out", dt, Q.device, "[H, N, d] of Q")
        k = v = ko = vo = None
        kh = kt = vh = vt = 0
        if K is not None:
            k, (kh, kt, inner) = K.data_ptr(), K.stride()
            if inner != 1 or not (K.dtype is dt and K.get_device() == index and K.shape == shape):
                _refuse_rows(K, "K", dt, Q.device)
            if K_out is None:
                K_out = _empty(shape, dt, Q.device, stream)
            if not (K_out.dtype is dt and K_out.get_device() == index and K_out.is_contiguous()
                    and K_out.shape == shape):
                _refuse(K_out, "K_out", dt, Q.device, "[H, N, d] of Q")
            ko = K_out.data_ptr()
        elif K_out is not None or k_weight is not None:
            raise ValueError("K_out and k_weight need K")
        if V is not None:
            v, (vh, vt, inner) = V.data_ptr(), V.stride()
            if inner != 1 or not (V.dtype is dt and V.get_device() == index and V.shape == shape):
                _refuse_rows(V, "V", dt, Q.device)
            if V_out is None:
                V_out = _empty(shape, dt, Q.device, stream)
            if not (V_out.dtype is dt and V_out.get_device() == index and V_out.is_contiguous()
                    and V_out.shape == shape):
                _refuse(V_out, "V_out", dt, Q.device, "[H, N, d] of Q")
            vo = V_out.data_ptr()
        elif V_out is not None:
            raise ValueError("V_out needs V")
        wq = wk = None
        if q_weight is not None:
            if not (q_weight.dtype is f32 and q_weight.get_device() == index
                    and q_weight.is_contiguous() and q_weight.numel() == d):
                _refuse(q_weight, "q_weight", f32, Q.device, "[d]")
            wq = q_weight.data_ptr()
        if k_weight is not None:
            if not (k_weight.dtype is f32 and k_weight.get_device() == index
                    and k_weight.is_contiguous() and k_weight.numel() == d):
                _refuse(k_weight, "k_weight", f32, Q.device, "[d]")
            wk = k_weight.data_ptr()
        pairs, naxes, counts, pos, freq, pos_f32 = 0, 0, None, None, None, False
        if inv_freq is not None:
            if positions is None:
                raise ValueError("inv_freq needs positions")
            pairs = inv_freq.numel()
            if not (inv_freq.dtype is f32 and inv_freq.get_device() == index
                    and inv_freq.is_contiguous()):
                _refuse(inv_freq, "inv_freq", f32, Q.device, "[pairs]")
            pos_f32 = positions.dtype is f32
            size = positions.shape
            naxes = size[1] if len(size) == 2 else 1
            if not ((pos_f32 or positions.dtype is torch.int32)
                    and positions.get_device() == index and positions.is_contiguous()
                    and 1 <= len(size) <= 2 and size[0] == N):
                _refuse(positions, "positions", (torch.int32, f32), Q.device, "[N, axes]")
            total, counts = _axes((pairs,) if axis_pairs is None else axis_pairs)
            if total != pairs or len(counts) != naxes:
                raise ValueError("axis_pairs must give every axis of positions its pairs of "
                                 "inv_freq")
            pos, freq = positions.data_ptr(), inv_freq.data_ptr()
        elif positions is not None or axis_pairs is not None:
            raise ValueError("positions and axis_pairs need inv_freq")
    except AttributeError:
        _type_error(("Q",), Q=Q, K=K, V=V, q_weight=q_weight, k_weight=k_weight,
                    positions=positions, inv_freq=inv_freq, Q_out=Q_out, K_out=K_out, V_out=V_out)
        raise
    st = _launch(index, lib().spark_qk_norm_rope, q, k, v, code, H, N, d,
                 _Strides(qh, qt, kh, kt, vh, vt), wq, wk, eps, pos, pos_f32, naxes, counts, pairs,
                 freq, bool(interleaved), rope_scale, Q_out.data_ptr(), ko, vo,
                 _stream_of(index, stream))
    if st:
        _check("spark_qk_norm_rope", st)
    return Q_out, K_out, V_out


def spark_attend_ranges(nq, q_offsets, k_offsets=None, c_offsets=None, prefix=None, causal=False,
                        ranges=None, err=None, stream=None):
    """Key ranges [nq, 4] int32 of packed segments' query rows, from int32 offsets [segments + 1]
    of their queries, video keys and context keys; causal ends a row's context range behind its
    own place or the segment's prefix."""
    i32 = torch.int32
    _need(q_offsets, "q_offsets", i32)
    index, n = q_offsets.get_device(), q_offsets.numel()
    try:
        k = c = p = e = None
        if k_offsets is not None:
            if not (k_offsets.dtype is i32 and k_offsets.get_device() == index
                    and k_offsets.is_contiguous() and k_offsets.numel() == n):
                _refuse(k_offsets, "k_offsets", i32, q_offsets.device, f"[{n}]")
            k = k_offsets.data_ptr()
        if c_offsets is not None:
            if not (c_offsets.dtype is i32 and c_offsets.get_device() == index
                    and c_offsets.is_contiguous() and c_offsets.numel() == n):
                _refuse(c_offsets, "c_offsets", i32, q_offsets.device, f"[{n}]")
            c = c_offsets.data_ptr()
        if prefix is not None:
            if not causal:
                raise ValueError("prefix needs causal")
            if not (prefix.dtype is i32 and prefix.get_device() == index
                    and prefix.is_contiguous() and prefix.numel() == n - 1):
                _refuse(prefix, "prefix", i32, q_offsets.device, f"[{n - 1}]")
            p = prefix.data_ptr()
        if ranges is None:
            ranges = _empty((max(int(nq), 0), 4), i32, q_offsets.device, stream)
        if not (ranges.dtype is i32 and ranges.get_device() == index and ranges.is_contiguous()
                and ranges.shape == (nq, 4)):
            _refuse(ranges, "ranges", i32, q_offsets.device, "[nq, 4]")
        if err is not None:
            _need(err, "err", i32, q_offsets.device)
            e = err.data_ptr()
    except AttributeError:
        _type_error((), k_offsets=k_offsets, c_offsets=c_offsets, prefix=prefix, ranges=ranges)
        raise
    st = _launch(index, lib().spark_attend_ranges, nq, n - 1, q_offsets.data_ptr(), k, c, p,
                 bool(causal), ranges.data_ptr(), e, _stream_of(index, stream))
    if st:
        _check("spark_attend_ranges", st)
    return ranges


def spark_attend_dense_workspace_size(H, nq, nk, nc, d) -> int:
    return int(lib().spark_attend_dense_workspace_size(H, nq, nk, nc, d))


def spark_attend_dense(Q, K, V, Kc=None, Vc=None, ranges=None, out_dtype=torch.bfloat16, out=None,
                       lse=None, workspace=None, err=None, stream=None):
    """Dense attention of the rows of Q [H, nq, d] over the video keys K, V [H, nk, d] and the
    context keys Kc, Vc [H, nc, d] (bf16), each row over its ranges ([nq, 4] int32, None: all);
    returns (out, lse)."""
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    try:
        index, shape = Q.get_device(), Q.shape
        if not (Q.dtype is bf and index >= 0 and Q.is_contiguous() and len(shape) == 3):
            _refuse(Q, "Q", bf, None, "[H, nq, d]")
        H, nq, d = shape
        if not (K.dtype is bf and K.get_device() == index and K.is_contiguous() and K.dim() == 3):
            _refuse(K, "K", bf, Q.device, "[H, nk, d]")
        keys = K.shape
        nk, nc, kc, vc, rg, e = keys[1], 0, None, None, None, None
        if keys[0] != H or keys[2] != d:
            raise ValueError("K and V must have the shape [H, nk, d]")
        if not (V.dtype is bf and V.get_device() == index and V.is_contiguous()
                and V.shape == keys):
            _refuse(V, "V", bf, Q.device, "[H, nk, d]")
        if Kc is not None or Vc is not None:
            if not (Kc.dtype is bf and Kc.get_device() == index and Kc.is_contiguous()
                    and Kc.dim() == 3):
                _refuse(Kc, "Kc", bf, Q.device, "[H, nc, d]")
            keys = Kc.shape
            if keys[0] != H or keys[2] != d:
                raise ValueError("Kc and Vc must have the shape [H, nc, d]")
            if not (Vc.dtype is bf and Vc.get_device() == index and Vc.is_contiguous()
                    and Vc.shape == keys):
                _refuse(Vc, "Vc", bf, Q.device, "[H, nc, d]")
            nc, kc, vc = keys[1], Kc.data_ptr(), Vc.data_ptr()
        if ranges is not None:
            if not (ranges.dtype is i32 and ranges.get_device() == index
                    and ranges.is_contiguous() and ranges.shape == (nq, 4)):
                _refuse(ranges, "ranges", i32, Q.device, "[nq, 4]")
            rg = ranges.data_ptr()
        if out is None:
            out = _empty(shape, out_dtype, Q.device, stream)
        code = _code(out.dtype)
        if not (out.get_device() == index and out.is_contiguous() and out.shape == shape):
            _refuse(out, "out", out.dtype, Q.device, "[H, nq, d] of Q")
        if lse is None:
            lse = _empty((H, nq), f32, Q.device, stream)
        if not (lse.dtype is f32 and lse.get_device() == index and lse.is_contiguous()
                and lse.shape == (H, nq)):
            _refuse(lse, "lse", f32, Q.device, "[H, nq]")
        if workspace is None:
            workspace = _empty(spark_attend_dense_workspace_size(H, nq, nk, nc, d), torch.uint8,
                               Q.device, stream)
        if not (workspace.dtype is torch.uint8 and workspace.get_device() == index
                and workspace.is_contiguous()):
            _need(workspace, "workspace", torch.uint8, Q.device)
        if err is not None:
            _need(err, "err", i32, Q.device)
            e = err.data_ptr()
    except AttributeError:
        both = () if Kc is None and Vc is None else ("Kc", "Vc")
        _type_error(("Q", "K", "V", *both), Q=Q, K=K, V=V, Kc=Kc, Vc=Vc, ranges=ranges, out=out,
                    lse=lse, workspace=workspace)
        raise
    st = _launch(index, lib().spark_attend_dense, Q.data_ptr(), K.data_ptr(), V.data_ptr(), kc, vc,
                 H, nq, nk, nc, d, rg, out.data_ptr(), code, lse.data_ptr(), workspace.data_ptr(),
                 workspace.numel(), e, _stream_of(index, stream))
    if st:
        _check("spark_attend_dense", st)
    return out, lse


def spark_bsa_workspace_size_joint(H, N, d, nqb, nkb, topk_ratio, nc) -> int:
    return int(lib().spark_bsa_workspace_size_joint(H, N, d, nqb, nkb, float(topk_ratio), nc))


def spark_bsa_forward_joint(Q, K, V, Qc, Kc, Vc, q_perm, k_perm, q_offsets, k_offsets, topk_ratio,
                            out=None, out_c=None, workspace=None, stream=None):
    """spark_bsa_forward_ctx for the video queries and dense attention for the context queries
    Qc [H, nc, d]; returns (out, out_c, workspace, layout)."""
    _need(Q, "Q", (torch.bfloat16, torch.float32))
    dev = Q.device
    H, N, d = Q.shape
    for n, t in (("K", K), ("V", V), ("Qc", Qc)):
        _need(t, n, Q.dtype, dev)
    if K.shape != Q.shape or V.shape != Q.shape:
        raise ValueError("Q, K, V must share the shape [H, N, d]")
    _need(Kc, "Kc", Q.dtype, dev)
    Kc, Vc, nc = _context_args(Kc, Vc, H, d, Q.dtype, dev)
    if Qc.shape != Kc.shape:
        raise ValueError("Qc, Kc and Vc must share the shape [H, nc, d]")
    for n, t in (("q_perm", q_perm), ("k_perm", k_perm)):
        _need(t, n, torch.int32, dev)
        if t.shape != (H, N):
            raise ValueError(f"{n} must have shape [H, N]")
    for n, t in (("q_offsets", q_offsets), ("k_offsets", k_offsets)):
        _need(t, n, torch.int32, dev)
    nqb, nkb = q_offsets.numel() - 1, k_offsets.numel() - 1
    layout = spark_bsa_workspace_layout(H, N, d, nqb, nkb, topk_ratio)
    if out is None:
        out = _empty(Q.shape, Q.dtype, dev, stream)
    if out_c is None:
        out_c = _empty(Qc.shape, Q.dtype, dev, stream)
    _need(out, "out", Q.dtype, dev)
    _need(out_c, "out_c", Q.dtype, dev)
    if out.shape != Q.shape or out_c.shape != Qc.shape:
        raise ValueError("out and out_c must have the shapes of Q and Qc")
    if workspace is None:
        size = spark_bsa_workspace_size_joint(H, N, d, nqb, nkb, topk_ratio, nc)
        workspace = _empty(size, torch.uint8, dev, stream)
    _need(workspace, "workspace", torch.uint8, dev)
    st = _launch(dev.index, lib().spark_bsa_forward_joint, _ptr(Q), _ptr(K), _ptr(V), _ptr(Qc),
                 _ptr(Kc), _ptr(Vc), nc, _code(Q.dtype), H, N, d, _ptr(q_perm), _ptr(k_perm),
                 _ptr(q_offsets), nqb, _ptr(k_offsets), nkb, float(topk_ratio), _ptr(out),
                 _ptr(out_c), _ptr(workspace), workspace.numel(), _stream_of(dev.index, stream))
    _check("spark_bsa_forward_joint", st)
    return out, out_c, workspace, layout
