"""Python binding of the C ABI in ``include/gdn.h`` (argument marshalling only).

Every function here has the name of the C entry point it calls.  The binding
checks tensor devices, dtypes, shapes and contiguity, passes raw device
pointers and the current CUDA stream, and turns status codes into
exceptions.  It computes nothing itself and has no fallback: if ``libgdn.so``
is missing or CUDA is unavailable it raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libgdn.so")

GDN_OK = 0
(GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_WORKSPACE, GDN_ERR_CUDA, GDN_ERR_TIMEOUT,
 GDN_ERR_BAD_SEQLENS, GDN_ERR_DEVICE_CHECK, GDN_ERR_NO_PAGES) = range(1, 9)
STATUS_NAMES = {0: "GDN_OK", 1: "GDN_ERR_INVALID_ARG", 2: "GDN_ERR_UNSUPPORTED",
                3: "GDN_ERR_WORKSPACE", 4: "GDN_ERR_CUDA", 5: "GDN_ERR_TIMEOUT",
                6: "GDN_ERR_BAD_SEQLENS", 7: "GDN_ERR_DEVICE_CHECK", 8: "GDN_ERR_NO_PAGES"}
GDN_F32, GDN_BF16 = 0, 1
GDN_QK_L2NORM = 1 << 0
GDN_FORCE_SIMT = 1 << 1
GDN_GATE_SIGMOID = 1 << 2
GDN_BETA_LOGITS = 1 << 3
GDN_DEBUG_CHECKS = 1 << 4
GDN_SEQ_SPLIT = 1 << 5
GDN_NORM_SILU = 1 << 6
# site codes of a GDN_ERR_DEVICE_CHECK record (gdn_check_record)
DEBUG_SITES = {1: "q", 2: "k", 3: "v", 4: "g", 5: "beta", 6: "o", 7: "initial_state",
               8: "final_state", 9: "out_gate", 10: "tma_x"}
CHUNK_SIZE = 64

# Every symbol include/gdn.h declares.
EXPORTED = ("gdn_fwd_workspace_size", "gdn_workspace_init", "gdn_fwd", "gdn_check",
            "gdn_status_string", "gdn_fwd_kernel_name", "gdn_fwd_static_scratch",
            "gdn_decode", "gdn_diag_workspace_size", "gdn_diag_fwd", "gdn_conv_silu",
            "gdn_bwd_workspace_size", "gdn_bwd", "gdn_fwd_debug", "gdn_check_record",
            "gdn_fwd_kernel_name_chunk", "gdn_fwd_split_segments", "gdn_fwd_split_workspace_size",
            "gdn_diag_delta_workspace_size", "gdn_diag_delta_fwd",
            "gdn_lin_workspace_size", "gdn_lin_fwd", "gdn_lin_bwd", "gdn_lin_decode",
            "gdn_group_norm_workspace_size", "gdn_group_norm", "gdn_group_norm_bwd",
            "gdn_pages_workspace_size", "gdn_pages_copy", "gdn_pages_fork", "gdn_pages_free",
            "gdn_pages_compact")
# ... and include/gdn_debug.h (self-tests of the failure reporting).
DEBUG_EXPORTED = ("gdn_debug_wait_timeout",)

_lib = None
_lock = threading.Lock()


class GdnError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


def lib() -> ctypes.CDLL:
    """Load ``libgdn.so`` (raises if it was not built; there is no fallback)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} not found: build it with "
                    "`python -m linear_attention_recurrence_gated_gb300.build`")
            L = ctypes.CDLL(LIB_PATH)
            vp, i32, u32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_uint32, ctypes.c_size_t
            L.gdn_fwd_workspace_size.restype = sz
            L.gdn_fwd_workspace_size.argtypes = [i32, i32, i32, i32, u32]
            L.gdn_workspace_init.restype = ctypes.c_int
            L.gdn_workspace_init.argtypes = [vp, sz, vp]
            L.gdn_fwd.restype = ctypes.c_int
            L.gdn_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                  i32, i32, i32, i32, i32, i32, i32, ctypes.c_int, u32,
                                  vp, sz, vp]
            L.gdn_check.restype = ctypes.c_int
            L.gdn_check.argtypes = [vp, vp]
            L.gdn_check_record.restype = ctypes.c_int
            L.gdn_check_record.argtypes = [vp, vp, ctypes.POINTER(i32), ctypes.POINTER(i32),
                                           ctypes.POINTER(i32)]
            L.gdn_fwd_debug.restype = ctypes.c_int
            L.gdn_fwd_debug.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                        i32, i32, i32, i32, i32, i32, i32, ctypes.c_int, u32,
                                        vp, sz, ctypes.POINTER(GdnExtents), vp]
            L.gdn_debug_wait_timeout.restype = ctypes.c_int
            L.gdn_debug_wait_timeout.argtypes = [vp, sz, vp]
            L.gdn_status_string.restype = ctypes.c_char_p
            L.gdn_status_string.argtypes = [i32]
            L.gdn_fwd_kernel_name.restype = ctypes.c_char_p
            L.gdn_fwd_kernel_name.argtypes = [i32, i32, ctypes.c_int, u32]
            L.gdn_fwd_kernel_name_chunk.restype = ctypes.c_char_p
            L.gdn_fwd_kernel_name_chunk.argtypes = [i32, i32, i32, ctypes.c_int, u32]
            L.gdn_fwd_split_workspace_size.restype = sz
            L.gdn_fwd_split_workspace_size.argtypes = [i32, i32, i32, i32, i32]
            L.gdn_fwd_split_segments.restype = i32
            L.gdn_fwd_split_segments.argtypes = [i32, i32, i32, i32, i32, i32, ctypes.c_int, u32,
                                                 i32]
            L.gdn_fwd_static_scratch.restype = ctypes.c_int
            L.gdn_fwd_static_scratch.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                                 i32, i32, i32, i32, i32, i32, i32,
                                                 ctypes.c_int, u32, i32, vp]
            L.gdn_decode.restype = ctypes.c_int
            L.gdn_decode.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp,
                                     i32, i32, i32, i32, ctypes.c_int, u32, vp]
            L.gdn_bwd_workspace_size.restype = sz
            L.gdn_bwd_workspace_size.argtypes = [i32, i32, i32, i32, i32]
            L.gdn_bwd.restype = ctypes.c_int
            L.gdn_bwd.argtypes = [vp] * 15 + [i32] * 6 + [ctypes.c_int, u32, vp, sz, vp]
            L.gdn_conv_silu.restype = ctypes.c_int
            L.gdn_conv_silu.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, ctypes.c_int, vp]
            L.gdn_diag_workspace_size.restype = sz
            L.gdn_diag_workspace_size.argtypes = [i32, i32, i32, i32, i32]
            L.gdn_diag_fwd.restype = ctypes.c_int
            L.gdn_diag_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                       i32, i32, i32, i32, i32, ctypes.c_int, u32, vp, sz, vp]
            L.gdn_diag_delta_workspace_size.restype = sz
            L.gdn_diag_delta_workspace_size.argtypes = [i32, i32, i32, i32, i32]
            L.gdn_diag_delta_fwd.restype = ctypes.c_int
            L.gdn_diag_delta_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp,
                                             i32, i32, i32, i32, i32, ctypes.c_int, u32, vp, sz,
                                             vp]
            i64, st = ctypes.c_int64, ctypes.c_int
            for name, res, args in (
                    ("gdn_lin_workspace_size", sz, [i32] * 5 + [u32]),
                    ("gdn_lin_fwd", st, [vp] * 8 + [i32] * 6 + [i64] * 3 + [st, u32, vp, sz, vp]),
                    ("gdn_lin_bwd", st, [vp] * 12 + [i32] * 6 + [i64] * 3 + [st, u32, vp, sz, vp]),
                    ("gdn_lin_decode", st, [vp] * 8 + [i32] * 5 + [i64, st, u32, vp, sz, vp]),
                    ("gdn_group_norm_workspace_size", sz, [i32] * 4),
                    ("gdn_group_norm", st, [vp] * 7 + [i32] * 4 + [ctypes.c_float, st, u32, vp, sz,
                                                                   vp]),
                    ("gdn_group_norm_bwd", st, [vp] * 11 + [i32] * 4 + [st, u32, vp, sz, vp]),
                    ("gdn_pages_workspace_size", sz, [i32] * 3),
                    ("gdn_pages_copy", st, [vp, i64, i32, vp, vp, i32, vp, sz, vp]),
                    ("gdn_pages_fork", st, [vp, i64, i32, vp, vp, vp, i32, i32, vp, vp, i32, vp, vp,
                                            vp, vp, vp, sz, vp]),
                    ("gdn_pages_free", st, [vp] * 3 + [i32] * 3 + [vp, i32] + [vp] * 4 + [sz, vp]),
                    ("gdn_pages_compact", st, [vp, i64, i32, vp, vp, vp, i32, i32, vp, vp, vp, vp,
                                               sz, vp])):
                getattr(L, name).restype = res
                getattr(L, name).argtypes = args
            _lib = L
    return _lib


class GdnExtents(ctypes.Structure):
    """``gdn_extents``: elements each buffer of a forward call holds."""
    _fields_ = [(n, ctypes.c_int64) for n in ("q", "k", "v", "g", "beta", "o", "initial_state",
                                              "final_state", "out_gate")]


def status_string(status: int) -> str:
    try:
        return lib().gdn_status_string(int(status)).decode()
    except RuntimeError:
        return STATUS_NAMES.get(int(status), f"status {status}")


def _dtype_code(t: torch.dtype) -> int:
    if t == torch.float32:
        return GDN_F32
    if t == torch.bfloat16:
        return GDN_BF16
    raise TypeError(f"gdn: unsupported storage dtype {t} (float32 or bfloat16)")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream_handle(stream) -> ctypes.c_void_p:
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def gdn_fwd_workspace_size(num_seqs: int, num_heads: int, head_dim_k: int, head_dim_v: int,
                           flags: int = 0) -> int:
    return int(lib().gdn_fwd_workspace_size(num_seqs, num_heads, head_dim_k, head_dim_v, flags))


def gdn_workspace_init(workspace: torch.Tensor, stream=None) -> None:
    st = lib().gdn_workspace_init(_ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream_handle(stream))
    if st != GDN_OK:
        raise GdnError(st, "gdn_workspace_init")


def gdn_fwd_split_workspace_size(num_seqs: int, seq_len: int, num_heads: int, head_dim_k: int,
                                 head_dim_v: int) -> int:
    return int(lib().gdn_fwd_split_workspace_size(num_seqs, seq_len, num_heads, head_dim_k,
                                                  head_dim_v))


def new_workspace(num_seqs, num_heads, head_dim_k, head_dim_v, flags=0, device=None,
                  seq_len=None):
    """A zeroed workspace of the size gdn_fwd needs (the caller keeps it).
    With GDN_SEQ_SPLIT in ``flags`` pass ``seq_len`` (tokens per sequence of a
    dense call): a split call keeps per-token maps in the workspace."""
    if (flags & GDN_SEQ_SPLIT) and seq_len is not None:
        n = gdn_fwd_split_workspace_size(num_seqs, seq_len, num_heads, head_dim_k, head_dim_v)
    else:
        n = gdn_fwd_workspace_size(num_seqs, num_heads, head_dim_k, head_dim_v, flags)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def gdn_check(workspace: torch.Tensor, stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word."""
    return int(lib().gdn_check(_ptr(workspace), _stream_handle(stream)))


def gdn_check_record(workspace: torch.Tensor, stream=None):
    """gdn_check that also returns where the error arose:
    ``(status, seq, head, site)`` (site codes in ``DEBUG_SITES``)."""
    seq, head, site = ctypes.c_int32(), ctypes.c_int32(), ctypes.c_int32()
    st = lib().gdn_check_record(_ptr(workspace), _stream_handle(stream), ctypes.byref(seq),
                                ctypes.byref(head), ctypes.byref(site))
    return int(st), seq.value, head.value, site.value


def gdn_debug_wait_timeout(workspace: torch.Tensor, stream=None) -> int:
    """Enqueue the self-test whose bounded waits must give up (about 2 s) and
    report GDN_ERR_TIMEOUT in the workspace status word; returns the launch
    status (read the device status with gdn_check)."""
    return int(lib().gdn_debug_wait_timeout(_ptr(workspace),
                                            workspace.numel() * workspace.element_size(),
                                            _stream_handle(stream)))


def gdn_fwd_kernel_name(head_dim_k, head_dim_v, dtype: torch.dtype, flags: int = 0,
                        chunk_size: int = CHUNK_SIZE):
    r = lib().gdn_fwd_kernel_name_chunk(head_dim_k, head_dim_v, chunk_size, _dtype_code(dtype),
                                        flags)
    return None if r is None else r.decode()


def gdn_fwd_split_segments(num_seqs, seq_len, num_heads, head_dim_k, head_dim_v,
                           dtype: torch.dtype, flags: int = 0, chunk_size: int = CHUNK_SIZE,
                           varlen: bool = False) -> int:
    """Segments per sequence a gdn_fwd call with these sizes is cut into on the
    current device (1: not split, one kernel launch; >= 3: three launches);
    0 for sizes gdn_fwd rejects."""
    return int(lib().gdn_fwd_split_segments(num_seqs, seq_len, num_heads, head_dim_k,
                                            head_dim_v, chunk_size, _dtype_code(dtype), flags,
                                            1 if varlen else 0))


def _check_fwd_tensors(where, q, k, v, g, beta, initial_state, cu_seqlens, o, final_state,
                       D_skip=None, out_gate=None):
    """The tensor checks every forward entry point makes before it calls the
    library: device, contiguity, dtypes and shapes of inputs and of any output
    passed in.  Returns (N, H, dk, dv)."""
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError(f"{where}: q, k, v must be [B, T, H, D]")
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    tensors = [q, k, v, g, beta] + [t for t in (initial_state, cu_seqlens, o, final_state,
                                                D_skip, out_gate) if t is not None]
    for t in tensors:
        if not t.is_cuda:
            raise ValueError(f"{where}: every tensor must be on a CUDA device")
        if not t.is_contiguous():
            raise ValueError(f"{where}: every tensor must be contiguous")
    _dtype_code(q.dtype)
    if k.dtype != q.dtype or v.dtype != q.dtype or beta.dtype != q.dtype:
        raise TypeError(f"{where}: q, k, v and beta must share one storage dtype")
    if g.dtype != torch.float32:
        raise TypeError(f"{where}: g must be float32")
    if k.shape != q.shape or v.shape[:3] != q.shape[:3] or g.shape != (B, T, H) or \
            beta.shape != (B, T, H):
        raise ValueError(f"{where}: shape mismatch among q, k, v, g, beta")
    if initial_state is not None and (initial_state.dtype != torch.float32 or
                                      initial_state.shape != (N, H, dk, dv)):
        raise ValueError(f"{where}: initial_state must be float32 [N, H, dk, dv]")
    if cu_seqlens is not None and cu_seqlens.dtype != torch.int32:
        raise TypeError(f"{where}: cu_seqlens must be int32")
    if o is not None and (o.shape != v.shape or o.dtype != v.dtype):
        raise ValueError(f"{where}: o must match v in shape and dtype")
    if final_state is not None and (final_state.dtype != torch.float32 or
                                    final_state.shape != (N, H, dk, dv)):
        raise ValueError(f"{where}: final_state must be float32 [N, H, dk, dv]")
    if D_skip is not None and (D_skip.dtype != torch.float32 or tuple(D_skip.shape) != (H,)):
        raise ValueError(f"{where}: D_skip must be float32 [H]")
    if out_gate is not None and (out_gate.dtype != torch.float32 or out_gate.shape != (B, T, H)):
        raise ValueError(f"{where}: out_gate must be float32 [B, T, H]")
    return N, H, dk, dv


def _fwd_flags(qk_l2norm, beta_logits, force_simt, debug_checks, seq_split=False):
    return (GDN_QK_L2NORM if qk_l2norm else 0) | (GDN_FORCE_SIMT if force_simt else 0) | \
        (GDN_BETA_LOGITS if beta_logits else 0) | (GDN_DEBUG_CHECKS if debug_checks else 0) | \
        (GDN_SEQ_SPLIT if seq_split else 0)


def gdn_fwd(q, k, v, g, beta, initial_state=None, cu_seqlens=None, *, o=None,
            final_state=None, output_final_state=True, workspace=None, D_skip=None,
            out_gate=None, qk_l2norm=False, beta_logits=False, force_simt=False,
            chunk_size=CHUNK_SIZE, stream=None, check=False, debug_checks=False,
            seq_split=False):
    """Forward pass of the gated delta rule through the C ABI.

    q, k ``[B, T, H, dk]``; v ``[B, T, H, dv]``; g ``[B, T, H]`` fp32; beta
    ``[B, T, H]``; all CUDA, contiguous, q/k/v/beta/o in one storage dtype
    (float32 or bfloat16).  initial_state ``[N, H, dk, dv]`` fp32 or None;
    cu_seqlens int32 ``[N+1]`` on the device (then B must be 1) or None.
    ``o`` / ``final_state`` may be given to write into preallocated outputs
    (``final_state`` may be ``initial_state``).  ``chunk_size`` is 32, 64 (the
    default) or 128.  Returns ``(o, final_state)``.
    ``D_skip`` ``[H]`` and ``out_gate`` ``[B, T, H]`` (fp32, optional) fuse the
    block epilogue o <- (o + D_skip[h] v) * out_gate; ``beta_logits`` makes the
    kernel use sigmoid(beta); ``qk_l2norm`` normalises q and k in-kernel.
    ``debug_checks`` sets GDN_DEBUG_CHECKS (range checks before every access);
    ``seq_split`` sets GDN_SEQ_SPLIT (long dense sequences with head_dim_k 128
    cut into segments computed in parallel; a given ``workspace`` must be sized
    by ``gdn_fwd_split_workspace_size``, e.g. ``new_workspace(..., GDN_SEQ_SPLIT,
    seq_len=T)``).
    With ``check=True`` the call synchronises and raises on a device-side error.
    """
    N, H, dk, dv = _check_fwd_tensors("gdn_fwd", q, k, v, g, beta, initial_state, cu_seqlens,
                                      o, final_state, D_skip, out_gate)
    if o is None:
        o = torch.empty_like(v)
    if final_state is None and output_final_state:
        final_state = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
    B, T = q.shape[:2]
    dcode = _dtype_code(q.dtype)
    flags = _fwd_flags(qk_l2norm, beta_logits, force_simt, debug_checks, seq_split)
    if workspace is None:
        workspace = new_workspace(N, H, dk, dv, flags, device=q.device,
                                  seq_len=T if cu_seqlens is None else None)
    st = lib().gdn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
                       _ptr(cu_seqlens), _ptr(o), _ptr(final_state), _ptr(D_skip),
                       _ptr(out_gate), B, T, H, dk, dv, N, chunk_size, dcode, flags, _ptr(workspace),
                       workspace.numel() * workspace.element_size(), _stream_handle(stream))
    if st != GDN_OK:
        raise GdnError(st, "gdn_fwd")
    if check:
        st = gdn_check(workspace, stream)
        if st != GDN_OK:
            raise GdnError(st, "gdn_fwd (device)")
    return o, final_state


def gdn_fwd_static_scratch(q, k, v, g, beta, initial_state, cu_seqlens, o, final_state, *,
                           D_skip=None, out_gate=None, qk_l2norm=False, beta_logits=False,
                           force_simt=False, check=True, stream=None,
                           debug_checks=False) -> int:
    """Forward pass for callers that cannot allocate device memory.

    Same tensors as ``gdn_fwd`` but every output must be passed in (this call
    allocates nothing, not even through torch) and there is no workspace: the
    library's own 256-byte device array holds the status record.  With
    ``check`` the call synchronises and returns the device status code; the
    status is returned, not raised, so the caller decides.
    """
    if o is None:
        raise ValueError("gdn_fwd_static_scratch: o must be passed in (the call allocates nothing)")
    N, H, dk, dv = _check_fwd_tensors("gdn_fwd_static_scratch", q, k, v, g, beta,
                                      initial_state, cu_seqlens, o, final_state, D_skip,
                                      out_gate)
    B, T = q.shape[:2]
    flags = _fwd_flags(qk_l2norm, beta_logits, force_simt, debug_checks)
    return int(lib().gdn_fwd_static_scratch(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state), _ptr(cu_seqlens),
        _ptr(o), _ptr(final_state), _ptr(D_skip), _ptr(out_gate), B, T, H, dk, dv, N, CHUNK_SIZE,
        _dtype_code(q.dtype),
        flags, 1 if check else 0, _stream_handle(stream)))


def gdn_fwd_debug(q, k, v, g, beta, initial_state, cu_seqlens, o, final_state, workspace, *,
                  declared=None, D_skip=None, out_gate=None, qk_l2norm=False,
                  beta_logits=False, force_simt=False, chunk_size=CHUNK_SIZE, stream=None):
    """``gdn_fwd_debug``: the forward pass with GDN_DEBUG_CHECKS against
    declared extents.  ``declared`` maps buffer names (``GdnExtents`` fields)
    to element counts; missing names take the count of the tensor passed (0
    for None).  Outputs and workspace are passed in.  Returns the host status;
    read the device record with ``gdn_check_record``."""
    N, H, dk, dv = _check_fwd_tensors("gdn_fwd_debug", q, k, v, g, beta, initial_state,
                                      cu_seqlens, o, final_state, D_skip, out_gate)
    B, T = q.shape[:2]
    ext = None
    if declared is not None:
        have = dict(q=q, k=k, v=v, g=g, beta=beta, o=o, initial_state=initial_state,
                    final_state=final_state, out_gate=out_gate)
        unknown = set(declared) - set(have)
        if unknown:
            raise ValueError(f"gdn_fwd_debug: unknown extents {sorted(unknown)}")
        ext = GdnExtents(**{n: int(declared.get(n, 0 if t is None else t.numel()))
                            for n, t in have.items()})
    flags = _fwd_flags(qk_l2norm, beta_logits, force_simt, True)
    return int(lib().gdn_fwd_debug(
        _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state), _ptr(cu_seqlens),
        _ptr(o), _ptr(final_state), _ptr(D_skip), _ptr(out_gate), B, T, H, dk, dv, N,
        chunk_size, _dtype_code(q.dtype), flags, _ptr(workspace),
        workspace.numel() * workspace.element_size(),
        None if ext is None else ctypes.byref(ext), _stream_handle(stream)))


def gdn_decode(q, k, v, g, beta, state=None, *, o=None, state_out=None, qk_l2norm=False,
               stream=None):
    """One recurrent step per (sequence, head) through the C ABI.

    q, k ``[N, H, dk]``; v ``[N, H, dv]``; g ``[N, H]`` fp32; beta ``[N, H]``;
    q/k/v/beta/o in one storage dtype (float32 or bfloat16).  ``state``
    ``[N, H, dk, dv]`` fp32 or None (zeros).  ``state_out`` may be given
    (``state_out=state`` updates the state in place); otherwise a new tensor is
    returned.  Returns ``(o, state_out)``.
    """
    N, H, dk = q.shape
    dv = v.shape[-1]
    for t in [q, k, v, g, beta] + [t for t in (state, o, state_out) if t is not None]:
        if not t.is_cuda:
            raise ValueError("gdn_decode: every tensor must be on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("gdn_decode: every tensor must be contiguous")
    dcode = _dtype_code(q.dtype)
    if k.dtype != q.dtype or v.dtype != q.dtype or beta.dtype != q.dtype:
        raise TypeError("gdn_decode: q, k, v and beta must share one storage dtype")
    if g.dtype != torch.float32:
        raise TypeError("gdn_decode: g must be float32")
    if k.shape != q.shape or v.shape[:2] != (N, H) or g.shape != (N, H) or beta.shape != (N, H):
        raise ValueError("gdn_decode: shape mismatch among q, k, v, g, beta")
    for name, t in (("state", state), ("state_out", state_out)):
        if t is not None and (t.dtype != torch.float32 or t.shape != (N, H, dk, dv)):
            raise ValueError(f"gdn_decode: {name} must be float32 [N, H, dk, dv]")
    if o is None:
        o = torch.empty_like(v)
    elif o.shape != v.shape or o.dtype != v.dtype:
        raise ValueError("gdn_decode: o must match v in shape and dtype")
    if state_out is None:
        state_out = torch.empty((N, H, dk, dv), dtype=torch.float32, device=q.device)
    st = lib().gdn_decode(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(state),
                          _ptr(state_out), _ptr(o), N, H, dk, dv, dcode,
                          GDN_QK_L2NORM if qk_l2norm else 0, _stream_handle(stream))
    if st != GDN_OK:
        raise GdnError(st, "gdn_decode")
    return o, state_out


def gdn_diag_workspace_size(batch: int, seq_len: int, num_heads: int, d_state: int,
                            head_dim: int) -> int:
    return int(lib().gdn_diag_workspace_size(batch, seq_len, num_heads, d_state, head_dim))


def new_diag_workspace(batch, seq_len, num_heads, d_state, head_dim, device=None):
    """A zeroed workspace of the size gdn_diag_fwd needs (the caller keeps it)."""
    n = gdn_diag_workspace_size(batch, seq_len, num_heads, d_state, head_dim)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def gdn_diag_fwd(v, b, c, g, A_log, initial_state=None, *, D_skip=None, out_gate=None,
                 gate_sigmoid=False, o=None, final_state=None, output_final_state=True,
                 workspace=None, stream=None, check=False):
    """The pages' diagonal-decay recurrence through the C ABI.

    v ``[B, T, H, D]``; b, c ``[B, T, H, S]`` (v, b, c and o in one storage
    dtype, float32 or bfloat16); g ``[B, T, H]`` fp32; A_log ``[H, S]`` fp32;
    initial_state ``[B, H, S, D]`` fp32 or None.  ``D_skip`` ``[H]`` and
    ``out_gate`` ``[B, T, H]`` (fp32) fuse the block epilogue
    o <- (o + D_skip v) * out_gate; ``gate_sigmoid`` makes g the logits of the
    decay gate (g = sigmoid(g) in the kernel).  Returns ``(o, final_state)``
    (``final_state`` None when ``output_final_state`` is False and none is given).
    A workspace made by ``new_diag_workspace`` for the same sizes may be reused
    across calls on one stream.
    """
    B, T, H, D = v.shape
    S = b.shape[-1]
    for t in [v, b, c, g, A_log] + [t for t in (initial_state, o, final_state, D_skip, out_gate)
                                    if t is not None]:
        if not t.is_cuda:
            raise ValueError("gdn_diag_fwd: every tensor must be on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("gdn_diag_fwd: every tensor must be contiguous")
    dcode = _dtype_code(v.dtype)
    if b.dtype != v.dtype or c.dtype != v.dtype:
        raise TypeError("gdn_diag_fwd: v, b and c must share one storage dtype")
    if g.dtype != torch.float32 or A_log.dtype != torch.float32:
        raise TypeError("gdn_diag_fwd: g and A_log must be float32")
    if b.shape != (B, T, H, S) or c.shape != (B, T, H, S) or g.shape != (B, T, H) or \
            A_log.shape != (H, S):
        raise ValueError("gdn_diag_fwd: shape mismatch among v, b, c, g, A_log")
    for name, t in (("initial_state", initial_state), ("final_state", final_state)):
        if t is not None and (t.dtype != torch.float32 or t.shape != (B, H, S, D)):
            raise ValueError(f"gdn_diag_fwd: {name} must be float32 [B, H, S, D]")
    if D_skip is not None and (D_skip.dtype != torch.float32 or D_skip.shape != (H,)):
        raise ValueError("gdn_diag_fwd: D_skip must be float32 [H]")
    if out_gate is not None and (out_gate.dtype != torch.float32 or out_gate.shape != (B, T, H)):
        raise ValueError("gdn_diag_fwd: out_gate must be float32 [B, T, H]")
    if o is None:
        o = torch.empty_like(v)
    elif o.shape != v.shape or o.dtype != v.dtype:
        raise ValueError("gdn_diag_fwd: o must match v in shape and dtype")
    if final_state is None and output_final_state:
        final_state = torch.empty((B, H, S, D), dtype=torch.float32, device=v.device)
    if workspace is None:
        workspace = new_diag_workspace(B, T, H, S, D, device=v.device)
    st = lib().gdn_diag_fwd(_ptr(v), _ptr(b), _ptr(c), _ptr(g), _ptr(A_log), _ptr(D_skip),
                            _ptr(out_gate), _ptr(initial_state), _ptr(o), _ptr(final_state),
                            B, T, H, S, D, dcode, GDN_GATE_SIGMOID if gate_sigmoid else 0,
                            _ptr(workspace),
                            workspace.numel() * workspace.element_size(),
                            _stream_handle(stream))
    if st != GDN_OK:
        raise GdnError(st, "gdn_diag_fwd")
    if check:
        st = gdn_check(workspace, stream)
        if st != GDN_OK:
            raise GdnError(st, "gdn_diag_fwd (device)")
    return o, final_state


def gdn_diag_delta_workspace_size(batch: int, seq_len: int, num_heads: int, d_state: int,
                                  head_dim: int) -> int:
    return int(lib().gdn_diag_delta_workspace_size(batch, seq_len, num_heads, d_state,
                                                   head_dim))


def new_diag_delta_workspace(batch, seq_len, num_heads, d_state, head_dim, device=None):
    """A zeroed workspace of the size gdn_diag_delta_fwd needs (the caller keeps it)."""
    n = gdn_diag_delta_workspace_size(batch, seq_len, num_heads, d_state, head_dim)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def gdn_diag_delta_fwd(v, b, c, g, A_log, beta, initial_state=None, *, D_skip=None,
                       out_gate=None, gate_sigmoid=False, beta_logits=False, o=None,
                       final_state=None, output_final_state=True, workspace=None, stream=None,
                       check=False):
    """The pages' diagonal decay combined with the delta rule, through the C ABI.

    Tensors as ``gdn_diag_fwd`` plus beta ``[B, T, H]`` in the storage dtype of
    v, b, c.  ``beta_logits`` makes beta the logits of the write strength
    (sigmoid in the kernel).  Returns ``(o, final_state)``.  A workspace made by
    ``new_diag_delta_workspace`` for the same sizes may be reused across calls
    on one stream.
    """
    B, T, H, D = v.shape
    S = b.shape[-1]
    for t in [v, b, c, g, A_log, beta] + [t for t in (initial_state, o, final_state, D_skip,
                                                      out_gate) if t is not None]:
        if not t.is_cuda:
            raise ValueError("gdn_diag_delta_fwd: every tensor must be on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("gdn_diag_delta_fwd: every tensor must be contiguous")
    dcode = _dtype_code(v.dtype)
    if b.dtype != v.dtype or c.dtype != v.dtype or beta.dtype != v.dtype:
        raise TypeError("gdn_diag_delta_fwd: v, b, c and beta must share one storage dtype")
    if g.dtype != torch.float32 or A_log.dtype != torch.float32:
        raise TypeError("gdn_diag_delta_fwd: g and A_log must be float32")
    if b.shape != (B, T, H, S) or c.shape != (B, T, H, S) or g.shape != (B, T, H) or \
            beta.shape != (B, T, H) or A_log.shape != (H, S):
        raise ValueError("gdn_diag_delta_fwd: shape mismatch among v, b, c, g, beta, A_log")
    for name, t in (("initial_state", initial_state), ("final_state", final_state)):
        if t is not None and (t.dtype != torch.float32 or t.shape != (B, H, S, D)):
            raise ValueError(f"gdn_diag_delta_fwd: {name} must be float32 [B, H, S, D]")
    if D_skip is not None and (D_skip.dtype != torch.float32 or D_skip.shape != (H,)):
        raise ValueError("gdn_diag_delta_fwd: D_skip must be float32 [H]")
    if out_gate is not None and (out_gate.dtype != torch.float32 or out_gate.shape != (B, T, H)):
        raise ValueError("gdn_diag_delta_fwd: out_gate must be float32 [B, T, H]")
    if o is None:
        o = torch.empty_like(v)
    elif o.shape != v.shape or o.dtype != v.dtype:
        raise ValueError("gdn_diag_delta_fwd: o must match v in shape and dtype")
    if final_state is None and output_final_state:
        final_state = torch.empty((B, H, S, D), dtype=torch.float32, device=v.device)
    if workspace is None:
        workspace = new_diag_delta_workspace(B, T, H, S, D, device=v.device)
    flags = (GDN_GATE_SIGMOID if gate_sigmoid else 0) | (GDN_BETA_LOGITS if beta_logits else 0)
    st = lib().gdn_diag_delta_fwd(_ptr(v), _ptr(b), _ptr(c), _ptr(g), _ptr(A_log), _ptr(beta),
                                  _ptr(D_skip), _ptr(out_gate), _ptr(initial_state), _ptr(o),
                                  _ptr(final_state), B, T, H, S, D, dcode, flags,
                                  _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream_handle(stream))
    if st != GDN_OK:
        raise GdnError(st, "gdn_diag_delta_fwd")
    if check:
        st = gdn_check(workspace, stream)
        if st != GDN_OK:
            raise GdnError(st, "gdn_diag_delta_fwd (device)")
    return o, final_state


def gdn_conv_silu(x, w, x_prev=None, *, y=None, x_tail=None, stream=None):
    """Causal depthwise conv1d + SiLU through the C ABI (the GDN block prologue).

    x ``[B, T, C]`` (float32 or bfloat16); w ``[C, K]`` fp32 (PyTorch's Conv1d
    weight ``[C, 1, K]`` squeezed); x_prev ``[B, K-1, C]`` or None (zeros).
    ``x_tail`` (``[B, K-1, C]``, x's dtype) receives the last K-1 inputs when
    given.  Returns ``y``.
    """
    B, T, C = x.shape
    K = w.shape[-1]
    for t in [x, w] + [t for t in (x_prev, y, x_tail) if t is not None]:
        if not t.is_cuda:
            raise ValueError("gdn_conv_silu: every tensor must be on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("gdn_conv_silu: every tensor must be contiguous")
    dcode = _dtype_code(x.dtype)
    if w.dtype != torch.float32 or w.shape != (C, K):
        raise ValueError("gdn_conv_silu: w must be float32 [C, K]")
    for name, t in (("x_prev", x_prev), ("x_tail", x_tail)):
        if t is not None and (t.dtype != x.dtype or t.shape != (B, K - 1, C)):
            raise ValueError(f"gdn_conv_silu: {name} must be [B, K-1, C] in x's dtype")
    if y is None:
        y = torch.empty_like(x)
    elif y.shape != x.shape or y.dtype != x.dtype:
        raise ValueError("gdn_conv_silu: y must match x")
    st = lib().gdn_conv_silu(_ptr(x), _ptr(w), _ptr(x_prev), _ptr(y), _ptr(x_tail), B, T, C, K,
                             dcode, _stream_handle(stream))
    if st != GDN_OK:
        raise GdnError(st, "gdn_conv_silu")
    return y


def gdn_bwd_workspace_size(num_seqs: int, seq_len: int, num_heads: int, head_dim_k: int,
                           head_dim_v: int) -> int:
    return int(lib().gdn_bwd_workspace_size(num_seqs, seq_len, num_heads, head_dim_k, head_dim_v))


def gdn_bwd(q, k, v, g, beta, d_o, initial_state=None, cu_seqlens=None, d_final_state=None, *,
            grads=None, workspace=None, stream=None, check=False):
    """Backward pass of ``gdn_fwd`` through the C ABI.

    Inputs as ``gdn_fwd`` plus ``d_o`` (like v) and ``d_final_state``
    (``[N, H, dk, dv]`` fp32 or None).  Returns a dict of fp32 tensors
    ``dq, dk, dv, dg, dbeta, dh0`` (``grads`` may supply them preallocated).
    """
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    for t in [q, k, v, g, beta, d_o] + [t for t in (initial_state, cu_seqlens, d_final_state)
                                        if t is not None]:
        if not t.is_cuda:
            raise ValueError("gdn_bwd: every tensor must be on a CUDA device")
        if not t.is_contiguous():
            raise ValueError("gdn_bwd: every tensor must be contiguous")
    dcode = _dtype_code(q.dtype)
    if k.dtype != q.dtype or v.dtype != q.dtype or beta.dtype != q.dtype or d_o.dtype != q.dtype:
        raise TypeError("gdn_bwd: q, k, v, beta and d_o must share one storage dtype")
    if g.dtype != torch.float32:
        raise TypeError("gdn_bwd: g must be float32")
    if d_o.shape != v.shape:
        raise ValueError("gdn_bwd: d_o must match v")
    for name, t in (("initial_state", initial_state), ("d_final_state", d_final_state)):
        if t is not None and (t.dtype != torch.float32 or t.shape != (N, H, dk, dv)):
            raise ValueError(f"gdn_bwd: {name} must be float32 [N, H, dk, dv]")
    f32 = dict(dtype=torch.float32, device=q.device)
    if grads is None:
        grads = {"dq": torch.empty((B, T, H, dk), **f32), "dk": torch.empty((B, T, H, dk), **f32),
                 "dv": torch.empty((B, T, H, dv), **f32), "dg": torch.empty((B, T, H), **f32),
                 "dbeta": torch.empty((B, T, H), **f32),
                 "dh0": torch.empty((N, H, dk, dv), **f32)}
    if workspace is None:
        n = gdn_bwd_workspace_size(N, T, H, dk, dv)
        workspace = torch.zeros(n, dtype=torch.uint8, device=q.device)
    st = lib().gdn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), _ptr(initial_state),
                       _ptr(cu_seqlens), _ptr(d_o), _ptr(d_final_state), _ptr(grads["dq"]),
                       _ptr(grads["dk"]), _ptr(grads["dv"]), _ptr(grads["dg"]),
                       _ptr(grads["dbeta"]), _ptr(grads.get("dh0")), B, T, H, dk, dv, N, dcode,
                       0, _ptr(workspace), workspace.numel() * workspace.element_size(),
                       _stream_handle(stream))
    if st != GDN_OK:
        raise GdnError(st, "gdn_bwd")
    if check:
        st = gdn_check(workspace, stream)
        if st != GDN_OK:
            raise GdnError(st, "gdn_bwd (device)")
    return grads


# ---------------------------------------------------------------------------
# Linear attention with a decay for each head, group norm, pages of states
#
# These calls are also made for single tokens, where a step takes a few
# microseconds on the GPU: each looks its arguments over in one expression and
# names what is wrong (`_explain`) only if something is.
# ---------------------------------------------------------------------------
_F32, _I32, _U8 = torch.float32, torch.int32, torch.uint8
_CODES = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}
_calls = {}


def _call(name):
    """The library's function of this name."""
    f = _calls.get(name)
    if f is None:
        f = _calls[name] = getattr(lib(), name)
    return f


_current_device = getattr(torch._C, "_cuda_getDevice", None)   # (a build without CUDA)


def _elsewhere(name, device, *args):
    with torch.cuda.device(device):
        return _call(name)(*args)


def _on(name, device):
    """The library's function of this name, called with the tensors' device current:
    kernels are launched on the current device, whatever the stream's."""
    if device < 0 or _current_device() == device:
        return _call(name)
    return functools.partial(_elsewhere, name, device)


def _dense(device, *tensors):
    """Every tensor given (None: not given) is a contiguous CUDA tensor on this device."""
    for t in tensors:
        if t is not None and not (t.get_device() == device and t.is_contiguous() and
                                  (device >= 0 or t.is_cuda)):
            return False
    return True


def _explain(where, device, tensors, specs, lists=()):
    """Raise for the first thing wrong: ``tensors`` name -> tensor (or None) that
    must be contiguous on CUDA device ``device``; ``specs`` name -> (tensor, shape, dtype);
    ``lists``: names whose tensors must be lists of one length."""
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{where}: {name} must be on a CUDA device")
        if t.get_device() != device:
            raise ValueError(f"{where}: {name} must be on the device of the other tensors")
        if not t.is_contiguous():
            raise ValueError(f"{where}: {name} must be contiguous")
    for name, (t, shape, dtype) in specs.items():
        if t is not None and (t.dtype != dtype or tuple(t.shape) != tuple(shape)):
            kind = TypeError if t.dtype != dtype and dtype == _I32 else ValueError
            raise kind(f"{where}: {name} must be {str(dtype).split('.')[-1]} {list(shape)}")
    raise ValueError(f"{where}: {', '.join(lists) or 'arguments'} do not match in shape or dtype")


def _fits(t, shape, dtype):
    return t is None or (t.dtype == dtype and t.shape == shape)


def _raw_stream(stream, device):
    """The CUDA stream handle: of ``stream``, or the device's current one."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    if stream.device_index != device:
        raise ValueError(f"gdn: a stream of device {stream.device_index} for tensors on {device}")
    return stream.cuda_stream


def _p(t):
    return None if t is None else t.data_ptr()


def _empty(stream, like, shape, dtype):
    """A new tensor for the call's results, made on the stream that the call runs
    on, so that the allocator orders its reuse after it."""
    # (torch.empty takes 1.7 us where new_empty takes 3, empty_like 1.3)
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _like_new(stream, t):
    if not t.is_contiguous():
        return _empty(stream, t, t.shape, t.dtype)
    if stream is None:
        return torch.empty_like(t)
    with torch.cuda.stream(stream):
        return torch.empty_like(t)


def _workspace(stream, like, given, size, status):
    """``given``, or a new one; its status word is zeroed if it will be read."""
    if given is not None:
        if not _dense(like.get_device(), given):
            raise ValueError("gdn: the workspace must be contiguous, on the device of the tensors")
        return given
    ws = _empty(stream, like, (size,), _U8)
    if status:
        if stream is None:
            ws[:256].zero_()
        else:
            with torch.cuda.stream(stream):
                ws[:256].zero_()
    return ws


def _nbytes(t):
    return t.numel() * t.element_size()


def _done(where, st, check, workspace, stream):
    if st:
        raise GdnError(st, where)
    if check:
        with torch.cuda.device(workspace.get_device()):
            st = gdn_check(workspace, stream)
        if st:
            raise GdnError(st, f"{where} (device)")


def _stride(where, name, t):
    """Elements from one token row of ``t`` ``[B, T, H, D]`` to the next (rows
    contiguous, the rows of a batch one after the other); 0: packed."""
    if t.is_contiguous():
        return 0
    B, T, H, D = t.shape
    s = t.stride(1) if T > 1 else (t.stride(0) if B > 1 else H * D)
    if (D > 1 and t.stride(3) != 1) or (H > 1 and t.stride(2) != D) or s < H * D or \
            (B > 1 and T > 0 and t.stride(0) != T * s):
        raise ValueError(f"{where}: {name} must have contiguous rows [H, D] at one stride")
    if s * t.element_size() % 16:
        raise ValueError(f"{where}: the row stride of {name} must be a multiple of 16 bytes")
    return s


def _lin_check(where, q, k, v, log_decay, cu_seqlens, dense, specs):
    """Checks shared by gdn_lin_fwd and gdn_lin_bwd; ``specs``: further tensors,
    name -> (tensor, 0: the state's shape and fp32, 1: like q, 2: like v)."""
    if q.dim() != 4 or v.dim() != 4:
        raise ValueError(f"{where}: q, k, v must be [B, T, H, D]")
    B, T, H, dk = q.shape
    dv = v.shape[3]
    N = B if cu_seqlens is None else cu_seqlens.numel() - 1
    dt = q.dtype
    state = (N, H, dk, dv)
    dev = q.get_device()
    ok = k.get_device() == dev == v.get_device() and \
        (dev >= 0 or (q.is_cuda and k.is_cuda and v.is_cuda)) and dt in _CODES and k.dtype == dt and \
        v.dtype == dt and k.shape == q.shape and v.shape[:3] == q.shape[:3] and \
        _dense(dev, log_decay, cu_seqlens, *dense) and log_decay.dtype == _F32 and \
        log_decay.shape == (H,) and (cu_seqlens is None or (cu_seqlens.dtype == _I32 and
                                                            cu_seqlens.dim() == 1))
    if ok:
        for t, kind in specs.values():
            if t is not None and not (_fits(t, state, _F32) if kind == 0 else
                                      _fits(t, q.shape if kind == 1 else v.shape, dt)):
                ok = False
                break
    if not ok:
        _dtype_code(dt)
        if k.dtype != dt or v.dtype != dt:
            raise TypeError(f"{where}: q, k and v must share one storage dtype")
        if k.shape != q.shape or v.shape[:3] != q.shape[:3]:
            raise ValueError(f"{where}: shape mismatch among q, k, v")
        for name, t in (("q", q), ("k", k), ("v", v)):
            if not t.is_cuda:
                raise ValueError(f"{where}: {name} must be on a CUDA device")
            if t.get_device() != dev:
                raise ValueError(f"{where}: {name} must be on the device of q")
        full = {n: (t, state if kind == 0 else q.shape if kind == 1 else v.shape,
                    _F32 if kind == 0 else dt) for n, (t, kind) in specs.items()}
        full["log_decay"] = (log_decay, (H,), _F32)
        full["cu_seqlens"] = (cu_seqlens, (N + 1,), _I32)
        _explain(where, dev, {n: e[0] for n, e in full.items()}, full)
    return B, T, H, dk, dv, N


@functools.lru_cache(maxsize=256)
def gdn_lin_workspace_size(num_seqs: int, seq_len: int, num_heads: int, head_dim_k: int,
                           head_dim_v: int, flags: int = 0) -> int:
    return int(lib().gdn_lin_workspace_size(num_seqs, seq_len, num_heads, head_dim_k, head_dim_v,
                                            flags))


def gdn_lin_fwd(q, k, v, log_decay, initial_state=None, cu_seqlens=None, *, o=None,
                final_state=None, output_final_state=True, workspace=None, force_simt=False,
                stream=None, check=False):
    """Linear attention with a decay for each head, through the C ABI:
    S_t = exp(log_decay[h]) S_{t-1} + k_t v_t^T, o_t = S_t^T q_t.

    q, k ``[B, T, H, dk]``, v ``[B, T, H, dv]`` (float32 or bfloat16; slices of
    one projection are taken as they are: rows ``[H, D]`` contiguous, one stride
    between tokens); log_decay ``[H]`` fp32; initial_state ``[N, H, dk, dv]``
    fp32 or None; cu_seqlens int32 ``[N+1]`` on the device (then B must be 1) or
    None.  ``o`` / ``final_state`` may be given (``final_state`` may be
    ``initial_state``).  Returns ``(o, final_state)``.  With ``check=True`` the
    call synchronises and raises on a device-side error."""
    w = "gdn_lin_fwd"
    B, T, H, dk, dv, N = _lin_check(
        w, q, k, v, log_decay, cu_seqlens, (initial_state, o, final_state),
        dict(initial_state=(initial_state, 0), o=(o, 2), final_state=(final_state, 0)))
    if o is None:
        o = _like_new(stream, v)
    if final_state is None and output_final_state:
        final_state = _empty(stream, v, (N, H, dk, dv), _F32)
    flags = GDN_FORCE_SIMT if force_simt else 0
    ws = _workspace(stream, v, workspace, gdn_lin_workspace_size(N, T, H, dk, dv, flags), check)
    dev = q.get_device()
    st = _on(w, dev)(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _p(initial_state),
        _p(cu_seqlens), o.data_ptr(), _p(final_state), B, T, H, dk, dv, N, _stride(w, "q", q),
        _stride(w, "k", k), _stride(w, "v", v), _CODES[q.dtype], flags, ws.data_ptr(), _nbytes(ws),
        _raw_stream(stream, dev))
    if st or check:
        _done(w, st, check, ws, stream)
    return o, final_state


def gdn_lin_bwd(q, k, v, log_decay, d_o, initial_state=None, cu_seqlens=None, d_final_state=None,
                *, grads=None, workspace=None, force_simt=False, stream=None, check=False):
    """Backward pass of ``gdn_lin_fwd`` through the C ABI.

    Inputs as ``gdn_lin_fwd`` plus ``d_o`` (like o) and ``d_final_state``
    (``[N, H, dk, dv]`` fp32 or None).  Returns a dict ``dq, dk, dv`` (storage
    dtype) and ``dh0`` (fp32) (``grads`` may supply them; one without ``dh0``
    leaves it out)."""
    w = "gdn_lin_bwd"
    given = grads or {}
    dq_, dk_, dv_, dh_ = (given.get(n) for n in ("dq", "dk", "dv", "dh0"))
    B, T, H, dk, dv, N = _lin_check(
        w, q, k, v, log_decay, cu_seqlens, (d_o, initial_state, d_final_state, dq_, dk_, dv_, dh_),
        dict(d_o=(d_o, 2), initial_state=(initial_state, 0), d_final_state=(d_final_state, 0),
             dq=(dq_, 1), dk=(dk_, 1), dv=(dv_, 2), dh0=(dh_, 0)))
    if grads is None:
        grads = {"dq": _like_new(stream, q), "dk": _like_new(stream, k), "dv": _like_new(stream, v),
                 "dh0": _empty(stream, q, (N, H, dk, dv), _F32)}
    flags = GDN_FORCE_SIMT if force_simt else 0
    ws = _workspace(stream, v, workspace, gdn_lin_workspace_size(N, T, H, dk, dv, flags), check)
    dev = q.get_device()
    st = _on(w, dev)(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _p(initial_state),
        _p(cu_seqlens), d_o.data_ptr(), _p(d_final_state), grads["dq"].data_ptr(),
        grads["dk"].data_ptr(), grads["dv"].data_ptr(), _p(grads.get("dh0")), B, T, H, dk, dv, N,
        _stride(w, "q", q), _stride(w, "k", k), _stride(w, "v", v), _CODES[q.dtype], flags,
        ws.data_ptr(), _nbytes(ws), _raw_stream(stream, dev))
    if st or check:
        _done(w, st, check, ws, stream)
    return grads


def gdn_lin_decode(q, k, v, log_decay, state, pages=None, *, o=None, state_out=None,
                   workspace=None, stream=None, check=False):
    """One token per (sequence, head) of ``gdn_lin_fwd``'s recurrence.

    q, k ``[N, H, dk]``; v ``[N, H, dv]``; log_decay ``[H]`` fp32; ``state``
    ``[P, H, dk, dv]`` fp32: the pages of a pool, each contiguous, at any stride
    (``pool[:, layer]``), or None (zeros; then give ``state_out``).  ``pages``
    int32 ``[N]``: the page of each sequence (-1: a padded row, o = 0), or None
    (sequence n has page n).  The pages are updated in place unless
    ``state_out`` (laid out like ``state``) is given.  Returns
    ``(o, state_out)``.  With ``check=True`` the call synchronises and raises if
    a page number was out of range."""
    w = "gdn_lin_decode"
    N, H, dk = q.shape
    dv = v.shape[2]
    dt = q.dtype
    if state_out is None:
        if state is None:
            raise ValueError(f"{w}: give state, or state_out")
        state_out = state
    P = state_out.shape[0]
    stride = state_out.stride(0) if P > 1 else 0
    page = (H, dk, dv)
    dev = q.get_device()
    ok = _dense(dev, q, k, v, log_decay, pages, o) and dt in _CODES and k.dtype == dt and \
        v.dtype == dt and k.shape == q.shape and v.shape == (N, H, dv) and \
        log_decay.dtype == _F32 and log_decay.shape == (H,) and \
        _fits(pages, (N,), _I32) and _fits(o, v.shape, dt)
    if ok:
        for t in (state_out,) if state is state_out or state is None else (state_out, state):
            # a page is contiguous: [H, dk, dv] packed at every stride(0)
            if not (t.get_device() == dev and (dev >= 0 or t.is_cuda) and t.dtype == _F32 and
                    t.shape == (P, *page) and (P <= 1 or t.stride(0) == stride) and
                    (t.is_contiguous() or (P > 0 and t[0].is_contiguous()))):
                ok = False
    if not ok:
        _dtype_code(dt)
        if k.dtype != dt or v.dtype != dt:
            raise TypeError(f"{w}: q, k and v must share one storage dtype")
        if k.shape != q.shape or v.shape[:2] != (N, H):
            raise ValueError(f"{w}: shape mismatch among q, k, v")
        specs = dict(log_decay=(log_decay, (H,), _F32), pages=(pages, (N,), _I32),
                     o=(o, v.shape, dt), state=(state, (P, *page), _F32),
                     state_out=(state_out, (P, *page), _F32))
        for name in ("state", "state_out"):
            t = specs[name][0]
            if t is not None and t.is_cuda and t.dim() == 4 and P > 0 and \
                    (not t[0].is_contiguous() or (P > 1 and t.stride(0) != stride)):
                raise ValueError(f"{w}: {name} must have contiguous pages at one stride")
        one = lambda t: t if t is None or t.shape[0] == 0 else t[0]  # noqa: E731
        _explain(w, dev, dict(q=q, k=k, v=v, log_decay=log_decay, pages=pages, o=o,
                              state=one(state), state_out=one(state_out)), specs)
    if o is None:
        o = _like_new(stream, v)
    if check or workspace is not None:
        workspace = _workspace(stream, v, workspace, 256, check)
    st = _on(w, dev)(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), log_decay.data_ptr(), _p(state),
        state_out.data_ptr(), _p(pages), o.data_ptr(), N, H, dk, dv, P, stride, _CODES[dt], 0,
        _p(workspace), 0 if workspace is None else _nbytes(workspace), _raw_stream(stream, dev))
    if st or check:
        _done(w, st, check, workspace, stream)
    return o, state_out


@functools.lru_cache(maxsize=256)
def gdn_group_norm_workspace_size(batch: int, spatial: int, channels: int, groups: int) -> int:
    return int(lib().gdn_group_norm_workspace_size(batch, spatial, channels, groups))


def _norm_check(where, x, weight, bias, gate, groups, specs):
    """``specs``: name -> (tensor, 0: like x, 1: [N, groups] fp32, 2: [C] fp32)."""
    if x.dim() != 3:
        raise ValueError(f"{where}: x must be [N, S, C]")
    N, S, C = x.shape
    dt, stat, chan, dev = x.dtype, (N, groups), (C,), x.get_device()
    ok = dt in _CODES and _dense(dev, x, weight, bias, gate) and _fits(weight, chan, _F32) and \
        _fits(bias, chan, _F32) and _fits(gate, x.shape, dt)
    if ok:
        for t, kind in specs.values():
            if t is not None and not (_dense(dev, t) and
                                      (_fits(t, x.shape, dt) if kind == 0 else
                                       _fits(t, stat if kind == 1 else chan, _F32))):
                ok = False
                break
    if not ok:
        _dtype_code(dt)
        full = {n: (t, x.shape if kind == 0 else stat if kind == 1 else chan,
                    dt if kind == 0 else _F32) for n, (t, kind) in specs.items()}
        full.update(weight=(weight, chan, _F32), bias=(bias, chan, _F32), gate=(gate, x.shape, dt))
        _explain(where, dev, {"x": x, **{n: e[0] for n, e in full.items()}}, full)
    return N, S, C


def gdn_group_norm(x, weight, bias, groups, *, gate=None, silu=False, eps=1e-5, y=None, mean=None,
                   rstd=None, workspace=None, stream=None):
    """Group norm with an activation, channels last, through the C ABI.

    x ``[N, S, C]`` (float32 or bfloat16), ``groups`` groups of C / groups
    channels, statistics over the S rows and the group's channels; weight, bias
    ``[C]`` fp32 or None.  y = act(u) * silu(gate) with u the normalised, scaled
    value, act = SiLU with ``silu`` (else the identity) and ``gate`` like x, or
    None (no factor).  Returns ``(y, mean, rstd)``, the last two ``[N, groups]``
    fp32 (kept for the backward pass)."""
    w = "gdn_group_norm"
    N, S, C = _norm_check(w, x, weight, bias, gate, groups,
                          dict(y=(y, 0), mean=(mean, 1), rstd=(rstd, 1)))
    y = _like_new(stream, x) if y is None else y
    mean = _empty(stream, x, (N, groups), _F32) if mean is None else mean
    rstd = _empty(stream, x, (N, groups), _F32) if rstd is None else rstd
    ws = _workspace(stream, x, workspace, gdn_group_norm_workspace_size(N, S, C, groups), False)
    dev = x.get_device()
    st = _on(w, dev)(
        x.data_ptr(), _p(weight), _p(bias), _p(gate), y.data_ptr(), mean.data_ptr(),
        rstd.data_ptr(), N, S, C, groups, eps, _CODES[x.dtype], GDN_NORM_SILU if silu else 0,
        ws.data_ptr(), _nbytes(ws), _raw_stream(stream, dev))
    if st:
        raise GdnError(st, w)
    return y, mean, rstd


def gdn_group_norm_bwd(x, weight, bias, groups, mean, rstd, d_y, *, gate=None, silu=False,
                       grads=None, workspace=None, stream=None):
    """Backward pass of ``gdn_group_norm`` from the ``mean`` and ``rstd`` it
    returned.  Returns a dict ``dx``, ``dgate`` (storage dtype; dgate None
    without a gate), ``dweight``, ``dbias`` (fp32 ``[C]``); ``grads`` may supply
    them."""
    w = "gdn_group_norm_bwd"
    given = grads or {}
    N, S, C = _norm_check(w, x, weight, bias, gate, groups,
                          dict(mean=(mean, 1), rstd=(rstd, 1), d_y=(d_y, 0),
                               dx=(given.get("dx"), 0), dgate=(given.get("dgate"), 0),
                               dweight=(given.get("dweight"), 2), dbias=(given.get("dbias"), 2)))
    if grads is None:
        grads = {"dx": _like_new(stream, x),
                 "dgate": None if gate is None else _like_new(stream, gate),
                 "dweight": _empty(stream, x, (C,), _F32), "dbias": _empty(stream, x, (C,), _F32)}
    ws = _workspace(stream, x, workspace, gdn_group_norm_workspace_size(N, S, C, groups), False)
    dev = x.get_device()
    st = _on(w, dev)(
        x.data_ptr(), _p(weight), _p(bias), _p(gate), mean.data_ptr(), rstd.data_ptr(),
        d_y.data_ptr(), grads["dx"].data_ptr(), _p(grads.get("dgate")), _p(grads.get("dweight")),
        _p(grads.get("dbias")), N, S, C, groups, _CODES[x.dtype], GDN_NORM_SILU if silu else 0,
        ws.data_ptr(), _nbytes(ws), _raw_stream(stream, dev))
    if st:
        raise GdnError(st, w)
    return grads


@functools.lru_cache(maxsize=256)
def gdn_pages_workspace_size(num_pages: int, num_rows: int, n: int) -> int:
    return int(lib().gdn_pages_workspace_size(num_pages, num_rows, n))


def _pages_fine(pool, table, counts, refs, rows, own, table_out, counts_out, refs_out):
    """The bookkeeping of a call matches (the quick look before _pages_check): all
    tensors dense, ``rows`` (may be None) a list; no output is given (``own``: the
    call's own one) but inputs updated in place."""
    return own is None and (table_out is None or table_out is table) and \
        (counts_out is None or counts_out is counts) and \
        (refs_out is None or refs_out is refs) and \
        _dense(table.get_device(), pool, table, counts, refs, rows) and \
        table.dtype == _I32 and counts.dtype == _I32 and refs.dtype == _I32 and \
        table.dim() == 2 and refs.dim() == 1 and counts.shape == table.shape[:1] and \
        (pool is None or pool.shape[0] == refs.shape[0]) and \
        (rows is None or (rows.dtype == _I32 and rows.dim() == 1))


def _pages_check(where, pool, table, counts, refs, lists, outs):
    """``lists`` and ``outs``: name -> tensor.  Returns (page bytes, pages, rows,
    most pages of a row)."""
    R, M = (0, 1) if table is None else table.shape
    P = pool.shape[0] if table is None else refs.shape[0]
    n = None
    dev = (pool if table is None else table).get_device()
    ok = _dense(dev, pool, table, counts, refs, *lists.values(), *outs.values()) and \
        (pool is None or pool.shape[0] == P)
    if ok and table is not None:
        ok = table.dtype == _I32 and _fits(counts, (R,), _I32) and _fits(refs, (P,), _I32)
    for t in lists.values():
        n = t.numel() if n is None else n
        ok = ok and t.dtype == _I32 and t.shape == (n,)
    shapes = dict(table_out=(R, M), counts_out=(R,), refs_out=(P,), fresh=(n,), num_live=(1,))
    for name, t in outs.items():
        ok = ok and _fits(t, shapes[name], _I32)
    if not ok:
        if pool is not None and pool.shape[0] != P:
            raise ValueError(f"{where}: refs must have one entry for each page of the pool")
        specs = {n_: (t, (n,), _I32) for n_, t in lists.items()}
        specs.update({n_: (t, shapes[n_], _I32) for n_, t in outs.items()})
        if table is not None:
            specs.update(table=(table, (R, M), _I32), counts=(counts, (R,), _I32),
                         refs=(refs, (P,), _I32))
        _explain(where, dev, dict(pool=pool, **{n_: e[0] for n_, e in specs.items()}), specs, lists)
    bytes_ = 16 if pool is None or P == 0 else _nbytes(pool) // P
    return bytes_, P, R, M


def gdn_pages_copy(pool, src, dst, *, workspace=None, stream=None, check=False):
    """Pages ``dst`` of ``pool`` ``[P, ...]`` become copies of pages ``src``
    (int32 ``[n]`` each).  Returns ``pool``."""
    w = "gdn_pages_copy"
    bytes_, P, _, _ = _pages_check(w, pool, None, None, None, dict(src=src, dst=dst), {})
    n = src.numel()
    ws = _workspace(stream, pool, workspace, gdn_pages_workspace_size(P, 0, n), check)
    dev = pool.get_device()
    st = _on(w, dev)(
        pool.data_ptr(), bytes_, P, src.data_ptr(), dst.data_ptr(), n, ws.data_ptr(), _nbytes(ws),
        _raw_stream(stream, dev))
    if st or check:
        _done(w, st, check, ws, stream)
    return pool


def gdn_pages_fork(pool, table, counts, refs, parents, children, *, fresh=None, table_out=None,
                   counts_out=None, refs_out=None, workspace=None, stream=None, check=False):
    """Fork rows of a page table: row ``children[i]`` shares the pages of row
    ``parents[i]`` but the last, of which it gets a copy in the lowest free page
    (parent -1: a new row with one page of zeros; parent = child: a snapshot,
    the row goes on in a copy of its last page).

    pool ``[P, ...]`` (pages a multiple of 16 bytes); table int32 ``[R, M]``;
    counts int32 ``[R]``; refs int32 ``[P]``; parents, children int32 ``[n]``.
    ``table_out`` / ``counts_out`` / ``refs_out`` may be the inputs (updated in
    place) and are new tensors if not given; the pool is updated in place.
    Returns ``(fresh, table_out, counts_out, refs_out)``, ``fresh[i]`` the new
    page of child i (-1: none).  With ``check=True`` the call synchronises and
    raises if a job was left out (a bad row or too few free pages)."""
    w = "gdn_pages_fork"
    if _pages_fine(pool, table, counts, refs, parents, fresh, table_out, counts_out, refs_out) and \
            _dense(table.get_device(), children) and children.dtype == _I32 and \
            children.shape == parents.shape:
        (R, M), P = table.shape, refs.shape[0]
        bytes_ = _nbytes(pool) // P if P else 16
    else:
        bytes_, P, R, M = _pages_check(w, pool, table, counts, refs,
                                       dict(parents=parents, children=children),
                                       dict(fresh=fresh, table_out=table_out,
                                            counts_out=counts_out, refs_out=refs_out))
    n = parents.shape[0]
    fresh = _like_new(stream, parents) if fresh is None else fresh
    table_out = _like_new(stream, table) if table_out is None else table_out
    counts_out = _like_new(stream, counts) if counts_out is None else counts_out
    refs_out = _like_new(stream, refs) if refs_out is None else refs_out
    ws = _workspace(stream, pool, workspace, gdn_pages_workspace_size(P, R, n), check)
    dev = pool.get_device()
    st = _on(w, dev)(
        pool.data_ptr(), bytes_, P, table.data_ptr(), counts.data_ptr(), refs.data_ptr(), R, M,
        parents.data_ptr(), children.data_ptr(), n, fresh.data_ptr(), table_out.data_ptr(),
        counts_out.data_ptr(), refs_out.data_ptr(), ws.data_ptr(), _nbytes(ws),
        _raw_stream(stream, dev))
    if st or check:
        _done(w, st, check, ws, stream)
    return fresh, table_out, counts_out, refs_out


def gdn_pages_free(table, counts, refs, rows, *, table_out=None, counts_out=None, refs_out=None,
                   workspace=None, stream=None, check=False):
    """Rows ``rows`` (int32 ``[n]``) give their pages back and are empty
    afterwards.  Tensors and outputs as ``gdn_pages_fork``.  Returns
    ``(table_out, counts_out, refs_out)``."""
    w = "gdn_pages_free"
    if _pages_fine(None, table, counts, refs, rows, None, table_out, counts_out, refs_out):
        (R, M), P = table.shape, refs.shape[0]
    else:
        _, P, R, M = _pages_check(w, None, table, counts, refs, dict(rows=rows),
                                  dict(table_out=table_out, counts_out=counts_out,
                                       refs_out=refs_out))
    n = rows.shape[0]
    table_out = _like_new(stream, table) if table_out is None else table_out
    counts_out = _like_new(stream, counts) if counts_out is None else counts_out
    refs_out = _like_new(stream, refs) if refs_out is None else refs_out
    ws = _workspace(stream, table, workspace, gdn_pages_workspace_size(P, R, n), check)
    dev = table.get_device()
    st = _on(w, dev)(
        table.data_ptr(), counts.data_ptr(), refs.data_ptr(), P, R, M, rows.data_ptr(), n,
        table_out.data_ptr(), counts_out.data_ptr(), refs_out.data_ptr(), ws.data_ptr(),
        _nbytes(ws), _raw_stream(stream, dev))
    if st or check:
        _done(w, st, check, ws, stream)
    return table_out, counts_out, refs_out


def gdn_pages_compact(pool, table, counts, refs, *, num_live=None, table_out=None, refs_out=None,
                      workspace=None, stream=None, check=False):
    """Move the live pages of ``pool`` to the lowest numbers and rewrite the
    table.  Tensors as ``gdn_pages_fork``.  Returns ``(num_live, table_out,
    refs_out)``, num_live int32 ``[1]`` on the device."""
    w = "gdn_pages_compact"
    if _pages_fine(pool, table, counts, refs, None, num_live, table_out, None, refs_out):
        (R, M), P = table.shape, refs.shape[0]
        bytes_ = _nbytes(pool) // P if P else 16
    else:
        bytes_, P, R, M = _pages_check(w, pool, table, counts, refs, {},
                                       dict(num_live=num_live, table_out=table_out,
                                            refs_out=refs_out))
    num_live = _empty(stream, pool, (1,), _I32) if num_live is None else num_live
    table_out = _like_new(stream, table) if table_out is None else table_out
    refs_out = _like_new(stream, refs) if refs_out is None else refs_out
    ws = _workspace(stream, pool, workspace, gdn_pages_workspace_size(P, R, 0), check)
    dev = pool.get_device()
    st = _on(w, dev)(
        pool.data_ptr(), bytes_, P, table.data_ptr(), counts.data_ptr(), refs.data_ptr(), R, M,
        num_live.data_ptr(), table_out.data_ptr(), refs_out.data_ptr(), ws.data_ptr(), _nbytes(ws),
        _raw_stream(stream, dev))
    if st or check:
        _done(w, st, check, ws, stream)
    return num_live, table_out, refs_out
