"""Python binding of libmoba.so (ctypes): argument marshalling only.

Every step of the MoBA forward pass runs in the library's CUDA kernels; PyTorch only provides
device memory and the current stream. The functions mirror the C entry points of include/moba.h
and raise if the library is missing or a call fails — there is no fallback path. The calls around
the paged cache, which a decode step makes in microseconds, marshal their arguments in csrc/bind.cpp
where these are plain (on the current stream, all as documented) and _bind.so loads; the checks here
handle the rest and say what is wrong.
"""
from __future__ import annotations

import ctypes
import os
import warnings
from typing import Optional, Sequence, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# MOBA_CHECKS=1 in the environment selects the build with device-side index checks
LIB_PATH = os.path.join(_HERE, "libmoba_checks.so" if os.environ.get("MOBA_CHECKS") == "1"
                        else "libmoba.so")

STATUS = {0: "MOBA_OK", -1: "MOBA_ERR_ARG", -2: "MOBA_ERR_UNSUPPORTED", -3: "MOBA_ERR_WORKSPACE",
          -4: "MOBA_ERR_CUDA", -5: "MOBA_ERR_DEVICE_CHECK", -6: "MOBA_ERR_TIMEOUT"}
KERNEL_CLASSES = ["centroid", "gate", "route_count", "route_scan", "route_scatter", "attention",
                  "merge", "plan", "densify", "decode", "bwd_dkdv", "bwd_dq", "bwd_aux"]

# every symbol include/moba.h declares
EXPORTS = ["moba_status_string", "moba_version", "moba_workspace_bytes", "moba_centroids",
           "moba_gate_topk", "moba_attn_fwd", "moba_device_status", "moba_timing_enable",
           "moba_timing_reset", "moba_timing_read", "moba_launch_count",
           "moba_attn_fwd_noalloc", "moba_noalloc_status", "moba_set_wait_limit_ns",
           "moba_centroids_kconv", "moba_attn_fwd_kconv", "moba_decode_workspace_bytes",
           "moba_decode_fwd", "moba_bwd_workspace_bytes", "moba_attn_bwd",
           "moba_set_diag_stall", "moba_qk_norm_rope", "moba_qk_norm_rope_bwd_workspace_bytes",
           "moba_qk_norm_rope_bwd", "moba_cache_append", "moba_cache_read",
           "moba_paged_workspace_bytes", "moba_paged_attn_fwd", "moba_paged_decode_fwd"]

NOALLOC_SCRATCH_BYTES = 64 << 20


class MobaError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what} failed: {STATUS.get(status, status)}")


_lib = None
_bind = None  # csrc/bind.cpp, once the library is loaded; None where it does not load


def _load_bind():
    """The native argument marshalling, or None with a warning: its calls then go through the checks
    of this file, with the same results and some microseconds more per call."""
    try:
        from . import _bind as bind
        made_for = bind.torch_version
    except (ImportError, AttributeError) as e:
        why = f"is missing or does not load ({e})"
    else:
        if made_for == torch.__version__:
            return bind
        why = f"was built for torch {made_for}, this is {torch.__version__}"
    warnings.warn(f"_bind.so {why}; the norm and paged-cache calls take the slower way. Build it "
                  "with `python -m block_sparse_long_moba_b200.build`", RuntimeWarning,
                  stacklevel=3)
    return None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libmoba.so, or libmoba_checks.so when MOBA_CHECKS=1 (build them with
    `python -m block_sparse_long_moba_b200.build [--checks]`)."""
    global _lib, _bind
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"libmoba.so not found at {path}; build it with "
                          "`python -m block_sparse_long_moba_b200.build`")
    lib = ctypes.CDLL(path)
    P, I, L, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_size_t
    lib.moba_status_string.argtypes = [I]
    lib.moba_status_string.restype = ctypes.c_char_p
    lib.moba_version.restype = I
    lib.moba_workspace_bytes.argtypes = [I, P, I, I, I, I, I]
    lib.moba_workspace_bytes.restype = S
    lib.moba_centroids.argtypes = [P, P, P, I, I, I, I, P, P]
    lib.moba_centroids.restype = I
    lib.moba_gate_topk.argtypes = [P, P, P, P, I, I, I, I, I, I, P, P]
    lib.moba_gate_topk.restype = I
    lib.moba_attn_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, P, P, P, P, P, S, P]
    lib.moba_attn_fwd.restype = I
    lib.moba_device_status.argtypes = [P, P]
    lib.moba_device_status.restype = I
    lib.moba_timing_enable.argtypes = [I]
    lib.moba_timing_enable.restype = I
    lib.moba_timing_reset.restype = I
    lib.moba_timing_read.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(L), I]
    lib.moba_timing_read.restype = I
    lib.moba_launch_count.restype = L
    lib.moba_attn_fwd_noalloc.argtypes = [P, P, P, P, P, I, I, I, I, I, I, F, P, P, P]
    lib.moba_attn_fwd_noalloc.restype = I
    lib.moba_centroids_kconv.argtypes = [P, P, I, P, P, I, I, I, I, P, P]
    lib.moba_centroids_kconv.restype = I
    lib.moba_attn_fwd_kconv.argtypes = [P, P, P, P, I, P, P, I, I, I, I, I, I, F, P, P, P, P, S, P]
    lib.moba_attn_fwd_kconv.restype = I
    lib.moba_decode_workspace_bytes.argtypes = [I, P, P, I, I, I, I, I]
    lib.moba_decode_workspace_bytes.restype = S
    lib.moba_decode_fwd.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, P, P, P, P, P, S,
                                    P]
    lib.moba_decode_fwd.restype = I
    lib.moba_bwd_workspace_bytes.argtypes = [I, P, I, I, I, I, I]
    lib.moba_bwd_workspace_bytes.restype = S
    lib.moba_attn_bwd.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, P, P, P, P, S, P]
    lib.moba_attn_bwd.restype = I
    lib.moba_noalloc_status.argtypes = [P]
    lib.moba_noalloc_status.restype = I
    lib.moba_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
    lib.moba_set_wait_limit_ns.restype = ctypes.c_ulonglong
    lib.moba_set_diag_stall.argtypes = [I]
    lib.moba_set_diag_stall.restype = I
    lib.moba_qk_norm_rope.argtypes = [P, L, P, L, P, P, P, I, I, P, I, I, I, I, F, I, P, P, P]
    lib.moba_qk_norm_rope.restype = I
    lib.moba_qk_norm_rope_bwd_workspace_bytes.argtypes = [I, I, I]
    lib.moba_qk_norm_rope_bwd_workspace_bytes.restype = S
    lib.moba_qk_norm_rope_bwd.argtypes = [P, L, P, L, P, P, P, I, I, P, P, P, I, I, I, I, F, I, P,
                                          P, P, P, P, S, P]
    lib.moba_qk_norm_rope_bwd.restype = I
    lib.moba_cache_append.argtypes = [P, P, L, P, L, P, I, P]
    lib.moba_cache_append.restype = I
    lib.moba_cache_read.argtypes = [P, P, I, P, P, P]
    lib.moba_cache_read.restype = I
    lib.moba_paged_workspace_bytes.argtypes = [P, I, I, I]
    lib.moba_paged_workspace_bytes.restype = S
    lib.moba_paged_attn_fwd.argtypes = [P, P, I, I, F, P, P, P, S, P]
    lib.moba_paged_attn_fwd.restype = I
    lib.moba_paged_decode_fwd.argtypes = [P, P, I, I, I, F, P, P, P, P, S, P]
    lib.moba_paged_decode_fwd.restype = I
    bind = _load_bind()
    if bind is not None:
        bind.init(*(ctypes.cast(f, P).value for f in (
            lib.moba_qk_norm_rope, lib.moba_qk_norm_rope_bwd,
            lib.moba_qk_norm_rope_bwd_workspace_bytes, lib.moba_cache_append,
            lib.moba_cache_read, lib.moba_paged_attn_fwd, lib.moba_paged_decode_fwd)))
    _lib, _bind = lib, bind
    return lib


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _check(status: int, what: str):
    if status != 0:
        raise MobaError(status, what)


_ANY_DEVICE = object()  # the device is checked separately (_current_device)


def _bad(what: str, why: str):
    raise MobaError(-1, f"{what}: {why}")


def _want(what: str, name: str, t: Optional[torch.Tensor], dtype, shape=None, device=None):
    """Checks one tensor argument before its pointer reaches the library: the kernels trust the
    layout (dtype, contiguity, shape) and launch on the current device, so a mismatch here would
    otherwise read or write the wrong memory."""
    if t is None:
        _bad(what, f"{name} is required")
    if not torch.is_tensor(t):
        _bad(what, f"{name} must be a torch tensor")
    if t.dtype != dtype:
        _bad(what, f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        _bad(what, f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        _bad(what, f"{name} must be contiguous")
    if device is None:
        if t.device.type != "cuda":
            _bad(what, f"{name} must be a CUDA tensor, got {t.device}")
    elif device is not _ANY_DEVICE and t.device != device:
        _bad(what, f"{name} is on {t.device}, the call runs on {device}")


def _current_device(what: str, t: torch.Tensor) -> torch.device:
    if t.device.type != "cuda":
        _bad(what, f"tensors must be CUDA tensors, got {t.device}")
    cur = torch.device("cuda", torch.cuda.current_device())
    if t.device != cur:
        _bad(what, f"tensors are on {t.device} but the current device is {cur}")
    return cur


def _want_cu(what: str, cu_seqlens: torch.Tensor, nseq: int, device):
    _want(what, "cu_seqlens", cu_seqlens, torch.int32, (nseq + 1,), device)


def _host_cu(cu_seqlens_host) -> Tuple[ctypes.Array, int]:
    vals = [int(x) for x in (cu_seqlens_host.tolist() if torch.is_tensor(cu_seqlens_host)
                             else cu_seqlens_host)]
    arr = (ctypes.c_int32 * len(vals))(*vals)
    return arr, len(vals) - 1


def num_blocks(cu_seqlens_host: Sequence[int], block_size: int) -> int:
    cu = [int(x) for x in cu_seqlens_host]
    return sum((cu[s + 1] - cu[s] + block_size - 1) // block_size for s in range(len(cu) - 1))


def moba_workspace_bytes(cu_seqlens_host, hq: int, hkv: int, d: int, block_size: int,
                         topk: int) -> int:
    arr, nseq = _host_cu(cu_seqlens_host)
    return int(load_library().moba_workspace_bytes(nseq, arr, hq, hkv, d, block_size, topk))


def moba_centroids(k: torch.Tensor, cu_seqlens: torch.Tensor, cu_seqlens_host, block_size: int,
                   out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Block centroids [NB, Hkv, d] fp32 of bf16 keys [T, Hkv, d]."""
    what = "moba_centroids"
    arr, nseq = _host_cu(cu_seqlens_host)
    if not torch.is_tensor(k) or k.dim() != 3:
        _bad(what, "k must be a [T, Hkv, d] tensor")
    T, hkv, d = k.shape
    _want(what, "k", k, torch.bfloat16, None, _ANY_DEVICE)
    dev = _current_device(what, k)
    _want_cu(what, cu_seqlens, nseq, dev)
    nb = num_blocks(list(arr), block_size)
    if out is None:
        out = torch.empty((nb, hkv, d), dtype=torch.float32, device=k.device)
    _want(what, "out", out, torch.float32, (nb, hkv, d), dev)
    st = load_library().moba_centroids(_ptr(k), _ptr(cu_seqlens), arr, nseq, hkv, d, block_size,
                                       _ptr(out), _stream(stream))
    _check(st, "moba_centroids")
    return out


def moba_centroids_kconv(k: torch.Tensor, conv_w: torch.Tensor, cu_seqlens: torch.Tensor,
                         cu_seqlens_host, block_size: int, out: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """Centroids [NB, Hkv, d] fp32 of keys passed through the in-block short convolution with
    weights conv_w [W, Hkv, d] fp32."""
    what = "moba_centroids_kconv"
    arr, nseq = _host_cu(cu_seqlens_host)
    if not torch.is_tensor(k) or k.dim() != 3 or not torch.is_tensor(conv_w) or conv_w.dim() != 3:
        _bad(what, "k must be [T, Hkv, d] and conv_w [W, Hkv, d]")
    T, hkv, d = k.shape
    _want(what, "k", k, torch.bfloat16, None, _ANY_DEVICE)
    dev = _current_device(what, k)
    _want(what, "conv_w", conv_w, torch.float32, (conv_w.shape[0], hkv, d), dev)
    _want_cu(what, cu_seqlens, nseq, dev)
    nb = num_blocks(list(arr), block_size)
    if out is None:
        out = torch.empty((nb, hkv, d), dtype=torch.float32, device=k.device)
    _want(what, "out", out, torch.float32, (nb, hkv, d), dev)
    st = load_library().moba_centroids_kconv(_ptr(k), _ptr(conv_w), conv_w.shape[0],
                                             _ptr(cu_seqlens), arr, nseq, hkv, d, block_size,
                                             _ptr(out), _stream(stream))
    _check(st, what)
    return out


def moba_gate_topk(q: torch.Tensor, centroids: torch.Tensor, cu_seqlens: torch.Tensor,
                   cu_seqlens_host, block_size: int, topk: int,
                   out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Routing [Hq, T, topk] int32 (ascending local block ids, -1 padded)."""
    what = "moba_gate_topk"
    arr, nseq = _host_cu(cu_seqlens_host)
    if not torch.is_tensor(q) or q.dim() != 3 or not torch.is_tensor(centroids) or \
            centroids.dim() != 3:
        _bad(what, "q must be [T, Hq, d] and centroids [NB, Hkv, d]")
    T, hq, d = q.shape
    hkv = centroids.shape[1]
    _want(what, "q", q, torch.bfloat16, None, _ANY_DEVICE)
    dev = _current_device(what, q)
    _want(what, "centroids", centroids, torch.float32,
          (num_blocks(list(arr), block_size), hkv, d), dev)
    _want_cu(what, cu_seqlens, nseq, dev)
    if out is None:
        out = torch.empty((hq, T, topk), dtype=torch.int32, device=q.device)
    _want(what, "out", out, torch.int32, (hq, T, topk), dev)
    st = load_library().moba_gate_topk(_ptr(q), _ptr(centroids), _ptr(cu_seqlens), arr, nseq, hq,
                                       hkv, d, block_size, topk, _ptr(out), _stream(stream))
    _check(st, "moba_gate_topk")
    return out


def _check_qkv(what, q, k, v, cu_seqlens, nseq):
    """q [T, Hq, d], k and v [T, Hkv, d], all bf16, contiguous, on the current device."""
    for name, t in (("q", q), ("k", k), ("v", v)):
        if not torch.is_tensor(t) or t.dim() != 3:
            _bad(what, f"{name} must be a 3-D tensor")
    T, hq, d = q.shape
    hkv = k.shape[1]
    _want(what, "q", q, torch.bfloat16, None, _ANY_DEVICE)
    dev = _current_device(what, q)
    _want(what, "k", k, torch.bfloat16, (T, hkv, d), dev)
    _want(what, "v", v, torch.bfloat16, (T, hkv, d), dev)
    _want_cu(what, cu_seqlens, nseq, dev)
    return dev, T, hq, hkv, d


def moba_attn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                  cu_seqlens_host, block_size: int, topk: int, scale: Optional[float] = None,
                  block_idx_in: Optional[torch.Tensor] = None,
                  block_idx_out: Optional[torch.Tensor] = None,
                  o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """MoBA forward: returns (o [T,Hq,d] bf16, lse [Hq,T] fp32). Buffers may be passed in."""
    what = "moba_attn_fwd"
    arr, nseq = _host_cu(cu_seqlens_host)
    dev, T, hq, hkv, d = _check_qkv(what, q, k, v, cu_seqlens, nseq)
    if scale is None:
        scale = d ** -0.5
    for name, t in (("block_idx_in", block_idx_in), ("block_idx_out", block_idx_out)):
        if t is not None:
            _want(what, name, t, torch.int32, (hq, T, topk), dev)
    lib = load_library()
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((hq, T), dtype=torch.float32, device=q.device)
    _want(what, "o", o, torch.bfloat16, (T, hq, d), dev)
    _want(what, "lse", lse, torch.float32, (hq, T), dev)
    if workspace is not None:
        _want(what, "workspace", workspace, torch.uint8, None, dev)
    if workspace is None:
        nbytes = int(lib.moba_workspace_bytes(nseq, arr, hq, hkv, d, block_size, topk))
        if nbytes == 0 and T > 0:
            raise MobaError(-1, "moba_workspace_bytes")
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=q.device)
    st = lib.moba_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), arr, nseq, hq, hkv, d,
                           block_size, topk, ctypes.c_float(scale), _ptr(block_idx_in),
                           _ptr(block_idx_out), _ptr(o), _ptr(lse), _ptr(workspace),
                           ctypes.c_size_t(workspace.numel()), _stream(stream))
    _check(st, "moba_attn_fwd")
    return o, lse


def moba_attn_fwd_kconv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                        conv_w: torch.Tensor, cu_seqlens: torch.Tensor, cu_seqlens_host,
                        block_size: int, topk: int, scale: Optional[float] = None,
                        block_idx_out: Optional[torch.Tensor] = None,
                        o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None):
    """MoBA forward with the routing computed on short-convolved keys (conv_w [W, Hkv, d] fp32);
    returns (o, lse)."""
    what = "moba_attn_fwd_kconv"
    arr, nseq = _host_cu(cu_seqlens_host)
    dev, T, hq, hkv, d = _check_qkv(what, q, k, v, cu_seqlens, nseq)
    if not torch.is_tensor(conv_w) or conv_w.dim() != 3:
        _bad(what, "conv_w must be [W, Hkv, d]")
    _want(what, "conv_w", conv_w, torch.float32, (conv_w.shape[0], hkv, d), dev)
    if scale is None:
        scale = d ** -0.5
    if block_idx_out is not None:
        _want(what, "block_idx_out", block_idx_out, torch.int32, (hq, T, topk), dev)
    lib = load_library()
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((hq, T), dtype=torch.float32, device=q.device)
    _want(what, "o", o, torch.bfloat16, (T, hq, d), dev)
    _want(what, "lse", lse, torch.float32, (hq, T), dev)
    if workspace is None:
        nbytes = int(lib.moba_workspace_bytes(nseq, arr, hq, hkv, d, block_size, topk))
        if nbytes == 0 and T > 0:
            raise MobaError(-1, "moba_workspace_bytes")
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=q.device)
    _want(what, "workspace", workspace, torch.uint8, None, dev)
    st = lib.moba_attn_fwd_kconv(_ptr(q), _ptr(k), _ptr(v), _ptr(conv_w), conv_w.shape[0],
                                 _ptr(cu_seqlens), arr, nseq, hq, hkv, d, block_size, topk,
                                 ctypes.c_float(scale), _ptr(block_idx_out), _ptr(o), _ptr(lse),
                                 _ptr(workspace), ctypes.c_size_t(workspace.numel()),
                                 _stream(stream))
    _check(st, what)
    return o, lse


def moba_decode_workspace_bytes(cu_seqlens_host, cu_seqlens_q_host, hq: int, hkv: int, d: int,
                                block_size: int, topk: int) -> int:
    arr, nseq = _host_cu(cu_seqlens_host)
    arq, nq = _host_cu(cu_seqlens_q_host)
    if nq != nseq:
        _bad("moba_decode_workspace_bytes", "cu_seqlens_q must have nseq + 1 entries")
    return int(load_library().moba_decode_workspace_bytes(nseq, arr, arq, hq, hkv, d, block_size,
                                                          topk))


def moba_decode_fwd(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    centroids: Optional[torch.Tensor], cu_seqlens: torch.Tensor, cu_seqlens_host,
                    cu_seqlens_q: torch.Tensor, cu_seqlens_q_host, block_size: int, topk: int,
                    scale: Optional[float] = None, block_idx_in: Optional[torch.Tensor] = None,
                    block_idx_out: Optional[torch.Tensor] = None,
                    o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None):
    """MoBA over the newest rows of a KV cache (decode: one row per sequence). q [Tq, Hq, d] are
    the last n_s tokens of each sequence (cu_seqlens_q); returns (o [Tq, Hq, d], lse [Hq, Tq])."""
    what = "moba_decode_fwd"
    arr, nseq = _host_cu(cu_seqlens_host)
    arq, nq = _host_cu(cu_seqlens_q_host)
    if nq != nseq:
        _bad(what, "cu_seqlens_q must have nseq + 1 entries")
    for name, t in (("q", q), ("k_cache", k_cache), ("v_cache", v_cache)):
        if not torch.is_tensor(t) or t.dim() != 3:
            _bad(what, f"{name} must be a 3-D tensor")
    Tq, hq, d = q.shape
    T, hkv = k_cache.shape[0], k_cache.shape[1]
    _want(what, "q", q, torch.bfloat16, None, _ANY_DEVICE)
    dev = _current_device(what, q)
    _want(what, "k_cache", k_cache, torch.bfloat16, (T, hkv, d), dev)
    _want(what, "v_cache", v_cache, torch.bfloat16, (T, hkv, d), dev)
    _want_cu(what, cu_seqlens, nseq, dev)
    _want(what, "cu_seqlens_q", cu_seqlens_q, torch.int32, (nseq + 1,), dev)
    if centroids is not None:
        _want(what, "centroids", centroids, torch.float32,
              (num_blocks(list(arr), block_size), hkv, d), dev)
    elif block_idx_in is None:
        _bad(what, "centroids are required unless a routing is given")
    for name, t in (("block_idx_in", block_idx_in), ("block_idx_out", block_idx_out)):
        if t is not None:
            _want(what, name, t, torch.int32, (hq, Tq, topk), dev)
    if scale is None:
        scale = d ** -0.5
    lib = load_library()
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((hq, Tq), dtype=torch.float32, device=q.device)
    _want(what, "o", o, torch.bfloat16, (Tq, hq, d), dev)
    _want(what, "lse", lse, torch.float32, (hq, Tq), dev)
    if workspace is None:
        nbytes = int(lib.moba_decode_workspace_bytes(nseq, arr, arq, hq, hkv, d, block_size, topk))
        if nbytes == 0 and Tq > 0:
            raise MobaError(-1, "moba_decode_workspace_bytes")
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=q.device)
    _want(what, "workspace", workspace, torch.uint8, None, dev)
    st = lib.moba_decode_fwd(_ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(centroids),
                             _ptr(cu_seqlens), arr, _ptr(cu_seqlens_q), arq, nseq, hq, hkv, d,
                             block_size, topk, ctypes.c_float(scale), _ptr(block_idx_in),
                             _ptr(block_idx_out), _ptr(o), _ptr(lse), _ptr(workspace),
                             ctypes.c_size_t(workspace.numel()), _stream(stream))
    _check(st, what)
    return o, lse


def moba_bwd_workspace_bytes(cu_seqlens_host, hq: int, hkv: int, d: int, block_size: int,
                             topk: int) -> int:
    arr, nseq = _host_cu(cu_seqlens_host)
    return int(load_library().moba_bwd_workspace_bytes(nseq, arr, hq, hkv, d, block_size, topk))


def moba_attn_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                  lse: torch.Tensor, d_o: torch.Tensor, block_idx: torch.Tensor,
                  cu_seqlens: torch.Tensor, cu_seqlens_host, block_size: int, topk: int,
                  scale: Optional[float] = None, dq: Optional[torch.Tensor] = None,
                  dk: Optional[torch.Tensor] = None, dv: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients (dq, dk, dv) of the routed attention with the routing held fixed; o and lse are
    the forward pass's outputs and block_idx the routing it used."""
    what = "moba_attn_bwd"
    arr, nseq = _host_cu(cu_seqlens_host)
    dev, T, hq, hkv, d = _check_qkv(what, q, k, v, cu_seqlens, nseq)
    _want(what, "o", o, torch.bfloat16, (T, hq, d), dev)
    _want(what, "d_o", d_o, torch.bfloat16, (T, hq, d), dev)
    _want(what, "lse", lse, torch.float32, (hq, T), dev)
    _want(what, "block_idx", block_idx, torch.int32, (hq, T, topk), dev)
    if scale is None:
        scale = d ** -0.5
    lib = load_library()
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    _want(what, "dq", dq, torch.bfloat16, (T, hq, d), dev)
    _want(what, "dk", dk, torch.bfloat16, (T, hkv, d), dev)
    _want(what, "dv", dv, torch.bfloat16, (T, hkv, d), dev)
    if workspace is None:
        nbytes = int(lib.moba_bwd_workspace_bytes(nseq, arr, hq, hkv, d, block_size, topk))
        if nbytes == 0 and T > 0:
            raise MobaError(-1, "moba_bwd_workspace_bytes")
        workspace = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=q.device)
    _want(what, "workspace", workspace, torch.uint8, None, dev)
    st = lib.moba_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(o), _ptr(lse), _ptr(d_o),
                           _ptr(block_idx), _ptr(cu_seqlens), arr, nseq, hq, hkv, d, block_size,
                           topk, ctypes.c_float(scale), _ptr(dq), _ptr(dk), _ptr(dv),
                           _ptr(workspace), ctypes.c_size_t(workspace.numel()), _stream(stream))
    _check(st, what)
    return dq, dk, dv


def moba_attn_fwd_noalloc(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                          cu_seqlens: torch.Tensor, cu_seqlens_host, block_size: int, topk: int,
                          scale: Optional[float] = None, o: Optional[torch.Tensor] = None,
                          lse: Optional[torch.Tensor] = None, stream=None):
    """moba_attn_fwd without a workspace: the library's static scratch array is used instead
    (for callers that cannot allocate device memory; see include/moba.h). The outputs may be
    passed in so that the call itself allocates nothing."""
    what = "moba_attn_fwd_noalloc"
    arr, nseq = _host_cu(cu_seqlens_host)
    dev, T, hq, hkv, d = _check_qkv(what, q, k, v, cu_seqlens, nseq)
    if scale is None:
        scale = d ** -0.5
    if o is None:
        o = torch.empty_like(q)
    if lse is None:
        lse = torch.empty((hq, T), dtype=torch.float32, device=q.device)
    _want(what, "o", o, torch.bfloat16, (T, hq, d), dev)
    _want(what, "lse", lse, torch.float32, (hq, T), dev)
    st = load_library().moba_attn_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), arr,
                                              nseq, hq, hkv, d, block_size, topk,
                                              ctypes.c_float(scale), _ptr(o), _ptr(lse),
                                              _stream(stream))
    _check(st, "moba_attn_fwd_noalloc")
    return o, lse


def _is(t, dtype, shape, device) -> bool:
    """The conditions of _want as one expression: the calls of a decode step take microseconds, so
    they ask this first and _want says what is wrong."""
    return (torch.is_tensor(t) and t.dtype is dtype and t.shape == shape and t.device == device
            and t.is_contiguous())


def _raw_stream(device: torch.device) -> int:
    """The cudaStream_t of the device's current stream."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _done(result, what: str):
    """What a call through csrc/bind.cpp returned: its outputs, or a status that is not MOBA_OK."""
    if type(result) is int:
        _check(result, what)
    return result


def _rows(what: str, name: str, t: torch.Tensor, heads: Optional[int] = None,
          d: Optional[int] = None) -> int:
    """Checks bf16 [T, heads, d] whose heads are packed and whose tokens may lie further apart
    (a slice of a fused projection); returns the token stride in elements."""
    if not torch.is_tensor(t) or t.dim() != 3:
        _bad(what, f"{name} must be a 3-D tensor")
    if t.dtype is not torch.bfloat16:
        _bad(what, f"{name} must be {torch.bfloat16}, got {t.dtype}")
    T, h, w = t.shape
    if (heads is not None and h != heads) or (d is not None and w != d):
        _bad(what, f"{name} must have shape {(T, heads, d)}, got {tuple(t.shape)}")
    s0, s1, s2 = t.stride()
    if (w > 1 and s2 != 1) or (h > 1 and s1 != w):
        _bad(what, f"{name}: the heads of a token must be packed, strides are {t.stride()}")
    return s0 if T > 1 else h * w


def _workspace(nbytes: int, device) -> torch.Tensor:
    """A workspace for one call. The calls below run on the current stream (one that is given is
    made current first), so that what they allocate is memory of the stream that uses it."""
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def rope_table(n_pos: int, rot_dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """fp32 [n_pos, rot_dim] table for moba_qk_norm_rope: the cosines, then the sines, of
    p * base^(-2 i / rot_dim), computed in 64 bits (a far position's angle has no bits to spare)."""
    inv = float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device)
                          / rot_dim)
    a = torch.arange(n_pos, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _check_norm(what, q, k, q_weight, k_weight, rope, positions):
    q_ld = _rows(what, "q", q)
    T, hq, d = q.shape
    dev = _current_device(what, q)
    k_ld = _rows(what, "k", k, d=d)
    if k.shape[0] != T or k.device != dev:
        _bad(what, f"k must have {T} tokens on {dev}, got {tuple(k.shape)} on {k.device}")
    if not _is(q_weight, torch.float32, (d,), dev):
        _want(what, "q_weight", q_weight, torch.float32, (d,), dev)
    if not _is(k_weight, torch.float32, (d,), dev):
        _want(what, "k_weight", k_weight, torch.float32, (d,), dev)
    if not torch.is_tensor(rope) or rope.dim() != 2:
        _bad(what, "rope must be a [n_pos, rot_dim] tensor")
    if not _is(rope, torch.float32, rope.shape, dev):
        _want(what, "rope", rope, torch.float32, None, dev)
    if not _is(positions, torch.int32, (T,), dev):
        _want(what, "positions", positions, torch.int32, (T,), dev)
    return dev, T, hq, k.shape[1], d, q_ld, k_ld


def moba_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, q_weight: torch.Tensor,
                      k_weight: torch.Tensor, rope: torch.Tensor, positions: torch.Tensor,
                      eps: float = 1e-6, interleaved: bool = False,
                      q_out: Optional[torch.Tensor] = None, k_out: Optional[torch.Tensor] = None,
                      stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """RMS norm of every head of q [T, Hq, d] and k [T, Hkv, d] (tokens may be strided) times fp32
    weights [d], and the rotary position of positions [T] in a table from rope_table. Returns
    packed (q_out, k_out)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return moba_qk_norm_rope(q, k, q_weight, k_weight, rope, positions, eps,
                                     interleaved, q_out, k_out)
    what = "moba_qk_norm_rope"
    if _bind is not None:
        done = _bind.norm_rope(q, k, q_weight, k_weight, rope, positions, eps, interleaved, q_out,
                               k_out)
        if done is not None:
            return _done(done, what)
    dev, T, hq, hkv, d, q_ld, k_ld = _check_norm(what, q, k, q_weight, k_weight, rope, positions)
    if q_out is None:
        q_out = q.new_empty((T, hq, d))
    else:
        _want(what, "q_out", q_out, torch.bfloat16, (T, hq, d), dev)
    if k_out is None:
        k_out = k.new_empty((T, hkv, d))
    else:
        _want(what, "k_out", k_out, torch.bfloat16, (T, hkv, d), dev)
    st = load_library().moba_qk_norm_rope(
        q.data_ptr(), q_ld, k.data_ptr(), k_ld, q_weight.data_ptr(), k_weight.data_ptr(),
        rope.data_ptr(), rope.shape[0], rope.shape[1], positions.data_ptr(), T, hq, hkv, d, eps,
        1 if interleaved else 0, q_out.data_ptr(), k_out.data_ptr(), _raw_stream(dev))
    _check(st, what)
    return q_out, k_out


def moba_qk_norm_rope_bwd(q: torch.Tensor, k: torch.Tensor, q_weight: torch.Tensor,
                          k_weight: torch.Tensor, rope: torch.Tensor, positions: torch.Tensor,
                          d_q_out: torch.Tensor, d_k_out: torch.Tensor, eps: float = 1e-6,
                          interleaved: bool = False, dq: Optional[torch.Tensor] = None,
                          dk: Optional[torch.Tensor] = None,
                          d_q_weight: Optional[torch.Tensor] = None,
                          d_k_weight: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients (dq, dk, d_q_weight, d_k_weight) of moba_qk_norm_rope; nothing but its inputs is
    needed from the forward pass."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return moba_qk_norm_rope_bwd(q, k, q_weight, k_weight, rope, positions, d_q_out,
                                         d_k_out, eps, interleaved, dq, dk, d_q_weight,
                                         d_k_weight, workspace)
    what = "moba_qk_norm_rope_bwd"
    if (_bind is not None and dq is None and dk is None and d_q_weight is None
            and d_k_weight is None and workspace is None):
        done = _bind.norm_rope_bwd(q, k, q_weight, k_weight, rope, positions, d_q_out, d_k_out,
                                   eps, interleaved)
        if done is not None:
            return _done(done, what)
    dev, T, hq, hkv, d, q_ld, k_ld = _check_norm(what, q, k, q_weight, k_weight, rope, positions)
    _want(what, "d_q_out", d_q_out, torch.bfloat16, (T, hq, d), dev)
    _want(what, "d_k_out", d_k_out, torch.bfloat16, (T, hkv, d), dev)
    dq = torch.empty_like(d_q_out) if dq is None else dq
    dk = torch.empty_like(d_k_out) if dk is None else dk
    d_q_weight = torch.empty_like(q_weight) if d_q_weight is None else d_q_weight
    d_k_weight = torch.empty_like(k_weight) if d_k_weight is None else d_k_weight
    _want(what, "dq", dq, torch.bfloat16, (T, hq, d), dev)
    _want(what, "dk", dk, torch.bfloat16, (T, hkv, d), dev)
    _want(what, "d_q_weight", d_q_weight, torch.float32, (d,), dev)
    _want(what, "d_k_weight", d_k_weight, torch.float32, (d,), dev)
    lib = load_library()
    if workspace is None:
        workspace = _workspace(int(lib.moba_qk_norm_rope_bwd_workspace_bytes(hq, hkv, d)), dev)
    _want(what, "workspace", workspace, torch.uint8, None, dev)
    st = lib.moba_qk_norm_rope_bwd(
        q.data_ptr(), q_ld, k.data_ptr(), k_ld, q_weight.data_ptr(), k_weight.data_ptr(),
        rope.data_ptr(), rope.shape[0], rope.shape[1], positions.data_ptr(), d_q_out.data_ptr(),
        d_k_out.data_ptr(), T, hq, hkv, d, eps, 1 if interleaved else 0, dq.data_ptr(),
        dk.data_ptr(), d_q_weight.data_ptr(), d_k_weight.data_ptr(), workspace.data_ptr(),
        workspace.numel(), _raw_stream(dev))
    _check(st, what)
    return dq, dk, d_q_weight, d_k_weight


class _CacheStruct(ctypes.Structure):
    """moba_paged_cache of include/moba.h."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("k", "v", "k_scale", "v_scale", "block_sums",
                                               "page_table", "seq_lens")] + \
               [(n, ctypes.c_int32) for n in ("dtype", "nseq", "max_pages", "num_pages",
                                              "page_size", "Hkv", "d", "block_size")]


class PagedCache:
    """A paged key-value cache: the caller's tensors, checked once, as the cache calls take them.

    k, v: [num_pages, Hkv, page_size, d], bfloat16 or float8_e4m3fn; k_scale, v_scale (e4m3 only):
    uint8 [num_pages, Hkv, page_size]; page_table: int32 [nseq, max_pages]; seq_lens: int32 [nseq];
    block_sums (for moba_paged_decode_fwd): float32 [num_pages, Hkv, d] with its block_size. The
    tensors are kept by reference and their contents may change between calls; see
    include/moba.h for the layout and its limits.
    """

    def __init__(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor,
                 seq_lens: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None,
                 block_sums: Optional[torch.Tensor] = None, block_size: Optional[int] = None):
        what = "PagedCache"
        if not torch.is_tensor(k) or k.dim() != 4:
            _bad(what, "k must be a [num_pages, Hkv, page_size, d] tensor")
        if k.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            _bad(what, f"k must be torch.bfloat16 or torch.float8_e4m3fn, got {k.dtype}")
        _want(what, "k", k, k.dtype, None, _ANY_DEVICE)
        dev = _current_device(what, k)
        pages, hkv, page, d = k.shape
        _want(what, "v", v, k.dtype, (pages, hkv, page, d), dev)
        if not torch.is_tensor(page_table) or page_table.dim() != 2:
            _bad(what, "page_table must be a [nseq, max_pages] tensor")
        _want(what, "page_table", page_table, torch.int32, None, dev)
        nseq = page_table.shape[0]
        _want(what, "seq_lens", seq_lens, torch.int32, (nseq,), dev)
        fp8 = k.dtype == torch.float8_e4m3fn
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if fp8:
                _want(what, name, t, torch.uint8, (pages, hkv, page), dev)
            elif t is not None:
                _bad(what, f"{name} goes with an e4m3 cache")
        if block_sums is not None:
            _want(what, "block_sums", block_sums, torch.float32, (pages, hkv, d), dev)
            if not isinstance(block_size, int) or block_size < 1:
                _bad(what, "block_sums need a block_size")
        self.tensors = (k, v, k_scale, v_scale, block_sums, page_table, seq_lens)
        self.device, self.nseq, self.hkv, self.d = dev, nseq, hkv, d
        self._index = -1 if dev.index is None else dev.index
        load_library()
        self.block_size = block_size if block_sums is not None else 0
        ptr = [None if t is None else t.data_ptr() for t in self.tensors]
        self._c = _CacheStruct(*ptr, 1 if fp8 else 0, nseq, page_table.shape[1], pages, page, hkv,
                               d, self.block_size)
        self._ref = ctypes.addressof(self._c)
        self._bytes = {}

    def workspace_bytes(self, hq: int, rows_per_seq: int = 1, topk: int = 0) -> int:
        """Bytes of workspace for attention over this cache (topk 0: moba_paged_attn_fwd)."""
        key = (hq, rows_per_seq, topk)
        if key not in self._bytes:
            self._bytes[key] = int(load_library().moba_paged_workspace_bytes(
                self._ref, hq, rows_per_seq, topk))
        return self._bytes[key]

    def _here(self, what: str) -> torch.device:
        """The cache's device, which has to be the current one."""
        if torch.cuda.current_device() != self.device.index:
            _bad(what, f"the cache is on {self.device} but the current device is "
                       f"cuda:{torch.cuda.current_device()}")
        return self.device


def _cache(what: str, cache) -> PagedCache:
    if not isinstance(cache, PagedCache):
        _bad(what, "cache must be a PagedCache")
    return cache


def moba_cache_append(cache: PagedCache, k: torch.Tensor, v: torch.Tensor,
                      cu_seqlens_q: torch.Tensor, stream=None) -> None:
    """Writes the newest rows k, v [Tq, Hkv, d] bf16 (tokens may be strided) of every sequence
    (cu_seqlens_q [nseq + 1]; cache.seq_lens already counts them) into the cache's pages, rounded
    to 8 bits where the cache is e4m3, and adds the keys to their blocks' sums."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return moba_cache_append(cache, k, v, cu_seqlens_q)
    what = "moba_cache_append"
    if _bind is not None and type(cache) is PagedCache:
        done = _bind.append(cache._ref, cache._index, k, v, cu_seqlens_q)
        if done is not None:
            return _check(done, what)
    dev = _cache(what, cache)._here(what)
    k_ld = _rows(what, "k", k, cache.hkv, cache.d)
    v_ld = _rows(what, "v", v, cache.hkv, cache.d)
    if v.shape[0] != k.shape[0]:
        _bad(what, f"k and v must have the same rows, got {k.shape[0]} and {v.shape[0]}")
    if k.device != dev or v.device != dev:
        _bad(what, f"k is on {k.device} and v on {v.device}, the cache on {dev}")
    if not _is(cu_seqlens_q, torch.int32, (cache.nseq + 1,), dev):
        _want(what, "cu_seqlens_q", cu_seqlens_q, torch.int32, (cache.nseq + 1,), dev)
    _check(load_library().moba_cache_append(cache._ref, k.data_ptr(), k_ld, v.data_ptr(), v_ld,
                                            cu_seqlens_q.data_ptr(), k.shape[0],
                                            _raw_stream(dev)), what)


def moba_cache_read(cache: PagedCache, cu_seqlens: torch.Tensor, cu_seqlens_host,
                    k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None,
                    stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The first cu[s+1] - cu[s] cached tokens of every sequence, packed: (k, v) [T, Hkv, d] bf16
    as moba_attn_fwd takes them."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return moba_cache_read(cache, cu_seqlens, cu_seqlens_host, k, v)
    what = "moba_cache_read"
    dev = _cache(what, cache)._here(what)
    if len(cu_seqlens_host) != cache.nseq + 1:
        _bad(what, f"cu_seqlens_host must have {cache.nseq + 1} entries")
    if _bind is not None:
        done = _bind.read(cache._ref, cache._index, cu_seqlens, int(cu_seqlens_host[-1]), k, v)
        if done is not None:
            return _done(done, what)
    _want(what, "cu_seqlens", cu_seqlens, torch.int32, (cache.nseq + 1,), dev)
    shape = (int(cu_seqlens_host[-1]), cache.hkv, cache.d)
    if shape[0] < 0:
        _bad(what, "cu_seqlens_host must not be negative")
    k = torch.empty(shape, dtype=torch.bfloat16, device=dev) if k is None else k
    v = torch.empty(shape, dtype=torch.bfloat16, device=dev) if v is None else v
    _want(what, "k", k, torch.bfloat16, shape, dev)
    _want(what, "v", v, torch.bfloat16, shape, dev)
    _check(load_library().moba_cache_read(cache._ref, cu_seqlens.data_ptr(), shape[0],
                                          k.data_ptr(), v.data_ptr(), _raw_stream(dev)), what)
    return k, v


def _paged_plain(cache, q, rows_per_seq, topk, scale, idx, o, lse, workspace):
    """The call through csrc/bind.cpp, or None where its arguments are not plain."""
    if (_bind is None or type(cache) is not PagedCache
            or not torch.is_tensor(q) or q.dim() != 3):
        return None
    nbytes = 0 if workspace is not None else cache.workspace_bytes(q.shape[1], rows_per_seq, topk)
    return _bind.paged(cache._ref, cache._index, q, rows_per_seq, topk, scale, idx, o, lse,
                       workspace, nbytes)


def _paged(what, cache, q, rows_per_seq, topk, o, lse, workspace):
    """Checks and buffers that both attention calls over a paged cache share."""
    dev = _cache(what, cache)._here(what)
    if not torch.is_tensor(q) or q.dim() != 3:
        _bad(what, "q must be a 3-D tensor")
    n, hq, d = q.shape
    if rows_per_seq < 1 or n != cache.nseq * rows_per_seq or d != cache.d:
        _bad(what, f"q must have shape {(cache.nseq * rows_per_seq, hq, cache.d)}, "
                   f"got {tuple(q.shape)}")
    if not _is(q, torch.bfloat16, q.shape, dev):
        _want(what, "q", q, torch.bfloat16, None, dev)
    if o is None:
        o = torch.empty_like(q)
    else:
        _want(what, "o", o, torch.bfloat16, (n, hq, d), dev)
    if lse is None:
        lse = torch.empty((hq, n), dtype=torch.float32, device=dev)
    else:
        _want(what, "lse", lse, torch.float32, (hq, n), dev)
    if workspace is None:
        workspace = _workspace(cache.workspace_bytes(hq, rows_per_seq, topk), dev)
    else:
        _want(what, "workspace", workspace, torch.uint8, None, dev)
    return dev, n, hq, o, lse, workspace


def moba_paged_attn_fwd(cache: PagedCache, q: torch.Tensor, rows_per_seq: int = 1,
                        scale: Optional[float] = None, o: Optional[torch.Tensor] = None,
                        lse: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None):
    """Full attention of the last rows_per_seq tokens of every cached sequence: q
    [nseq * rows_per_seq, Hq, d] bf16; returns (o like q, lse [Hq, rows] fp32)."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return moba_paged_attn_fwd(cache, q, rows_per_seq, scale, o, lse, workspace)
    what = "moba_paged_attn_fwd"
    if scale is None:
        scale = _cache(what, cache).d ** -0.5
    done = _paged_plain(cache, q, rows_per_seq, 0, scale, None, o, lse, workspace)
    if done is not None:
        return _done(done, what)
    dev, n, hq, o, lse, ws = _paged(what, cache, q, rows_per_seq, 0, o, lse, workspace)
    st = load_library().moba_paged_attn_fwd(
        cache._ref, q.data_ptr(), hq, rows_per_seq, scale, o.data_ptr(),
        lse.data_ptr(), ws.data_ptr(), ws.numel(), _raw_stream(dev))
    _check(st, what)
    return o, lse


def moba_paged_decode_fwd(cache: PagedCache, q: torch.Tensor, topk: int, rows_per_seq: int = 1,
                          scale: Optional[float] = None,
                          block_idx_out: Optional[torch.Tensor] = None,
                          o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None):
    """MoBA attention of the last rows_per_seq tokens of every cached sequence: routing by the
    cache's block_sums, then attention over the selected blocks. Returns (o, lse) as
    moba_paged_attn_fwd; block_idx_out [Hq, rows, topk] int32 receives the routing."""
    if stream is not None:
        with torch.cuda.stream(stream):
            return moba_paged_decode_fwd(cache, q, topk, rows_per_seq, scale, block_idx_out, o,
                                         lse, workspace)
    what = "moba_paged_decode_fwd"
    if topk < 1 or not _cache(what, cache).block_size:
        _bad(what, "topk must be positive and the cache have block_sums")
    if scale is None:
        scale = cache.d ** -0.5
    done = _paged_plain(cache, q, rows_per_seq, topk, scale, block_idx_out, o, lse, workspace)
    if done is not None:
        return _done(done, what)
    dev, n, hq, o, lse, ws = _paged(what, cache, q, rows_per_seq, topk, o, lse, workspace)
    if block_idx_out is not None and not _is(block_idx_out, torch.int32, (hq, n, topk), dev):
        _want(what, "block_idx_out", block_idx_out, torch.int32, (hq, n, topk), dev)
    st = load_library().moba_paged_decode_fwd(
        cache._ref, q.data_ptr(), hq, rows_per_seq, topk, scale,
        None if block_idx_out is None else block_idx_out.data_ptr(), o.data_ptr(), lse.data_ptr(),
        ws.data_ptr(), ws.numel(), _raw_stream(dev))
    _check(st, what)
    return o, lse


def moba_device_status(workspace: torch.Tensor, stream=None) -> int:
    return int(load_library().moba_device_status(_ptr(workspace), _stream(stream)))


def moba_noalloc_status(stream=None) -> int:
    """Status word of the last moba_attn_fwd_noalloc call on the current device (synchronises)."""
    return int(load_library().moba_noalloc_status(_stream(stream)))


def set_wait_limit_ns(ns: int) -> int:
    """Diagnostics: limit of one pipeline wait in the attention kernel (0 = built-in 2 s);
    returns the previous limit."""
    return int(load_library().moba_set_wait_limit_ns(ctypes.c_ulonglong(int(ns))))


def set_diag_stall(on: bool) -> bool:
    """Diagnostics: make the attention kernel's MMA issuer wait on a barrier nothing arrives on
    (so that a short wait limit runs out); returns the previous setting."""
    return bool(load_library().moba_set_diag_stall(1 if on else 0))


def timing_enable(on: bool = True):
    load_library().moba_timing_enable(1 if on else 0)


def timing_reset():
    load_library().moba_timing_reset()


def timing_read() -> dict:
    lib = load_library()
    n = len(KERNEL_CLASSES)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_longlong * n)()
    r = lib.moba_timing_read(ms, cnt, n)
    if r < 0:
        raise MobaError(r, "moba_timing_read")
    return {KERNEL_CLASSES[i]: (float(ms[i]), int(cnt[i])) for i in range(n)}


def launch_count() -> int:
    return int(load_library().moba_launch_count())
