"""Python binding of the B200 CKDA library (``libckda.so``, C ABI in ``include/ckda.h``).

Argument marshalling only: every step of the computation runs in the library's CUDA kernels.
PyTorch supplies device memory and the current stream.  There is no CPU fallback: if the
compiled library is missing or no CUDA device is present, the calls raise.

Build the library with ``python -m gated_delta_rule_82_b200.build``.
"""
from __future__ import annotations

import ctypes
import functools
import os

import torch

__all__ = ["CkdaError", "library_path", "abi_version", "qk_prologue", "workspace_bytes",
           "fwd_chunked", "varlen_workspace_bytes", "fwd_varlen", "decode_step", "selftest_umma",
           "last_device_status", "set_wait_limit_ns", "bwd_workspace_bytes", "bwd_chunked",
           "linattn_fwd_workspace_bytes", "linattn_fwd_chunked", "linattn_bwd_workspace_bytes",
           "linattn_bwd_chunked", "linattn_decode_step", "block_norm", "block_norm_bwd",
           "block_norm_bwd_workspace_bytes", "PATHS"]

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libckda.so")
_lib = None

PATHS = {"auto": 0, "simt": 1, "tc": 2}
_F32, _BF16 = 0, 1


class CkdaError(RuntimeError):
    def __init__(self, func, status):
        self.status = status
        msg = _load().ckda_strerror(status).decode()
        super().__init__(f"{func} failed: status {status} ({msg})")


class _Flags(ctypes.Structure):
    _fields_ = [("l2norm", ctypes.c_int), ("rope_theta", ctypes.c_float),
                ("rope_convention", ctypes.c_int), ("scale", ctypes.c_float),
                ("path", ctypes.c_int), ("stages", ctypes.c_int), ("gate_logits", ctypes.c_int),
                ("rope_dims", ctypes.c_int), ("qk_heads", ctypes.c_int)]


class _NormFlags(ctypes.Structure):
    _fields_ = [("post_group", ctypes.c_int), ("gate_act", ctypes.c_int),
                ("res_scale", ctypes.c_float), ("eps", ctypes.c_float)]


def library_path() -> str:
    return _LIB_PATH


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise RuntimeError(f"CKDA CUDA library not built: {_LIB_PATH} is missing "
                           "(run python -m gated_delta_rule_82_b200.build)")
    lib = ctypes.CDLL(_LIB_PATH)
    P, I, LL, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t
    lib.ckda_abi_version.restype = I
    lib.ckda_abi_version.argtypes = []
    lib.ckda_strerror.restype = ctypes.c_char_p
    lib.ckda_strerror.argtypes = [I]
    lib.ckda_qk_prologue.restype = I
    lib.ckda_qk_prologue.argtypes = [P, P, P, P, I, I, I, I, _Flags, I, LL, P]
    lib.ckda_fwd_workspace_bytes.restype = SZ
    lib.ckda_fwd_workspace_bytes.argtypes = [I, I, I, I, I, I, I, I]
    lib.ckda_fwd_chunked.restype = I
    lib.ckda_fwd_chunked.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, _Flags, I, LL, P,
                                     SZ, P]
    lib.ckda_fwd_segmented_workspace_bytes.restype = SZ
    lib.ckda_fwd_segmented_workspace_bytes.argtypes = [I] * 6
    lib.ckda_fwd_segmented.restype = I
    lib.ckda_fwd_segmented.argtypes = [P] * 8 + [I] * 5 + [_Flags, I, LL, I, P, SZ, P]
    lib.ckda_fwd_simt_workspace_bytes.restype = SZ
    lib.ckda_fwd_simt_workspace_bytes.argtypes = [I] * 5
    lib.ckda_fwd_segments_auto.restype = I
    lib.ckda_fwd_segments_auto.argtypes = [I, I, I]
    lib.ckda_fwd_varlen_workspace_bytes.restype = SZ
    lib.ckda_fwd_varlen_workspace_bytes.argtypes = [P, I, I, I, I, I, I, I]
    lib.ckda_fwd_varlen.restype = I
    lib.ckda_fwd_varlen.argtypes = [P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, _Flags, I, LL, P,
                                    SZ, P]
    lib.ckda_decode_step.restype = I
    lib.ckda_decode_step.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, _Flags, I, P]
    lib.ckda_selftest_umma.restype = I
    lib.ckda_selftest_umma.argtypes = [P, P, P, I, I, I, I, P]
    lib.ckda_bwd_workspace_bytes.restype = SZ
    lib.ckda_bwd_workspace_bytes.argtypes = [I, I, I, I, I]
    lib.ckda_bwd_chunked.restype = I
    lib.ckda_bwd_chunked.argtypes = [P] * 14 + [I] * 5 + [_Flags, I, LL, P, SZ, P]
    lib.ckda_linattn_fwd_workspace_bytes.restype = SZ
    lib.ckda_linattn_fwd_workspace_bytes.argtypes = [I, I, P, I, I, I, I]
    lib.ckda_linattn_fwd_chunked.restype = I
    lib.ckda_linattn_fwd_chunked.argtypes = [P, P, P, P, I, P, P, P, I, I, P, P, I, I, I, I, _Flags,
                                             I, P, SZ, P]
    lib.ckda_linattn_bwd_workspace_bytes.restype = SZ
    lib.ckda_linattn_bwd_workspace_bytes.argtypes = [I, I, P, I, I, I, I, I]
    lib.ckda_linattn_bwd_chunked.restype = I
    lib.ckda_linattn_bwd_chunked.argtypes = [P, P, P, P, I] + [P] * 8 + [I, I, P, P, I, I, I, I,
                                                                       _Flags, I, P, SZ, P]
    lib.ckda_linattn_decode_step.restype = I
    lib.ckda_linattn_decode_step.argtypes = [P, P, P, P, I, P, P, I, I, I, I, _Flags, I, P]
    lib.ckda_block_norm.restype = I
    lib.ckda_block_norm.argtypes = [P] * 8 + [LL, I, _NormFlags, I, P]
    lib.ckda_block_norm_bwd_workspace_bytes.restype = SZ
    lib.ckda_block_norm_bwd_workspace_bytes.argtypes = [LL, I, I]
    lib.ckda_block_norm_bwd.restype = I
    lib.ckda_block_norm_bwd.argtypes = [P] * 14 + [LL, I, _NormFlags, I, P, SZ, P]
    lib.ckda_last_device_status.restype = I
    lib.ckda_last_device_status.argtypes = [P, ctypes.POINTER(I)]
    lib.ckda_set_wait_limit_ns.restype = I
    lib.ckda_set_wait_limit_ns.argtypes = [ctypes.c_ulonglong]
    _lib = lib
    return lib


def abi_version() -> int:
    return _load().ckda_abi_version()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return _BF16
    if t.dtype == torch.float32:
        return _F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def _check(t: torch.Tensor, name: str, dtype=None, shape=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _room(workspace, device):
    """(address, bytes) of a workspace that a caller gave, or (None, 0)."""
    if workspace is None:
        return None, 0
    if not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if workspace.device != device:
        raise ValueError(f"workspace is on {workspace.device}, expected {device}")
    if not workspace.is_contiguous():     # (its bytes are counted by its elements)
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _flags(l2norm, rope_theta, rope_convention, scale, path=0, stages=0, gate_logits=False,
           qk_heads=0, rope_dims=0):
    return _Flags(int(bool(l2norm)), float(rope_theta), int(rope_convention), float(scale),
                  int(path), int(stages), int(bool(gate_logits)), int(rope_dims), int(qk_heads))


def _raise(func, status):
    if status != 0:
        raise CkdaError(func, status)


def qk_prologue(q, k, *, l2norm=True, rope_theta=0.0, rope_convention=0, pos_offset=0,
                q_out=None, k_out=None, rope_dims=0):
    """Rotation at positions pos_offset + t, then per-head L2 norm, of q and k [B, T, H, dk]."""
    _check(q, "q")
    _check(k, "k", dtype=q.dtype, shape=q.shape)
    B, T, H, dk = q.shape
    q_out = torch.empty_like(q) if q_out is None else q_out
    k_out = torch.empty_like(k) if k_out is None else k_out
    _check(q_out, "q_out", dtype=q.dtype, shape=q.shape)
    _check(k_out, "k_out", dtype=q.dtype, shape=q.shape)
    st = _load().ckda_qk_prologue(_ptr(q), _ptr(k), _ptr(q_out), _ptr(k_out), B, T, H, dk,
                                  _flags(l2norm, rope_theta, rope_convention, 0.0,
                                         rope_dims=rope_dims),
                                  _dtype_code(q), int(pos_offset), _stream(q.device))
    _raise("ckda_qk_prologue", st)
    return q_out, k_out


def workspace_bytes(B, T, H, dk, dv, chunk=64, dtype=torch.bfloat16, path="auto") -> int:
    code = _BF16 if dtype == torch.bfloat16 else _F32
    n = _load().ckda_fwd_workspace_bytes(B, T, H, dk, dv, chunk, code, PATHS[path])
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("unsupported problem for ckda_fwd_chunked")
    return int(n)


def fwd_chunked(q, k, v, alpha, beta, h0=None, *, chunk=64, l2norm=True, rope_theta=0.0,
                rope_convention=0, scale=0.0, pos_offset=0, path="auto", want_state=True,
                out=None, hT=None, workspace=None, stages=0, gate_logits=False, rope_dims=0):
    """Chunked CKDA forward.  Returns (out [B, T, H, dv], hT [B, H, dk, dv] or None).

    q, k: [B, T, Hk, dk] (bf16 or fp32); v: [B, T, H, dv] same dtype, H a multiple of Hk (grouped
    value heads when H > Hk: value head h reads q/k head h // (H // Hk)); alpha: [B, T, H, dk]
    fp32; beta: [B, T, H] fp32; h0: [B, H, dk, dv] fp32 or None.  With gate_logits, alpha holds
    logits a in q's dtype and beta fp32 logits b; the kernels use alpha = 2 sigma(a) - 1 and
    beta = 2 sigma(b).
    """
    _check(q, "q")
    B, T, Hk, dk = q.shape
    _check(v, "v", dtype=q.dtype)
    if v.dim() != 4 or v.shape[:2] != (B, T):
        raise ValueError(f"v: expected [B={B}, T={T}, H, dv], got {tuple(v.shape)}")
    H, dv = v.shape[2], v.shape[3]
    if H % Hk:
        raise ValueError(f"v has {H} heads, not a multiple of q's {Hk}")
    _check(k, "k", dtype=q.dtype, shape=q.shape)
    _check(alpha, "alpha", dtype=q.dtype if gate_logits else torch.float32, shape=(B, T, H, dk))
    _check(beta, "beta", dtype=torch.float32, shape=(B, T, H))
    if h0 is not None:
        _check(h0, "h0", dtype=torch.float32, shape=(B, H, dk, dv))
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    _check(out, "out", dtype=q.dtype, shape=(B, T, H, dv))
    if want_state and hT is None:
        hT = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    if hT is not None:
        _check(hT, "hT", dtype=torch.float32, shape=(B, H, dk, dv))
    code = _dtype_code(q)
    if workspace is None:   # (a workspace given is checked against the need by the library)
        need = workspace_bytes(B, T, H, dk, dv, chunk, q.dtype, path)
        if need == 0:   # the CUDA-core path: the workspace of its record form
            need = int(_load().ckda_fwd_simt_workspace_bytes(B, T, H, dk, dv))
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    room = _room(workspace, q.device)
    st = _load().ckda_fwd_chunked(
        _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(h0), _ptr(out), _ptr(hT),
        B, T, H, dk, dv, int(chunk), _flags(l2norm, rope_theta, rope_convention, scale,
                                           PATHS[path], stages, gate_logits,
                                           Hk if Hk != H else 0, rope_dims),
        code, int(pos_offset), *room, _stream(q.device))
    _raise("ckda_fwd_chunked", st)
    return out, hT


def simt_workspace_bytes(B, T, H, dk, dv) -> int:
    """Bytes of the optional workspace that selects the record form of the CUDA-core path."""
    n = _load().ckda_fwd_simt_workspace_bytes(B, T, H, dk, dv)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("unsupported problem for the CUDA-core path")
    return int(n)


def segments_auto(B, T, H) -> int:
    """Segment count ckda_fwd_segments_auto picks for a batch of B x H sequences of T tokens on the
    current device (1: the single fused launch is expected to be faster)."""
    return int(_load().ckda_fwd_segments_auto(B, T, H))


def segmented_workspace_bytes(B, T, H, dk, dv, segments) -> int:
    n = _load().ckda_fwd_segmented_workspace_bytes(B, T, H, dk, dv, segments)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("unsupported problem for ckda_fwd_segmented")
    return int(n)


def fwd_segmented(q, k, v, alpha, beta, h0=None, *, segments=0, l2norm=True, rope_theta=0.0,
                  rope_convention=0, scale=0.0, pos_offset=0, want_state=True, out=None, hT=None,
                  workspace=None, gate_logits=False, rope_dims=0):
    """Tensor-core forward with the segment-parallel state pass (ckda_fwd_segmented): arguments
    and results as fwd_chunked (bf16, dk = dv = 128).  segments = 0 takes segments_auto's count.
    Returns (out, hT)."""
    _check(q, "q")
    B, T, Hk, dk = q.shape
    _check(v, "v", dtype=q.dtype)
    if v.dim() != 4 or v.shape[:2] != (B, T):
        raise ValueError(f"v: expected [B={B}, T={T}, H, dv], got {tuple(v.shape)}")
    H, dv = v.shape[2], v.shape[3]
    if H % Hk:
        raise ValueError(f"v has {H} heads, not a multiple of q's {Hk}")
    _check(k, "k", dtype=q.dtype, shape=q.shape)
    _check(alpha, "alpha", dtype=q.dtype if gate_logits else torch.float32, shape=(B, T, H, dk))
    _check(beta, "beta", dtype=torch.float32, shape=(B, T, H))
    if h0 is not None:
        _check(h0, "h0", dtype=torch.float32, shape=(B, H, dk, dv))
    if segments == 0:
        segments = segments_auto(B, T, H)
    if out is None:
        out = torch.empty((B, T, H, dv), dtype=q.dtype, device=q.device)
    _check(out, "out", dtype=q.dtype, shape=(B, T, H, dv))
    if want_state and hT is None:
        hT = torch.empty((B, H, dk, dv), dtype=torch.float32, device=q.device)
    if hT is not None:
        _check(hT, "hT", dtype=torch.float32, shape=(B, H, dk, dv))
    if workspace is None:
        workspace = torch.empty(segmented_workspace_bytes(B, T, H, dk, dv, segments),
                                dtype=torch.uint8, device=q.device)
    room = _room(workspace, q.device)
    st = _load().ckda_fwd_segmented(
        _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(h0), _ptr(out), _ptr(hT),
        B, T, H, dk, dv, _flags(l2norm, rope_theta, rope_convention, scale, PATHS["tc"], 0,
                                gate_logits, Hk if Hk != H else 0, rope_dims),
        _dtype_code(q), int(pos_offset), int(segments), *room,
        _stream(q.device))
    _raise("ckda_fwd_segmented", st)
    return out, hT


def _offsets(host):
    """Host offsets as int32 (the library reads them where they lie)."""
    if not isinstance(host, torch.Tensor):
        raise TypeError("cu_seqlens_cpu must be a torch.Tensor")
    if host.device.type != "cpu":
        raise ValueError("cu_seqlens_cpu is not on the CPU")
    if host.numel() < 2:
        raise ValueError("cu_seqlens_cpu: expected [n + 1] token offsets, n >= 1")
    return host.to(torch.int32).contiguous()


def _host_offsets(cu_seqlens, cu_seqlens_cpu):
    """int32 offsets on the device (as given) and a host copy (given, or read back: a sync)."""
    _check(cu_seqlens, "cu_seqlens", dtype=torch.int32)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2:
        raise ValueError("cu_seqlens: expected [n + 1] token offsets, n >= 1")
    host = _offsets(cu_seqlens.cpu() if cu_seqlens_cpu is None else cu_seqlens_cpu)
    if tuple(host.shape) != tuple(cu_seqlens.shape):
        raise ValueError("cu_seqlens_cpu must have the shape of cu_seqlens")
    return host


def varlen_workspace_bytes(cu_seqlens_cpu, H, dk, dv, chunk, dtype, path="auto") -> int:
    """Device workspace bytes of fwd_varlen for these host offsets (0 when none is needed)."""
    host = _offsets(cu_seqlens_cpu)
    code = _BF16 if dtype == torch.bfloat16 else _F32
    n = _load().ckda_fwd_varlen_workspace_bytes(ctypes.c_void_p(host.data_ptr()), host.numel() - 1,
                                                H, dk, dv, chunk, code, PATHS[path])
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("unsupported sizes or invalid offsets for the packed forward")
    return n


def fwd_varlen(q, k, v, alpha, beta, cu_seqlens, h0=None, *, cu_seqlens_cpu=None, chunk=64,
               l2norm=True, rope_theta=0.0, rope_convention=0, scale=0.0, pos_offset=0,
               path="auto", want_state=True, out=None, hT=None, workspace=None, stages=0,
               gate_logits=False, rope_dims=0):
    """Chunked CKDA forward over packed sequences of different lengths.  Returns (out, hT).

    q, k: [1, T, Hk, dk] or [T, Hk, dk]; v: [.., T, H, dv]; alpha: [.., T, H, dk]; beta:
    [.., T, H] (the layouts of fwd_chunked with a batch of 1, or without the batch axis);
    cu_seqlens: int32 [n + 1] on the device, token offsets of the n sequences (0 first,
    non-decreasing, T last); cu_seqlens_cpu: the same offsets on the host (read back from the
    device when omitted); h0 / hT: [n, H, dk, dv] fp32.  Each sequence starts from its own h0,
    ends in its own hT, and its rotary positions start again at pos_offset.
    """
    _check(q, "q")
    lead = q.dim() == 4
    if lead and q.shape[0] != 1:
        raise ValueError("packed sequences take a batch axis of 1 (or none)")
    T, Hk, dk = q.shape[-3:]
    _check(v, "v", dtype=q.dtype)
    if v.dim() != q.dim() or v.shape[-3] != T:
        raise ValueError(f"v: expected [.., T={T}, H, dv], got {tuple(v.shape)}")
    H, dv = v.shape[-2], v.shape[-1]
    if H % Hk:
        raise ValueError(f"v has {H} heads, not a multiple of q's {Hk}")
    pre = (1,) if lead else ()
    _check(k, "k", dtype=q.dtype, shape=q.shape)
    _check(alpha, "alpha", dtype=q.dtype if gate_logits else torch.float32, shape=pre + (T, H, dk))
    _check(beta, "beta", dtype=torch.float32, shape=pre + (T, H))
    host = _host_offsets(cu_seqlens, cu_seqlens_cpu)
    n = host.numel() - 1
    if int(host[-1]) != T:
        raise ValueError(f"cu_seqlens ends at {int(host[-1])}, but the token axis holds {T}")
    if h0 is not None:
        _check(h0, "h0", dtype=torch.float32, shape=(n, H, dk, dv))
    if out is None:
        out = torch.empty(pre + (T, H, dv), dtype=q.dtype, device=q.device)
    _check(out, "out", dtype=q.dtype, shape=pre + (T, H, dv))
    if want_state and hT is None:
        hT = torch.empty((n, H, dk, dv), dtype=torch.float32, device=q.device)
    if hT is not None:
        _check(hT, "hT", dtype=torch.float32, shape=(n, H, dk, dv))
    if workspace is None:   # (a workspace given is checked against the need by the library)
        need = varlen_workspace_bytes(host, H, dk, dv, chunk, q.dtype, path)
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    room = _room(workspace, q.device)
    st = _load().ckda_fwd_varlen(
        _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(h0), _ptr(out), _ptr(hT),
        _ptr(cu_seqlens), ctypes.c_void_p(host.data_ptr()), n, H, dk, dv, int(chunk),
        _flags(l2norm, rope_theta, rope_convention, scale, PATHS[path], stages, gate_logits,
               Hk if Hk != H else 0, rope_dims),
        _dtype_code(q), int(pos_offset), *room, _stream(q.device))
    _raise("ckda_fwd_varlen", st)
    return out, hT


def decode_step(q, k, v, alpha, beta, state, pos=None, *, l2norm=True, rope_theta=0.0,
                rope_convention=0, scale=0.0, out=None, gate_logits=False, rope_dims=0):
    """One decode step, in place on state [N, H, dk, dv] fp32.  Returns out [N, H, dv].
    q, k: [N, Hk, dk] with H a multiple of Hk (grouped value heads when H > Hk).  With
    gate_logits, alpha holds logits a in q's dtype and beta fp32 logits b."""
    _check(q, "q")
    N, Hk, dk = q.shape
    _check(v, "v", dtype=q.dtype)
    if v.dim() != 3 or v.shape[0] != N:
        raise ValueError(f"v: expected [N={N}, H, dv], got {tuple(v.shape)}")
    H, dv = v.shape[1], v.shape[2]
    if H % Hk:
        raise ValueError(f"v has {H} heads, not a multiple of q's {Hk}")
    _check(k, "k", dtype=q.dtype, shape=q.shape)
    _check(alpha, "alpha", dtype=q.dtype if gate_logits else torch.float32, shape=(N, H, dk))
    _check(beta, "beta", dtype=torch.float32, shape=(N, H))
    _check(state, "state", dtype=torch.float32, shape=(N, H, dk, dv))
    if pos is not None:
        _check(pos, "pos", dtype=torch.int64, shape=(N,))
    if out is None:
        out = torch.empty((N, H, dv), dtype=q.dtype, device=q.device)
    _check(out, "out", dtype=q.dtype, shape=(N, H, dv))
    st = _load().ckda_decode_step(
        _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(state), _ptr(out), _ptr(pos),
        N, H, dk, dv, _flags(l2norm, rope_theta, rope_convention, scale, 0, 0, gate_logits,
                             Hk if Hk != H else 0, rope_dims),
        _dtype_code(q),
        _stream(q.device))
    _raise("ckda_decode_step", st)
    return out


def bwd_workspace_bytes(B, T, H, dk, dv) -> int:
    n = _load().ckda_bwd_workspace_bytes(B, T, H, dk, dv)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("unsupported problem for ckda_bwd_chunked")
    return int(n)


def bwd_chunked(q, k, v, alpha, beta, h0, dout, dhT=None, *, l2norm=True, rope_theta=0.0,
                rope_convention=0, scale=0.0, pos_offset=0, gate_logits=False, rope_dims=0,
                workspace=None, want_dh0=True):
    """Gradients of <dout, out> + <dhT, hT> for fwd_chunked with the same inputs and flags.

    Returns a dict of fp32 tensors: dq, dk ([B, T, Hk, dk]), dv, dalpha, dbeta and dh0 (None
    when want_dh0 is False).  dout has the dtype of q; dhT is fp32 [B, H, dk, dv] or None.
    """
    _check(q, "q")
    B, T, Hk, dk = q.shape
    _check(v, "v", dtype=q.dtype)
    H, dv = v.shape[2], v.shape[3]
    if H % Hk:
        raise ValueError(f"v has {H} heads, not a multiple of q's {Hk}")
    _check(k, "k", dtype=q.dtype, shape=q.shape)
    _check(alpha, "alpha", dtype=q.dtype if gate_logits else torch.float32, shape=(B, T, H, dk))
    _check(beta, "beta", dtype=torch.float32, shape=(B, T, H))
    _check(dout, "dout", dtype=q.dtype, shape=(B, T, H, dv))
    if h0 is not None:
        _check(h0, "h0", dtype=torch.float32, shape=(B, H, dk, dv))
    if dhT is not None:
        _check(dhT, "dhT", dtype=torch.float32, shape=(B, H, dk, dv))
    f32 = dict(dtype=torch.float32, device=q.device)
    g = {"dq": torch.empty((B, T, Hk, dk), **f32), "dk": torch.empty((B, T, Hk, dk), **f32),
         "dv": torch.empty((B, T, H, dv), **f32), "dalpha": torch.empty((B, T, H, dk), **f32),
         "dbeta": torch.empty((B, T, H), **f32),
         "dh0": torch.empty((B, H, dk, dv), **f32) if want_dh0 else None}
    if workspace is None:
        workspace = torch.empty(bwd_workspace_bytes(B, T, H, dk, dv), dtype=torch.uint8,
                                device=q.device)
    room = _room(workspace, q.device)
    st = _load().ckda_bwd_chunked(
        _ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(h0), _ptr(dout), _ptr(dhT),
        _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["dalpha"]), _ptr(g["dbeta"]),
        _ptr(g["dh0"]), B, T, H, dk, dv,
        _flags(l2norm, rope_theta, rope_convention, scale, 0, 0, gate_logits,
               Hk if Hk != H else 0, rope_dims),
        _dtype_code(q), int(pos_offset), *room, _stream(q.device))
    _raise("ckda_bwd_chunked", st)
    return g


# The calls below are used token by token and layer by layer, where the marshalling costs as much as
# a small kernel: pointers go to ctypes as plain integers, and checks that pass are made inline.

def _need(t, name, dtype, shape, device):
    """t is a contiguous CUDA tensor of this type and shape on this device."""
    if type(t) is torch.Tensor and t.dtype is dtype and t.shape == shape and t.device == device \
            and t.is_contiguous():
        return
    _check(t, name, dtype=dtype, shape=shape)
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _p(t):
    return None if t is None else t.data_ptr()


# (the handle alone: building a Stream object costs as much as the launch)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(fn, device, *args):
    """fn(*args, stream) with `device` current, on its current stream."""
    if torch.cuda.current_device() == device.index:
        return fn(*args, _raw_stream(device.index))
    with torch.cuda.device(device):
        return fn(*args, _raw_stream(device.index))


@functools.lru_cache(maxsize=256)
def _linattn_flags(scale, qk_heads):
    return _flags(False, 0.0, 0, scale, qk_heads=qk_heads)


@functools.lru_cache(maxsize=256)
def _linattn_rows_bytes(backward, B, T, H, Hk, dk, dv):
    """Workspace bytes for B rows of T tokens (a function of the sizes alone)."""
    return (linattn_bwd_workspace_bytes(B, T, H, Hk, dk, dv) if backward
            else linattn_fwd_workspace_bytes(B, T, H, dk, dv))


def _linattn_shapes(q, k, v, log_decay, cu_seqlens, cu_seqlens_cpu):
    """(B, T, n, lead, H, Hk, dk, dv, per_token, host offsets) of the chunked calls' arguments."""
    _check(q, "q")
    dev = q.device
    packed = cu_seqlens is not None
    if not packed and q.dim() != 4:
        raise ValueError(f"q: expected [B, T, Hk, dk], got {tuple(q.shape)}")
    if packed and q.dim() not in (3, 4):
        raise ValueError(f"q: expected [T, Hk, dk] or [1, T, Hk, dk], got {tuple(q.shape)}")
    if packed and q.dim() == 4 and q.shape[0] != 1:
        raise ValueError("packed sequences take a batch axis of 1 (or none)")
    *lead, Hk, dk = q.shape
    lead = tuple(lead)
    if not isinstance(v, torch.Tensor) or v.dim() != q.dim():
        raise ValueError(f"v: expected {lead + ('H', 'dv')}")
    H, dv = v.shape[-2:]
    if Hk < 1 or H < 1 or H % Hk:
        raise ValueError(f"v has {H} heads, not a multiple of q's {Hk}")
    _need(v, "v", q.dtype, lead + (H, dv), dev)
    _need(k, "k", q.dtype, q.shape, dev)
    per_token = isinstance(log_decay, torch.Tensor) and log_decay.dim() != 1
    _need(log_decay, "log_decay", torch.float32, lead + (H,) if per_token else (H,), dev)
    if not packed:
        return *lead, lead[0], lead, H, Hk, dk, dv, per_token, None
    host = _host_offsets(cu_seqlens, cu_seqlens_cpu)
    if cu_seqlens.device != dev:
        raise ValueError(f"cu_seqlens is on {cu_seqlens.device}, q on {dev}")
    if int(host[-1]) != lead[-1]:
        raise ValueError(f"cu_seqlens ends at {int(host[-1])}, but the token axis holds {lead[-1]}")
    return 1, lead[-1], host.numel() - 1, lead, H, Hk, dk, dv, per_token, host


def linattn_fwd_workspace_bytes(B, T, H, dk, dv, cu_seqlens_cpu=None) -> int:
    """Device workspace bytes of linattn_fwd_chunked: B rows of T tokens, or (B and T ignored)
    packed sequences with these host offsets.  0 when none is needed."""
    host = None if cu_seqlens_cpu is None else _offsets(cu_seqlens_cpu)
    n = _load().ckda_linattn_fwd_workspace_bytes(B, T, _ptr(host),
                                                 0 if host is None else host.numel() - 1, H, dk, dv)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("unsupported problem for ckda_linattn_fwd_chunked")
    return int(n)


def linattn_fwd_chunked(q, k, v, log_decay, h0=None, *, cu_seqlens=None, cu_seqlens_cpu=None,
                        scale=0.0, want_state=True, out=None, hT=None, workspace=None):
    """Chunked linear attention with a decay for each head:
    S_t = exp(log_decay_t) S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.  Returns (out, hT or None).

    q, k: [B, T, Hk, dk] (bf16 or fp32); v: [B, T, H, dv] same dtype, H a multiple of Hk (value
    head h reads q/k head h // (H // Hk)); log_decay: fp32, [B, T, H] or [H] (fixed per head),
    <= 0, -inf resets the state; h0 / hT: [B, H, dk, dv] fp32.  With cu_seqlens (int32 [n + 1] on
    the device; cu_seqlens_cpu the same on the host, read back when omitted) the token axis holds n
    packed sequences: [T, ..] or [1, T, ..] inputs, h0 / hT [n, H, dk, dv].  q and k are used as
    they are (qk_prologue rotates and normalises them).
    """
    B, T, n, lead, H, Hk, dk, dv, per_token, host = _linattn_shapes(q, k, v, log_decay, cu_seqlens,
                                                                    cu_seqlens_cpu)
    dev, shape, states = q.device, lead + (H, dv), (n, H, dk, dv)
    if h0 is not None:
        _need(h0, "h0", torch.float32, states, dev)
    if out is None:
        out = torch.empty(shape, dtype=q.dtype, device=dev)
    else:
        _need(out, "out", q.dtype, shape, dev)
    if hT is not None:
        _need(hT, "hT", torch.float32, states, dev)
    elif want_state:
        hT = torch.empty(states, dtype=torch.float32, device=dev)
    if workspace is None:   # (a workspace given is checked against the need by the library)
        need = (_linattn_rows_bytes(False, B, T, H, Hk, dk, dv) if host is None
                else linattn_fwd_workspace_bytes(B, T, H, dk, dv, host))
        if need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    room = _room(workspace, dev)
    st = _call(_load().ckda_linattn_fwd_chunked, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(),
               log_decay.data_ptr(), int(per_token), _p(h0), out.data_ptr(), _p(hT), B, T,
               _p(cu_seqlens), _p(host), 0 if host is None else n, H, dk, dv,
               _linattn_flags(float(scale), Hk if Hk != H else 0), _dtype_code(q), *room)
    _raise("ckda_linattn_fwd_chunked", st)
    return out, hT


def linattn_bwd_workspace_bytes(B, T, H, Hk, dk, dv, cu_seqlens_cpu=None) -> int:
    """Device workspace bytes of linattn_bwd_chunked (arguments as the forward's query)."""
    host = None if cu_seqlens_cpu is None else _offsets(cu_seqlens_cpu)
    n = _load().ckda_linattn_bwd_workspace_bytes(B, T, _ptr(host),
                                                 0 if host is None else host.numel() - 1, H, Hk, dk,
                                                 dv)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("unsupported problem for ckda_linattn_bwd_chunked")
    return int(n)


def linattn_bwd_chunked(q, k, v, log_decay, h0, dout, dhT=None, *, cu_seqlens=None,
                        cu_seqlens_cpu=None, scale=0.0, want_dlog_decay=True, want_dh0=True,
                        workspace=None):
    """Gradients of <dout, out> + <dhT, hT> for linattn_fwd_chunked with the same inputs.

    Returns a dict: dq, dk, dv in the inputs' dtype and layouts (a grouped q/k head receives the
    sum over its value heads), dlog_decay (fp32, log_decay's shape) and dh0 (fp32); the last two
    are None when not wanted.  dout has out's dtype and layout, dhT is fp32 or None.
    """
    B, T, n, lead, H, Hk, dk, dv, per_token, host = _linattn_shapes(q, k, v, log_decay, cu_seqlens,
                                                                    cu_seqlens_cpu)
    dev, states = q.device, (n, H, dk, dv)
    _need(dout, "dout", q.dtype, lead + (H, dv), dev)
    if h0 is not None:
        _need(h0, "h0", torch.float32, states, dev)
    if dhT is not None:
        _need(dhT, "dhT", torch.float32, states, dev)
    g = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
         "dlog_decay": torch.empty_like(log_decay) if want_dlog_decay else None,
         "dh0": torch.empty(states, dtype=torch.float32, device=dev) if want_dh0 else None}
    if workspace is None:
        need = (_linattn_rows_bytes(True, B, T, H, Hk, dk, dv) if host is None
                else linattn_bwd_workspace_bytes(B, T, H, Hk, dk, dv, host))
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    room = _room(workspace, dev)
    st = _call(_load().ckda_linattn_bwd_chunked, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(),
               log_decay.data_ptr(), int(per_token), _p(h0), dout.data_ptr(), _p(dhT),
               g["dq"].data_ptr(), g["dk"].data_ptr(), g["dv"].data_ptr(), _p(g["dlog_decay"]),
               _p(g["dh0"]), B, T, _p(cu_seqlens), _p(host), 0 if host is None else n, H, dk, dv,
               _linattn_flags(float(scale), Hk if Hk != H else 0), _dtype_code(q), *room)
    _raise("ckda_linattn_bwd_chunked", st)
    return g


def linattn_decode_step(q, k, v, log_decay, state, *, scale=0.0, out=None):
    """One token of the linear attention for N sequences, in place on state [N, H, dk, dv] fp32:
    S <- exp(log_decay) S + k v^T, out = scale S^T q [N, H, dv].  q, k: [N, Hk, dk]; v: [N, H, dv];
    log_decay: fp32 [N, H] or [H]."""
    _check(q, "q")
    if q.dim() != 3:
        raise ValueError(f"q: expected [N, Hk, dk], got {tuple(q.shape)}")
    N, Hk, dk = q.shape
    if not isinstance(v, torch.Tensor) or v.dim() != 3:
        raise ValueError(f"v: expected [N={N}, H, dv]")
    H, dv = v.shape[1:]
    if Hk < 1 or H % Hk:
        raise ValueError(f"v has {H} heads, not a multiple of q's {Hk}")
    dev = q.device
    _need(k, "k", q.dtype, q.shape, dev)
    _need(v, "v", q.dtype, (N, H, dv), dev)
    per_token = isinstance(log_decay, torch.Tensor) and log_decay.dim() != 1
    _need(log_decay, "log_decay", torch.float32, (N, H) if per_token else (H,), dev)
    _need(state, "state", torch.float32, (N, H, dk, dv), dev)
    if out is None:
        out = torch.empty_like(v)
    else:
        _need(out, "out", q.dtype, v.shape, dev)
    st = _call(_load().ckda_linattn_decode_step, dev, q.data_ptr(), k.data_ptr(), v.data_ptr(),
               log_decay.data_ptr(), int(per_token), state.data_ptr(), out.data_ptr(), N, H, dk, dv,
               _linattn_flags(float(scale), Hk if Hk != H else 0), _dtype_code(q))
    _raise("ckda_linattn_decode_step", st)
    return out


GATE_ACTS = {"none": 0, "sigmoid": 1, "silu": 2}


@functools.lru_cache(maxsize=256)
def _norm_flags(post_group, gate_act, res_scale, eps):
    return _NormFlags(post_group, GATE_ACTS[gate_act], res_scale, eps)


def _norm_args(y, gate, gate_act, residual, post_group, post_weight, res_scale, res_vector, eps,
               pre_weight):
    """(rows, D, flags) of the block norms' shared arguments."""
    _check(y, "y")
    if y.dim() < 1 or y.numel() == 0:
        raise ValueError(f"y: expected [.., D] with at least one row, got {tuple(y.shape)}")
    D, dev = y.shape[-1], y.device
    if gate is not None:
        _need(gate, "gate", y.dtype, y.shape, dev)
    if residual is not None:
        _need(residual, "residual", y.dtype, y.shape, dev)
    if gate_act not in GATE_ACTS:
        raise ValueError(f"gate_act: expected one of {sorted(GATE_ACTS)}, got {gate_act!r}")
    if (gate is None) != (gate_act == "none"):
        raise ValueError("gate and gate_act go together (gate_act 'none' without a gate)")
    if post_weight is not None:
        if not post_group:
            raise ValueError("post_weight without a first norm (post_group = 0)")
        _need(post_weight, "post_weight", torch.float32, (post_group,), dev)
    if res_vector is not None:
        _need(res_vector, "res_vector", torch.float32, (D,), dev)
    if pre_weight is not None:
        _need(pre_weight, "pre_weight", torch.float32, (D,), dev)
    return y.numel() // D, D, _norm_flags(int(post_group), gate_act, float(res_scale), float(eps))


def block_norm(y, *, gate=None, gate_act="none", residual=None, post_group=0, post_weight=None,
               res_scale=1.0, res_vector=None, pre_norm=False, pre_weight=None, eps=1e-5, h=None,
               n=None):
    """The norms around a block, fused with its gate, scale and the residual add, for y [.., D]:

        u = rms_norm(y, over groups of post_group channels) * post_weight   (post_group 0: u = y)
        h = residual + res_scale * res_vector * u * act(gate)
        n = rms_norm(h, over D) * pre_weight                                 (with pre_norm)

    Returns (h, n or None) in y's dtype (bf16 or fp32).  post_group: 0, D, or 16, 32, 64, 128
    dividing D (a norm per head, one weight [post_group] for all); gate, residual: y's shape or
    None; gate_act "sigmoid" or "silu" with a gate; weights fp32, None for ones.  An attention
    head's output norm with its gate is block_norm(out.flatten(-2), post_group=dv, gate=..., ...).
    """
    rows, D, flags = _norm_args(y, gate, gate_act, residual, post_group, post_weight, res_scale,
                                res_vector, eps, pre_weight)
    if pre_weight is not None and not pre_norm:
        raise ValueError("pre_weight without pre_norm")
    if n is not None and not pre_norm:
        raise ValueError("n without pre_norm")
    if h is None:
        h = torch.empty_like(y)
    else:
        _need(h, "h", y.dtype, y.shape, y.device)
    if pre_norm:
        if n is None:
            n = torch.empty_like(y)
        else:
            _need(n, "n", y.dtype, y.shape, y.device)
    st = _call(_load().ckda_block_norm, y.device, y.data_ptr(), _p(gate), _p(residual),
               _p(post_weight), _p(res_vector), _p(pre_weight), h.data_ptr(), _p(n), rows, D, flags,
               _dtype_code(y))
    _raise("ckda_block_norm", st)
    return h, n


@functools.lru_cache(maxsize=256)
def block_norm_bwd_workspace_bytes(rows, D, post_group=0) -> int:
    n = _load().ckda_block_norm_bwd_workspace_bytes(rows, D, post_group)
    if n == ctypes.c_size_t(-1).value:
        raise ValueError("unsupported problem for ckda_block_norm_bwd")
    return int(n)


def block_norm_bwd(y, dh, dn=None, *, gate=None, gate_act="none", residual=None, post_group=0,
                   post_weight=None, res_scale=1.0, res_vector=None, pre_norm=False,
                   pre_weight=None, eps=1e-5, workspace=None):
    """Gradients of <dh, h> + <dn, n> for block_norm with the same arguments (dh or dn may be None,
    not both; dn only with pre_norm).

    Returns a dict: dy, and dgate and dresidual where there is a gate and a residual, in y's dtype;
    dpost_weight, dres_vector and dpre_weight (fp32) where those vectors were given; else None.
    """
    rows, D, flags = _norm_args(y, gate, gate_act, residual, post_group, post_weight, res_scale,
                                res_vector, eps, pre_weight)
    if dn is not None and not pre_norm:
        raise ValueError("dn without pre_norm")
    if dh is None and dn is None:
        raise ValueError("dh and dn are both missing")
    if pre_weight is not None and not pre_norm:
        raise ValueError("pre_weight without pre_norm")
    if dh is not None:
        _need(dh, "dh", y.dtype, y.shape, y.device)
    if dn is not None:
        _need(dn, "dn", y.dtype, y.shape, y.device)
    like = lambda t: None if t is None else torch.empty_like(t)
    g = {"dy": torch.empty_like(y), "dgate": like(gate), "dresidual": like(residual),
         "dpost_weight": like(post_weight), "dres_vector": like(res_vector), "dpre_weight": None}
    if pre_weight is not None:
        g["dpre_weight"] = torch.empty_like(pre_weight) if dn is not None else \
            torch.zeros_like(pre_weight)
    sums = post_weight is not None or res_vector is not None or pre_weight is not None
    if workspace is None and sums:
        workspace = torch.empty(block_norm_bwd_workspace_bytes(rows, D, post_group),
                                dtype=torch.uint8, device=y.device)
    room = _room(workspace, y.device)
    st = _call(_load().ckda_block_norm_bwd, y.device, y.data_ptr(), _p(gate), _p(residual),
               _p(post_weight), _p(res_vector), _p(pre_weight), _p(dh), _p(dn), g["dy"].data_ptr(),
               _p(g["dgate"]), _p(g["dresidual"]), _p(g["dpost_weight"]), _p(g["dres_vector"]),
               _p(g["dpre_weight"]) if dn is not None else None, rows, D, flags, _dtype_code(y),
               *room)
    _raise("ckda_block_norm_bwd", st)
    return g


def last_device_status(device=None) -> int:
    """Wait for the current stream of `device` (or of the current one), then read and clear the
    library's status word there:
    0 = no failure recorded; 1 / 2 = a bounded wait of the tensor-core forward ran out (factor
    work / state pass); 3 = packed-sequence offsets on the device disagreed with the host copy; 4 = a
    bounded wait of the linear attention's tensor-core kernels ran out."""
    code = ctypes.c_int(0)
    with torch.cuda.device(device):     # (each device has a word of its own)
        st = _load().ckda_last_device_status(_stream(device), ctypes.byref(code))
    if st not in (0, 8):   # CKDA_OK, CKDA_ERR_DEVICE_STATUS
        raise CkdaError("ckda_last_device_status", st)
    return int(code.value)


def set_wait_limit_ns(ns: int = 0) -> None:
    """Upper bound of one wait of the tensor-core forward's state pass on the current device
    (0 restores the default of 4 s).  A diagnostic: a short limit makes a wait give up sooner."""
    _raise("ckda_set_wait_limit_ns", _load().ckda_set_wait_limit_ns(int(ns)))


def selftest_umma(A, B, b_mn_major=False, a_tmem=False):
    """fp32 A @ B^T (b_mn_major=False, B [N, K]) or A @ B (B [K, N]) via the library's tcgen05
    wrappers, for bf16 A [M, K] and B.  a_tmem: False (A from shared memory), True or "cp" (A
    copied into Tensor Memory by tcgen05.cp), "st" (A written into Tensor Memory by tcgen05.st)."""
    _check(A, "A", dtype=torch.bfloat16)
    _check(B, "B", dtype=torch.bfloat16)
    M, K = A.shape
    N = B.shape[1] if b_mn_major else B.shape[0]
    D = torch.empty((M, N), dtype=torch.float32, device=A.device)
    mode = int(bool(b_mn_major)) | (4 if a_tmem == "st" else 2 if a_tmem else 0)
    st = _load().ckda_selftest_umma(_ptr(A), _ptr(B), _ptr(D), M, N, K, mode,
                                    _stream(A.device))
    _raise("ckda_selftest_umma", st)
    return D
