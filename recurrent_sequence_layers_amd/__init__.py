"""Python binding of libqdelta.so, the gfx950 Q-Delta layer library.

Argument marshalling only: every step of the layer runs in the HIP kernels behind
the C ABI declared in ``include/qdelta.h``.  PyTorch supplies device memory and the
HIP stream: every wrapper takes ``stream=None`` (torch's current stream) or a
``torch.cuda.Stream``, enqueues the kernels on it and allocates any output or workspace
it creates while that stream is current.  If the library is not built, the functions raise; there is no
fallback path.

    qdelta_chunk_fwd(q, k, v, alpha, beta, lam, S0=None, C=64, o=None, S_T=None)
        -> (o, S_T)
    qdelta_step(q, k, v, alpha, beta, lam, S, o=None) -> o        (S updated in place)
    qdelta_chunk_bwd(q, k, v, alpha, beta, lam, S0, d_o, dS_T=None, C=64)
        -> dict(dq, dk, dv, dalpha, dbeta, dlam, dS0)

The operators around the recurrence (a short causal convolution before it, a selective state
space scan beside it, a gated group norm after it), each forward, backward and, where it
carries a state, for one token:

    qdelta_conv_fwd / qdelta_conv_step / qdelta_conv_bwd
    qdelta_ssm_fwd / qdelta_ssm_step / qdelta_ssm_bwd
    qdelta_group_norm_fwd / qdelta_group_norm_bwd

Beside the delta rules, linear attention with a decay for each head, and around a block its RMS
norms with the gate, the scale and the residual sum:

    qdelta_linattn_fwd / qdelta_linattn_step / qdelta_linattn_bwd
    qdelta_block_norm_fwd / qdelta_block_norm_bwd
"""
import contextlib
import ctypes
import math
import os

from . import inputs  # noqa: F401  (seeded workload generators)

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqdelta.so")

QD_F32, QD_BF16 = 0, 1
# bytes of device scratch qdelta_chunk_fwd_noalloc holds per device (QDELTA_NOALLOC_SCRATCH_BYTES)
NOALLOC_SCRATCH_BYTES = 32 << 20
_lib = None
# torch's own current device and stream handle, without the checks around them; set with the library
_get_device = _raw_stream = None


class QDeltaError(RuntimeError):
    pass


def load_library():
    """Load libqdelta.so (built in-tree by ``python -m recurrent_sequence_layers_amd.build``)."""
    global _lib, _get_device, _raw_stream
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise QDeltaError(f"{LIB_PATH} is missing: build it with "
                          "`python -m recurrent_sequence_layers_amd.build` (no CPU fallback exists)")
    lib = ctypes.CDLL(LIB_PATH)
    vp, fp, i, sz = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    lib.qdelta_abi_version.restype = i
    lib.qdelta_abi_version.argtypes = []
    lib.qdelta_status_string.restype = ctypes.c_char_p
    lib.qdelta_status_string.argtypes = [i]
    lib.qdelta_chunk_fwd_workspace_bytes.restype = sz
    lib.qdelta_chunk_fwd_workspace_bytes.argtypes = [i] * 7
    lib.qdelta_chunk_fwd.restype = i
    lib.qdelta_chunk_fwd.argtypes = [vp, vp, vp, fp, fp, fp, fp, vp, fp] + [i] * 7 + [vp, sz, vp]
    lib.qdelta_chunk_fwd_noalloc.restype = i
    lib.qdelta_chunk_fwd_noalloc.argtypes = [vp, vp, vp, fp, fp, fp, fp, vp, fp] + [i] * 7 + [vp]
    lib.qdelta_chunk_fwd_raw.restype = i
    lib.qdelta_chunk_fwd_raw.argtypes = [vp, vp, vp, fp, fp, fp, fp, vp, fp] + [i] * 7 + [vp, sz, vp]
    lib.qdelta_step.restype = i
    lib.qdelta_step.argtypes = [vp, vp, vp, fp, fp, fp, fp, vp] + [i] * 5 + [vp]
    lib.qdelta_step_raw.restype = i
    lib.qdelta_step_raw.argtypes = [vp, vp, vp, fp, fp, fp, fp, vp] + [i] * 5 + [vp]
    lib.qdelta_qed_chunk_fwd.restype = i
    lib.qdelta_qed_chunk_fwd.argtypes = [vp] * 10 + [i] * 7 + [vp]
    lib.qdelta_qed_step.restype = i
    lib.qdelta_qed_step.argtypes = [vp] * 9 + [i] * 5 + [vp]
    lib.qdelta_eda_chunk_fwd_workspace_bytes.restype = sz
    lib.qdelta_eda_chunk_fwd_workspace_bytes.argtypes = [i] * 7
    lib.qdelta_eda_chunk_fwd.restype = i
    lib.qdelta_eda_chunk_fwd.argtypes = [vp] * 7 + [i] * 7 + [vp, sz, vp]
    lib.qdelta_eda_step.restype = i
    lib.qdelta_eda_step.argtypes = [vp] * 6 + [i] * 5 + [vp]
    lib.qdelta_chunk_bwd_workspace_bytes.restype = sz
    lib.qdelta_chunk_bwd_workspace_bytes.argtypes = [i] * 7
    lib.qdelta_chunk_bwd.restype = i
    lib.qdelta_chunk_bwd.argtypes = [vp] * 16 + [i] * 7 + [vp, sz, vp]
    f = ctypes.c_float
    for name, restype, argtypes in (
            ("conv_fwd", i, [vp] * 7 + [i] * 6 + [vp]),
            ("conv_step", i, [vp] * 5 + [i] * 5 + [vp]),
            ("conv_bwd_workspace_bytes", sz, [i] * 5),
            ("conv_bwd", i, [vp] * 11 + [i] * 6 + [vp, sz, vp]),
            ("ssm_fwd_workspace_bytes", sz, [i] * 6),
            ("ssm_fwd", i, [vp] * 12 + [i] * 7 + [vp, sz, vp]),
            ("ssm_step", i, [vp] * 10 + [i] * 6 + [vp]),
            ("ssm_bwd_workspace_bytes", sz, [i] * 6),
            ("ssm_bwd", i, [vp] * 21 + [i] * 7 + [vp, sz, vp]),
            ("group_norm_fwd_workspace_bytes", sz, [i] * 5),
            ("group_norm_fwd", i, [vp] * 6 + [i] * 4 + [f] + [i] * 2 + [vp, sz, vp]),
            ("group_norm_bwd_workspace_bytes", sz, [i] * 5),
            ("group_norm_bwd", i, [vp] * 10 + [i] * 6 + [vp, sz, vp]),
            ("linattn_fwd_workspace_bytes", sz, [i] * 6),
            ("linattn_fwd", i, [vp] * 8 + [i] * 7 + [vp, sz, vp]),
            ("linattn_step", i, [vp] * 6 + [i] * 6 + [vp]),
            ("linattn_bwd_workspace_bytes", sz, [i] * 7),
            ("linattn_bwd", i, [vp] * 13 + [i] * 7 + [vp, sz, vp]),
            ("block_norm_fwd", i, [vp] * 9 + [i] * 2 + [f] + [i] * 2 + [vp]),
            ("block_norm_bwd_workspace_bytes", sz, [i] * 4),
            ("block_norm_bwd", i, [vp] * 15 + [i] * 4 + [vp, sz, vp])):
        fn = getattr(lib, "qdelta_" + name)
        fn.restype, fn.argtypes = restype, argtypes
    import torch
    _get_device, _raw_stream = (getattr(torch._C, n, None) for n in ("_cuda_getDevice", "_cuda_getCurrentRawStream"))
    _lib = lib
    return lib


def qdelta_abi_version() -> int:
    return load_library().qdelta_abi_version()


def qdelta_status_string(status: int) -> str:
    return load_library().qdelta_status_string(int(status)).decode()


def qdelta_chunk_fwd_workspace_bytes(B, T, H, d_k, d_v, C, dtype) -> int:
    return int(load_library().qdelta_chunk_fwd_workspace_bytes(B, T, H, d_k, d_v, C, _dtype_code(dtype)))


def _dtype_code(dt) -> int:
    import torch
    if dt in (QD_F32, QD_BF16):
        return dt
    if dt == torch.float32:
        return QD_F32
    if dt == torch.bfloat16:
        return QD_BF16
    raise QDeltaError(f"unsupported dtype {dt}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _check(t, name, dtype=None, shape=None):
    import torch
    if t is None:
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise QDeltaError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise QDeltaError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise QDeltaError(f"{name} must be {dtype}, got {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise QDeltaError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _launch_stream(stream, device):
    """The stream the kernels are enqueued on: torch's current stream, or the given
    torch.cuda.Stream.  Wrappers allocate their outputs and workspaces while that stream
    is current, so the caching allocator ties those blocks to it: a workspace released on
    return is handed out again only to work ordered after these kernels."""
    import torch
    if stream is None:
        return torch.cuda.current_stream(device)
    if not isinstance(stream, torch.cuda.Stream):
        raise QDeltaError("stream must be a torch.cuda.Stream or None")
    if device.type == "cuda" and stream.device != device:     # its kernels could not reach the tensors
        raise QDeltaError(f"stream must be on {device}, got one on {stream.device}")
    return stream


def _raise(rc, fn):
    if rc != 0:
        raise QDeltaError(f"{fn}: {qdelta_status_string(rc)} (status {rc})")


def qdelta_chunk_fwd(q, k, v, alpha, beta, lam, S0=None, C: int = 64, o=None, S_T=None,
                     want_state: bool = True, stream=None, workspace=None, raw: bool = False):
    """Layer forward, chunkwise WY/UT form.  q, k [B,T,H,d_k], v [B,T,H,d_v] (fp32 or
    bf16, same dtype); alpha, beta, lam [B,T,H] fp32 (alpha None means 1, lam None
    means 0); S0 [B,H,d_v,d_k] fp32 or None.  Returns (o, S_T); S_T is None when
    want_state is False.  S_T may be passed as S0 for an in-place state update.
    workspace: a device tensor of at least qdelta_chunk_fwd_workspace_bytes(...) bytes
    (long sequences over few heads run a segmented schedule that needs one); when None
    and one is needed, it is allocated here.
    raw: q and k unnormalised and alpha, beta, lam given as logits (qdelta_chunk_fwd_raw:
    the layer's normalisation and gate maps run inside the kernel)."""
    import torch
    lib = load_library()
    s = _launch_stream(stream, q.device)
    with torch.cuda.stream(s):
        B, T, H, dk = q.shape
        dv = v.shape[-1]
        dt = q.dtype
        _check(q, "q", dt); _check(k, "k", dt, q.shape); _check(v, "v", dt, (B, T, H, dv))
        for name, g in (("alpha", alpha), ("beta", beta), ("lam", lam)):
            _check(g, name, torch.float32, (B, T, H))
        _check(S0, "S0", torch.float32, (B, H, dv, dk))
        if o is None:
            o = torch.empty((B, T, H, dv), dtype=dt, device=q.device)
        _check(o, "o", dt, (B, T, H, dv))
        if S_T is None and want_state:
            S_T = torch.empty((B, H, dv, dk), dtype=torch.float32, device=q.device)
        _check(S_T, "S_T", torch.float32, (B, H, dv, dk))
        code = _dtype_code(dt)
        ws = lib.qdelta_chunk_fwd_workspace_bytes(B, T, H, dk, dv, C, code)
        if ws and workspace is None:
            workspace = torch.empty(ws, dtype=torch.uint8, device=q.device)
        ws_ptr, ws_bytes = (None, 0) if workspace is None else (_ptr(workspace), workspace.numel() * workspace.element_size())
        fn = lib.qdelta_chunk_fwd_raw if raw else lib.qdelta_chunk_fwd
        rc = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(lam), _ptr(S0),
                _ptr(o), _ptr(S_T), B, T, H, dk, dv, int(C), code, ws_ptr, ws_bytes, ctypes.c_void_p(s.cuda_stream))
        _raise(rc, "qdelta_chunk_fwd_raw" if raw else "qdelta_chunk_fwd")
        return o, S_T


def qdelta_chunk_fwd_noalloc(q, k, v, alpha, beta, lam, S0, o, S_T, C: int = 64, stream=None):
    """qdelta_chunk_fwd for callers that cannot allocate: o and S_T (or None) are supplied
    by the caller and nothing is allocated, here or in the library; the segmented schedule,
    when the sizes call for it, runs in the library's per-device scratch (calls that overlap
    in time on one GPU race on it).  Raises when the sizes need more than
    NOALLOC_SCRATCH_BYTES of it."""
    import torch
    lib = load_library()
    s = _launch_stream(stream, q.device)
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dt = q.dtype
    _check(q, "q", dt); _check(k, "k", dt, q.shape); _check(v, "v", dt, (B, T, H, dv))
    for name, g in (("alpha", alpha), ("beta", beta), ("lam", lam)):
        _check(g, name, torch.float32, (B, T, H))
    _check(S0, "S0", torch.float32, (B, H, dv, dk))
    if o is None:
        raise QDeltaError("qdelta_chunk_fwd_noalloc: o must be supplied (nothing is allocated)")
    _check(o, "o", dt, (B, T, H, dv))
    _check(S_T, "S_T", torch.float32, (B, H, dv, dk))
    rc = lib.qdelta_chunk_fwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(lam), _ptr(S0),
                                      _ptr(o), _ptr(S_T), B, T, H, dk, dv, int(C), _dtype_code(dt),
                                      ctypes.c_void_p(s.cuda_stream))
    _raise(rc, "qdelta_chunk_fwd_noalloc")
    return o, S_T


def qdelta_chunk_bwd_workspace_bytes(B, T, H, d_k, d_v, C, dtype) -> int:
    return int(load_library().qdelta_chunk_bwd_workspace_bytes(B, T, H, d_k, d_v, C, _dtype_code(dtype)))


def qdelta_chunk_bwd(q, k, v, alpha, beta, lam, S0, d_o, dS_T=None, C: int = 64, want_dS0: bool = True,
                     out=None, workspace=None, stream=None):
    """Layer backward: gradients of sum(o * d_o) + sum(S_T * dS_T) for the forward of
    ``qdelta_chunk_fwd`` on the same inputs.  d_o [B,T,H,d_v] in the input dtype; dS_T
    [B,H,d_v,d_k] fp32 or None.  Returns a dict with dq, dk (like q), dv (like v), dbeta,
    and dalpha / dlam (fp32 [B,T,H], None when alpha / lam are None) and dS0 (fp32, None
    unless want_dS0).  ``out`` may supply any of those tensors; ``workspace`` a device
    buffer of at least qdelta_chunk_bwd_workspace_bytes(...) bytes (allocated when None)."""
    import torch
    lib = load_library()
    s = _launch_stream(stream, q.device)
    with torch.cuda.stream(s):
        B, T, H, dk = q.shape
        dv = v.shape[-1]
        dt = q.dtype
        dev = q.device
        _check(q, "q", dt); _check(k, "k", dt, q.shape); _check(v, "v", dt, (B, T, H, dv))
        _check(d_o, "d_o", dt, (B, T, H, dv))
        for name, g in (("alpha", alpha), ("beta", beta), ("lam", lam)):
            _check(g, name, torch.float32, (B, T, H))
        _check(S0, "S0", torch.float32, (B, H, dv, dk))
        _check(dS_T, "dS_T", torch.float32, (B, H, dv, dk))
        out = dict(out or {})
        shapes = dict(dq=((B, T, H, dk), dt), dk=((B, T, H, dk), dt), dv=((B, T, H, dv), dt),
                      dbeta=((B, T, H), torch.float32), dalpha=((B, T, H), torch.float32),
                      dlam=((B, T, H), torch.float32), dS0=((B, H, dv, dk), torch.float32))
        wanted = dict(dq=True, dk=True, dv=True, dbeta=True, dalpha=alpha is not None, dlam=lam is not None,
                      dS0=want_dS0)
        for name, (shape, dtype) in shapes.items():
            if not wanted[name]:
                out[name] = None
                continue
            if out.get(name) is None:
                out[name] = torch.empty(shape, dtype=dtype, device=dev)
            _check(out[name], name, dtype, shape)
        code = _dtype_code(dt)
        ws = lib.qdelta_chunk_bwd_workspace_bytes(B, T, H, dk, dv, C, code)
        if ws and workspace is None:
            workspace = torch.empty(ws, dtype=torch.uint8, device=dev)
        ws_ptr, ws_bytes = (None, 0) if workspace is None else (_ptr(workspace), workspace.numel() * workspace.element_size())
        rc = lib.qdelta_chunk_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(lam), _ptr(S0), _ptr(d_o),
                                  _ptr(dS_T), _ptr(out["dq"]), _ptr(out["dk"]), _ptr(out["dv"]), _ptr(out["dalpha"]),
                                  _ptr(out["dbeta"]), _ptr(out["dlam"]), _ptr(out["dS0"]), B, T, H, dk, dv, int(C), code,
                                  ws_ptr, ws_bytes, ctypes.c_void_p(s.cuda_stream))
        _raise(rc, "qdelta_chunk_bwd")
        return out


def qdelta_qed_chunk_fwd(q, k, v, g, b, w, lam_h, S0=None, C: int = 32, o=None, S_T=None, want_state=True,
                         stream=None):
    """QED / GDN-2 layer forward.  q, k [B,T,H,d_k], v [B,T,H,d_v] (fp32 or bf16); g, b
    [B,T,H,d_k], w [B,T,H,d_v], lam_h [H], S0 [B,H,d_v,d_k] fp32.  Returns (o, S_T)."""
    import torch
    lib = load_library()
    s = _launch_stream(stream, q.device)
    with torch.cuda.stream(s):
        B, T, H, dk = q.shape
        dv = v.shape[-1]
        dt = q.dtype
        _check(q, "q", dt); _check(k, "k", dt, q.shape); _check(v, "v", dt, (B, T, H, dv))
        _check(g, "g", torch.float32, (B, T, H, dk)); _check(b, "b", torch.float32, (B, T, H, dk))
        _check(w, "w", torch.float32, (B, T, H, dv)); _check(lam_h, "lam_h", torch.float32, (H,))
        _check(S0, "S0", torch.float32, (B, H, dv, dk))
        if o is None:
            o = torch.empty((B, T, H, dv), dtype=dt, device=q.device)
        _check(o, "o", dt, (B, T, H, dv))
        if S_T is None and want_state:
            S_T = torch.empty((B, H, dv, dk), dtype=torch.float32, device=q.device)
        _check(S_T, "S_T", torch.float32, (B, H, dv, dk))
        rc = lib.qdelta_qed_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(w), _ptr(lam_h), _ptr(S0),
                                      _ptr(o), _ptr(S_T), B, T, H, dk, dv, int(C), _dtype_code(dt), ctypes.c_void_p(s.cuda_stream))
        _raise(rc, "qdelta_qed_chunk_fwd")
        return o, S_T


def qdelta_qed_step(q, k, v, g, b, w, lam_h, S, o=None, stream=None):
    """One QED / GDN-2 decode step.  q, k [N,H,d_k], v [N,H,d_v]; g, b [N,H,d_k], w [N,H,d_v],
    lam_h [H] fp32; S [N,H,d_v,d_k] fp32 updated in place.  Returns o [N,H,d_v]."""
    import torch
    lib = load_library()
    s = _launch_stream(stream, q.device)
    with torch.cuda.stream(s):
        N, H, dk = q.shape
        dv = v.shape[-1]
        dt = q.dtype
        _check(q, "q", dt); _check(k, "k", dt, q.shape); _check(v, "v", dt, (N, H, dv))
        _check(g, "g", torch.float32, (N, H, dk)); _check(b, "b", torch.float32, (N, H, dk))
        _check(w, "w", torch.float32, (N, H, dv)); _check(lam_h, "lam_h", torch.float32, (H,))
        _check(S, "S", torch.float32, (N, H, dv, dk))
        if o is None:
            o = torch.empty((N, H, dv), dtype=dt, device=q.device)
        _check(o, "o", dt, (N, H, dv))
        rc = lib.qdelta_qed_step(_ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(b), _ptr(w), _ptr(lam_h), _ptr(S), _ptr(o),
                                 N, H, dk, dv, _dtype_code(dt), ctypes.c_void_p(s.cuda_stream))
        _raise(rc, "qdelta_qed_step")
        return o


def qdelta_eda_chunk_fwd(q, k, v, e, S0=None, C: int = 64, o=None, S_T=None, want_state=True, workspace=None,
                         stream=None):
    """Erase-then-Delta layer forward.  q, k, e [B,T,H,d_k] (unit-norm), v [B,T,H,d_v], same
    dtype; S0 [B,H,d_v,d_k] fp32.  Returns (o, S_T).  workspace: a device buffer of at least
    qdelta_eda_chunk_fwd_workspace_bytes(...) bytes (allocated here when None)."""
    import torch
    lib = load_library()
    s = _launch_stream(stream, q.device)
    with torch.cuda.stream(s):
        B, T, H, dk = q.shape
        dv = v.shape[-1]
        dt = q.dtype
        _check(q, "q", dt); _check(k, "k", dt, q.shape); _check(e, "e", dt, q.shape); _check(v, "v", dt, (B, T, H, dv))
        _check(S0, "S0", torch.float32, (B, H, dv, dk))
        if o is None:
            o = torch.empty((B, T, H, dv), dtype=dt, device=q.device)
        _check(o, "o", dt, (B, T, H, dv))
        if S_T is None and want_state:
            S_T = torch.empty((B, H, dv, dk), dtype=torch.float32, device=q.device)
        _check(S_T, "S_T", torch.float32, (B, H, dv, dk))
        code = _dtype_code(dt)
        ws = lib.qdelta_eda_chunk_fwd_workspace_bytes(B, T, H, dk, dv, C, code)
        if ws and workspace is None:
            workspace = torch.empty(ws, dtype=torch.uint8, device=q.device)
        ws_ptr, ws_bytes = (None, 0) if workspace is None else (_ptr(workspace), workspace.numel() * workspace.element_size())
        rc = lib.qdelta_eda_chunk_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(e), _ptr(S0), _ptr(o), _ptr(S_T), B, T, H, dk, dv,
                                      int(C), code, ws_ptr, ws_bytes, ctypes.c_void_p(s.cuda_stream))
        _raise(rc, "qdelta_eda_chunk_fwd")
        return o, S_T


def qdelta_eda_chunk_fwd_workspace_bytes(B, T, H, d_k, d_v, C, dtype) -> int:
    return int(load_library().qdelta_eda_chunk_fwd_workspace_bytes(B, T, H, d_k, d_v, C, _dtype_code(dtype)))


def qdelta_eda_step(q, k, v, e, S, o=None, stream=None):
    """One Erase-then-Delta decode step.  q, k, e [N,H,d_k], v [N,H,d_v]; S [N,H,d_v,d_k] fp32,
    updated in place.  Returns o [N,H,d_v]."""
    import torch
    lib = load_library()
    s = _launch_stream(stream, q.device)
    with torch.cuda.stream(s):
        N, H, dk = q.shape
        dv = v.shape[-1]
        dt = q.dtype
        _check(q, "q", dt); _check(k, "k", dt, q.shape); _check(e, "e", dt, q.shape); _check(v, "v", dt, (N, H, dv))
        _check(S, "S", torch.float32, (N, H, dv, dk))
        if o is None:
            o = torch.empty((N, H, dv), dtype=dt, device=q.device)
        _check(o, "o", dt, (N, H, dv))
        rc = lib.qdelta_eda_step(_ptr(q), _ptr(k), _ptr(v), _ptr(e), _ptr(S), _ptr(o), N, H, dk, dv, _dtype_code(dt),
                                 ctypes.c_void_p(s.cuda_stream))
        _raise(rc, "qdelta_eda_step")
        return o


def qdelta_step(q, k, v, alpha, beta, lam, S, o=None, stream=None, raw: bool = False):
    """One decode step for N sequences x H heads.  q, k [N,H,d_k], v [N,H,d_v];
    alpha, beta, lam [N,H] fp32 (alpha None means 1, lam None means 0);
    S [N,H,d_v,d_k] fp32, updated in place.  Returns o [N,H,d_v].
    raw: q and k unnormalised and the gates as logits (qdelta_step_raw)."""
    import torch
    lib = load_library()
    s = _launch_stream(stream, q.device)
    with torch.cuda.stream(s):
        N, H, dk = q.shape
        dv = v.shape[-1]
        dt = q.dtype
        _check(q, "q", dt); _check(k, "k", dt, q.shape); _check(v, "v", dt, (N, H, dv))
        for name, g in (("alpha", alpha), ("beta", beta), ("lam", lam)):
            _check(g, name, torch.float32, (N, H))
        _check(S, "S", torch.float32, (N, H, dv, dk))
        if o is None:
            o = torch.empty((N, H, dv), dtype=dt, device=q.device)
        _check(o, "o", dt, (N, H, dv))
        fn = lib.qdelta_step_raw if raw else lib.qdelta_step
        rc = fn(_ptr(q), _ptr(k), _ptr(v), _ptr(alpha), _ptr(beta), _ptr(lam), _ptr(S), _ptr(o),
                N, H, dk, dv, _dtype_code(dt), ctypes.c_void_p(s.cuda_stream))
        _raise(rc, "qdelta_step_raw" if raw else "qdelta_step")
        return o


# ---------------------------------------------------------------- around the recurrence
def _int_sizes(sizes):
    """Refuses what the library's 32-bit sizes cannot hold: ctypes would pass the low 32 bits on."""
    if max(sizes) > 0x7fffffff:
        raise QDeltaError(f"sizes must be below 2**31, got {tuple(sizes)}")
    return sizes


def _shape(t, name, dims):
    """Shape of a device tensor with `dims` dimensions."""
    if not getattr(t, "is_cuda", False):
        raise QDeltaError(f"{name} must be a device tensor")
    shape = t.shape
    if len(shape) != dims:
        raise QDeltaError(f"{name} must have {dims} dimensions, got {len(shape)}")
    return _int_sizes(shape)


def _check_all(device, checks):
    """_check for each (tensor, name, dtype, shape), and that every tensor is on `device`.  A
    decode step is a few microseconds on the GPU, so what is right costs four comparisons."""
    index = device.index
    for t, name, dtype, shape in checks:
        if t is None:
            continue
        try:
            if t.dtype is dtype and t.get_device() == index and (shape is None or t.shape == shape) and t.is_contiguous():
                continue
        except AttributeError:
            pass
        _check(t, name, dtype, shape)
        if t.device != device:
            raise QDeltaError(f"{name} must be on {device}, got {t.device}")


_NO_CONTEXT = contextlib.nullcontext()


def _enter(stream, device):
    """(context, stream handle) for a call's allocations and launches: `device` and the stream
    current, and no context at all where they are already."""
    import torch
    if stream is None and device.index == (_get_device or torch.cuda.current_device)():
        # the handle without a Stream object around it
        return _NO_CONTEXT, _raw_stream(device.index) if _raw_stream else torch.cuda.current_stream(device).cuda_stream
    s = _launch_stream(stream, device)
    return torch.cuda.stream(s), s.cuda_stream


def _result(t, name, like, device, empty=True):
    """The caller's t, checked, or a new tensor.  `like` is a tensor of the same shape and type, or
    (shape, dtype).  Not empty: new ones are zeros, where a kernel leaves rows of padding unwritten."""
    import torch
    tensor = isinstance(like, torch.Tensor)
    if t is not None:
        shape, dtype = (like.shape, like.dtype) if tensor else like
        _check_all(device, [(t, name, dtype, shape)])
        return t
    if tensor:
        return torch.empty_like(like) if empty else torch.zeros_like(like)
    return torch.empty(like[0], dtype=like[1], device=device)


def _results(out, specs, device):
    """The tensors that specs {name: like, or None where not wanted} names, from out or new."""
    got = dict(out or {})
    for name, like in specs.items():
        got[name] = None if like is None else _result(got.get(name), name, like, device)
    return got


def _workspace(workspace, need, device):
    """(address, bytes) of the caller's workspace, or of a new one, and the tensor itself."""
    import torch
    if workspace is None:
        if not need:
            return None, 0, None
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        return workspace.data_ptr(), need, workspace
    _check(workspace, "workspace")
    _check_all(device, [(workspace, "workspace", workspace.dtype, None)])
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _at(t):
    return None if t is None else t.data_ptr()


def qdelta_conv_fwd(x, w, bias=None, S0=None, silu: bool = True, lens=None, y=None, S_T=None,
                    want_state: bool = True, stream=None):
    """Short causal depthwise convolution over x [B,T,D] (fp32 or bf16), y = silu(pre) or pre.
    w [D,W] and bias [D] fp32, W in 2..4; S0 [B,W-1,D] like x, the inputs before the first
    token (None: zeros).  lens [B] int32: the tokens of each right-padded sequence; rows of y
    past them are left as they were (zeros in a y allocated here).  Returns (y, S_T); S_T is None when want_state is False,
    and may be passed as S0."""
    import torch
    lib = load_library()
    B, T, D = _shape(x, "x", 3)
    W = _shape(w, "w", 2)[1]
    context, handle = _enter(stream, x.device)
    with context:
        dt, dev, f32 = x.dtype, x.device, torch.float32
        code = _dtype_code(dt)
        state = ((B, W - 1, D), dt)
        _check_all(dev, [(x, "x", dt, None), (w, "w", f32, (D, W)), (bias, "bias", f32, (D,)),
                         (S0, "S0", dt, state[0]), (lens, "lens", torch.int32, (B,))])
        y = _result(y, "y", x, dev, empty=lens is None)
        if want_state or S_T is not None:
            S_T = _result(S_T, "S_T", state if S0 is None else S0, dev)
        rc = lib.qdelta_conv_fwd(_at(x), _at(w), _at(bias), _at(S0), _at(lens), _at(y), _at(S_T), B, T, D, W,
                                 int(silu), code, handle)
        _raise(rc, "qdelta_conv_fwd")
        return y, S_T


def qdelta_conv_step(x, w, bias, S, silu: bool = True, y=None, stream=None):
    """One token of the short convolution for N sequences: x [N,D]; S [N,W-1,D] like x, the
    last inputs, shifted in place.  Returns y [N,D]."""
    import torch
    lib = load_library()
    N, D = _shape(x, "x", 2)
    W = _shape(w, "w", 2)[1]
    context, handle = _enter(stream, x.device)
    with context:
        dt, dev, f32 = x.dtype, x.device, torch.float32
        code = _dtype_code(dt)
        _check_all(dev, [(x, "x", dt, None), (w, "w", f32, (D, W)), (bias, "bias", f32, (D,)), (S, "S", dt, (N, W - 1, D))])
        y = _result(y, "y", x, dev)
        rc = lib.qdelta_conv_step(_at(x), _at(w), _at(bias), _at(S), _at(y), N, D, W, int(silu), code, handle)
        _raise(rc, "qdelta_conv_step")
        return y


def qdelta_conv_bwd_workspace_bytes(B, T, D, W, dtype) -> int:
    return int(load_library().qdelta_conv_bwd_workspace_bytes(*_int_sizes((B, T, D, W)), _dtype_code(dtype)))


def qdelta_conv_bwd(x, w, bias, S0, dy, dS_T=None, silu: bool = True, want_dS0: bool = True, lens=None, out=None,
                    workspace=None, stream=None):
    """Gradients of sum(y * dy) + sum(S_T * dS_T) for qdelta_conv_fwd on the same inputs.  With
    lens, rows past a sequence's end are not read, dy's neither, and their dx is zero.  Returns a dict with dx, dw, dbias (None without bias) and dS0 (None unless want_dS0; also
    given when S0 is None).  ``out`` may supply any of them; ``workspace`` a device buffer of
    at least qdelta_conv_bwd_workspace_bytes(...) bytes (allocated when None)."""
    import torch
    lib = load_library()
    B, T, D = _shape(x, "x", 3)
    W = _shape(w, "w", 2)[1]
    context, handle = _enter(stream, x.device)
    with context:
        dt, dev, f32 = x.dtype, x.device, torch.float32
        code = _dtype_code(dt)
        _check_all(dev, [(x, "x", dt, None), (w, "w", f32, (D, W)), (bias, "bias", f32, (D,)),
                         (S0, "S0", dt, (B, W - 1, D)), (lens, "lens", torch.int32, (B,)), (dy, "dy", dt, (B, T, D)),
                         (dS_T, "dS_T", dt, (B, W - 1, D))])
        dS0 = S0 if S0 is not None else ((B, W - 1, D), dt)
        out = _results(out, dict(dx=x, dw=w, dbias=bias, dS0=dS0 if want_dS0 else None), dev)
        p, n, workspace = _workspace(workspace, lib.qdelta_conv_bwd_workspace_bytes(B, T, D, W, code), dev)
        rc = lib.qdelta_conv_bwd(_at(x), _at(w), _at(bias), _at(S0), _at(lens), _at(dy), _at(dS_T),
                                 _at(out["dx"]), _at(out["dw"]), _at(out["dbias"]), _at(out["dS0"]), B, T, D, W,
                                 int(silu), code, p, n, handle)
        _raise(rc, "qdelta_conv_bwd")
        return out


def _ssm_inputs(u, dt, A, Bm, Cm, D, z, dt_bias, token_dims):
    """Sizes (tokens.., channels, G, N) and the checks of the inputs that a token has."""
    import torch
    shape = tuple(_shape(u, "u", token_dims + 1))
    G, N = _shape(Bm, "Bm", token_dims + 2)[token_dims:]
    f32, e, ch = torch.float32, u.dtype, shape[-1]
    if G < 1 or ch % G:
        raise QDeltaError(f"the {ch} channels of u must divide into the {G} groups of Bm")
    bc = shape[:-1] + (G, N)
    return shape + (G, N), [(u, "u", e, None), (dt, "dt", e, shape), (A, "A", f32, (ch, N)), (Bm, "Bm", e, bc),
                            (Cm, "Cm", e, bc), (D, "D", f32, (ch,)), (z, "z", e, shape), (dt_bias, "dt_bias", f32, (ch,))]


def qdelta_ssm_fwd_workspace_bytes(B, T, D, G, N, dtype) -> int:
    return int(load_library().qdelta_ssm_fwd_workspace_bytes(*_int_sizes((B, T, D, G, N)), _dtype_code(dtype)))


def qdelta_ssm_fwd(u, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, S0=None, softplus: bool = True, lens=None, o=None,
                   S_T=None, want_state: bool = True, workspace=None, stream=None):
    """Selective state space scan.  u, dt, z [B,T,D] and Bm, Cm [B,T,G,N] (fp32 or bf16, same
    dtype); A [D,N], D [D], dt_bias [D], S0 [B,D,N] fp32, all but A optional; N in 16, 32, 64.
    softplus: delta = softplus(dt + dt_bias), else dt + dt_bias.  lens [B] int32: the tokens of
    each right-padded sequence; rows of o past them are left as they were (zeros in an o
    allocated here).  Returns (o, S_T);
    S_T is None when want_state is False, and may be passed as S0.  workspace: at least
    qdelta_ssm_fwd_workspace_bytes(...) bytes, allocated here when None and needed."""
    import torch
    lib = load_library()
    (B, T, ch, G, N), checks = _ssm_inputs(u, dt, A, Bm, Cm, D, z, dt_bias, 2)
    context, handle = _enter(stream, u.device)
    with context:
        dev, f32, code = u.device, torch.float32, _dtype_code(u.dtype)
        state = ((B, ch, N), f32)
        _check_all(dev, checks + [(S0, "S0", f32, state[0]), (lens, "lens", torch.int32, (B,))])
        o = _result(o, "o", u, dev, empty=lens is None)
        if want_state or S_T is not None:
            S_T = _result(S_T, "S_T", state if S0 is None else S0, dev)
        p, n, workspace = _workspace(workspace, lib.qdelta_ssm_fwd_workspace_bytes(B, T, ch, G, N, code), dev)
        rc = lib.qdelta_ssm_fwd(_at(u), _at(dt), _at(A), _at(Bm), _at(Cm), _at(D), _at(z), _at(dt_bias), _at(S0),
                                _at(lens), _at(o), _at(S_T), B, T, ch, G, N, int(softplus), code, p, n, handle)
        _raise(rc, "qdelta_ssm_fwd")
        return o, S_T


def qdelta_ssm_step(u, dt, A, Bm, Cm, D, z, dt_bias, S, softplus: bool = True, o=None, stream=None):
    """One token of the selective scan for N sequences: u, dt, z [N,D], Bm, Cm [N,G,states];
    S [N,D,states] fp32, updated in place.  Returns o [N,D]."""
    import torch
    lib = load_library()
    (n_seq, ch, G, N), checks = _ssm_inputs(u, dt, A, Bm, Cm, D, z, dt_bias, 1)
    context, handle = _enter(stream, u.device)
    with context:
        dev, code = u.device, _dtype_code(u.dtype)
        _check_all(dev, checks + [(S, "S", torch.float32, (n_seq, ch, N))])
        o = _result(o, "o", u, dev)
        rc = lib.qdelta_ssm_step(_at(u), _at(dt), _at(A), _at(Bm), _at(Cm), _at(D), _at(z), _at(dt_bias), _at(S),
                                 _at(o), n_seq, ch, G, N, int(softplus), code, handle)
        _raise(rc, "qdelta_ssm_step")
        return o


def qdelta_ssm_bwd_workspace_bytes(B, T, D, G, N, dtype) -> int:
    return int(load_library().qdelta_ssm_bwd_workspace_bytes(*_int_sizes((B, T, D, G, N)), _dtype_code(dtype)))


def qdelta_ssm_bwd(u, dt, A, Bm, Cm, D, z, dt_bias, S0, d_o, dS_T=None, softplus: bool = True, want_dS0: bool = True,
                   lens=None, out=None, workspace=None, stream=None):
    """Gradients of sum(o * d_o) + sum(S_T * dS_T) for qdelta_ssm_fwd on the same inputs.  With
    lens, rows past a sequence's end are not read, d_o's neither, and their gradients are zero.
    Returns a dict with du, ddt, dB, dC (like their inputs), dA, and, None where the input is
    None, dD, dz, ddt_bias, and dS0 (None unless want_dS0; also given when S0 is None).
    ``out`` may supply any of them; ``workspace`` a device buffer of at least
    qdelta_ssm_bwd_workspace_bytes(...) bytes (allocated when None)."""
    import torch
    lib = load_library()
    (B, T, ch, G, N), checks = _ssm_inputs(u, dt, A, Bm, Cm, D, z, dt_bias, 2)
    context, handle = _enter(stream, u.device)
    with context:
        dev, f32, e, code = u.device, torch.float32, u.dtype, _dtype_code(u.dtype)
        _check_all(dev, checks + [(S0, "S0", f32, (B, ch, N)), (lens, "lens", torch.int32, (B,)),
                                  (d_o, "d_o", e, (B, T, ch)), (dS_T, "dS_T", f32, (B, ch, N))])
        dS0 = S0 if S0 is not None else ((B, ch, N), f32)
        out = _results(out, dict(du=u, ddt=dt, dA=A, dB=Bm, dC=Cm, dD=D, dz=z, ddt_bias=dt_bias,
                                 dS0=dS0 if want_dS0 else None), dev)
        if not ch:
            for name in ("dB", "dC"):
                out[name].zero_()                      # sums over no channels: no kernel writes them
        p, n, workspace = _workspace(workspace, lib.qdelta_ssm_bwd_workspace_bytes(B, T, ch, G, N, code), dev)
        rc = lib.qdelta_ssm_bwd(_at(u), _at(dt), _at(A), _at(Bm), _at(Cm), _at(D), _at(z), _at(dt_bias), _at(S0),
                                _at(lens), _at(d_o), _at(dS_T), _at(out["du"]), _at(out["ddt"]), _at(out["dA"]),
                                _at(out["dB"]), _at(out["dC"]), _at(out["dD"]), _at(out["dz"]), _at(out["ddt_bias"]),
                                _at(out["dS0"]), B, T, ch, G, N, int(softplus), code, p, n, handle)
        _raise(rc, "qdelta_ssm_bwd")
        return out


def _norm_sizes(x, groups):
    """(samples, positions, channels) of x [N, .., C]: the dimensions between are the positions."""
    import torch
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise QDeltaError("x must be a device tensor")
    if x.dim() < 2:
        raise QDeltaError("x must have at least 2 dimensions")
    n, c = x.shape[0], x.shape[-1]
    length = 1
    for d in x.shape[1:-1]:
        length *= d
    if groups < 1 or c % groups:
        raise QDeltaError(f"the {c} channels of x must divide into {groups} groups")
    return _int_sizes((n, length, c))


def qdelta_group_norm_fwd_workspace_bytes(N, L, C, G, dtype) -> int:
    return int(load_library().qdelta_group_norm_fwd_workspace_bytes(*_int_sizes((N, L, C, G)), _dtype_code(dtype)))


def qdelta_group_norm_fwd(x, groups: int, weight=None, bias=None, gate=None, silu: bool = False, eps: float = 1e-5,
                          y=None, stats=None, want_stats: bool = True, workspace=None, stream=None):
    """Group norm of x [N,..,C] (fp32 or bf16), channels last: statistics per sample and group
    over the dimensions between and C / groups channels; weight, bias [C] fp32 (None: 1, 0).
    silu applies SiLU to the normed value; gate, like x, multiplies it by silu(gate).  The
    output norm of a layer's o [B,T,H,d] per token and head is
    ``qdelta_group_norm_fwd(o.view(B * T, H * d), H, ...)``.  Returns (y, stats), stats
    [N,groups,2] the mean and 1/std the backward needs (None when want_stats is False; zeros for
    groups without elements)."""
    import torch
    lib = load_library()
    N, L, C = _norm_sizes(x, groups)
    context, handle = _enter(stream, x.device)
    with context:
        dt, dev, f32, code = x.dtype, x.device, torch.float32, _dtype_code(x.dtype)
        _check_all(dev, [(x, "x", dt, None), (weight, "weight", f32, (C,)), (bias, "bias", f32, (C,)),
                         (gate, "gate", dt, x.shape)])
        y = _result(y, "y", x, dev)
        if want_stats or stats is not None:
            stats = _result(stats, "stats", ((N, groups, 2), f32), dev)
        if stats is not None and not L * C:
            stats.zero_()                              # no elements: no kernel writes them
        p, n, workspace = _workspace(workspace, lib.qdelta_group_norm_fwd_workspace_bytes(N, L, C, groups, code), dev)
        rc = lib.qdelta_group_norm_fwd(_at(x), _at(weight), _at(bias), _at(gate), _at(y), _at(stats), N, L, C, groups,
                                       float(eps), int(silu), code, p, n, handle)
        _raise(rc, "qdelta_group_norm_fwd")
        return y, stats


def qdelta_group_norm_bwd_workspace_bytes(N, L, C, G, dtype) -> int:
    return int(load_library().qdelta_group_norm_bwd_workspace_bytes(*_int_sizes((N, L, C, G)), _dtype_code(dtype)))


def qdelta_group_norm_bwd(x, groups: int, weight, bias, gate, stats, dy, silu: bool = False, out=None, workspace=None,
                          stream=None):
    """Gradients of sum(y * dy) for qdelta_group_norm_fwd on the same inputs, whose stats are
    given.  Returns a dict with dx and, None where the input is None, dweight, dbias, dgate.
    ``out`` may supply any of them; ``workspace`` a device buffer of at least
    qdelta_group_norm_bwd_workspace_bytes(...) bytes (allocated when None)."""
    import torch
    lib = load_library()
    N, L, C = _norm_sizes(x, groups)
    context, handle = _enter(stream, x.device)
    with context:
        dt, dev, f32, code = x.dtype, x.device, torch.float32, _dtype_code(x.dtype)
        if stats is None:
            raise QDeltaError("stats must be the forward's")
        _check_all(dev, [(x, "x", dt, None), (weight, "weight", f32, (C,)), (bias, "bias", f32, (C,)),
                         (gate, "gate", dt, x.shape), (stats, "stats", f32, (N, groups, 2)), (dy, "dy", dt, x.shape)])
        out = _results(out, dict(dx=x, dweight=weight, dbias=bias, dgate=gate), dev)
        p, n, workspace = _workspace(workspace, lib.qdelta_group_norm_bwd_workspace_bytes(N, L, C, groups, code), dev)
        rc = lib.qdelta_group_norm_bwd(_at(x), _at(weight), _at(bias), _at(gate), _at(stats), _at(dy), _at(out["dx"]),
                                       _at(out["dweight"]), _at(out["dbias"]), _at(out["dgate"]), N, L, C, groups,
                                       int(silu), code, p, n, handle)
        _raise(rc, "qdelta_group_norm_bwd")
        return out


# ---------------------------------------------------------------- linear attention with a decay for each head
def _linattn_inputs(q, k, v, g, token_dims):
    """Sizes (tokens.., heads, d_k, d_v), whether g is per head, and the checks of what a token has."""
    import torch
    shape, value = _shape(q, "q", token_dims + 2), _shape(v, "v", token_dims + 2)
    dt, head = q.dtype, shape[:-1]
    per_head = g is not None and len(getattr(g, "shape", ())) == 1
    return (*shape, value[-1]), per_head, [(q, "q", dt, None), (k, "k", dt, shape),
                                           (v, "v", dt, value if value[:-1] == head else (*head, value[-1])),
                                           (g, "g", torch.float32, head[-1:] if per_head else head)]


def qdelta_linattn_fwd_workspace_bytes(B, T, H, d_k, d_v, dtype) -> int:
    return int(load_library().qdelta_linattn_fwd_workspace_bytes(*_int_sizes((B, T, H, d_k, d_v)), _dtype_code(dtype)))


def qdelta_linattn_fwd(q, k, v, g=None, S0=None, lens=None, o=None, S_T=None, want_state: bool = True, workspace=None,
                       stream=None):
    """Linear attention with a decay for each head, S_t = exp(g_t) S_{t-1} + v_t k_t^T, o_t = S_t q_t.
    q, k [B,T,H,d_k], v [B,T,H,d_v] (fp32 or bf16, same dtype; d_k, d_v in 64, 128); g the log
    decays, fp32 [B,T,H], or [H] for every token alike, or None (no decay); S0 [B,H,d_v,d_k] fp32 or
    None.  lens [B] int32: the tokens of each right-padded sequence; rows of o past them are left as
    they were (zeros in an o allocated here).  Returns (o, S_T); S_T is None when want_state is
    False (in bf16 the last bits of o depend on that), and may be passed as S0.  workspace: at least qdelta_linattn_fwd_workspace_bytes(...)
    bytes, allocated here when None and needed."""
    import torch
    lib = load_library()
    (B, T, H, d_k, d_v), per_head, checks = _linattn_inputs(q, k, v, g, 2)
    context, handle = _enter(stream, q.device)
    with context:
        dev, f32, code = q.device, torch.float32, _dtype_code(q.dtype)
        state = ((B, H, d_v, d_k), f32)
        _check_all(dev, checks + [(S0, "S0", f32, state[0]), (lens, "lens", torch.int32, (B,))])
        o = _result(o, "o", v, dev, empty=lens is None)
        if want_state or S_T is not None:
            S_T = _result(S_T, "S_T", state if S0 is None else S0, dev)
        p, n, workspace = _workspace(workspace, lib.qdelta_linattn_fwd_workspace_bytes(B, T, H, d_k, d_v, code), dev)
        rc = lib.qdelta_linattn_fwd(_at(q), _at(k), _at(v), _at(g), _at(S0), _at(lens), _at(o), _at(S_T), B, T, H, d_k, d_v,
                                    int(per_head), code, p, n, handle)
        _raise(rc, "qdelta_linattn_fwd")
        return o, S_T


def qdelta_linattn_step(q, k, v, g, S, o=None, stream=None):
    """One token of linear attention for N sequences x H heads: q, k [N,H,d_k], v [N,H,d_v]; g fp32
    [N,H], or [H], or None; S [N,H,d_v,d_k] fp32, updated in place.  Returns o [N,H,d_v]."""
    import torch
    lib = load_library()
    (N, H, d_k, d_v), per_head, checks = _linattn_inputs(q, k, v, g, 1)
    context, handle = _enter(stream, q.device)
    with context:
        dev, code = q.device, _dtype_code(q.dtype)
        _check_all(dev, checks + [(S, "S", torch.float32, (N, H, d_v, d_k))])
        o = _result(o, "o", v, dev)
        rc = lib.qdelta_linattn_step(_at(q), _at(k), _at(v), _at(g), _at(S), _at(o), N, H, d_k, d_v, int(per_head), code, handle)
        _raise(rc, "qdelta_linattn_step")
        return o


def qdelta_linattn_bwd_workspace_bytes(B, T, H, d_k, d_v, want_dg, dtype) -> int:
    return int(load_library().qdelta_linattn_bwd_workspace_bytes(*_int_sizes((B, T, H, d_k, d_v)), int(want_dg),
                                                                 _dtype_code(dtype)))


def qdelta_linattn_bwd(q, k, v, g, S0, d_o, dS_T=None, want_dS0: bool = True, want_dg: bool = True, lens=None, out=None,
                       workspace=None, stream=None):
    """Gradients of sum(o * d_o) + sum(S_T * dS_T) for qdelta_linattn_fwd on the same inputs.  With
    lens, rows past a sequence's end are not read, d_o's neither, and their gradients are zero.
    Returns a dict with dq, dk, dv (like their inputs), dg (like g, fp32; for a g of [H] summed over
    tokens and sequences; None without g or unless want_dg; zero where g is -inf, elsewhere as exact
    as the terms around the token are, not as itself) and dS0 (None unless want_dS0; also given when
    S0 is None).  In bf16 the last bits of dq, dk and dv depend on want_dg and want_dS0.  ``out`` may supply any of them; ``workspace`` a device buffer of at
    least qdelta_linattn_bwd_workspace_bytes(...) bytes (allocated when None)."""
    import torch
    lib = load_library()
    (B, T, H, d_k, d_v), per_head, checks = _linattn_inputs(q, k, v, g, 2)
    context, handle = _enter(stream, q.device)
    with context:
        dev, f32, dt, code = q.device, torch.float32, q.dtype, _dtype_code(q.dtype)
        state = (B, H, d_v, d_k)
        if d_o is None:
            raise QDeltaError("d_o must be given")
        _check_all(dev, checks + [(S0, "S0", f32, state), (lens, "lens", torch.int32, (B,)), (d_o, "d_o", dt, v.shape),
                                  (dS_T, "dS_T", f32, state)])
        dS0 = S0 if S0 is not None else (state, f32)
        out = _results(out, dict(dq=q, dk=k, dv=v, dg=g if want_dg else None, dS0=dS0 if want_dS0 else None), dev)
        need = lib.qdelta_linattn_bwd_workspace_bytes(B, T, H, d_k, d_v, int(out["dg"] is not None), code)
        p, n, workspace = _workspace(workspace, need, dev)
        rc = lib.qdelta_linattn_bwd(_at(q), _at(k), _at(v), _at(g), _at(S0), _at(lens), _at(d_o), _at(dS_T), _at(out["dq"]),
                                    _at(out["dk"]), _at(out["dv"]), _at(out["dg"]), _at(out["dS0"]), B, T, H, d_k, d_v,
                                    int(per_head), code, p, n, handle)
        _raise(rc, "qdelta_linattn_bwd")
        return out


# ---------------------------------------------------------------- norms around a block
_GATE_ACTS = {"linear": 0, "sigmoid": 1, "silu": 2}


def _block_norm_sizes(y, act):
    """(rows, channels) of y [..,C] and the gate's code."""
    if not getattr(y, "is_cuda", False):
        raise QDeltaError("y must be a device tensor")
    shape = y.shape
    if not shape:
        raise QDeltaError("y must have at least 1 dimension")
    if act not in _GATE_ACTS:
        raise QDeltaError(f"act must be one of {', '.join(_GATE_ACTS)}, got {act!r}")
    return *_int_sizes((math.prod(shape[:-1]), shape[-1])), _GATE_ACTS[act]


def qdelta_block_norm_fwd(y, x=None, post=None, gate=None, scale=None, pre=None, act: str = "silu", eps: float = 1e-5, h=None,
                          n=None, stats=None, want_stats: bool = True, stream=None):
    """RMS norms after and before a block with its gate, scale and residual sum, over the last
    dimension: f = rms(y) * post (y itself when post is None), h = x + scale * act(gate) * f, n =
    rms(h) * pre of h as stored.  y, x, gate [..,C] (fp32 or bf16, same dtype), post, scale, pre [C]
    fp32; all but y optional.  act: "silu", "sigmoid" or "linear" (the gate itself).  The gated RMS
    norm of a layer's o [B,T,H,d] per head is ``qdelta_block_norm_fwd(o, post=weight, gate=z)``.
    Returns (h, n, stats): n is None without pre; stats [rows,2] are the 1/rms of both norms, zero
    for one that is not taken, which the backward needs (None when want_stats is False)."""
    import torch
    lib = load_library()
    N, C, code_act = _block_norm_sizes(y, act)
    context, handle = _enter(stream, y.device)
    with context:
        dt, dev, f32, code = y.dtype, y.device, torch.float32, _dtype_code(y.dtype)
        rows, channels = y.shape, (C,)
        _check_all(dev, [(y, "y", dt, None), (x, "x", dt, rows), (gate, "gate", dt, rows), (post, "post", f32, channels),
                         (scale, "scale", f32, channels), (pre, "pre", f32, channels)])
        h = _result(h, "h", y, dev)
        if pre is not None:
            n = _result(n, "n", y, dev)
        elif n is not None:
            raise QDeltaError("n is only written with pre")
        if want_stats or stats is not None:
            stats = _result(stats, "stats", ((N, 2), f32), dev)
        if stats is not None and not C:
            stats.zero_()                              # no elements: no kernel writes them
        rc = lib.qdelta_block_norm_fwd(_at(y), _at(x), _at(post), _at(gate), _at(scale), _at(pre), _at(h), _at(n), _at(stats),
                                       N, C, float(eps), code_act, code, handle)
        _raise(rc, "qdelta_block_norm_fwd")
        return h, n, stats


def qdelta_block_norm_bwd_workspace_bytes(N, C, want_sums, dtype) -> int:
    return int(load_library().qdelta_block_norm_bwd_workspace_bytes(*_int_sizes((N, C)), int(want_sums), _dtype_code(dtype)))


def qdelta_block_norm_bwd(y, h, post, gate, scale, pre, stats, dh, dn=None, act: str = "silu", want_dx: bool = True, out=None,
                          workspace=None, stream=None):
    """Gradients of sum(h * dh) + sum(n * dn) for qdelta_block_norm_fwd on the same inputs, whose h
    (needed with dn) and stats (needed with dn or post) are given; either of dh and dn may be None.
    Returns a dict with dx (None unless want_dx), dy, and, None where the input is None, dgate,
    dpost, dscale, dpre.  ``out`` may supply any of them; ``workspace`` a device buffer of at least
    qdelta_block_norm_bwd_workspace_bytes(...) bytes (allocated when None)."""
    import torch
    lib = load_library()
    N, C, code_act = _block_norm_sizes(y, act)
    context, handle = _enter(stream, y.device)
    with context:
        dt, dev, f32, code = y.dtype, y.device, torch.float32, _dtype_code(y.dtype)
        _check_all(dev, [(y, "y", dt, None), (h, "h", dt, y.shape), (gate, "gate", dt, y.shape), (post, "post", f32, (C,)),
                         (scale, "scale", f32, (C,)), (pre, "pre", f32, (C,)), (stats, "stats", f32, (N, 2)),
                         (dh, "dh", dt, y.shape), (dn, "dn", dt, y.shape)])
        out = _results(out, dict(dx=y if want_dx else None, dy=y, dgate=gate, dpost=post, dscale=scale, dpre=pre), dev)
        sums = post is not None or scale is not None or pre is not None
        p, n, workspace = _workspace(workspace, lib.qdelta_block_norm_bwd_workspace_bytes(N, C, int(sums), code), dev)
        rc = lib.qdelta_block_norm_bwd(_at(y), _at(h), _at(post), _at(gate), _at(scale), _at(pre), _at(stats), _at(dh), _at(dn),
                                       _at(out["dx"]), _at(out["dy"]), _at(out["dgate"]), _at(out["dpost"]),
                                       _at(out["dscale"]), _at(out["dpre"]), N, C, code_act, code, p, n, handle)
        _raise(rc, "qdelta_block_norm_bwd")
        return out
