"""Python binding of libgradlev.so, the B200 GradLev scan library.

Argument marshalling only: every step of the scans runs in the library's CUDA
kernels. PyTorch provides device memory and the stream. The functions carry
the names of the C entry points declared in ``include/gradlev.h``.

If the shared library is missing or cannot be loaded, every call raises
``GradlevError``; there is no fallback.
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os

__all__ = [
    "GradlevError", "lib", "gradlev_status_string", "gradlev_scan_supported",
    "gradlev_scan_workspace_bytes", "gradlev_scan_ckpt_bytes", "gradlev_scan_fwd",
    "gradlev_scan_bwd", "gradlev_scan_fwd_state", "gradlev_scan_bwd_state",
    "gradlev_decode_step", "gradlev_consistency_workspace_bytes", "gradlev_consistency_step",
    "gradlev_mlp2_workspace_bytes", "gradlev_mlp2_recon", "gradlev_delta_supported",
    "gradlev_delta_workspace_bytes", "gradlev_delta_ckpt_bytes", "gradlev_delta_fwd",
    "gradlev_delta_bwd", "gradlev_delta_step", "gradlev_qk_norm_rope_workspace_bytes",
    "gradlev_qk_norm_rope_fwd", "gradlev_qk_norm_rope_bwd", "gradlev_device_status",
    "gradlev_last_launch_count", "F32", "BF16", "LIB_PATH",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgradlev.so")
F32 = 0
BF16 = 1

_ENTRY_POINTS = (
    "gradlev_status_string", "gradlev_scan_supported", "gradlev_scan_workspace_bytes",
    "gradlev_scan_ckpt_bytes", "gradlev_scan_fwd", "gradlev_scan_bwd",
    "gradlev_scan_fwd_state", "gradlev_scan_bwd_state", "gradlev_decode_step",
    "gradlev_consistency_workspace_bytes", "gradlev_consistency_step",
    "gradlev_mlp2_workspace_bytes", "gradlev_mlp2_recon", "gradlev_delta_supported",
    "gradlev_delta_workspace_bytes", "gradlev_delta_ckpt_bytes", "gradlev_delta_fwd",
    "gradlev_delta_bwd", "gradlev_delta_step", "gradlev_qk_norm_rope_workspace_bytes",
    "gradlev_qk_norm_rope_fwd", "gradlev_qk_norm_rope_bwd", "gradlev_device_status",
    "gradlev_last_launch_count",
)


class GradlevError(RuntimeError):
    """A C entry point returned a non-OK status, or the library is unavailable."""

    def __init__(self, msg, status=None):
        super().__init__(msg)
        self.status = status


_lib = None


def lib():
    """The loaded ctypes library (loads it on first use; raises GradlevError if absent)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise GradlevError(f"libgradlev.so not built ({LIB_PATH}); run "
                           "`python -m token_weight_scans_b200.build`")
    try:
        L = ctypes.CDLL(LIB_PATH)
    except OSError as e:  # pragma: no cover - depends on the box
        raise GradlevError(f"cannot load {LIB_PATH}: {e}") from e
    I, Z, P = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p
    L.gradlev_status_string.argtypes = [I]
    L.gradlev_status_string.restype = ctypes.c_char_p
    L.gradlev_scan_supported.argtypes = [I] * 6
    L.gradlev_scan_supported.restype = I
    L.gradlev_scan_workspace_bytes.argtypes = [I] * 7
    L.gradlev_scan_workspace_bytes.restype = Z
    L.gradlev_scan_ckpt_bytes.argtypes = [I] * 6
    L.gradlev_scan_ckpt_bytes.restype = Z
    L.gradlev_scan_fwd.argtypes = [I] * 6 + [P] * 8 + [Z, P]
    L.gradlev_scan_fwd.restype = I
    L.gradlev_scan_bwd.argtypes = [I] * 6 + [P] * 13 + [Z, P]
    L.gradlev_scan_bwd.restype = I
    L.gradlev_scan_fwd_state.argtypes = [I] * 6 + [P] * 10 + [Z, P]
    L.gradlev_scan_fwd_state.restype = I
    L.gradlev_scan_bwd_state.argtypes = [I] * 6 + [P] * 16 + [Z, P]
    L.gradlev_scan_bwd_state.restype = I
    L.gradlev_decode_step.argtypes = [I] * 6 + [P] * 9
    L.gradlev_decode_step.restype = I
    L.gradlev_consistency_workspace_bytes.argtypes = [I] * 6
    L.gradlev_consistency_workspace_bytes.restype = Z
    L.gradlev_consistency_step.argtypes = ([I] * 6 + [P] * 6 + [ctypes.c_float] + [P] * 11 +
                                           [Z, P])
    L.gradlev_consistency_step.restype = I
    L.gradlev_mlp2_workspace_bytes.argtypes = [I] * 7
    L.gradlev_mlp2_workspace_bytes.restype = Z
    L.gradlev_mlp2_recon.argtypes = [I] * 7 + [P] * 8 + [I] + [P] * 7 + [Z, P]
    L.gradlev_mlp2_recon.restype = I
    F, LL = ctypes.c_float, ctypes.POINTER(ctypes.c_longlong)
    L.gradlev_delta_supported.argtypes = [I] * 7
    L.gradlev_delta_supported.restype = I
    L.gradlev_delta_workspace_bytes.argtypes = [I] * 8
    L.gradlev_delta_workspace_bytes.restype = Z
    L.gradlev_delta_ckpt_bytes.argtypes = [I] * 7
    L.gradlev_delta_ckpt_bytes.restype = Z
    L.gradlev_delta_fwd.argtypes = [I] * 7 + [P] * 5 + [F] + [P] * 5 + [Z, P]
    L.gradlev_delta_fwd.restype = I
    L.gradlev_delta_bwd.argtypes = [I] * 7 + [P] * 5 + [F] + [P] * 11 + [Z, P]
    L.gradlev_delta_bwd.restype = I
    L.gradlev_delta_step.argtypes = [I] * 7 + [P] * 5 + [F, P, I] + [P] * 3
    L.gradlev_delta_step.restype = I
    L.gradlev_qk_norm_rope_workspace_bytes.argtypes = [I] * 6
    L.gradlev_qk_norm_rope_workspace_bytes.restype = Z
    L.gradlev_qk_norm_rope_fwd.argtypes = [I] * 8 + [F, P, LL, P, LL] + [P] * 7
    L.gradlev_qk_norm_rope_fwd.restype = I
    L.gradlev_qk_norm_rope_bwd.argtypes = ([I] * 8 + [F, P, P, P, LL, P, LL] + [P] * 4 +
                                           [P, LL, P, LL] + [P] * 3 + [Z, P])
    L.gradlev_qk_norm_rope_bwd.restype = I
    L.gradlev_device_status.argtypes = [P, P]
    L.gradlev_device_status.restype = I
    L.gradlev_last_launch_count.argtypes = []
    L.gradlev_last_launch_count.restype = I
    L.gradlev_debug_inject_timeout.argtypes = [I, I]
    L.gradlev_debug_inject_timeout.restype = None
    L.gradlev_debug_summary_rescale.argtypes = [ctypes.c_float]
    L.gradlev_debug_summary_rescale.restype = None
    _lib = L
    return L


def gradlev_status_string(status: int) -> str:
    return lib().gradlev_status_string(int(status)).decode()


def _check(status: int, what: str):
    if status != 0:
        raise GradlevError(f"{what}: {gradlev_status_string(status)}", status)


def _dt_code(dtype) -> int:
    import torch
    if dtype == torch.float32:
        return F32
    if dtype == torch.bfloat16:
        return BF16
    raise GradlevError(f"unsupported I/O dtype {dtype}")


def gradlev_scan_supported(B, H, T, d_in, d_out, dt) -> int:
    return int(lib().gradlev_scan_supported(B, H, T, d_in, d_out, dt))


def gradlev_scan_workspace_bytes(B, H, T, d_in, d_out, dt, is_bwd) -> int:
    return int(lib().gradlev_scan_workspace_bytes(B, H, T, d_in, d_out, dt, int(is_bwd)))


def gradlev_scan_ckpt_bytes(B, H, T, d_in, d_out, dt) -> int:
    return int(lib().gradlev_scan_ckpt_bytes(B, H, T, d_in, d_out, dt))


def gradlev_last_launch_count() -> int:
    return int(lib().gradlev_last_launch_count())


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream_ptr(stream, device=None):
    """The stream as a cudaStream_t: the given one, which must belong to `device`, or the
    current stream of `device` (of the current device when `device` is None)."""
    import torch
    if stream is None:
        return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)
    if device is not None and stream.device != device:
        raise GradlevError(f"stream is on {stream.device}, the tensors on {device}")
    return ctypes.c_void_p(stream.cuda_stream)


def _on_stream(call, stream, *args, **named):
    """`call` with the given stream current, so that what it allocates comes from that stream's
    memory: a block of the current stream's may still be in use by kernels queued there, which the
    given stream does not wait for. The tensors that come back are used by the caller's stream as
    well, and what the caller lent by the given one, so both hold their memory until they are done
    with it."""
    import torch
    dev = _cuda_device(args[0])
    if stream.device != dev:
        raise GradlevError(f"stream is on {stream.device}, the tensors on {dev}")
    with torch.cuda.stream(stream):
        result = call(*args, **named)
    held = result.values() if isinstance(result, dict) else \
        result if isinstance(result, tuple) else (result,)
    for t in (*held, named.get("ckpt"), named.get("workspace")):
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
            t.record_stream(torch.cuda.current_stream(dev))
    return result


def _cuda_device(x):
    """The device of x, which must be a CUDA device: the library's kernels dereference
    every pointer on the GPU, so host memory is refused here, before any call."""
    if not getattr(x, "is_cuda", False):
        raise GradlevError(f"tensors must be on a CUDA device, got {getattr(x, 'device', type(x))}")
    return x.device


def _check_tensor(name, t, shape, dtype, device):
    if t.shape != tuple(shape):
        raise GradlevError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if t.dtype != dtype:
        raise GradlevError(f"{name}: dtype {t.dtype} != {dtype}")
    if t.device != device:
        raise GradlevError(f"{name}: device {t.device} != {device}")
    if not t.is_contiguous():
        raise GradlevError(f"{name}: must be contiguous")


def _check_buffer(name, t, nbytes, device):
    """A caller's byte buffer (workspace, checkpoints): on the call's device, contiguous,
    at least nbytes long."""
    if t.device != device:
        raise GradlevError(f"{name}: device {t.device} != {device}")
    if not t.is_contiguous():
        raise GradlevError(f"{name}: must be contiguous")
    if t.numel() * t.element_size() < nbytes:
        raise GradlevError(f"{name} too small: {t.numel() * t.element_size()} < {nbytes} bytes")


def _workspace(nbytes, device, workspace):
    import torch
    if workspace is None:
        return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    _check_buffer("workspace", workspace, nbytes, device)
    return workspace


def _check_ckpt(ckpt, B, H, T, d_in, d_out, code, device):
    if ckpt is not None:
        _check_buffer("ckpt", ckpt, gradlev_scan_ckpt_bytes(B, H, T, d_in, d_out, code), device)


def _check_out(out, spec, device):
    """Caller-supplied outputs: every tensor of `spec` (name -> (shape, dtype)) present and
    matching; None entries allowed only where spec says so (dtype None)."""
    for k, (shape, dtype) in spec.items():
        t = out.get(k)
        if t is None:
            if dtype is None:
                continue
            raise GradlevError(f"out[{k!r}] missing")
        _check_tensor(f"out[{k!r}]", t, shape, t.dtype if dtype is None else dtype, device)


def _dims(x, g):
    if x.dim() != 4 or g.dim() != 4:
        raise GradlevError("x and g must be [B,H,T,d] tensors")
    B, H, T, d_in = x.shape
    d_out = g.shape[-1]
    return B, H, T, d_in, d_out


def gradlev_scan_fwd(x, g, eta, alpha, W0, *, y=None, ckpt=None, workspace=None, stream=None):
    """Forward scan on the GPU. Returns y [B,H,T,d_out] (dtype of x)."""
    if stream is not None:
        return _on_stream(gradlev_scan_fwd, stream, x, g, eta, alpha, W0, y=y, ckpt=ckpt,
                          workspace=workspace)
    import torch
    B, H, T, d_in, d_out = _dims(x, g)
    dev, dt = _cuda_device(x), x.dtype
    f32 = torch.float32
    _check_tensor("g", g, (B, H, T, d_out), dt, dev)
    _check_tensor("eta", eta, (B, H, T), f32, dev)
    _check_tensor("alpha", alpha, (B, H, T), f32, dev)
    _check_tensor("W0", W0, (H, d_out, d_in), f32, dev)
    _check_tensor("x", x, (B, H, T, d_in), dt, dev)
    code = _dt_code(dt)
    _check(gradlev_scan_supported(B, H, T, d_in, d_out, code), "gradlev_scan_fwd")
    if y is None:
        y = torch.empty((B, H, T, d_out), dtype=dt, device=dev)
    _check_tensor("y", y, (B, H, T, d_out), dt, dev)
    _check_ckpt(ckpt, B, H, T, d_in, d_out, code, dev)
    nws = gradlev_scan_workspace_bytes(B, H, T, d_in, d_out, code, 0)
    ws = _workspace(nws, dev, workspace)
    with torch.cuda.device(dev):  # launches go to the tensors' device
        st = lib().gradlev_scan_fwd(B, H, T, d_in, d_out, code, _ptr(x), _ptr(g), _ptr(eta),
                                    _ptr(alpha), _ptr(W0), _ptr(y), _ptr(ckpt), _ptr(ws),
                                    ws.numel() * ws.element_size(), _stream_ptr(None, dev))
    _check(st, "gradlev_scan_fwd")
    return y


def gradlev_scan_bwd(x, g, eta, alpha, W0, dy, *, ckpt=None, workspace=None, stream=None,
                     out=None):
    """Reverse scan on the GPU. Returns dict dx, dg, deta, dalpha, dW0."""
    if stream is not None:
        return _on_stream(gradlev_scan_bwd, stream, x, g, eta, alpha, W0, dy, ckpt=ckpt,
                          workspace=workspace, out=out)
    import torch
    B, H, T, d_in, d_out = _dims(x, g)
    dev, dt = _cuda_device(x), x.dtype
    f32 = torch.float32
    _check_tensor("x", x, (B, H, T, d_in), dt, dev)
    _check_tensor("g", g, (B, H, T, d_out), dt, dev)
    _check_tensor("dy", dy, (B, H, T, d_out), dt, dev)
    _check_tensor("eta", eta, (B, H, T), f32, dev)
    _check_tensor("alpha", alpha, (B, H, T), f32, dev)
    _check_tensor("W0", W0, (H, d_out, d_in), f32, dev)
    code = _dt_code(dt)
    _check(gradlev_scan_supported(B, H, T, d_in, d_out, code), "gradlev_scan_bwd")
    if out is None:
        out = dict(dx=torch.empty_like(x), dg=torch.empty_like(g),
                   deta=torch.empty((B, H, T), dtype=f32, device=dev),
                   dalpha=torch.empty((B, H, T), dtype=f32, device=dev),
                   dW0=torch.empty((H, d_out, d_in), dtype=f32, device=dev))
    _check_out(out, dict(dx=((B, H, T, d_in), dt), dg=((B, H, T, d_out), dt),
                         deta=((B, H, T), f32), dalpha=((B, H, T), f32),
                         dW0=((H, d_out, d_in), f32)), dev)
    _check_ckpt(ckpt, B, H, T, d_in, d_out, code, dev)
    nws = gradlev_scan_workspace_bytes(B, H, T, d_in, d_out, code, 1)
    ws = _workspace(nws, dev, workspace)
    with torch.cuda.device(dev):  # launches go to the tensors' device
        st = lib().gradlev_scan_bwd(B, H, T, d_in, d_out, code, _ptr(x), _ptr(g), _ptr(eta),
                                    _ptr(alpha), _ptr(W0), _ptr(dy), _ptr(out["dx"]),
                                    _ptr(out["dg"]), _ptr(out["deta"]), _ptr(out["dalpha"]),
                                    _ptr(out["dW0"]), _ptr(ckpt), _ptr(ws),
                                    ws.numel() * ws.element_size(), _stream_ptr(None, dev))
    _check(st, "gradlev_scan_bwd")
    return out


def _state_tensor(name, t, B, H, d_in, d_out, dev):
    import torch
    if t is not None:
        _check_tensor(name, t, (B, H, d_out, d_in), torch.float32, dev)
    return t


def gradlev_scan_fwd_state(x, g, eta, alpha, W0, S0=None, *, y=None, ST=None, ckpt=None,
                           workspace=None, stream=None):
    """Forward scan continuing from the carried deviation S0 ([B,H,d_out,d_in] float32,
    None = 0). Returns (y, ST), ST the deviation after the last token."""
    if stream is not None:
        return _on_stream(gradlev_scan_fwd_state, stream, x, g, eta, alpha, W0, S0, y=y, ST=ST,
                          ckpt=ckpt, workspace=workspace)
    import torch
    B, H, T, d_in, d_out = _dims(x, g)
    dev, dt = _cuda_device(x), x.dtype
    f32 = torch.float32
    _check_tensor("x", x, (B, H, T, d_in), dt, dev)
    _check_tensor("g", g, (B, H, T, d_out), dt, dev)
    _check_tensor("eta", eta, (B, H, T), f32, dev)
    _check_tensor("alpha", alpha, (B, H, T), f32, dev)
    _check_tensor("W0", W0, (H, d_out, d_in), f32, dev)
    _state_tensor("S0", S0, B, H, d_in, d_out, dev)
    code = _dt_code(dt)
    _check(gradlev_scan_supported(B, H, T, d_in, d_out, code), "gradlev_scan_fwd_state")
    if y is None:
        y = torch.empty((B, H, T, d_out), dtype=dt, device=dev)
    _check_tensor("y", y, (B, H, T, d_out), dt, dev)
    if ST is None:
        ST = torch.empty((B, H, d_out, d_in), dtype=f32, device=dev)
    _state_tensor("ST", ST, B, H, d_in, d_out, dev)
    _check_ckpt(ckpt, B, H, T, d_in, d_out, code, dev)
    nws = gradlev_scan_workspace_bytes(B, H, T, d_in, d_out, code, 0)
    ws = _workspace(nws, dev, workspace)
    with torch.cuda.device(dev):  # launches go to the tensors' device
        st = lib().gradlev_scan_fwd_state(B, H, T, d_in, d_out, code, _ptr(x), _ptr(g), _ptr(eta),
                                          _ptr(alpha), _ptr(W0), _ptr(S0), _ptr(y), _ptr(ST),
                                          _ptr(ckpt), _ptr(ws), ws.numel() * ws.element_size(),
                                          _stream_ptr(None, dev))
    _check(st, "gradlev_scan_fwd_state")
    return y, ST


def gradlev_scan_bwd_state(x, g, eta, alpha, W0, dy, S0=None, LamT=None, *, ckpt=None,
                           workspace=None, stream=None, out=None):
    """Reverse scan with the carried state: S0 the start deviation of the forward (read only
    without ckpt), LamT the adjoint flowing in after the last token (both [B,H,d_out,d_in]
    float32, None = 0). Returns dict dx, dg, deta, dalpha, dW0, dS0."""
    if stream is not None:
        return _on_stream(gradlev_scan_bwd_state, stream, x, g, eta, alpha, W0, dy, S0, LamT,
                          ckpt=ckpt, workspace=workspace, out=out)
    import torch
    B, H, T, d_in, d_out = _dims(x, g)
    dev, dt = _cuda_device(x), x.dtype
    f32 = torch.float32
    _check_tensor("x", x, (B, H, T, d_in), dt, dev)
    _check_tensor("g", g, (B, H, T, d_out), dt, dev)
    _check_tensor("dy", dy, (B, H, T, d_out), dt, dev)
    _check_tensor("eta", eta, (B, H, T), f32, dev)
    _check_tensor("alpha", alpha, (B, H, T), f32, dev)
    _check_tensor("W0", W0, (H, d_out, d_in), f32, dev)
    _state_tensor("S0", S0, B, H, d_in, d_out, dev)
    _state_tensor("LamT", LamT, B, H, d_in, d_out, dev)
    code = _dt_code(dt)
    _check(gradlev_scan_supported(B, H, T, d_in, d_out, code), "gradlev_scan_bwd_state")
    if out is None:
        out = dict(dx=torch.empty_like(x), dg=torch.empty_like(g),
                   deta=torch.empty((B, H, T), dtype=f32, device=dev),
                   dalpha=torch.empty((B, H, T), dtype=f32, device=dev),
                   dW0=torch.empty((H, d_out, d_in), dtype=f32, device=dev),
                   dS0=torch.empty((B, H, d_out, d_in), dtype=f32, device=dev))
    _check_out(out, dict(dx=((B, H, T, d_in), dt), dg=((B, H, T, d_out), dt),
                         deta=((B, H, T), f32), dalpha=((B, H, T), f32),
                         dW0=((H, d_out, d_in), f32), dS0=((B, H, d_out, d_in), f32)), dev)
    _check_ckpt(ckpt, B, H, T, d_in, d_out, code, dev)
    nws = gradlev_scan_workspace_bytes(B, H, T, d_in, d_out, code, 1)
    ws = _workspace(nws, dev, workspace)
    with torch.cuda.device(dev):  # launches go to the tensors' device
        st = lib().gradlev_scan_bwd_state(B, H, T, d_in, d_out, code, _ptr(x), _ptr(g), _ptr(eta),
                                          _ptr(alpha), _ptr(W0), _ptr(S0), _ptr(dy), _ptr(LamT),
                                          _ptr(out["dx"]), _ptr(out["dg"]), _ptr(out["deta"]),
                                          _ptr(out["dalpha"]), _ptr(out["dW0"]), _ptr(out["dS0"]),
                                          _ptr(ckpt), _ptr(ws), ws.numel() * ws.element_size(),
                                          _stream_ptr(None, dev))
    _check(st, "gradlev_scan_bwd_state")
    return out


def gradlev_decode_step(x, v, eta, alpha, W0, S, *, y=None, g=None, want_g=True, stream=None):
    """Deployment decode of the T tokens of x in order, from the carried deviation S
    ([B,H,d_out,d_in] float32, updated in place). Returns (y, g): outputs and costates
    [B,H,T,d_out] (g is None when want_g is False and no buffer is given)."""
    if stream is not None:
        return _on_stream(gradlev_decode_step, stream, x, v, eta, alpha, W0, S, y=y, g=g,
                          want_g=want_g)
    import torch
    B, H, T, d_in, d_out = _dims(x, v)
    dev, dt = _cuda_device(x), x.dtype
    f32 = torch.float32
    _check_tensor("x", x, (B, H, T, d_in), dt, dev)
    _check_tensor("v", v, (B, H, T, d_out), dt, dev)
    _check_tensor("eta", eta, (B, H, T), f32, dev)
    _check_tensor("alpha", alpha, (B, H, T), f32, dev)
    _check_tensor("W0", W0, (H, d_out, d_in), f32, dev)
    _check_tensor("S", S, (B, H, d_out, d_in), f32, dev)
    if y is None:
        y = torch.empty((B, H, T, d_out), dtype=dt, device=dev)
    _check_tensor("y", y, (B, H, T, d_out), dt, dev)
    if g is None and want_g:
        g = torch.empty((B, H, T, d_out), dtype=dt, device=dev)
    if g is not None:
        _check_tensor("g", g, (B, H, T, d_out), dt, dev)
    with torch.cuda.device(dev):  # launches go to the tensors' device
        st = lib().gradlev_decode_step(B, H, T, d_in, d_out, _dt_code(dt), _ptr(x), _ptr(v),
                                       _ptr(eta), _ptr(alpha), _ptr(W0), _ptr(S), _ptr(y), _ptr(g),
                                       _stream_ptr(None, dev))
    _check(st, "gradlev_decode_step")
    return y, g


def gradlev_consistency_workspace_bytes(B, H, T, d_in, d_out, dt) -> int:
    return int(lib().gradlev_consistency_workspace_bytes(B, H, T, d_in, d_out, dt))


def gradlev_consistency_step(x, ghat, eta, alpha, W0, v, lam=1.0, *, want_dv=True,
                             workspace=None, stream=None, out=None):
    """One training step of the adapted layer from predicted costates ghat (see
    include/gradlev.h). Returns dict y, gtil, loss_tok, loss_c, dx, dghat, deta, dalpha, dW0
    and dv (None when want_dv is False)."""
    if stream is not None:
        return _on_stream(gradlev_consistency_step, stream, x, ghat, eta, alpha, W0, v, lam,
                          want_dv=want_dv, workspace=workspace, out=out)
    import torch
    B, H, T, d_in, d_out = _dims(x, ghat)
    dev, dt = _cuda_device(x), x.dtype
    f32 = torch.float32
    _check_tensor("x", x, (B, H, T, d_in), dt, dev)
    _check_tensor("ghat", ghat, (B, H, T, d_out), dt, dev)
    _check_tensor("v", v, (B, H, T, d_out), dt, dev)
    _check_tensor("eta", eta, (B, H, T), f32, dev)
    _check_tensor("alpha", alpha, (B, H, T), f32, dev)
    _check_tensor("W0", W0, (H, d_out, d_in), f32, dev)
    code = _dt_code(dt)
    nws = gradlev_consistency_workspace_bytes(B, H, T, d_in, d_out, code)
    if nws == 0:
        raise GradlevError("gradlev_consistency_step: unsupported shape", 2)
    if out is None:
        out = dict(y=torch.empty_like(ghat), gtil=torch.empty_like(ghat),
                   loss_tok=torch.empty((B, H, T), dtype=f32, device=dev),
                   loss_c=torch.empty((B, H, T), dtype=f32, device=dev),
                   dx=torch.empty_like(x), dghat=torch.empty_like(ghat),
                   deta=torch.empty((B, H, T), dtype=f32, device=dev),
                   dalpha=torch.empty((B, H, T), dtype=f32, device=dev),
                   dW0=torch.empty((H, d_out, d_in), dtype=f32, device=dev),
                   dv=torch.empty_like(ghat) if want_dv else None)
    _check_out(out, dict(y=((B, H, T, d_out), dt), gtil=((B, H, T, d_out), dt),
                         loss_tok=((B, H, T), f32), loss_c=((B, H, T), f32),
                         dx=((B, H, T, d_in), dt), dghat=((B, H, T, d_out), dt),
                         deta=((B, H, T), f32), dalpha=((B, H, T), f32),
                         dW0=((H, d_out, d_in), f32)), dev)
    if out.get("dv") is not None:
        _check_tensor("out['dv']", out["dv"], (B, H, T, d_out), dt, dev)
    ws = _workspace(nws, dev, workspace)
    with torch.cuda.device(dev):  # launches go to the tensors' device
        st = lib().gradlev_consistency_step(
            B, H, T, d_in, d_out, code, _ptr(x), _ptr(ghat), _ptr(eta), _ptr(alpha), _ptr(W0),
            _ptr(v), float(lam), _ptr(out["y"]), _ptr(out["gtil"]), _ptr(out["loss_tok"]),
            _ptr(out["loss_c"]), _ptr(out["dx"]), _ptr(out["dghat"]), _ptr(out["deta"]),
            _ptr(out["dalpha"]), _ptr(out["dW0"]), _ptr(out.get("dv")), _ptr(ws),
            ws.numel() * ws.element_size(), _stream_ptr(None, dev))
    _check(st, "gradlev_consistency_step")
    return out


def gradlev_mlp2_workspace_bytes(B, H, T, d_x, d_h, d_y, dt) -> int:
    return int(lib().gradlev_mlp2_workspace_bytes(B, H, T, d_x, d_h, d_y, dt))


def gradlev_mlp2_recon(x, g1hat, g2hat, v, eta, alpha, W1, W2, control=False, *,
                       workspace=None, stream=None, out=None):
    """Parallel reconstruction of the two-layer adapted MLP from given costates (see
    include/gradlev.h). Returns dict a, h, y, g2til, g1til, dW1."""
    if stream is not None:
        return _on_stream(gradlev_mlp2_recon, stream, x, g1hat, g2hat, v, eta, alpha, W1, W2,
                          control, workspace=workspace, out=out)
    import torch
    if x.dim() != 4 or v.dim() != 4 or W1.dim() != 3:
        raise GradlevError("x, v must be [B,H,T,d] and W1 [H,d_h,d_x]")
    B, H, T, d_x = x.shape
    d_y = v.shape[-1]
    d_h = W1.shape[1]
    dev, dt = _cuda_device(x), x.dtype
    f32 = torch.float32
    _check_tensor("x", x, (B, H, T, d_x), dt, dev)
    _check_tensor("g1hat", g1hat, (B, H, T, d_h), dt, dev)
    _check_tensor("g2hat", g2hat, (B, H, T, d_y), dt, dev)
    _check_tensor("v", v, (B, H, T, d_y), dt, dev)
    _check_tensor("eta", eta, (B, H, T), f32, dev)
    _check_tensor("alpha", alpha, (B, H, T), f32, dev)
    _check_tensor("W1", W1, (H, d_h, d_x), f32, dev)
    _check_tensor("W2", W2, (H, d_y, d_h), f32, dev)
    code = _dt_code(dt)
    nws = gradlev_mlp2_workspace_bytes(B, H, T, d_x, d_h, d_y, code)
    if nws == 0:
        raise GradlevError("gradlev_mlp2_recon: unsupported shape", 2)
    if out is None:
        out = dict(a=torch.empty_like(g1hat), h=torch.empty_like(g1hat), y=torch.empty_like(v),
                   g2til=torch.empty_like(v), g1til=torch.empty_like(g1hat),
                   dW1=torch.empty((B, H, d_h, d_x), dtype=f32, device=dev))
    _check_out(out, dict(a=((B, H, T, d_h), dt), h=((B, H, T, d_h), dt),
                         y=((B, H, T, d_y), dt), g2til=((B, H, T, d_y), dt),
                         g1til=((B, H, T, d_h), dt), dW1=((B, H, d_h, d_x), f32)), dev)
    ws = _workspace(nws, dev, workspace)
    with torch.cuda.device(dev):  # launches go to the tensors' device
        st = lib().gradlev_mlp2_recon(
            B, H, T, d_x, d_h, d_y, code, _ptr(x), _ptr(g1hat), _ptr(g2hat), _ptr(v), _ptr(eta),
            _ptr(alpha), _ptr(W1), _ptr(W2), 1 if control else 0, _ptr(out["a"]), _ptr(out["h"]),
            _ptr(out["y"]), _ptr(out["g2til"]), _ptr(out["g1til"]), _ptr(out["dW1"]), _ptr(ws),
            ws.numel() * ws.element_size(), _stream_ptr(None, dev))
    _check(st, "gradlev_mlp2_recon")
    return out


# The calls below are launch-bound at a token per request, so their checks and pointers
# avoid what torch's wrappers cost: the device is only switched when it is not current, the
# stream is read as a raw handle, and addresses are passed as integers.
_NO_SWITCH = contextlib.nullcontext()


def _on(dev):
    """Launches go to the tensors' device."""
    import torch
    return _NO_SWITCH if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _addr(t):
    return None if t is None else t.data_ptr()


def _stream_of(dev):
    """dev's current stream as a raw cudaStream_t."""
    import torch
    return torch._C._cuda_getCurrentRawStream(dev.index)


def _check_fast(name, t, shape, dtype, device):
    if (t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous()):
        _check_tensor(name, t, shape, dtype, device)


def gradlev_delta_supported(B, H, Hk, T, d_k, d_v, dt) -> int:
    return int(lib().gradlev_delta_supported(B, H, Hk, T, d_k, d_v, dt))


def gradlev_delta_workspace_bytes(B, H, Hk, T, d_k, d_v, dt, is_bwd) -> int:
    return int(lib().gradlev_delta_workspace_bytes(B, H, Hk, T, d_k, d_v, dt, int(is_bwd)))


def gradlev_delta_ckpt_bytes(B, H, Hk, T, d_k, d_v, dt) -> int:
    return int(lib().gradlev_delta_ckpt_bytes(B, H, Hk, T, d_k, d_v, dt))


def _delta_args(q, k, v, beta, log_alpha, scale):
    """Checks shared by the delta calls. Returns the sizes, the dtype code and the scale."""
    import torch
    qs, vs, dt = q.shape, v.shape, q.dtype
    if len(qs) != 4 or len(vs) != 4:
        raise GradlevError("q and v must be [B,H,T,d] tensors")
    B, Hk, T, d_k = qs
    H, d_v = vs[1], vs[3]
    dev, f32, gate = _cuda_device(q), torch.float32, (B, H, T)
    code = _dt_code(dt)
    # one expression for the usual case; the loop names what is wrong
    if not (k.shape == qs and vs == (B, H, T, d_v) and beta.shape == gate and
            log_alpha.shape == gate and k.dtype == dt and v.dtype == dt and beta.dtype == f32 and
            log_alpha.dtype == f32 and k.device == dev and v.device == dev and
            beta.device == dev and log_alpha.device == dev and q.is_contiguous() and
            k.is_contiguous() and v.is_contiguous() and beta.is_contiguous() and
            log_alpha.is_contiguous()):
        for name, t, shape, dtype in (("q", q, qs, dt), ("k", k, qs, dt),
                                      ("v", v, (B, H, T, d_v), dt), ("beta", beta, gate, f32),
                                      ("log_alpha", log_alpha, gate, f32)):
            _check_tensor(name, t, shape, dtype, dev)
    return (B, H, Hk, T, d_k, d_v, code), dev, dt, float(d_k ** -0.5 if scale is None else scale)


@functools.lru_cache(maxsize=256)
def _delta_need(size):
    """For sizes and a dtype: the status of gradlev_delta_supported, the workspace bytes of the
    forward and the backward, and the checkpoint bytes."""
    L = lib()
    return (int(L.gradlev_delta_supported(*size)), L.gradlev_delta_workspace_bytes(*size, 0),
            L.gradlev_delta_workspace_bytes(*size, 1), L.gradlev_delta_ckpt_bytes(*size))


def gradlev_delta_fwd(q, k, v, beta, log_alpha, S0=None, *, scale=None, y=None, ST=None,
                      want_ST=True, ckpt=None, workspace=None, stream=None):
    """Chunked gated delta rule (see include/gradlev.h): q, k [B,Hk,T,d_k], v [B,H,T,d_v],
    beta and log_alpha [B,H,T] float32, S0 [B,H,d_v,d_k] float32 or None (zero). scale None:
    d_k ** -0.5. Returns (y, ST), ST the float32 state after the last token (None when
    want_ST is False and no buffer is given)."""
    if stream is not None:
        return _on_stream(gradlev_delta_fwd, stream, q, k, v, beta, log_alpha, S0, scale=scale,
                          y=y, ST=ST, want_ST=want_ST, ckpt=ckpt, workspace=workspace)
    import torch
    size, dev, dt, scale = _delta_args(q, k, v, beta, log_alpha, scale)
    B, H, _, T, d_k, d_v, _ = size
    f32 = torch.float32
    supported, need, _, need_ckpt = _delta_need(size)
    _check(supported, "gradlev_delta_fwd")
    if S0 is not None:
        _check_fast("S0", S0, (B, H, d_v, d_k), f32, dev)
    if y is None:
        y = torch.empty_like(v)
    else:
        _check_tensor("y", y, (B, H, T, d_v), dt, dev)
    if ST is None and want_ST:
        ST = torch.empty((B, H, d_v, d_k), dtype=f32, device=dev)
    if ST is not None:
        _check_fast("ST", ST, (B, H, d_v, d_k), f32, dev)
    if ckpt is not None:
        _check_buffer("ckpt", ckpt, need_ckpt, dev)
    ws = _workspace(need, dev, workspace)
    with _on(dev):
        st = lib().gradlev_delta_fwd(*size, _addr(q), _addr(k), _addr(v), _addr(beta),
                                     _addr(log_alpha), scale, _addr(S0), _addr(y), _addr(ST),
                                     _addr(ckpt), _addr(ws), ws.numel() * ws.element_size(),
                                     _stream_of(dev))
    _check(st, "gradlev_delta_fwd")
    return y, ST


def gradlev_delta_bwd(q, k, v, beta, log_alpha, dy, S0=None, dST=None, *, scale=None, ckpt=None,
                      want_dS0=True, workspace=None, stream=None, out=None):
    """Gradients of the gated delta rule, all in the I/O dtype: dict dq, dk, dv, dbeta,
    dlog_alpha and dS0 (None when want_dS0 is False). dST [B,H,d_v,d_k] (I/O dtype, None = 0)
    is the gradient of the last state; ckpt the buffer a forward call on the same inputs
    filled (None: the states are recomputed from S0)."""
    if stream is not None:
        return _on_stream(gradlev_delta_bwd, stream, q, k, v, beta, log_alpha, dy, S0, dST,
                          scale=scale, ckpt=ckpt, want_dS0=want_dS0, workspace=workspace, out=out)
    import torch
    size, dev, dt, scale = _delta_args(q, k, v, beta, log_alpha, scale)
    B, H, _, T, d_k, d_v, _ = size
    supported, _, need, need_ckpt = _delta_need(size)
    _check(supported, "gradlev_delta_bwd")
    _check_fast("dy", dy, (B, H, T, d_v), dt, dev)
    if S0 is not None:
        _check_fast("S0", S0, (B, H, d_v, d_k), torch.float32, dev)
    if dST is not None:
        _check_fast("dST", dST, (B, H, d_v, d_k), dt, dev)
    if out is None:
        out = dict(dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
                   dbeta=torch.empty((B, H, T), dtype=dt, device=dev),
                   dlog_alpha=torch.empty((B, H, T), dtype=dt, device=dev),
                   dS0=torch.empty((B, H, d_v, d_k), dtype=dt, device=dev) if want_dS0 else None)
    else:
        _check_out(out, dict(dq=(q.shape, dt), dk=(k.shape, dt), dv=(v.shape, dt),
                             dbeta=((B, H, T), dt), dlog_alpha=((B, H, T), dt)), dev)
        if out.get("dS0") is not None:
            _check_fast("out['dS0']", out["dS0"], (B, H, d_v, d_k), dt, dev)
    if ckpt is not None:
        _check_buffer("ckpt", ckpt, need_ckpt, dev)
    ws = _workspace(need, dev, workspace)
    with _on(dev):
        st = lib().gradlev_delta_bwd(
            *size, _addr(q), _addr(k), _addr(v), _addr(beta), _addr(log_alpha), scale, _addr(S0),
            _addr(dy), _addr(dST), _addr(out["dq"]), _addr(out["dk"]), _addr(out["dv"]),
            _addr(out["dbeta"]), _addr(out["dlog_alpha"]), _addr(out.get("dS0")), _addr(ckpt),
            _addr(ws), ws.numel() * ws.element_size(), _stream_of(dev))
    _check(st, "gradlev_delta_bwd")
    return out


def gradlev_delta_step(q, k, v, beta, log_alpha, S, *, slots=None, scale=None, y=None,
                       stream=None):
    """The T tokens of q, k, v in order on the states S [pool,H,d_v,d_k] float32, updated in
    place. slots [B] int32 picks each batch row's state (None: row b); a row without a state
    of its own (slot outside the pool, or named by an earlier row) answers with zeros. S ends
    as the states after all T tokens. Returns y [B,H,T,d_v]."""
    if stream is not None:
        return _on_stream(gradlev_delta_step, stream, q, k, v, beta, log_alpha, S, slots=slots,
                          scale=scale, y=y)
    import torch
    size, dev, dt, scale = _delta_args(q, k, v, beta, log_alpha, scale)
    B, H, _, T, d_k, d_v, _ = size
    if S.dim() != 4:
        raise GradlevError("S must be a [pool,H,d_v,d_k] tensor")
    _check_fast("S", S, (S.shape[0], H, d_v, d_k), torch.float32, dev)
    if slots is not None:
        _check_fast("slots", slots, (B,), torch.int32, dev)
    if y is None:
        y = torch.empty_like(v)
    else:
        _check_tensor("y", y, (B, H, T, d_v), dt, dev)
    with _on(dev):
        st = lib().gradlev_delta_step(*size, _addr(q), _addr(k), _addr(v), _addr(beta),
                                      _addr(log_alpha), scale, _addr(slots), S.shape[0], _addr(S),
                                      _addr(y), _stream_of(dev))
    _check(st, "gradlev_delta_step")
    return y


_NORMS = {"l2": 0, "rms": 1}


def gradlev_qk_norm_rope_workspace_bytes(B, T, Hq, Hk, d, dt) -> int:
    return int(lib().gradlev_qk_norm_rope_workspace_bytes(B, T, Hq, Hk, d, dt))


def _strided(name, t, shape, dtype, device):
    """A [B,T,H,d] tensor whose columns are contiguous; its other strides as a C array."""
    if t.shape != tuple(shape):
        raise GradlevError(f"{name}: shape {tuple(t.shape)} != {tuple(shape)}")
    if t.dtype != dtype:
        raise GradlevError(f"{name}: dtype {t.dtype} != {dtype}")
    if t.device != device:
        raise GradlevError(f"{name}: device {t.device} != {device}")
    if t.stride(3) != 1 and t.shape[3] != 1:
        raise GradlevError(f"{name}: columns must be contiguous")
    return _c_strides(t.stride(), t.shape)


@functools.lru_cache(maxsize=256)
def _c_strides(stride, shape):
    """Strides of the first three axes as a C array; that of an axis of length 1 is unused."""
    return (ctypes.c_longlong * 3)(*[stride[i] if shape[i] > 1 else 0 for i in range(3)])


def _norm_args(q, k, wq, wk, pos, inv_freq, norm):
    import torch
    if q.dim() != 4 or k.dim() != 4:
        raise GradlevError("q and k must be [B,T,H,d] tensors")
    if norm not in _NORMS:
        raise GradlevError(f"norm: {norm!r} is not one of {sorted(_NORMS)}")
    qs, ks = q.shape, k.shape
    B, T, Hq, d = qs
    Hk = ks[2]
    dev, dt = _cuda_device(q), q.dtype
    qt, kt = q.stride(), k.stride()
    # one expression for the usual case; _strided names what is wrong
    if not (ks == (B, T, Hk, d) and k.dtype == dt and k.device == dev and
            (d == 1 or (qt[3] == 1 and kt[3] == 1))):
        _strided("q", q, (B, T, Hq, d), dt, dev)
        _strided("k", k, (B, T, Hk, d), dt, dev)
    sq, sk = _c_strides(qt, qs), _c_strides(kt, ks)
    for n, w in (("wq", wq), ("wk", wk)):
        if w is not None:
            _check_fast(n, w, (d,), torch.float32, dev)
    if pos is not None:
        _check_fast("pos", pos, (B, T), torch.int32, dev)
    rot = 0
    if inv_freq is not None:
        rot = 2 * inv_freq.numel()
        _check_fast("inv_freq", inv_freq, (rot // 2,), torch.float32, dev)
    return (B, T, Hq, Hk, d, rot, _dt_code(dt), _NORMS[norm]), dev, dt, sq, sk


def gradlev_qk_norm_rope_fwd(q, k, wq=None, wk=None, pos=None, inv_freq=None, *, norm="l2",
                             eps=1e-6, yq=None, yk=None, stream=None):
    """Norm per head and rotation by position of q [B,T,Hq,d] and k [B,T,Hk,d] (any strides
    with contiguous columns, e.g. views of one packed projection). Returns (yq [B,Hq,T,d],
    yk [B,Hk,T,d]), contiguous. norm "l2" or "rms"; wq, wk [d] float32 or None; pos [B,T]
    int32 or None (t); inv_freq [rot/2] float32 or None (no rotation)."""
    if stream is not None:
        return _on_stream(gradlev_qk_norm_rope_fwd, stream, q, k, wq, wk, pos, inv_freq,
                          norm=norm, eps=eps, yq=yq, yk=yk)
    import torch
    a, dev, dt, sq, sk = _norm_args(q, k, wq, wk, pos, inv_freq, norm)
    B, T, Hq, Hk, d = a[:5]
    if yq is None:
        yq = q.new_empty((B, Hq, T, d))
    else:
        _check_tensor("yq", yq, (B, Hq, T, d), dt, dev)
    if yk is None:
        yk = q.new_empty((B, Hk, T, d))
    else:
        _check_tensor("yk", yk, (B, Hk, T, d), dt, dev)
    with _on(dev):
        st = lib().gradlev_qk_norm_rope_fwd(*a, float(eps), _addr(q), sq, _addr(k), sk, _addr(wq),
                                            _addr(wk), _addr(pos), _addr(inv_freq), _addr(yq),
                                            _addr(yk), _stream_of(dev))
    _check(st, "gradlev_qk_norm_rope_fwd")
    return yq, yk


def gradlev_qk_norm_rope_bwd(dyq, dyk, q, k, wq=None, wk=None, pos=None, inv_freq=None, *,
                             norm="l2", eps=1e-6, workspace=None, stream=None, out=None):
    """Gradients of gradlev_qk_norm_rope_fwd from dyq [B,Hq,T,d] and dyk [B,Hk,T,d]. Returns
    dict dq, dk (shaped like q and k; strided when given in `out`) and dwq, dwk for the
    weights that are given."""
    if stream is not None:
        return _on_stream(gradlev_qk_norm_rope_bwd, stream, dyq, dyk, q, k, wq, wk, pos, inv_freq,
                          norm=norm, eps=eps, workspace=workspace, out=out)
    import torch
    a, dev, dt, sq, sk = _norm_args(q, k, wq, wk, pos, inv_freq, norm)
    B, T, Hq, Hk, d = a[:5]
    _check_fast("dyq", dyq, (B, Hq, T, d), dt, dev)
    _check_fast("dyk", dyk, (B, Hk, T, d), dt, dev)
    f32 = torch.float32
    if out is None:
        out = dict(dq=torch.empty((B, T, Hq, d), dtype=dt, device=dev),
                   dk=torch.empty((B, T, Hk, d), dtype=dt, device=dev))
        for n, w in (("dwq", wq), ("dwk", wk)):
            if w is not None:
                out[n] = torch.empty((d,), dtype=f32, device=dev)
    if out.get("dq") is None or out.get("dk") is None:
        raise GradlevError("out needs 'dq' and 'dk'")
    sdq = _strided("out['dq']", out["dq"], (B, T, Hq, d), dt, dev)
    sdk = _strided("out['dk']", out["dk"], (B, T, Hk, d), dt, dev)
    _check_out(out, {n: ((d,), f32) for n, w in (("dwq", wq), ("dwk", wk)) if w is not None}, dev)
    nws = gradlev_qk_norm_rope_workspace_bytes(B, T, Hq, Hk, d, a[6])
    ws = _workspace(nws, dev, workspace) if wq is not None or wk is not None else None
    with _on(dev):
        st = lib().gradlev_qk_norm_rope_bwd(
            *a, float(eps), _addr(dyq), _addr(dyk), _addr(q), sq, _addr(k), sk, _addr(wq), _addr(wk),
            _addr(pos), _addr(inv_freq), _addr(out["dq"]), sdq, _addr(out["dk"]), sdk,
            _addr(out["dwq"] if wq is not None else None),
            _addr(out["dwk"] if wk is not None else None), _addr(ws),
            ws.numel() * ws.element_size() if ws is not None else 0, _stream_of(dev))
    _check(st, "gradlev_qk_norm_rope_bwd")
    return out


def gradlev_device_status(workspace, stream=None) -> int:
    import torch
    with torch.cuda.device(workspace.device):
        return int(lib().gradlev_device_status(_ptr(workspace),
                                               _stream_ptr(stream, workspace.device)))
