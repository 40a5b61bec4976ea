"""Thin ctypes binding of ``libhla2.so`` (the C ABI in ``include/hla2.h``).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI.  PyTorch supplies device memory and the stream.  The
binding refuses to run without the compiled library (there is no fallback).
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libhla2.so")

HLA2_F32, HLA2_BF16 = 0, 1
HLA2_OK, HLA2_ERR_INVALID, HLA2_ERR_UNSUPPORTED, HLA2_ERR_WORKSPACE, HLA2_ERR_LAUNCH = 0, -1, -2, -3, -4

HLA2_GATE_LOG, HLA2_GATE_SIGMOID = 0, 1
HLA2_WINDOW_MAX_SINKS = 64
HLA2_GATED_SCAN_TILE = 256  # tokens between the saved states of hla2_gated_scan_forward

# every symbol include/hla2.h declares
EXPORTS = ("hla2_strerror", "hla2_abi_version", "hla2_forward_workspace_bytes", "hla2_forward_segments",
           "hla2_forward", "hla2_forward_ex_workspace_bytes", "hla2_forward_ex_segments", "hla2_forward_ex_plan",
           "hla2_forward_ex",
           "hla2_forward_timed", "hla2_decode_step", "hla2_state_floats", "hla2_forward_state_workspace_bytes",
           "hla2_forward_state", "hla2_backward_workspace_bytes", "hla2_backward",
           "hla2_ahla_forward_workspace_bytes", "hla2_ahla_forward", "hla2_ho3_forward_workspace_bytes",
           "hla2_ho3_forward", "hla2_forward_noalloc", "hla2_gated_scan_workspace_bytes",
           "hla2_gated_scan_forward", "hla2_gated_scan_backward", "hla2_gated_scan_step",
           "hla2_window_forward", "hla2_window_backward_workspace_bytes", "hla2_window_backward",
           "hla2_window_cache", "hla2_window_step_workspace_bytes", "hla2_window_step")
HLA2_NOALLOC_SCRATCH_BYTES = 96 << 20  # the fixed workspace of hla2_forward_noalloc (include/hla2.h)

_lock = threading.Lock()
_lib = None


class HLA2Error(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__("%s failed: %s (%d)" % (what, strerror(code) if _lib else "", code))


def lib():
    """Load libhla2.so (built beforehand by ``build.build()``); raise if absent."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError("libhla2.so is not built; run causal_prefix_scan_hla2_amd.build.build()")
            L = ctypes.CDLL(LIB_PATH)
            vp, i, f, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
            L.hla2_strerror.restype = ctypes.c_char_p
            L.hla2_strerror.argtypes = [i]
            L.hla2_abi_version.restype = i
            L.hla2_abi_version.argtypes = []
            L.hla2_forward_workspace_bytes.restype = sz
            L.hla2_forward_workspace_bytes.argtypes = [i, i, i, i, i, i]
            L.hla2_forward_segments.restype = i
            L.hla2_forward_segments.argtypes = [i, i, i, i, i, i]
            L.hla2_forward.restype = i
            L.hla2_forward.argtypes = [vp, vp, vp, vp, i, i, i, i, i, f, i, i, i, vp, vp, sz, vp]
            L.hla2_forward_ex_workspace_bytes.restype = sz
            L.hla2_forward_ex_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
            L.hla2_forward_ex_segments.restype = i
            L.hla2_forward_ex_segments.argtypes = [i, i, i, i, i, i, i]
            ip = ctypes.POINTER(ctypes.c_int)
            L.hla2_forward_ex_plan.restype = i
            L.hla2_forward_ex_plan.argtypes = [i, i, i, i, i, i, i, ip, ip, ip]
            L.hla2_forward_ex.restype = i
            L.hla2_forward_ex.argtypes = [vp, vp, vp, vp, i, i, i, i, i, f, i, i, i, vp, vp, sz, i, vp]
            L.hla2_forward_timed.restype = i
            L.hla2_forward_timed.argtypes = [vp, vp, vp, vp, i, i, i, i, i, f, i, i, i, vp, vp, sz, i, vp, vp]
            L.hla2_decode_step.restype = i
            L.hla2_decode_step.argtypes = [vp, vp, vp, vp, vp, i, i, i, i, f, i, i, vp]
            L.hla2_state_floats.restype = ctypes.c_long
            L.hla2_state_floats.argtypes = [i, i]
            L.hla2_forward_state_workspace_bytes.restype = sz
            L.hla2_forward_state_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
            L.hla2_forward_state.restype = i
            L.hla2_forward_state.argtypes = [vp, vp, vp, vp, i, i, i, i, i, f, i, i, i, vp, vp, vp, sz, i, vp]
            L.hla2_backward_workspace_bytes.restype = sz
            L.hla2_backward_workspace_bytes.argtypes = [i, i, i, i, i, i, i, i]
            L.hla2_ahla_forward_workspace_bytes.restype = sz
            L.hla2_ahla_forward_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
            L.hla2_ahla_forward.restype = i
            L.hla2_ahla_forward.argtypes = [vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, vp, sz, i, vp]
            L.hla2_ho3_forward_workspace_bytes.restype = sz
            L.hla2_ho3_forward_workspace_bytes.argtypes = [i, i, i, i, i, i, i]
            L.hla2_ho3_forward.restype = i
            L.hla2_ho3_forward.argtypes = [vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, vp, sz, i, vp]
            L.hla2_forward_noalloc.restype = i
            L.hla2_forward_noalloc.argtypes = [vp, vp, vp, vp, i, i, i, i, i, f, i, i, i, vp, vp]
            L.hla2_backward.restype = i
            L.hla2_backward.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, i, i, f, i, i, vp, sz, i, vp]
            L.hla2_gated_scan_workspace_bytes.restype = sz
            L.hla2_gated_scan_workspace_bytes.argtypes = [i, i, i, i, i]
            L.hla2_gated_scan_forward.restype = i
            L.hla2_gated_scan_forward.argtypes = [vp] * 7 + [i, i, i, i, i, i, vp, sz, vp]
            L.hla2_gated_scan_backward.restype = i
            L.hla2_gated_scan_backward.argtypes = [vp] * 10 + [i, i, i, i, i, i, vp, sz, vp]
            L.hla2_gated_scan_step.restype = i
            L.hla2_gated_scan_step.argtypes = [vp] * 5 + [i, i, i, i, i, vp]
            L.hla2_window_forward.restype = i
            L.hla2_window_forward.argtypes = [vp] * 6 + [i] * 8 + [f, i, vp]
            L.hla2_window_backward_workspace_bytes.restype = sz
            L.hla2_window_backward_workspace_bytes.argtypes = [i] * 9
            L.hla2_window_backward.restype = i
            L.hla2_window_backward.argtypes = [vp] * 10 + [i] * 8 + [f, i, vp, sz, vp]
            L.hla2_window_cache.restype = i
            L.hla2_window_cache.argtypes = [vp] * 5 + [i] * 8 + [vp]
            L.hla2_window_step_workspace_bytes.restype = sz
            L.hla2_window_step_workspace_bytes.argtypes = [i] * 8
            L.hla2_window_step.restype = i
            L.hla2_window_step.argtypes = [vp] * 7 + [i] * 7 + [f, i, vp, sz, vp]
            _lib = L
    return _lib


def strerror(code: int) -> str:
    return lib().hla2_strerror(int(code)).decode()


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        import torch
        return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return ctypes.c_void_p(stream)
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t):
    import torch
    if t.dtype == torch.float32:
        return HLA2_F32
    if t.dtype == torch.bfloat16:
        return HLA2_BF16
    raise TypeError("q, k, v must be float32 or bfloat16, got %s" % t.dtype)


def hla2_forward_workspace_bytes(B, H, n, d, dv, chunk, segments=0) -> int:
    return int(lib().hla2_forward_ex_workspace_bytes(B, H, n, d, dv, chunk, segments))


def hla2_forward_segments(B, H, n, d, dv, chunk, segments=0) -> int:
    return int(lib().hla2_forward_ex_segments(B, H, n, d, dv, chunk, segments))


def hla2_forward_plan(B, H, n, d, dv, chunk, segments=0):
    """The bf16 forward's segment plan: (nseg, chunks of segment 0, chunks of each later
    segment, lead) where lead says segment 0's outputs are walked beside the summary walks."""
    nseg, c0, cs = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    rc = lib().hla2_forward_ex_plan(B, H, n, d, dv, chunk, segments, ctypes.byref(nseg), ctypes.byref(c0),
                                    ctypes.byref(cs))
    if rc < 0:
        raise HLA2Error(rc, "hla2_forward_ex_plan")
    return nseg.value, c0.value, cs.value, bool(rc)


def hla2_state_floats(d, dv) -> int:
    return int(lib().hla2_state_floats(d, dv))


def hla2_forward(q, k, v, out, decay=1.0, normalize=False, chunk=64, den_out=None, workspace=None,
                 stream=None, segments=0, check=True, events=None) -> int:
    """Call the C forward pass on torch tensors q, k: [B,H,n,d]; v, out: [B,H,n,dv].

    ``hla2_forward`` when segments == 0, else ``hla2_forward_ex`` with that
    segment count; ``hla2_forward_timed`` when ``events`` (four created
    torch.cuda.Event objects, or None entries) is given.  ``workspace``: a
    uint8 device tensor of at least the required bytes; allocated here (torch
    caching allocator) when None.  Returns the C return code (and raises on
    error when check=True)."""
    _sizes(q, v)
    B, H, n, d = q.shape
    dv = v.shape[-1]
    for t in (q, k, v, out):
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
    need = hla2_forward_workspace_bytes(B, H, n, d, dv, chunk, segments)
    if workspace is None and need > 0:
        workspace = _scratch(need, q, stream)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = (_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, H, n, d, dv, float(decay), int(bool(normalize)), int(chunk),
            _dtype_code(q), _ptr(den_out), _ptr(workspace), wbytes)
    if events is not None:
        if len(events) != 4:
            raise ValueError("events must hold four entries")
        arr = (ctypes.c_void_p * 4)(*[None if e is None else e.cuda_event for e in events])
        rc = lib().hla2_forward_timed(*args, int(segments), arr, _stream(stream))
    elif segments:
        rc = lib().hla2_forward_ex(*args, int(segments), _stream(stream))
    else:
        rc = lib().hla2_forward(*args, _stream(stream))
    if check and rc != HLA2_OK:
        raise HLA2Error(rc, "hla2_forward")
    return rc


def hla2_forward_noalloc(q, k, v, out, decay=1.0, normalize=False, chunk=64, den_out=None, stream=None,
                         check=True) -> int:
    """Call the C forward pass that uses the library's fixed device workspace (no allocation here
    or in the library).  Same tensors and results as hla2_forward."""
    _sizes(q, v)
    B, H, n, d = q.shape
    dv = v.shape[-1]
    for t in (q, k, v, out):
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
    rc = lib().hla2_forward_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, H, n, d, dv, float(decay),
                                    int(bool(normalize)), int(chunk), _dtype_code(q), _ptr(den_out), _stream(stream))
    if check and rc != HLA2_OK:
        raise HLA2Error(rc, "hla2_forward_noalloc")
    return rc


def hla2_forward_state_workspace_bytes(B, H, n, d, dv, chunk, segments=0) -> int:
    return int(lib().hla2_forward_state_workspace_bytes(B, H, n, d, dv, chunk, segments))


def hla2_forward_state(q, k, v, out, state_out, decay=1.0, normalize=False, chunk=64, den_out=None,
                       workspace=None, stream=None, segments=0, check=True) -> int:
    """Call ``hla2_forward_state``: the forward pass of ``hla2_forward`` plus the
    final state, written to ``state_out`` (fp32 [B,H,state_floats], the layout
    ``hla2_decode_step`` reads).  ``workspace`` as for ``hla2_forward``."""
    import torch
    _sizes(q, v)
    B, H, n, d = q.shape
    dv = v.shape[-1]
    for t in (q, k, v, out, state_out):
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
    if state_out.dtype != torch.float32 or state_out.numel() != B * H * hla2_state_floats(d, dv):
        raise ValueError("state_out must be fp32 [B, H, state_floats]")
    need = hla2_forward_state_workspace_bytes(B, H, n, d, dv, chunk, segments)
    if workspace is None and need > 0:
        workspace = _scratch(need, q, stream)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().hla2_forward_state(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, H, n, d, dv, float(decay),
                                  int(bool(normalize)), int(chunk), _dtype_code(q), _ptr(den_out),
                                  _ptr(state_out), _ptr(workspace), wbytes, int(segments), _stream(stream))
    if check and rc != HLA2_OK:
        raise HLA2Error(rc, "hla2_forward_state")
    return rc


def hla2_backward_workspace_bytes(B, H, n, d, dv, normalize, dtype_code, segments=0) -> int:
    return int(lib().hla2_backward_workspace_bytes(B, H, n, d, dv, int(bool(normalize)), int(dtype_code), segments))


def hla2_backward(q, k, v, dout, grad_q, grad_k, grad_v, decay=1.0, normalize=False, out=None, den=None,
                  workspace=None, stream=None, segments=0, check=True) -> int:
    """Call ``hla2_backward``: gradients of sum(dout * out) w.r.t. q, k, v written to
    grad_q, grad_k: [B,H,n,d] and grad_v: [B,H,n,dv] (same dtype as q).  Under
    ``normalize`` the forward's ``out`` and fp32 ``den`` are required."""
    _sizes(q, v)
    B, H, n, d = q.shape
    dv = v.shape[-1]
    for t in (q, k, v, dout, grad_q, grad_k, grad_v) + ((out, den) if normalize else ()):
        if t is None or not t.is_contiguous():
            raise ValueError("tensors must be given and contiguous")
    code = _dtype_code(q)
    need = hla2_backward_workspace_bytes(B, H, n, d, dv, normalize, code, segments)
    if workspace is None and need > 0:
        workspace = _scratch(need, q, stream)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().hla2_backward(_ptr(q), _ptr(k), _ptr(v), _ptr(out) if normalize else None,
                             _ptr(den) if normalize else None, _ptr(dout), _ptr(grad_q), _ptr(grad_k), _ptr(grad_v),
                             B, H, n, d, dv, float(decay), int(bool(normalize)), code, _ptr(workspace), wbytes,
                             int(segments), _stream(stream))
    if check and rc != HLA2_OK:
        raise HLA2Error(rc, "hla2_backward")
    return rc


def hla2_ahla_forward_workspace_bytes(B, H, n, d, dv, dtype_code, segments=0) -> int:
    return int(lib().hla2_ahla_forward_workspace_bytes(B, H, n, d, dv, int(dtype_code), segments))


def hla2_ahla_forward(q, k, v, out, decay=1.0, normalize=False, den_out=None, workspace=None, stream=None,
                      segments=0, check=True) -> int:
    """Call ``hla2_ahla_forward`` (the asymmetric variant) on torch tensors q, k: [B,H,n,d];
    v, out: [B,H,n,dv]."""
    _sizes(q, v)
    B, H, n, d = q.shape
    dv = v.shape[-1]
    for t in (q, k, v, out):
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
    code = _dtype_code(q)
    need = hla2_ahla_forward_workspace_bytes(B, H, n, d, dv, code, segments)
    if workspace is None and need > 0:
        workspace = _scratch(need, q, stream)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().hla2_ahla_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, H, n, d, dv, float(decay),
                                 int(bool(normalize)), code, _ptr(den_out), _ptr(workspace), wbytes, int(segments),
                                 _stream(stream))
    if check and rc != HLA2_OK:
        raise HLA2Error(rc, "hla2_ahla_forward")
    return rc


def hla2_ho3_forward_workspace_bytes(B, H, n, d, dv, dtype_code, segments=0) -> int:
    return int(lib().hla2_ho3_forward_workspace_bytes(B, H, n, d, dv, int(dtype_code), segments))


def hla2_ho3_forward(q, k, v, out, decay=1.0, normalize=False, den_out=None, workspace=None, stream=None,
                     segments=0, check=True) -> int:
    """Call ``hla2_ho3_forward`` (third order) on torch tensors q, k: [B,H,n,d]; v, out: [B,H,n,dv]."""
    _sizes(q, v)
    B, H, n, d = q.shape
    dv = v.shape[-1]
    for t in (q, k, v, out):
        if not t.is_contiguous():
            raise ValueError("tensors must be contiguous")
    code = _dtype_code(q)
    need = hla2_ho3_forward_workspace_bytes(B, H, n, d, dv, code, segments)
    if workspace is None and need > 0:
        workspace = _scratch(need, q, stream)
    wbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    rc = lib().hla2_ho3_forward(_ptr(q), _ptr(k), _ptr(v), _ptr(out), B, H, n, d, dv, float(decay),
                                int(bool(normalize)), code, _ptr(den_out), _ptr(workspace), wbytes, int(segments),
                                _stream(stream))
    if check and rc != HLA2_OK:
        raise HLA2Error(rc, "hla2_ho3_forward")
    return rc


def hla2_decode_step(state, q, k, v, out, decay=1.0, normalize=False, stream=None, check=True) -> int:
    """Call ``hla2_decode_step``: state [N,H,state_floats] fp32 (in place);
    q, k: [N,H,d]; v, out: [N,H,dv]."""
    _sizes(q, v)
    N, H, d = q.shape
    dv = v.shape[-1]
    rc = lib().hla2_decode_step(_ptr(state), _ptr(q), _ptr(k), _ptr(v), _ptr(out), N, H, d, dv, float(decay),
                                int(bool(normalize)), _dtype_code(q), _stream(stream))
    if check and rc != HLA2_OK:
        raise HLA2Error(rc, "hla2_decode_step")
    return rc


def _launch(name, check, t, stream, *args):
    """The entry point `name`(*args, stream pointer) with t's device current (PyTorch's current stream of that
    device when no stream is given); tensors are passed by address, None as a null pointer."""
    import torch
    here = t.get_device()
    if here < 0:
        raise ValueError("tensors must be on the GPU")
    if stream is not None and getattr(stream, "device_index", here) != here:
        raise ValueError("stream must be one of the tensors' device")
    fn = getattr(_lib or lib(), name)
    # the raw handle, 0.2 us; building a Stream object for it takes 5 us, half of a small call
    s = torch._C._cuda_getCurrentRawStream(here) if stream is None else _stream(stream)
    if torch._C._cuda_getDevice() == here:
        rc = fn(*args, s)
    else:
        with torch.cuda.device(here):
            rc = fn(*args, s)
    if check and rc != HLA2_OK:
        raise HLA2Error(rc, name)
    return rc


def _at(t):
    """A tensor's address for an argument that may be absent."""
    return None if t is None else t.data_ptr()


def _expect(t, name, shape, dtype, device, optional=False):
    """A tensor argument as the C side takes it: contiguous, of this shape, type and device (an index)."""
    if t is None:
        if optional:
            return
        raise ValueError("%s must be given" % name)
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError("%s must be %s of shape %s, got %s of %s"
                         % (name, dtype, tuple(shape), t.dtype, tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    raise ValueError("%s must be on the device of the first tensor" % name)


def _expect_all(dtype, device, tensors):
    """_expect of each (tensor, name, shape) that must be given, in one loop: most of a small call's time on the
    host is such checks."""
    for t, name, shape in tensors:
        if t is None or t.dtype is not dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
            _expect(t, name, shape, dtype, device)


def _int(x, name):
    """x as a C int: ctypes would cut a larger one off silently."""
    x = int(x)
    if not -2147483648 <= x <= 2147483647:
        raise ValueError("%s must fit 32 bits, got %d" % (name, x))
    return x


def _sizes(*tensors):
    """The same for the sizes of tensors, which the calls take from their shapes."""
    for t in tensors:
        if t.numel() > 2147483647:  # else every size fits, or one is 0 and refused as that
            for size in t.shape:
                _int(size, "every size")


def _scratch(need, like, stream):
    """`need` bytes on like's device from the memory of the stream that the call runs on: what the allocator hands
    out there, and takes back when the call returns, is ordered with that stream's work alone.  (A block of the
    current stream's memory may still be in use by work that the given stream does not wait for.)"""
    import torch
    if stream is None or not like.is_cuda:
        return torch.empty(need, dtype=torch.uint8, device=like.device)
    handle = stream if isinstance(stream, int) else stream.cuda_stream
    with torch.cuda.stream(torch.cuda.ExternalStream(handle, device=like.device)):
        return torch.empty(need, dtype=torch.uint8, device=like.device)


def _workspace(workspace, need, like, stream):
    """(workspace tensor or None, its bytes); allocated here when the caller gives none."""
    if workspace is None:
        if need == 0:
            return None, 0
        workspace = _scratch(need, like, stream)
    elif not workspace.is_contiguous() or workspace.device != like.device:
        raise ValueError("workspace must be contiguous and on %s" % like.device)
    return workspace, workspace.numel() * workspace.element_size()


@functools.lru_cache(maxsize=256)
def hla2_gated_scan_workspace_bytes(B, H, n, d, dtype_code) -> int:
    sizes = (_int(x, "every size") for x in (B, H, n, d))
    return int(lib().hla2_gated_scan_workspace_bytes(*sizes, int(dtype_code)))


def _gated_shapes(x):
    import torch
    if x.dim() not in (3, 4):
        raise ValueError("x must be [B, H, n, d] or [B, n, d]")
    _sizes(x)
    B, n, d = x.shape[0], x.shape[-2], x.shape[-1]
    H = x.shape[1] if x.dim() == 4 else 1
    tiles = (n + HLA2_GATED_SCAN_TILE - 1) // HLA2_GATED_SCAN_TILE
    lead = x.shape[:-2]
    return B, H, n, d, (*lead, d), (*lead, tiles, d), torch.float32, torch.int32


def hla2_gated_scan_forward(x, g, out, gate=HLA2_GATE_LOG, s0=None, s_last=None, marks=None, lens=None,
                            workspace=None, stream=None, check=True) -> int:
    """Call ``hla2_gated_scan_forward`` on torch tensors x, g, out: [B,H,n,d] (or [B,n,d]).

    ``s0``, ``s_last``: fp32 [B,H,d] ([B,d]); ``marks``: fp32 [B,H,ceil(n/256),d], kept for the backward
    pass; ``lens``: int32 [B] on the device.  ``workspace`` as for ``hla2_forward``."""
    code = _dtype_code(x)
    B, H, n, d, ends, tiles, f32, i32 = _gated_shapes(x)
    shape, here = x.shape, x.get_device()
    _expect_all(x.dtype, here, ((x, "x", shape), (g, "g", shape), (out, "out", shape)))
    _expect(s0, "s0", ends, f32, here, True)
    _expect(s_last, "s_last", ends, f32, here, True)
    _expect(marks, "marks", tiles, f32, here, True)
    _expect(lens, "lens", (B,), i32, here, True)
    workspace, wbytes = _workspace(workspace, hla2_gated_scan_workspace_bytes(B, H, n, d, code), x, stream)
    return _launch("hla2_gated_scan_forward", check, x, stream, x.data_ptr(), g.data_ptr(), out.data_ptr(), _at(s0),
                   _at(s_last), _at(marks), _at(lens), B, H, n, d, _int(gate, "gate"), code, _at(workspace), wbytes)


def hla2_gated_scan_backward(x, g, dout, dx, dg, gate=HLA2_GATE_LOG, s0=None, marks=None, ds_last=None, ds0=None,
                             lens=None, workspace=None, stream=None, check=True) -> int:
    """Call ``hla2_gated_scan_backward``: gradients of sum(dout * out) + sum(ds_last * s_last) with respect to
    x, g and s0, written to dx, dg and ds0.  ``marks`` (from the forward call) is required when n > 256."""
    code = _dtype_code(x)
    B, H, n, d, ends, tiles, f32, i32 = _gated_shapes(x)
    shape, here = x.shape, x.get_device()
    _expect_all(x.dtype, here, ((x, "x", shape), (g, "g", shape), (dout, "dout", shape), (dx, "dx", shape),
                                (dg, "dg", shape)))
    for t, name in ((s0, "s0"), (ds_last, "ds_last"), (ds0, "ds0")):
        _expect(t, name, ends, f32, here, True)
    _expect(marks, "marks", tiles, f32, here, n <= HLA2_GATED_SCAN_TILE)
    _expect(lens, "lens", (B,), i32, here, True)
    workspace, wbytes = _workspace(workspace, hla2_gated_scan_workspace_bytes(B, H, n, d, code), x, stream)
    return _launch("hla2_gated_scan_backward", check, x, stream, x.data_ptr(), g.data_ptr(), _at(s0), _at(marks),
                   _at(lens), dout.data_ptr(), _at(ds_last), dx.data_ptr(), dg.data_ptr(), _at(ds0), B, H, n, d,
                   _int(gate, "gate"), code, _at(workspace), wbytes)


def hla2_gated_scan_step(state, x, g, out, gate=HLA2_GATE_LOG, pos=None, stream=None, check=True) -> int:
    """Call ``hla2_gated_scan_step``: state fp32 [N,H,d] (in place); x, g, out: [N,H,d] (or [N,d] throughout);
    ``pos``: int64 [N] on the device, negative for idle sequences."""
    import torch
    shape, here = x.shape, x.get_device()
    if len(shape) == 3:
        N, H, d = shape
    elif len(shape) == 2:
        (N, d), H = shape, 1
    else:
        raise ValueError("x must be [N, H, d] or [N, d]")
    _sizes(x)
    code = _dtype_code(x)
    _expect_all(x.dtype, here, ((x, "x", shape), (g, "g", shape), (out, "out", shape)))
    _expect(state, "state", shape, torch.float32, here)
    if pos is not None:
        _expect(pos, "pos", (N,), torch.int64, here)
    return _launch("hla2_gated_scan_step", check, x, stream, state.data_ptr(), x.data_ptr(), g.data_ptr(),
                   out.data_ptr(), _at(pos), N, H, d, _int(gate, "gate"), code)


def _window_shapes(q, k, v):
    """B, H, Hkv, n, d, dv of q [B,H,n,d], k [B,Hkv,n,d], v [B,Hkv,n,dv], checked against each other."""
    qs, ks, vs = q.shape, k.shape, v.shape
    if len(qs) != 4 or len(ks) != 4 or len(vs) != 4:
        raise ValueError("q, k, v must be [B, H, n, d], [B, Hkv, n, d], [B, Hkv, n, dv]")
    B, H, n, d = qs
    Hkv, dv = ks[1], vs[3]
    _sizes(q, k, v)
    _expect_all(q.dtype, q.get_device(), ((q, "q", qs), (k, "k", (B, Hkv, n, d)), (v, "v", (B, Hkv, n, dv))))
    return B, H, Hkv, n, d, dv


def hla2_window_forward(q, k, v, out, window, sinks=0, scale=None, lse=None, lens=None, stream=None,
                        check=True) -> int:
    """Call ``hla2_window_forward`` on torch tensors q: [B,H,n,d], k: [B,Hkv,n,d], v: [B,Hkv,n,dv],
    out: [B,H,n,dv]; ``scale`` 1/sqrt(d) when None; ``lse``: fp32 [B,H,n], kept for the backward pass;
    ``lens``: int32 [B] on the device."""
    import torch
    code, window, sinks = _dtype_code(q), _int(window, "window"), _int(sinks, "sinks")
    B, H, Hkv, n, d, dv = _window_shapes(q, k, v)
    here = q.get_device()
    _expect(out, "out", (B, H, n, dv), q.dtype, here)
    _expect(lse, "lse", (B, H, n), torch.float32, here, True)
    _expect(lens, "lens", (B,), torch.int32, here, True)
    scale = d ** -0.5 if scale is None else float(scale)
    return _launch("hla2_window_forward", check, q, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                   _at(lse), _at(lens), B, H, Hkv, n, d, dv, window, sinks, scale, code)


@functools.lru_cache(maxsize=256)
def hla2_window_backward_workspace_bytes(B, H, Hkv, n, d, dv, window, sinks, dtype_code) -> int:
    sizes = (_int(x, "every size") for x in (B, H, Hkv, n, d, dv, window, sinks))
    return int(lib().hla2_window_backward_workspace_bytes(*sizes, int(dtype_code)))


def hla2_window_backward(q, k, v, out, lse, dout, dq, dk, dv, window, sinks=0, scale=None, lens=None, workspace=None,
                         stream=None, check=True) -> int:
    """Call ``hla2_window_backward``: gradients of sum(dout * out) with respect to q, k, v, written to
    dq, dk, dv; ``out`` and ``lse`` are the forward call's.  ``workspace`` as for ``hla2_forward``."""
    import torch
    code, window, sinks = _dtype_code(q), _int(window, "window"), _int(sinks, "sinks")
    B, H, Hkv, n, d, dvd = _window_shapes(q, k, v)
    here = q.get_device()
    _expect_all(q.dtype, here, ((out, "out", (B, H, n, dvd)), (dout, "dout", (B, H, n, dvd)), (dq, "dq", q.shape),
                                (dk, "dk", k.shape), (dv, "dv", v.shape)))
    _expect(lse, "lse", (B, H, n), torch.float32, here)
    _expect(lens, "lens", (B,), torch.int32, here, True)
    scale = d ** -0.5 if scale is None else float(scale)
    need = hla2_window_backward_workspace_bytes(B, H, Hkv, n, d, dvd, window, sinks, code)
    workspace, wbytes = _workspace(workspace, need, q, stream)
    return _launch("hla2_window_backward", check, q, stream, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(),
                   _at(lse), dout.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _at(lens), B, H, Hkv, n, d,
                   dvd, window, sinks, scale, code, _at(workspace), wbytes)


def hla2_window_cache(k, v, cache_k, cache_v, window, sinks=0, lens=None, stream=None, check=True) -> int:
    """Call ``hla2_window_cache``: the cache [B,Hkv,window+sinks,d], [.., dv] after the tokens of k: [B,Hkv,n,d],
    v: [B,Hkv,n,dv], as ``hla2_window_step`` continues it."""
    import torch
    code, window, sinks = _dtype_code(k), _int(window, "window"), _int(sinks, "sinks")
    _, _, Hkv, n, d, dv = _window_shapes(k, k, v)
    B, slots = k.shape[0], window + sinks
    here = k.get_device()
    _expect_all(k.dtype, here, ((cache_k, "cache_k", (B, Hkv, slots, d)), (cache_v, "cache_v", (B, Hkv, slots, dv))))
    _expect(lens, "lens", (B,), torch.int32, here, True)
    return _launch("hla2_window_cache", check, k, stream, k.data_ptr(), v.data_ptr(), cache_k.data_ptr(),
                   cache_v.data_ptr(), _at(lens), B, Hkv, n, d, dv, window, sinks, code)


@functools.lru_cache(maxsize=256)
def hla2_window_step_workspace_bytes(N, H, Hkv, d, dv, window, sinks, dtype_code) -> int:
    sizes = (_int(x, "every size") for x in (N, H, Hkv, d, dv, window, sinks))
    return int(lib().hla2_window_step_workspace_bytes(*sizes, int(dtype_code)))


def hla2_window_step(cache_k, cache_v, pos, q, k, v, out, window, sinks=0, scale=None, workspace=None, stream=None,
                     check=True) -> int:
    """Call ``hla2_window_step``: token pos[i] (int64 [N] on the device; negative: idle) of each sequence,
    q: [N,H,d], k: [N,Hkv,d], v: [N,Hkv,dv], out: [N,H,dv]; the cache is updated in place."""
    import torch
    code, window, sinks = _dtype_code(q), _int(window, "window"), _int(sinks, "sinks")
    qs, ks, vs = q.shape, k.shape, v.shape
    if len(qs) != 3 or len(ks) != 3 or len(vs) != 3:
        raise ValueError("q, k, v must be [N, H, d], [N, Hkv, d], [N, Hkv, dv]")
    N, H, d = qs
    Hkv, dv, slots = ks[1], vs[2], window + sinks
    _sizes(q, k, v)
    here = q.get_device()
    _expect_all(q.dtype, here, ((q, "q", qs), (k, "k", (N, Hkv, d)), (v, "v", (N, Hkv, dv)),
                                (out, "out", (N, H, dv)), (cache_k, "cache_k", (N, Hkv, slots, d)),
                                (cache_v, "cache_v", (N, Hkv, slots, dv))))
    _expect(pos, "pos", (N,), torch.int64, here)
    scale = d ** -0.5 if scale is None else float(scale)
    need = hla2_window_step_workspace_bytes(N, H, Hkv, d, dv, window, sinks, code)
    workspace, wbytes = _workspace(workspace, need, q, stream)
    return _launch("hla2_window_step", check, q, stream, cache_k.data_ptr(), cache_v.data_ptr(), _at(pos),
                   q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), N, H, Hkv, d, dv, window, sinks, scale,
                   code, _at(workspace), wbytes)
