"""GB300 (sm_103a) decode-linear weight streaming: Python binding.

y[M, N] = x[M, K] . W[N, K]^T (+ bias) for M = 1..16 decode tokens, with bf16
weights or weight-only FP8 (e4m3, one fp32 scale per 128x128 block).  Every
step runs in the CUDA kernels of ``libdecode_linear.so`` behind the C ABI in
``include/dl_linear.h``; this module only checks torch tensors and passes raw
device pointers, sizes and the current stream through ctypes.  There is no CPU
fallback: if the library has not been built, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading
from dataclasses import dataclass

import torch

__all__ = [
    "BF16", "FP8_B128", "KERNEL_AUTO", "KERNEL_SIMT", "KERNEL_MMA", "DLError", "Layer",
    "library_path", "load", "version", "workspace_bytes", "Workspace", "linear_bf16",
    "linear_swiglu", "linear_argmax", "interleave_gate_up", "ABI_VERSION",
    "linear_bf16_static_scratch", "STATIC_SCRATCH_BYTES", "WORKSPACE_ZERO_BYTES",
    "linear_fp8_block128", "decode_stream", "decode_stream_workspace_bytes",
    "decode_stream_launches", "graph_cache_clear", "graph_cache_size", "set_wait_test",
    "set_override", "PagedKVCache", "kv_append", "attention_paged", "attention_workspace_bytes",
    "verify_draft",
    "device_status", "exported_symbols", "header_symbols",
]

BF16 = 0
FP8_B128 = 1
KERNEL_AUTO, KERNEL_SIMT, KERNEL_MMA, KERNEL_TC = 0, 1, 2, 3

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB_PATH = os.path.join(_HERE, "libdecode_linear.so")
_HEADER = os.path.join(os.path.dirname(_HERE), "include", "dl_linear.h")
_lock = threading.Lock()
_lib = None
_native: dict = {}       # the calls of _binding, once the library is loaded

_STATUS = {0: "DL_OK", 1: "DL_ERR_INVALID_ARG", 2: "DL_ERR_UNSUPPORTED_SHAPE",
           3: "DL_ERR_MISALIGNED", 4: "DL_ERR_WORKSPACE", 5: "DL_ERR_CUDA", 6: "DL_ERR_DEVICE"}


class DLError(RuntimeError):
    """A non-OK dl_status; ``.status`` holds the code."""

    def __init__(self, status: int, message: str):
        super().__init__(f"{_STATUS.get(status, status)}: {message}")
        self.status = status


class _Layer(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int), ("M", ctypes.c_int), ("N", ctypes.c_int),
                ("K", ctypes.c_int), ("x", ctypes.c_void_p), ("W", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("bias", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("act", ctypes.c_int)]

class _KVCache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("page_stride", ctypes.c_longlong),
                ("head_stride", ctypes.c_longlong), ("scale_page_stride", ctypes.c_longlong),
                ("scale_head_stride", ctypes.c_longlong), ("num_pages", ctypes.c_int),
                ("num_heads", ctypes.c_int), ("page_size", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("block", ctypes.c_int)]


ABI_VERSION = 4   # DL_VERSION this binding marshals for


def library_path() -> str:
    return _LIB_PATH


def load():
    """Load the shared library (raises if it is missing: there is no fallback)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(f"{_LIB_PATH} is missing: build it with "
                               "`python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(_LIB_PATH)
        vp, sz, i = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
        lib.dl_version.restype = i
        lib.dl_last_error.restype = ctypes.c_char_p
        lib.dl_workspace_bytes.argtypes = [i, i, i, i]
        lib.dl_workspace_bytes.restype = sz
        lib.dl_linear_bf16.argtypes = [vp, vp, vp, vp, vp, i, i, i, vp, sz, vp]
        lib.dl_linear_bf16.restype = i
        lib.dl_linear_fp8_block128.argtypes = [vp, vp, vp, vp, vp, vp, i, i, i, vp, sz, vp]
        lib.dl_linear_fp8_block128.restype = i
        lib.dl_decode_stream.argtypes = [ctypes.POINTER(_Layer), i, vp, sz, vp, i]
        lib.dl_decode_stream.restype = i
        lib.dl_graph_cache_clear.restype = None
        lib.dl_graph_cache_size.restype = i
        lib.dl_set_wait_test.argtypes = [ctypes.c_longlong, i]
        lib.dl_set_wait_test.restype = i
        lib.dl_decode_stream_workspace_bytes.argtypes = [ctypes.POINTER(_Layer), i]
        lib.dl_decode_stream_workspace_bytes.restype = sz
        lib.dl_decode_stream_launches.argtypes = [ctypes.POINTER(_Layer), i, sz]
        lib.dl_decode_stream_launches.restype = i
        lib.dl_linear_swiglu.argtypes = [i, vp, vp, vp, vp, vp, vp, i, i, i, vp, sz, vp]
        lib.dl_linear_argmax.argtypes = [i, vp, vp, vp, vp, vp, vp, vp, vp, i, i, i, vp, sz, vp]
        lib.dl_linear_argmax.restype = i
        lib.dl_linear_swiglu.restype = i
        lib.dl_attention_workspace_bytes.argtypes = [i, i, i, i, i, i]
        lib.dl_attention_workspace_bytes.restype = sz
        lib.dl_set_override.argtypes = [i, i, i]
        lib.dl_set_override.restype = i
        lib.dl_device_status.argtypes = [ctypes.POINTER(ctypes.c_uint)]
        lib.dl_device_status.restype = i
        if lib.dl_version() != ABI_VERSION:
            raise RuntimeError(f"{_LIB_PATH} is ABI version {lib.dl_version()}, this binding "
                               f"marshals version {ABI_VERSION}: rebuild the library")
        from . import _binding
        address = lambda f: ctypes.cast(f, vp).value   # noqa: E731
        _binding.bind(torch.Tensor, torch.bfloat16, torch.int32, torch.float32,
                      torch._C._cuda_getCurrentRawStream, address(lib.cudaGetDevice),
                      address(lib.dl_kv_append), address(lib.dl_attention_paged), address(lib.dl_verify_draft))
        _native.update(append=_binding.append, attention=_binding.attention, verify=_binding.verify)
        _lib = lib
        return lib


def _check(status: int):
    if status != 0:
        raise DLError(status, load().dl_last_error().decode(errors="replace"))


def version() -> int:
    return load().dl_version()


def header_symbols() -> list[str]:
    """Function names declared in include/dl_linear.h."""
    text = open(_HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(dl_[a-z0-9_]+)\s*\(", text)))


def exported_symbols() -> list[str]:
    lib = load()
    return [s for s in header_symbols() if hasattr(lib, s)]


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _handle(stream, device) -> int:
    """The address of the stream that a call runs on: a stream, an address, or None (the current one)."""
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    try:
        return int(getattr(stream, "cuda_stream", stream))
    except TypeError:
        raise ValueError("stream must be a stream or its address") from None


def _stream(stream, device):
    return ctypes.c_void_p(_handle(stream, device))


def _empty(shape, dtype, device, stream):
    """An output of a call that runs on `stream`.  It is that stream's memory, so that what the
    current stream has freed and may still use is not written, and it is held until the current
    stream, on which the caller goes on, has done with it."""
    if stream is None or device.type != "cuda":
        return torch.empty(shape, dtype=dtype, device=device)
    handle, current = _handle(stream, device), torch.cuda.current_stream(device)
    if handle == current.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(current)
    return t


def _need(t, name, dtype, device=None):
    if type(t) is torch.Tensor and t.dtype is dtype and t.is_contiguous() and \
            (t.is_cuda if device is None else t.device == device):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (there is no CPU path)")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def workspace_bytes(M: int, N: int, K: int, dtype: int) -> int:
    """Workspace one call needs on the current device (0 = invalid shape)."""
    return int(load().dl_workspace_bytes(M, N, K, dtype))


class Workspace:
    """A device buffer for the arrival counters (its first WORKSPACE_ZERO_BYTES,
    zero-filled here once; every call leaves them zero) and the calls' scratch
    (split-K partial sums, the FP8 activation copy).  Do not share one
    Workspace between streams that may run at the same time; a call without
    one takes the default of the stream that it runs on.
    """

    def __init__(self, nbytes: int, device="cuda"):
        self.nbytes = max(int(nbytes), 256)
        self.tensor = torch.zeros(self.nbytes, dtype=torch.uint8, device=device)
        # the zeros must be in place before a kernel on any stream reads them
        torch.cuda.synchronize(self.tensor.device)
        self.addr = self.tensor.data_ptr()

    @classmethod
    def for_shapes(cls, shapes, device="cuda"):
        """Workspace large enough for every (M, N, K, dtype) in `shapes`."""
        with torch.cuda.device(torch.device(device)):
            n = max(workspace_bytes(*s) for s in shapes)
        return cls(n, device)

    @classmethod
    def for_stream(cls, layers, device=None):
        """Workspace with which decode_stream makes the activation copies of all
        FP8 layers whose x no earlier layer writes in one launch at the start."""
        n = decode_stream_workspace_bytes(layers)
        return cls(n, device if device is not None else layers[0].x.device)

    def reset(self):
        self.tensor.zero_()
        torch.cuda.synchronize(self.tensor.device)

    @property
    def ptr(self):
        return ctypes.c_void_p(self.tensor.data_ptr())


_default_ws: dict = {}
_outgrown: list = []     # default workspaces that larger ones replaced: calls under way and graphs name them


def _workspace(ws, need: int, device, stream):
    """`ws`, or the default one of the stream that the call runs on."""
    if ws is not None:
        return ws
    key = (device.index, _handle(stream, device))
    cur = _default_ws.get(key)
    if cur is None or cur.nbytes < need:
        if cur is not None:
            _outgrown.append(cur)
        cur = Workspace(need, device)
        _default_ws[key] = cur
    return cur


def _out(out, out_f32, M, N, device, stream):
    if out is None:
        out = _empty((M, N), torch.bfloat16, device, stream)
    _need(out, "out", torch.bfloat16, device)
    if out.numel() != M * N:
        raise ValueError("out must hold M*N elements")
    if out_f32 is not None:
        _need(out_f32, "out_f32", torch.float32, device)
        if out_f32.numel() != M * N:
            raise ValueError("out_f32 must hold M*N elements")
    return out


def linear_bf16(x, w, bias=None, *, out=None, out_f32=None, workspace: Workspace | None = None,
                stream=None):
    """out[M, N] (bf16) = x[M, K] . w[N, K]^T (+ bias[N]); bf16 weights."""
    _need(x, "x", torch.bfloat16)
    dev = x.device
    _need(w, "w", torch.bfloat16, dev)
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, dev)
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError("x must be [M, K] and w [N, K]")
    M, K = x.shape
    N = w.shape[0]
    if bias is not None and bias.numel() != N:
        raise ValueError("bias must be [N]")
    out = _out(out, out_f32, M, N, dev, stream)
    with torch.cuda.device(dev):
        need = workspace_bytes(M, N, K, BF16)
        ws = _workspace(workspace, need, dev, stream)
        _check(load().dl_linear_bf16(_ptr(x), _ptr(w), _ptr(bias), _ptr(out), _ptr(out_f32),
                                     M, N, K, ws.ptr, ws.nbytes, _stream(stream, dev)))
    return out


def linear_swiglu(x, w, scales=None, bias=None, *, out=None, out_f32=None,
                  workspace: Workspace | None = None, stream=None):
    """out[M, N/2] = silu(g) * u: gate_up projection with the SwiGLU epilogue.

    w: [N, K] bf16, or e4m3 codes (uint8 / float8_e4m3fn) with fp32 `scales`,
    its gate and up rows interleaved in groups of 16 (rows 16b..16b+7 gate,
    16b+8..16b+15 up, of outputs 8b..8b+7); see interleave_gate_up.
    """
    if isinstance(w, torch.Tensor) and w.dtype == torch.float8_e4m3fn:
        w = w.view(torch.uint8)
    _need(x, "x", torch.bfloat16)
    dev = x.device
    fp8 = scales is not None
    _need(w, "w", torch.uint8 if fp8 else torch.bfloat16, dev)
    if fp8:
        _need(scales, "scales", torch.float32, dev)
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, dev)
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError("x must be [M, K] and w [N, K]")
    M, K = x.shape
    N = w.shape[0]
    if N % 16:
        raise ValueError("SwiGLU needs N % 16 == 0")
    out = _out(out, out_f32, M, N // 2, dev, stream)
    dt = FP8_B128 if fp8 else BF16
    with torch.cuda.device(dev):
        ws = _workspace(workspace, workspace_bytes(M, N, K, dt), dev, stream)
        _check(load().dl_linear_swiglu(dt, _ptr(x), _ptr(w), _ptr(scales), _ptr(bias), _ptr(out),
                                       _ptr(out_f32), M, N, K, ws.ptr, ws.nbytes, _stream(stream, dev)))
    return out


def linear_argmax(x, w, scales=None, bias=None, *, out_idx=None, out_max=None, out=None,
                  out_f32=None, workspace: Workspace | None = None, stream=None):
    """idx[M] (int32) = argmax over n of x . w^T (+ bias), lowest index among
    ties, decided on the fp32 values (NaN largest).  out_max (fp32 [M]) gets the
    largest value; out / out_f32 get the logits only if given."""
    if isinstance(w, torch.Tensor) and w.dtype == torch.float8_e4m3fn:
        w = w.view(torch.uint8)
    _need(x, "x", torch.bfloat16)
    dev = x.device
    fp8 = scales is not None
    _need(w, "w", torch.uint8 if fp8 else torch.bfloat16, dev)
    if fp8:
        _need(scales, "scales", torch.float32, dev)
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, dev)
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError("x must be [M, K] and w [N, K]")
    M, K = x.shape
    N = w.shape[0]
    if out_idx is None:
        out_idx = _empty((M,), torch.int32, dev, stream)
    _need(out_idx, "out_idx", torch.int32, dev)
    if out_max is not None:
        _need(out_max, "out_max", torch.float32, dev)
    if out is not None:
        _need(out, "out", torch.bfloat16, dev)
    if out_f32 is not None:
        _need(out_f32, "out_f32", torch.float32, dev)
    dt = FP8_B128 if fp8 else BF16
    with torch.cuda.device(dev):
        ws = _workspace(workspace, workspace_bytes(M, N, K, dt), dev, stream)
        _check(load().dl_linear_argmax(dt, _ptr(x), _ptr(w), _ptr(scales), _ptr(bias), _ptr(out_idx),
                                       _ptr(out_max), _ptr(out), _ptr(out_f32), M, N, K, ws.ptr,
                                       ws.nbytes, _stream(stream, dev)))
    return out_idx


def interleave_gate_up(gate: torch.Tensor, up: torch.Tensor) -> torch.Tensor:
    """[I, K] gate and up matrices (any dtype) -> the [2I, K] row order of
    linear_swiglu: rows 16b..16b+7 = gate rows 8b..8b+7, rows 16b+8..16b+15 =
    the matching up rows.  I % 8 == 0.  A one-time layout step for weights
    (plain tensor indexing, not part of the decode path)."""
    if gate.shape != up.shape or gate.shape[0] % 8:
        raise ValueError("gate and up must have the same [I, K] shape, I % 8 == 0")
    I, K = gate.shape
    return torch.stack([gate.reshape(I // 8, 8, K), up.reshape(I // 8, 8, K)], dim=1).reshape(2 * I, K)


STATIC_SCRATCH_BYTES = 16 << 20   # DL_STATIC_SCRATCH_BYTES of include/dl_linear.h
WORKSPACE_ZERO_BYTES = 256 + 16384 * 4   # DL_WORKSPACE_ZERO_BYTES: zero before the first call


def linear_bf16_static_scratch(x, w, bias=None, *, out, out_f32=None, stream=None):
    """linear_bf16 through dl_linear_bf16_static_scratch: no workspace argument;
    the library's static device scratch (STATIC_SCRATCH_BYTES per device) holds
    the split-K state and nothing is allocated on the call path, so `out` (and
    `out_f32`, if wanted) must be passed in.  Calls that may overlap on the GPU
    share that scratch and race; calls ordered on one stream do not."""
    if out is None:
        raise ValueError("out is required: this entry point allocates nothing")
    _need(x, "x", torch.bfloat16)
    dev = x.device
    _need(w, "w", torch.bfloat16, dev)
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, dev)
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError("x must be [M, K] and w [N, K]")
    M, K = x.shape
    N = w.shape[0]
    if bias is not None and bias.numel() != N:
        raise ValueError("bias must be [N]")
    out = _out(out, out_f32, M, N, dev, stream)
    lib = load()
    fn = lib.dl_linear_bf16_static_scratch
    vp, i = ctypes.c_void_p, ctypes.c_int
    fn.argtypes = [vp, vp, vp, vp, vp, i, i, i, vp]
    fn.restype = i
    with torch.cuda.device(dev):
        _check(fn(_ptr(x), _ptr(w), _ptr(bias), _ptr(out), _ptr(out_f32), M, N, K,
                  _stream(stream, dev)))
    return out


def linear_fp8_block128(x, wq, scales, bias=None, *, out=None, out_f32=None,
                        workspace: Workspace | None = None, stream=None):
    """out[M, N] (bf16) = x . (e4m3(wq) * scales[n/128, k/128])^T (+ bias).

    wq: uint8 e4m3 codes [N, K] (a torch.float8_e4m3fn tensor is accepted and
    viewed as bytes); scales: fp32 [ceil(N/128), K/128].
    """
    if isinstance(wq, torch.Tensor) and wq.dtype == torch.float8_e4m3fn:
        wq = wq.view(torch.uint8)
    _need(x, "x", torch.bfloat16)
    dev = x.device
    _need(wq, "wq", torch.uint8, dev)
    _need(scales, "scales", torch.float32, dev)
    if bias is not None:
        _need(bias, "bias", torch.bfloat16, dev)
    if x.dim() != 2 or wq.dim() != 2 or x.shape[1] != wq.shape[1]:
        raise ValueError("x must be [M, K] and wq [N, K]")
    M, K = x.shape
    N = wq.shape[0]
    if scales.numel() != ((N + 127) // 128) * ((K + 127) // 128):
        raise ValueError("scales must be [ceil(N/128), ceil(K/128)]")
    if bias is not None and bias.numel() != N:
        raise ValueError("bias must be [N]")
    out = _out(out, out_f32, M, N, dev, stream)
    with torch.cuda.device(dev):
        need = workspace_bytes(M, N, K, FP8_B128)
        ws = _workspace(workspace, need, dev, stream)
        _check(load().dl_linear_fp8_block128(_ptr(x), _ptr(wq), _ptr(scales), _ptr(bias),
                                             _ptr(out), _ptr(out_f32), M, N, K, ws.ptr,
                                             ws.nbytes, _stream(stream, dev)))
    return out


@dataclass
class Layer:
    """One entry of a decode weight stream (all tensors on one CUDA device)."""

    dtype: int
    x: torch.Tensor
    w: torch.Tensor
    y: torch.Tensor
    scales: torch.Tensor | None = None
    bias: torch.Tensor | None = None
    act: int = 0          # 1: SwiGLU epilogue (see linear_swiglu): y is [M, N/2];
                          # 2: argmax (see linear_argmax): y is int32 [M], no logits

    def shape(self):
        return (self.x.shape[0], self.w.shape[0], self.x.shape[1], self.dtype)


def _layer_struct(L: Layer) -> _Layer:
    M, N, K, dt = L.shape()
    w = L.w.view(torch.uint8) if L.w.dtype == torch.float8_e4m3fn else L.w
    for t, n in ((L.x, "x"), (w, "w"), (L.y, "y")):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"layer {n} must be a contiguous CUDA tensor")
    return _Layer(dt, M, N, K, L.x.data_ptr(), w.data_ptr(),
                  None if L.scales is None else L.scales.data_ptr(),
                  None if L.bias is None else L.bias.data_ptr(), L.y.data_ptr(), int(L.act))


def decode_stream(layers, workspace: Workspace, *, use_graph: bool = False, stream=None):
    """Run the layers back to back on one stream (optionally as a cached CUDA graph)."""
    arr = (_Layer * max(1, len(layers)))(*[_layer_struct(L) for L in layers])
    dev = layers[0].x.device if layers else torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        _check(load().dl_decode_stream(arr, len(layers), workspace.ptr, workspace.nbytes,
                                       _stream(stream, dev), 1 if use_graph else 0))


def decode_stream_workspace_bytes(layers) -> int:
    """Workspace bytes for decode_stream over `layers` with the FP8 activation
    copies made without per-layer prep launches where possible: ahead for the
    layers whose x is ready at the start, by the layer before for a layer fed
    by a plain linear's whole y (see dl_linear.h)."""
    arr = (_Layer * max(1, len(layers)))(*[_layer_struct(L) for L in layers])
    dev = layers[0].x.device if layers else torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        n = load().dl_decode_stream_workspace_bytes(arr, len(layers))
    if n == 0:
        raise ValueError("invalid layer list: " + load().dl_last_error().decode())
    return n


def decode_stream_launches(layers, workspace: Workspace) -> int:
    """Kernels one decode_stream call over `layers` enqueues with this workspace."""
    arr = (_Layer * max(1, len(layers)))(*[_layer_struct(L) for L in layers])
    dev = layers[0].x.device if layers else torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        n = load().dl_decode_stream_launches(arr, len(layers), workspace.nbytes)
    if n < 0:
        raise ValueError("invalid layer list: " + load().dl_last_error().decode())
    return n


class PagedKVCache:
    """A paged cache of keys and values in 8 bits (see dl_kv_cache in dl_linear.h).

    k, v              e4m3 codes (uint8 or float8_e4m3fn) [num_pages, kv_heads, page_size, head_dim];
                      a page's tokens and dims are dense, its page and head strides are free
                      (multiples of 16, the same for both), so k and v may be views of one buffer
    k_scale, v_scale  fp32 [num_pages, kv_heads, page_size // block], dense in the last dim: one
                      scale for each block of tokens and head

    The object holds the tensors and is made once; the calls below read and
    write them in place.  ``PagedKVCache.empty`` makes them.
    """

    def __init__(self, k, v, k_scale, v_scale):
        for t, n in ((k, "k"), (v, "v"), (k_scale, "k_scale"), (v_scale, "v_scale")):
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{n} must be a torch.Tensor")
            if not t.is_cuda or t.device != k.device:
                raise ValueError("the cache must be CUDA tensors of one device (there is no CPU path)")
        # one page, or one head, has no next one: its stride says nothing
        steps = lambda t: [s for s, n in zip(t.stride(), t.shape) if n != 1]   # noqa: E731
        for t, n in ((k, "k"), (v, "v")):
            if t.dtype not in (torch.uint8, torch.float8_e4m3fn):
                raise ValueError(f"{n} must be e4m3 codes (uint8 or float8_e4m3fn), got {t.dtype}")
            if t.dim() != 4 or t.shape != k.shape or steps(t) != steps(k):
                raise ValueError("k and v must be [num_pages, kv_heads, page_size, head_dim] with equal strides")
            if t.numel() and (t.stride(3) != 1 or t.stride(2) != t.shape[3]):
                raise ValueError(f"a page of {n} must be dense in its tokens and dims")
        pages, heads, page, dim = k.shape
        for t, n in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t.dtype != torch.float32:
                raise ValueError(f"{n} must be torch.float32, got {t.dtype}")
            if t.dim() != 3 or t.shape != k_scale.shape or steps(t) != steps(k_scale) or \
                    t.shape[:2] != (pages, heads) or t.shape[2] < 1 or page % t.shape[2]:
                raise ValueError("k_scale and v_scale must be [num_pages, kv_heads, page_size // block] "
                                 "with equal strides")
            if t.shape[2] > 1 and t.stride(2) != 1:
                raise ValueError(f"{n} must be dense in its last dim")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = pages, heads, page, dim
        self.block = page // k_scale.shape[2]
        self.device = k.device
        blocks = k_scale.shape[2]
        self._struct = _KVCache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                                k.stride(0) if pages > 1 else heads * page * dim,
                                k.stride(1) if heads > 1 else page * dim,
                                k_scale.stride(0) if pages > 1 else heads * blocks,
                                k_scale.stride(1) if heads > 1 else blocks,
                                pages, heads, page, dim, self.block)
        # what a call passes of it: its description's address, its device, heads and dims
        self._args = (ctypes.addressof(self._struct), self.device.index, heads, dim)

    @classmethod
    def empty(cls, num_pages, kv_heads, head_dim, *, page_size=64, block=16, device="cuda"):
        """A cache with nothing in it (codes and scales zero)."""
        shape = (num_pages, kv_heads, page_size, head_dim)
        k, v = (torch.zeros(shape, dtype=torch.uint8, device=device) for _ in range(2))
        ks, vs = (torch.zeros((num_pages, kv_heads, page_size // block), dtype=torch.float32,
                              device=device) for _ in range(2))
        return cls(k, v, ks, vs)


def _call(name, device, *args):
    """A call of _binding: True once it is enqueued, False if an argument is not in order (nothing was
    called then); raises for a call that the library refuses."""
    if not _native:
        load()
    fn = _native[name]
    status = fn(*args)
    if status == -2:                # another device is current
        with torch.cuda.device(device):
            status = fn(*args)
    if status > 0:
        _check(status)
    return status == 0


def _need_sequences(cache, block_table, seq_lens, q_start):
    dev = cache.device
    _need(block_table, "block_table", torch.int32, dev)
    _need(seq_lens, "seq_lens", torch.int32, dev)
    _need(q_start, "q_start", torch.int32, dev)
    B = seq_lens.numel()
    if block_table.dim() != 2 or block_table.shape[0] != B or q_start.numel() != B + 1:
        raise ValueError("block_table must be [batch, pages], seq_lens [batch], q_start [batch + 1]")


def _need_rows(t, name, heads, dim, device):
    """bf16 [tokens, heads, dim], a token's heads dense, any stride between tokens; returns tokens."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must be a CUDA tensor on {device} (there is no CPU path)")
    if t.dim() != 3 or t.shape[2] != dim or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [tokens, {'heads' if heads is None else heads}, {dim}]")
    if t.numel() and (t.stride(2) != 1 or (t.shape[1] > 1 and t.stride(1) != dim)):
        raise ValueError(f"{name} must be dense in a token's heads and dims")
    return t.shape[0]


def kv_append(q, k, v, cache: PagedKVCache, block_table, seq_lens, q_start, *, max_q: int, cos=None,
              sin=None, positions=None, out_q=None, stream=None):
    """Rotate the new tokens' queries and keys and append keys and values to `cache`.

    q [tokens, q_heads, head_dim] (or None), k, v [tokens, kv_heads, head_dim]: bf16, possibly
    views of the fused QKV output.  seq_lens [batch] counts the cached tokens including the
    new ones, which are rows q_start[b] .. q_start[b + 1] - 1; max_q bounds a sequence's new
    tokens.  cos, sin: fp32 [positions, rotary_dim / 2] (None: no rotation); positions: int32
    [tokens] (None: the place in the cache).  Returns the rotated queries (`out_q`, which may
    be q; None without q).  See dl_kv_append for the scales and the rounding.
    """
    if q is not None and out_q is None and isinstance(q, torch.Tensor):
        out_q = torch.empty_like(q, memory_format=torch.contiguous_format) if stream is None else \
            _empty(q.shape, q.dtype, q.device, stream)
    if not _call("append", cache.device, *cache._args, q, k, v, block_table, seq_lens, q_start, max_q, cos, sin,
                 positions, out_q, stream):
        _explain_append(q, k, v, cache, block_table, seq_lens, q_start, cos, sin, positions, out_q)
    return out_q


def _explain_append(q, k, v, cache, block_table, seq_lens, q_start, cos, sin, positions, out_q):
    """Raise for the first argument of a kv_append call that is not in order."""
    dev, D = cache.device, cache.head_dim
    T = _need_rows(k, "k", cache.kv_heads, D, dev)
    Tq = Tv = _need_rows(v, "v", cache.kv_heads, D, dev)
    _need_sequences(cache, block_table, seq_lens, q_start)
    if q is not None:
        Tq = _need_rows(q, "q", None, D, dev)
        _need(out_q, "out_q", torch.bfloat16, dev)
    elif out_q is not None:
        raise ValueError("out_q needs q")
    if Tv != T or Tq != T or (q is not None and out_q.shape != q.shape):
        raise ValueError("q, k, v and out_q must have the same tokens")
    if cos is not None or sin is not None:
        _need(cos, "cos", torch.float32, dev)
        _need(sin, "sin", torch.float32, dev)
        if cos.dim() != 2 or cos.shape != sin.shape:
            raise ValueError("cos and sin must be [positions, rotary_dim / 2]")
    if positions is not None:
        _need(positions, "positions", torch.int32, dev)
        if positions.numel() != T:
            raise ValueError("positions must be [tokens]")
    raise ValueError("max_q and stream must be integers, sizes below 2^31")


def attention_workspace_bytes(batch: int, tokens: int, q_heads: int, kv_heads: int, head_dim: int,
                              *, max_q: int) -> int:
    """Workspace attention_paged needs on the current device (0 = invalid sizes)."""
    return int(load().dl_attention_workspace_bytes(batch, tokens, q_heads, kv_heads, head_dim, max_q))


def attention_paged(q, cache: PagedKVCache, block_table, seq_lens, q_start, *, max_q: int, scale=None,
                    out=None, out_lse=None, workspace: Workspace | None = None, stream=None):
    """Attention of the new tokens (q, bf16 [tokens, q_heads, head_dim]) over `cache`, which
    already holds them; causal among them.  Returns out, bf16 like q but dense; out_lse (fp32
    [tokens, q_heads]) gets the log-sum-exp of the scaled scores.  scale: head_dim ** -0.5 if
    None.  The sequences are described as for kv_append; see dl_attention_paged.
    """
    if not isinstance(q, torch.Tensor):
        raise TypeError("q must be a torch.Tensor")
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format) if stream is None else \
            _empty(q.shape, q.dtype, q.device, stream)
    if workspace is None:
        _explain_attention(q, cache, block_table, seq_lens, q_start, out, out_lse)
        with torch.cuda.device(cache.device):
            workspace = _workspace(None, attention_workspace_bytes(
                seq_lens.numel(), q.shape[0], q.shape[1], cache.kv_heads, cache.head_dim, max_q=max_q), cache.device,
                stream)
    elif workspace.tensor.device != cache.device:
        raise ValueError(f"workspace is on {workspace.tensor.device}, expected {cache.device}")
    if not _call("attention", cache.device, *cache._args, q, block_table, seq_lens, q_start, max_q,
                 cache.head_dim ** -0.5 if scale is None else scale, out, out_lse, workspace.addr,
                 workspace.nbytes, stream):
        _explain_attention(q, cache, block_table, seq_lens, q_start, out, out_lse)
        raise ValueError("max_q and stream must be integers, scale a number, sizes below 2^31")
    return out


def _explain_attention(q, cache, block_table, seq_lens, q_start, out, out_lse):
    """Raise for the first argument of an attention_paged call that is not in order."""
    dev, D = cache.device, cache.head_dim
    T = _need_rows(q, "q", None, D, dev)
    _need_sequences(cache, block_table, seq_lens, q_start)
    _need(out, "out", torch.bfloat16, dev)
    if out.numel() != q.numel():
        raise ValueError("out must hold tokens * q_heads * head_dim elements")
    if out_lse is not None:
        _need(out_lse, "out_lse", torch.float32, dev)
        if out_lse.numel() != T * q.shape[1]:
            raise ValueError("out_lse must hold tokens * q_heads elements")


def verify_draft(draft_tokens, target_probs, u_accept, u_next, *, draft_probs=None, draft_lens=None,
                 out_tokens=None, out_count=None, stream=None):
    """Accept a prefix of the drafted tokens and draw the next one (see dl_verify_draft).

    draft_tokens int32 [batch, drafts]; target_probs [batch, drafts + 1, vocab] and draft_probs
    [batch, drafts, vocab] (None: the draft was deterministic), both fp32 or both bf16;
    u_accept fp32 [batch, drafts] and u_next fp32 [batch], random numbers in [0, 1);
    draft_lens int32 [batch] or None.  Returns (tokens int32 [batch, drafts + 1]: accepted
    tokens, the next one, then -1; count int32 [batch]: how many were accepted).
    """
    if not isinstance(target_probs, torch.Tensor) or not isinstance(draft_tokens, torch.Tensor):
        raise TypeError("target_probs and draft_tokens must be torch.Tensors")
    if not target_probs.is_cuda:
        raise ValueError("target_probs must be a CUDA tensor (there is no CPU path)")
    if draft_tokens.dim() != 2:
        raise ValueError("draft_tokens must be [batch, drafts]")
    dev, (B, S) = target_probs.device, draft_tokens.shape
    if out_tokens is None:
        out_tokens = torch.empty((B, S + 1), dtype=torch.int32, device=dev) if stream is None else \
            _empty((B, S + 1), torch.int32, dev, stream)
    if out_count is None:
        out_count = torch.empty((B,), dtype=torch.int32, device=dev) if stream is None else \
            _empty((B,), torch.int32, dev, stream)
    if not _call("verify", dev, dev.index, draft_tokens, target_probs, u_accept, u_next, draft_probs, draft_lens,
                 out_tokens, out_count, stream):
        _explain_verify(draft_tokens, target_probs, u_accept, u_next, draft_probs, draft_lens, out_tokens, out_count)
    return out_tokens, out_count


def _explain_verify(draft_tokens, target_probs, u_accept, u_next, draft_probs, draft_lens, out_tokens, out_count):
    """Raise for the first argument of a verify_draft call that is not in order."""
    kind, dev, (B, S) = target_probs.dtype, target_probs.device, draft_tokens.shape
    if kind not in (torch.float32, torch.bfloat16):
        raise ValueError(f"target_probs must be torch.float32 or torch.bfloat16, got {kind}")
    _need(target_probs, "target_probs", kind)
    _need(draft_tokens, "draft_tokens", torch.int32, dev)
    _need(u_accept, "u_accept", torch.float32, dev)
    _need(u_next, "u_next", torch.float32, dev)
    if target_probs.dim() != 3 or target_probs.shape[:2] != (B, S + 1):
        raise ValueError("target_probs must be [batch, drafts + 1, vocab]")
    if u_accept.numel() != B * S or u_next.numel() != B:
        raise ValueError("u_accept must be [batch, drafts] and u_next [batch]")
    if draft_probs is not None:
        _need(draft_probs, "draft_probs", kind, dev)
        if draft_probs.shape != (B, S, target_probs.shape[2]):
            raise ValueError("draft_probs must be [batch, drafts, vocab]")
    if draft_lens is not None:
        _need(draft_lens, "draft_lens", torch.int32, dev)
        if draft_lens.numel() != B:
            raise ValueError("draft_lens must be [batch]")
    _need(out_tokens, "out_tokens", torch.int32, dev)
    _need(out_count, "out_count", torch.int32, dev)
    if out_tokens.numel() != B * (S + 1) or out_count.numel() != B:
        raise ValueError("out_tokens must be [batch, drafts + 1] and out_count [batch]")
    raise ValueError("stream must be an integer or a stream, sizes below 2^31")


def graph_cache_clear():
    load().dl_graph_cache_clear()


def graph_cache_size() -> int:
    """Graphs currently cached by decode_stream(use_graph=True)."""
    return int(load().dl_graph_cache_size())


def set_wait_test(wait_limit_ns: int = 0, withhold_stage: int = 0):
    """Test hooks of the bounded device waits (see dl_set_wait_test): the wait
    limit of later launches and a stage CTA 0 withholds; (0, 0) turns them off."""
    _check(load().dl_set_wait_test(int(wait_limit_ns), int(withhold_stage)))


def set_override(kernel: int = 0, ctas_per_sm: int = 0, max_ctas: int = 0):
    """Force a kernel family / grid shape (0 = automatic).  Process-wide."""
    _check(load().dl_set_override(kernel, ctas_per_sm, max_ctas))


def device_status() -> int:
    """Synchronise, read and clear the device error word; returns it (0 = no error)."""
    flags = ctypes.c_uint(0)
    st = load().dl_device_status(ctypes.byref(flags))
    if st != 0 and st != 6:
        _check(st)
    return int(flags.value)
