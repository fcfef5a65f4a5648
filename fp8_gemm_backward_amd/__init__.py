"""Backward of block-scaled low-precision linear and grouped matmuls on MI355X.

A thin Python binding over the C-ABI library `liblp.so` (declared in
`include/lp.h`).  The functions below keep the C names; they only marshal
torch tensors (device memory) and the current HIP stream into the C calls.
With stream= (a torch stream or a raw handle) a call runs on that stream, and
what it allocates comes from that stream's memory; the caller orders his own
tensors, the results among them, between the streams.
Every step of the computation runs in the library's HIP kernels; there is no
fallback, and importing this package fails if the library is not built
(`python fp8_gemm_backward_amd/build.py`).

Formats (see include/lp.h): "bf16", "mxfp4", "nvfp4", "fp8_b128", "mxfp8",
the per-tensor scaled "fp8t_e4m3", "fp8t_e5m2", and "fp8_r128" (E4M3 with an
fp32 scale per run of 128, the counterpart of an "fp8_b128" weight in FP8
products).  include/lp_train.h declares the quantizers of the last two, the
forwards that quantize their own input, and the AdamW step.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
import re
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblp.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "lp.h")

FMT = {"bf16": 0, "mxfp4": 1, "nvfp4": 2, "fp8_b128": 3, "mxfp8": 4, "fp8t_e4m3": 5, "fp8t_e5m2": 6, "fp8_r128": 8}
STATUS = {0: "LP_OK", 1: "LP_ERR_NULL", 2: "LP_ERR_SHAPE", 3: "LP_ERR_FORMAT", 4: "LP_ERR_ALIGN",
          5: "LP_ERR_HIP"}


class LpError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)}")


class _QTensorC(ctypes.Structure):
    _fields_ = [("fmt", ctypes.c_int32), ("scale_axis", ctypes.c_int32), ("batch", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("codes", ctypes.c_void_p),
                ("scales", ctypes.c_void_p), ("tensor_scale", ctypes.c_void_p)]


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run `python fp8_gemm_backward_amd/build.py`")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.POINTER(_QTensorC)
    v = ctypes.c_void_p
    i64, i32 = ctypes.c_int64, ctypes.c_int32
    lib.lp_dequant.argtypes = [P, v, v]
    lib.lp_mx_quant.argtypes = [v, i64, i64, i64, i32, i32, v, v, v]
    lib.lp_mx_quant_dual.argtypes = [v, i64, i64, i64, i32, v, v, v, v, v]
    lib.lp_linear_bwd.argtypes = [P, P, P, v, v, v]
    lib.lp_grouped_bwd.argtypes = [P, P, P, v, i64, v, v, v]
    lib.lp_linear_bwd_workspace.argtypes = [P, P, P, v, v, ctypes.POINTER(ctypes.c_size_t)]
    lib.lp_linear_bwd_ws.argtypes = [P, P, P, v, v, v, ctypes.c_size_t, v]
    lib.lp_linear_bwd_noalloc.argtypes = [P, P, P, v, v, v]
    lib.lp_grouped_dx_deferred.argtypes = [P, v, i64, v, i64, i64, v, v, v, v]
    lib.lp_tensor_amax.argtypes = [v, i64, v, v]
    lib.lp_tensor_quant.argtypes = [v, i64, i32, v, v, v, v]
    lib.lp_scale_from_history.argtypes = [v, i32, i32, i32, v, v]
    lib.lp_tensor_quant_delayed.argtypes = [v, i64, i32, v, i32, i32, i32, v, v, v]
    lib.lp_linear_fwd.argtypes = [P, P, v, v]
    lib.lp_grouped_fwd.argtypes = [P, P, v, i64, v, v]
    lib.lp_r128_quant.argtypes = [v, i64, i64, i64, i32, v, i64, v, v, v]
    lib.lp_r128_quant_dual.argtypes = [v, i64, i64, i64, v, i64, v, v, v, v, v]
    lib.lp_b128_quant.argtypes = [v, i64, i64, i64, v, v, v]
    lib.lp_linear_fwd_dyn.argtypes = [v, i64, P, v, v, v, v]
    lib.lp_grouped_fwd_dyn.argtypes = [v, i64, P, v, i64, v, v, v, v]
    f64 = ctypes.c_double
    lib.lp_adamw_plan.argtypes = [v, i64, i32, i32, i32, v, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(i64)]
    lib.lp_adamw.argtypes = [v, i64, i64, i32, i32, i32, f64, f64, f64, f64, i64, v, v]
    lib.lp_status_string.argtypes = [i32]
    lib.lp_status_string.restype = ctypes.c_char_p
    for f in ("lp_dequant", "lp_mx_quant", "lp_mx_quant_dual", "lp_linear_bwd", "lp_grouped_bwd",
              "lp_linear_bwd_workspace", "lp_linear_bwd_ws", "lp_linear_bwd_noalloc", "lp_grouped_dx_deferred", "lp_tensor_amax", "lp_tensor_quant",
              "lp_scale_from_history", "lp_linear_fwd", "lp_grouped_fwd", "lp_tensor_quant_delayed",
              "lp_r128_quant", "lp_r128_quant_dual", "lp_b128_quant", "lp_linear_fwd_dyn", "lp_grouped_fwd_dyn",
              "lp_adamw_plan", "lp_adamw"):
        getattr(lib, f).restype = ctypes.c_int32
    return lib


lib = _load()


_CODE_BITS = {"bf16": 16, "mxfp4": 4, "nvfp4": 4, "fp8_b128": 8, "mxfp8": 8, "fp8t_e4m3": 8, "fp8t_e5m2": 8,
              "fp8_r128": 8}
_NAMES = {f: (f"{f} codes", f"{f} scales", f"{f} tensor scale") for f in FMT}


def _scale_bytes(fmt: str, axis: int, b: int, r: int, c: int, groups: int = 0) -> int:
    """Bytes of scales that a call reads, over `groups` groups of rows (0: a call without offsets)."""
    """Bytes of a tensor's block scales (include/lp.h, formats)."""
    if fmt == "mxfp4" or (fmt == "mxfp8" and axis == -1):
        return b * r * (c // 32)
    if fmt == "mxfp8":
        return b * (r // 32) * c
    if fmt == "nvfp4":
        return b * r * (c // 16)
    if fmt == "fp8_b128":
        return b * (-(-r // 128)) * (-(-c // 128)) * 4
    if fmt == "fp8_r128":
        if axis == -1:
            return 4 * b * (-(-c // 128)) * r
        # Runs that restart at every group: group g's begin at its first row / 128 + g.
        return 4 * b * (r // 128 + groups if groups > 1 else -(-r // 128)) * c
    return 0


def _device(t: Optional[torch.Tensor], name, nbytes: int, dtype=None) -> None:
    """A tensor the library reads or writes `nbytes` of: on the GPU,
    contiguous, large enough (and of `dtype` where its element count is what
    the call passes).  Checked here because the C calls take bare pointers:
    a host pointer or a short buffer would reach a kernel as it is.  name: a
    string, or a list's name and an index."""
    if nbytes <= 0:
        return
    if t is not None and t.is_cuda and (dtype is None or t.dtype == dtype) and t.is_contiguous() and t.nbytes >= nbytes:
        return
    if isinstance(name, tuple):
        name = "%s[%d]" % name
    if t is None:
        raise ValueError(f"{name}: a device tensor of {nbytes} bytes is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor, not on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    raise ValueError(f"{name} holds {t.nbytes} bytes, the call needs {nbytes}")


def header_functions() -> list[str]:
    """Names of the functions declared in include/lp.h."""
    text = open(HEADER_PATH).read()
    return re.findall(r"^\s*(?:lp_status|const char\*)\s+(lp_\w+)\s*\(", text, re.M)


@dataclasses.dataclass
class QTensor:
    """A (possibly block-scaled) tensor of logical shape [batch, rows, cols].

    codes: bf16 values (fmt "bf16"), uint8 E4M3 codes, or uint8 packed E2M1
    pairs; scales: uint8 E8M0 / E4M3 bytes or float32 block scales; for
    NVFP4 and the per-tensor FP8 formats `tensor_scale` is a one-element
    float32 device tensor.  run_groups: for "fp8_r128" along -2, the number of
    groups at whose first rows the runs restart (0: none do), as the
    quantizers set it; calls that would look for the runs elsewhere refuse the
    tensor.  None: not known, and not checked.
    """
    fmt: str
    codes: torch.Tensor
    scales: Optional[torch.Tensor] = None
    tensor_scale: Optional[torch.Tensor] = None
    shape: tuple = ()
    axis: int = -1
    run_groups: Optional[int] = None

    def __post_init__(self):
        if not self.shape:
            s = tuple(self.codes.shape)
            cols = s[-1] * (2 if self.fmt in ("mxfp4", "nvfp4") else 1)
            self.shape = (s[0] if len(s) == 3 else 1, s[-2], cols)
        if len(self.shape) == 2:
            self.shape = (1,) + tuple(self.shape)

    @property
    def rows(self) -> int:
        return self.shape[1]

    @property
    def cols(self) -> int:
        return self.shape[2]

    def c(self, groups: int = 0) -> _QTensorC:
        """The C descriptor, for a call over `groups` groups of rows (0: without offsets)."""
        b, r, c = self.shape
        n = b * r * c
        fmt, codes, scales, ts = self.fmt, self.codes, self.scales, self.tensor_scale
        made = self.run_groups                               # (one group: the layout without offsets)
        if made is not None and made != groups and (made > 1 or groups > 1):
            raise ValueError(f"{fmt} runs made for {made} groups, the call has {groups} (0: no offsets)")
        _device(codes, _NAMES[fmt][0], n * _CODE_BITS[fmt] // 8)
        _device(scales, _NAMES[fmt][1], _scale_bytes(fmt, self.axis, b, r, c, groups))
        if fmt in ("nvfp4", "fp8t_e4m3", "fp8t_e5m2"):
            _device(ts, _NAMES[fmt][2], 4 if n else 0, torch.float32)
        return _QTensorC(FMT[fmt], self.axis, b, r, c, None if codes is None else codes.data_ptr(),
                         None if scales is None else scales.data_ptr(), None if ts is None else ts.data_ptr())


# torch.cuda.current_stream().cuda_stream without the Stream object (2.7 us a
# call), where this torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> Optional[int]:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream if _raw_stream is None else _raw_stream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else stream


def _torch_stream(stream):
    """The torch stream of a stream argument (a torch stream, or a raw handle)."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = _stream(stream)
    # (ExternalStream(0) is a stream of torch's pool)
    return torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()


def _new(like: torch.Tensor, stream, result: bool = True):
    """new_empty(shape, dtype=) of like's device for a call on `stream` to write.
    On another stream than the current one the memory is that stream's: a block
    of the current stream's may still be used by work enqueued there before
    it was freed, which the call does not wait for.  result: returned to the
    caller, who uses it on the current stream."""
    if stream is None or not like.is_cuda or _stream(stream) == _stream(None):
        return like.new_empty

    def new(shape, dtype):
        current = torch.cuda.current_stream()
        torch.cuda.set_stream(_torch_stream(stream))         # (half the cost of the context manager)
        try:
            t = like.new_empty(shape, dtype=dtype)
        finally:
            torch.cuda.set_stream(current)
        if result:
            t.record_stream(current)
        return t
    return new


def _capturing(stream) -> bool:
    """Whether what is enqueued on the stream goes into a graph."""
    if stream is None or _stream(stream) == _stream(None):
        return torch.cuda.is_current_stream_capturing()
    current = torch.cuda.current_stream()
    torch.cuda.set_stream(_torch_stream(stream))
    try:
        return torch.cuda.is_current_stream_capturing()
    finally:
        torch.cuda.set_stream(current)


def _check(st: int, where: str):
    if st != 0:
        raise LpError(st, where)


def lp_dequant(src: QTensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Decode `src` to bf16 [batch, rows, cols] (bit-exact); not "fp8_r128"
    whose runs restart at groups."""
    if out is None:
        out = _new(src.codes, stream)(src.shape, dtype=torch.bfloat16)
    q = src.c()
    _device(out, "out", 2 * src.shape[0] * src.shape[1] * src.shape[2])
    _check(lib.lp_dequant(ctypes.byref(q), out.data_ptr(), _stream(stream)), "lp_dequant")
    return out


def lp_mx_quant(src: torch.Tensor, axis: int, fmt: str = "mxfp8", codes: Optional[torch.Tensor] = None,
                scales: Optional[torch.Tensor] = None, stream=None) -> QTensor:
    """MX-quantize a bf16 tensor [batch, rows, cols] (or [rows, cols]) along
    `axis` (-1 or -2) to "mxfp8" or "mxfp4"."""
    shape = tuple(src.shape) if src.dim() == 3 else (1,) + tuple(src.shape)
    b, r, c = shape
    if codes is None:
        codes = _new(src, stream)((b, r, c if fmt == "mxfp8" else c // 2), dtype=torch.uint8)
    if scales is None:
        sshape = (b, r, c // 32) if axis == -1 else (b, r // 32, c)
        scales = _new(src, stream)(sshape, dtype=torch.uint8)
    n = b * r * c
    _device(src, "src", 2 * n, torch.bfloat16)
    _device(codes, "codes", n if fmt == "mxfp8" else n // 2)
    _device(scales, "scales", _scale_bytes(fmt, axis, b, r, c))
    _check(lib.lp_mx_quant(src.data_ptr(), b, r, c, axis, FMT[fmt], codes.data_ptr(), scales.data_ptr(),
                           _stream(stream)), "lp_mx_quant")
    return QTensor(fmt, codes, scales, None, shape, axis)


def lp_mx_quant_dual(src: torch.Tensor, fmt: str = "mxfp8", stream=None) -> tuple:
    """MX-quantize a bf16 tensor [batch, rows, cols] (or [rows, cols]) along
    both axes in one pass: (copy scaled along -1, copy scaled along -2)."""
    shape = tuple(src.shape) if src.dim() == 3 else (1,) + tuple(src.shape)
    b, r, c = shape
    cb = c if fmt == "mxfp8" else c // 2
    _device(src, "src", 2 * b * r * c, torch.bfloat16)
    codes_c = _new(src, stream)((b, r, cb), dtype=torch.uint8)
    scales_c = _new(src, stream)((b, r, c // 32), dtype=torch.uint8)
    codes_r = _new(src, stream)((b, r, cb), dtype=torch.uint8)
    scales_r = _new(src, stream)((b, r // 32, c), dtype=torch.uint8)
    _check(lib.lp_mx_quant_dual(src.data_ptr(), b, r, c, FMT[fmt], codes_c.data_ptr(), scales_c.data_ptr(),
                                codes_r.data_ptr(), scales_r.data_ptr(), _stream(stream)), "lp_mx_quant_dual")
    return QTensor(fmt, codes_c, scales_c, None, shape, -1), QTensor(fmt, codes_r, scales_r, None, shape, -2)


def lp_tensor_amax(src: torch.Tensor, amax: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """max |x| of a bf16 tensor into a float32 device scalar (`amax` may be a
    one-element view into an amax history)."""
    if amax is None:
        amax = _new(src, stream)(1, dtype=torch.float32)
    _device(src, "src", 2 * src.numel(), torch.bfloat16)
    _device(amax, "amax", 4, torch.float32)
    _check(lib.lp_tensor_amax(src.data_ptr(), src.numel(), amax.data_ptr(), _stream(stream)), "lp_tensor_amax")
    return amax


def lp_tensor_quant(src: torch.Tensor, fmt: str, scale: torch.Tensor, amax: Optional[torch.Tensor] = None,
                    codes: Optional[torch.Tensor] = None, stream=None) -> QTensor:
    """Per-tensor FP8 quantization ("fp8t_e4m3" / "fp8t_e5m2") of a bf16
    tensor [batch, rows, cols] (or [rows, cols]) with the float32 device
    scalar `scale`; the input's amax goes to `amax` when given."""
    shape = tuple(src.shape) if src.dim() == 3 else (1,) + tuple(src.shape)
    if codes is None:
        codes = _new(src, stream)(shape, dtype=torch.uint8)
    _device(src, "src", 2 * src.numel(), torch.bfloat16)
    _device(codes, "codes", src.numel())
    _device(scale, "scale", 4, torch.float32)
    if amax is not None:
        _device(amax, "amax", 4, torch.float32)
    _check(lib.lp_tensor_quant(src.data_ptr(), src.numel(), FMT[fmt], scale.data_ptr(), codes.data_ptr(),
                               None if amax is None else amax.data_ptr(), _stream(stream)), "lp_tensor_quant")
    return QTensor(fmt, codes, None, scale, shape, -1)


def lp_tensor_quant_delayed(src: torch.Tensor, fmt: str, history: torch.Tensor, slot: int, margin: int = 0,
                            codes: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None,
                            stream=None) -> QTensor:
    """Delayed scaling in one call: scale from `history` (float32 device
    ring), quantization with it, the input's amax into history[slot]."""
    shape = tuple(src.shape) if src.dim() == 3 else (1,) + tuple(src.shape)
    if codes is None:
        codes = _new(src, stream)(shape, dtype=torch.uint8)
    if scale is None:
        scale = _new(src, stream)(1, dtype=torch.float32)
    _device(src, "src", 2 * src.numel(), torch.bfloat16)
    _device(codes, "codes", src.numel())
    _device(history, "history", 4 * max(history.numel(), 1), torch.float32)
    _device(scale, "scale", 4, torch.float32)
    _check(lib.lp_tensor_quant_delayed(src.data_ptr(), src.numel(), FMT[fmt], history.data_ptr(), history.numel(),
                                       slot, margin, codes.data_ptr(), scale.data_ptr(), _stream(stream)),
           "lp_tensor_quant_delayed")
    return QTensor(fmt, codes, None, scale, shape, -1)


def lp_scale_from_history(history: torch.Tensor, fmt: str, margin: int = 0, scale: Optional[torch.Tensor] = None,
                          stream=None) -> torch.Tensor:
    """Per-tensor scale (float32 device scalar) from a float32 amax history."""
    if scale is None:
        scale = _new(history, stream)(1, dtype=torch.float32)
    _device(history, "history", 4 * max(history.numel(), 1), torch.float32)
    _device(scale, "scale", 4, torch.float32)
    _check(lib.lp_scale_from_history(history.data_ptr(), history.numel(), FMT[fmt], margin, scale.data_ptr(),
                                     _stream(stream)), "lp_scale_from_history")
    return scale


def lp_linear_bwd(grad_out: QTensor, x: Optional[QTensor], w: Optional[QTensor], need_dx: bool = True,
                  need_dw: bool = True, grad_x: Optional[torch.Tensor] = None,
                  grad_w: Optional[torch.Tensor] = None, stream=None, workspace: Optional[torch.Tensor] = None):
    """(grad_X [M,K] or None, grad_W [N,K] or None) of a linear layer.
    `workspace`: a zero-filled uint8 device tensor of at least
    lp_linear_bwd_workspace(...) bytes lets the call split its contraction
    (lp_linear_bwd_ws); None calls lp_linear_bwd.  "fp8_r128" gradients need
    no zeroes, and get a workspace here when the call can use one."""
    _, M, N = grad_out.shape
    K = (w if need_dx else x).cols
    codes = grad_out.codes
    if need_dx:
        if grad_x is None:
            grad_x = _new(codes, stream)((M, K), dtype=torch.bfloat16)
        else:
            _device(grad_x, "grad_x", 2 * M * K)
    if need_dw:
        if grad_w is None:
            grad_w = _new(codes, stream)((N, K), dtype=torch.bfloat16)
        else:
            _device(grad_w, "grad_w", 2 * N * K)
    if workspace is not None:
        _device(workspace, "workspace", 1)
    g = grad_out.c()
    xc = x.c() if x is not None else None
    wc = w.c() if w is not None else None
    args = (ctypes.byref(g), ctypes.byref(xc) if xc else None, ctypes.byref(wc) if wc else None,
            grad_x.data_ptr() if need_dx else None, grad_w.data_ptr() if need_dw else None)
    if workspace is None and grad_out.fmt == "fp8_r128" and need_dx != need_dw:
        out_rows, depth = (M, N) if need_dx else (N, M)
        if depth > 31 * 128 and -(-out_rows // 128) * -(-K // 128) <= 128:     # else it would not split
            nbytes = ctypes.c_size_t(0)
            _check(lib.lp_linear_bwd_workspace(*args, ctypes.byref(nbytes)), "lp_linear_bwd_workspace")
            if nbytes.value:
                workspace = _new(codes, stream, result=False)(nbytes.value, dtype=torch.uint8)
    if workspace is None:
        st = lib.lp_linear_bwd(*args, _stream(stream))
        _check(st, "lp_linear_bwd")
    else:
        st = lib.lp_linear_bwd_ws(*args, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                  _stream(stream))
        _check(st, "lp_linear_bwd_ws")
    return (grad_x if need_dx else None), (grad_w if need_dw else None)


def lp_linear_bwd_noalloc(grad_out: QTensor, x: Optional[QTensor], w: Optional[QTensor], need_dx: bool = True,
                          need_dw: bool = True, grad_x: Optional[torch.Tensor] = None,
                          grad_w: Optional[torch.Tensor] = None, stream=None):
    """lp_linear_bwd with the split workspace held inside the library (no
    device allocation by the call; outputs are allocated here only when not
    given)."""
    M, N = grad_out.rows, grad_out.cols
    K = (w if need_dx else x).cols
    if need_dx and grad_x is None:
        grad_x = _new(grad_out.codes, stream)((M, K), dtype=torch.bfloat16)
    if need_dw and grad_w is None:
        grad_w = _new(grad_out.codes, stream)((N, K), dtype=torch.bfloat16)
    if need_dx:
        _device(grad_x, "grad_x", 2 * M * K)
    if need_dw:
        _device(grad_w, "grad_w", 2 * N * K)
    g = grad_out.c()
    xc = x.c() if x is not None else None
    wc = w.c() if w is not None else None
    st = lib.lp_linear_bwd_noalloc(ctypes.byref(g), ctypes.byref(xc) if xc else None,
                                   ctypes.byref(wc) if wc else None, grad_x.data_ptr() if need_dx else None,
                                   grad_w.data_ptr() if need_dw else None, _stream(stream))
    _check(st, "lp_linear_bwd_noalloc")
    return (grad_x if need_dx else None), (grad_w if need_dw else None)


def lp_grouped_dx_deferred(grad_out: QTensor, w: torch.Tensor, offsets: torch.Tensor, fuse_rows: int = 1536,
                           grad_x: Optional[torch.Tensor] = None, w_codes: Optional[torch.Tensor] = None,
                           w_scales: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """grad_X of the deferred MXFP8 recipe: grad_out (MXFP8 along -1) times
    the bf16 weight w [G, N, K] quantized to MXFP8 along N; groups of at most
    fuse_rows rows quantize their weight inside the product.  w_codes /
    w_scales (the weight's MXFP8 copy for the larger groups) are allocated
    here when not given and fuse_rows < M."""
    G, N, K = w.shape
    M = grad_out.rows
    if grad_x is None:
        grad_x = _new(grad_out.codes, stream)((M, K), dtype=torch.bfloat16)
    if fuse_rows < M or N % 512 or K % 32:
        if w_codes is None:
            w_codes = _new(w, stream, result=False)((G, N, K), dtype=torch.uint8)
        if w_scales is None:
            w_scales = _new(w, stream, result=False)((G, N // 32, K), dtype=torch.uint8)
        _device(w_codes, "w_codes", G * N * K)
        _device(w_scales, "w_scales", G * (N // 32) * K)
    _device(w, "w", 2 * G * N * K, torch.bfloat16)
    _device(offsets, "offsets", 4 * G, torch.int32)
    _device(grad_x, "grad_x", 2 * M * K)
    g = grad_out.c()
    st = lib.lp_grouped_dx_deferred(ctypes.byref(g), w.data_ptr(), K, offsets.data_ptr(), G, fuse_rows,
                                    grad_x.data_ptr(), None if w_codes is None else w_codes.data_ptr(),
                                    None if w_scales is None else w_scales.data_ptr(), _stream(stream))
    _check(st, "lp_grouped_dx_deferred")
    return grad_x


def lp_linear_bwd_workspace(grad_out: QTensor, x: Optional[QTensor], w: Optional[QTensor], need_dx: bool = True,
                            need_dw: bool = True) -> int:
    """Workspace bytes lp_linear_bwd_ws can use for this call (0: it does not split)."""
    g = grad_out.c()
    xc = x.c() if x is not None else None
    wc = w.c() if w is not None else None
    n = ctypes.c_size_t(0)
    st = lib.lp_linear_bwd_workspace(ctypes.byref(g), ctypes.byref(xc) if xc else None,
                                     ctypes.byref(wc) if wc else None, 1 if need_dx else None,
                                     1 if need_dw else None, ctypes.byref(n))
    _check(st, "lp_linear_bwd_workspace")
    return n.value


def lp_grouped_bwd(grad_out: QTensor, x: Optional[QTensor], w: Optional[QTensor], offsets: torch.Tensor,
                   need_dx: bool = True, need_dw: bool = True, grad_x: Optional[torch.Tensor] = None,
                   grad_w: Optional[torch.Tensor] = None, stream=None):
    """(grad_X [M,K] or None, grad_W [G,N,K] or None) of a grouped matmul.
    Rows of grad_X at or past offsets[-1] are left as they were in `grad_x`.  "fp8_r128" operands along -2: as
    lp_r128_quant with these offsets makes them."""
    _, M, N = grad_out.shape
    G = offsets.numel()
    K = (w if need_dx else x).cols
    codes = grad_out.codes
    if need_dx:
        if grad_x is None:
            grad_x = _new(codes, stream)((M, K), dtype=torch.bfloat16)
        else:
            _device(grad_x, "grad_x", 2 * M * K)
    if need_dw:
        if grad_w is None:
            grad_w = _new(codes, stream)((G, N, K), dtype=torch.bfloat16)
        else:
            _device(grad_w, "grad_w", 2 * G * N * K)
    _device(offsets, "offsets", 4 * G, torch.int32)
    g = grad_out.c(G)
    xc = x.c(G) if x is not None else None
    wc = w.c() if w is not None else None
    st = lib.lp_grouped_bwd(ctypes.byref(g), ctypes.byref(xc) if xc else None, ctypes.byref(wc) if wc else None,
                            offsets.data_ptr(), G, grad_x.data_ptr() if need_dx else None,
                            grad_w.data_ptr() if need_dw else None, _stream(stream))
    _check(st, "lp_grouped_bwd")
    return (grad_x if need_dx else None), (grad_w if need_dw else None)


def lp_linear_fwd(x: QTensor, w: QTensor, y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y [M, N] = x @ w^T: both "mxfp4" or both "mxfp8" (scaled along k),
    both "nvfp4", a "bf16" x with a "bf16", "fp8_b128" or "nvfp4" weight, or
    an "fp8_r128" x (along -1) with an "fp8_b128" weight."""
    if y is None:
        y = _new(x.codes, stream)((x.rows, w.rows), dtype=torch.bfloat16)
    _device(y, "y", 2 * x.rows * w.rows)
    xc, wc = x.c(), w.c()
    _check(lib.lp_linear_fwd(ctypes.byref(xc), ctypes.byref(wc), y.data_ptr(), _stream(stream)), "lp_linear_fwd")
    return y


def lp_grouped_fwd(x: QTensor, w: QTensor, offsets: torch.Tensor, y: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """y [M, N]: rows of group g are x[rows] @ w[g]^T; rows at or past
    offsets[-1] are left as they were in `y`."""
    if y is None:
        y = _new(x.codes, stream)((x.rows, w.rows), dtype=torch.bfloat16)
    _device(y, "y", 2 * x.rows * w.rows)
    _device(offsets, "offsets", 4 * offsets.numel(), torch.int32)
    xc, wc = x.c(), w.c()
    _check(lib.lp_grouped_fwd(ctypes.byref(xc), ctypes.byref(wc), offsets.data_ptr(), offsets.numel(), y.data_ptr(),
                              _stream(stream)), "lp_grouped_fwd")
    return y


def lp_status_string(status: int) -> str:
    return lib.lp_status_string(status).decode()


# ---------------------------------------------------------------- include/lp_train.h

def _shape3(src: torch.Tensor) -> tuple:
    return tuple(src.shape) if src.dim() == 3 else (1,) + tuple(src.shape)


def _runs(rows: int, offsets: Optional[torch.Tensor]) -> int:
    """Token runs of `rows` rows: per group when there are offsets."""
    if offsets is None:
        return -(-rows // 128)
    _device(offsets, "offsets", 4 * offsets.numel(), torch.int32)
    return rows // 128 + offsets.numel()


def _offsets(offsets: Optional[torch.Tensor]) -> tuple:
    if offsets is None:
        return None, 0
    if offsets.numel() == 0:                                 # its null address would mean no offsets
        raise LpError(2, "offsets of no group")
    return offsets.data_ptr(), offsets.numel()


def lp_r128_quant(src: torch.Tensor, axis: int = -1, offsets: Optional[torch.Tensor] = None, stream=None) -> QTensor:
    """Quantize a bf16 tensor [batch, rows, cols] (or [rows, cols]) to
    "fp8_r128" along `axis` (-1 or -2).  offsets (axis -2): int32 cumulative
    group ends; runs restart at every group's first row."""
    b, r, c = shape = _shape3(src)
    new, off = _new(src, stream), _offsets(offsets)
    codes = new(shape, dtype=torch.uint8)
    scales = new((b, -(-c // 128), r) if axis == -1 else (b, _runs(r, offsets), c), dtype=torch.float32)
    _device(src, "src", 2 * b * r * c, torch.bfloat16)
    _check(lib.lp_r128_quant(src.data_ptr(), b, r, c, axis, *off, codes.data_ptr(), scales.data_ptr(),
                             _stream(stream)), "lp_r128_quant")
    return QTensor("fp8_r128", codes, scales, None, shape, axis, off[1] if axis == -2 else None)


def lp_r128_quant_dual(src: torch.Tensor, offsets: Optional[torch.Tensor] = None, stream=None) -> tuple:
    """Both "fp8_r128" copies of a bf16 tensor from one read: (along -1, along
    -2); the second one's runs restart at each group of `offsets`.  Rows past
    the last offset are left unwritten in both."""
    b, r, c = shape = _shape3(src)
    new, off = _new(src, stream), _offsets(offsets)
    codes_c, codes_r = new(shape, dtype=torch.uint8), new(shape, dtype=torch.uint8)
    scales_c = new((b, -(-c // 128), r), dtype=torch.float32)
    scales_r = new((b, _runs(r, offsets), c), dtype=torch.float32)
    _device(src, "src", 2 * b * r * c, torch.bfloat16)
    _check(lib.lp_r128_quant_dual(src.data_ptr(), b, r, c, *off, codes_c.data_ptr(), scales_c.data_ptr(),
                                  codes_r.data_ptr(), scales_r.data_ptr(), _stream(stream)), "lp_r128_quant_dual")
    return (QTensor("fp8_r128", codes_c, scales_c, None, shape, -1),
            QTensor("fp8_r128", codes_r, scales_r, None, shape, -2, off[1]))


def lp_b128_quant(src: torch.Tensor, codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                  stream=None) -> QTensor:
    """Quantize a bf16 tensor [batch, rows, cols] (or [rows, cols]) to
    "fp8_b128" (into `codes` and `scales` when given)."""
    b, r, c = shape = _shape3(src)
    if codes is None:
        codes = _new(src, stream)(shape, dtype=torch.uint8)
    if scales is None:
        scales = _new(src, stream)((b, -(-r // 128), -(-c // 128)), dtype=torch.float32)
    _device(src, "src", 2 * b * r * c, torch.bfloat16)
    _device(codes, "codes", b * r * c)
    _device(scales, "scales", _scale_bytes("fp8_b128", -1, b, r, c), torch.float32)
    _check(lib.lp_b128_quant(src.data_ptr(), b, r, c, codes.data_ptr(), scales.data_ptr(), _stream(stream)),
           "lp_b128_quant")
    return QTensor("fp8_b128", codes, scales, None, shape)


def _fwd_dyn(x: torch.Tensor, w: QTensor, offsets: Optional[torch.Tensor], y: Optional[torch.Tensor], stream):
    M, K = x.shape
    if K != w.cols:
        raise ValueError(f"x has {K} columns, the weight {w.cols}")
    _device(x, "x", 2 * M * K, torch.bfloat16)
    if y is None:
        y = _new(x, stream)((M, w.rows), dtype=torch.bfloat16)
    else:
        _device(y, "y", 2 * M * w.rows)
    nb = -(-K // 128)
    if offsets is None and M <= 4 and M * nb <= 512:         # quantized inside the product
        codes = scales = None
    else:
        at = -(-4 * nb * M // 16) * 16                       # scratch: scales, then (16-byte aligned) codes
        scratch = _new(x, stream, result=False)(at + M * K, dtype=torch.uint8)
        scales = scratch.data_ptr()
        codes = scales + at
    args = (codes, scales, y.data_ptr(), _stream(stream))
    wc = w.c()
    if offsets is None:
        _check(lib.lp_linear_fwd_dyn(x.data_ptr(), M, ctypes.byref(wc), *args), "lp_linear_fwd_dyn")
    else:
        _device(offsets, "offsets", 4 * offsets.numel(), torch.int32)
        _check(lib.lp_grouped_fwd_dyn(x.data_ptr(), M, ctypes.byref(wc), offsets.data_ptr(), offsets.numel(), *args),
               "lp_grouped_fwd_dyn")
    return y


def lp_linear_fwd_dyn(x: torch.Tensor, w: QTensor, y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y [M, N] = x @ w^T: a bf16 x [M, K], quantized to "fp8_r128" in the
    call, times an "fp8_b128" weight."""
    return _fwd_dyn(x, w, None, y, stream)


def lp_grouped_fwd_dyn(x: torch.Tensor, w: QTensor, offsets: torch.Tensor, y: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """y [M, N]: rows of group g are x[rows] @ w[g]^T, x quantized in the
    call; rows at or past offsets[-1] are left as they were in `y`."""
    return _fwd_dyn(x, w, offsets, y, stream)


class _AdamWTensorC(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("exp_avg", ctypes.c_void_p),
                ("exp_avg_sq", ctypes.c_void_p), ("exp_avg_scales", ctypes.c_void_p),
                ("exp_avg_sq_scales", ctypes.c_void_p), ("param_copy", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("lr_scale", ctypes.c_float), ("weight_decay", ctypes.c_float)]


class AdamWPlan:
    """The tensors of an AdamW step, checked once: lists of equal length with
    each tensor's parameter (float32 or bfloat16), gradient (float32 or
    bfloat16) and moments.  Moments are float32 of the parameter's size, or
    uint8 E4M3 codes with float32 scales per 128 elements
    (exp_avg_sq_scales: of sqrt(v)).  copies: bfloat16 tensors that receive
    the new float32 parameters.  weight_decay, lr_scale: one number or one
    per tensor.  Tensors must not overlap (a tied weight is listed once).  The plan keeps the tensors alive and holds the device table
    that the step reads; set_grads makes a new one, so gradients that stay
    where they are from step to step are the cheaper way.

    A step can be captured into a graph, set_grads cannot.  The graph steps
    with the gradients, and the step number, of its capture whatever set_grads
    does later; the plan keeps the table and the gradients of captured steps,
    and has to live as long as the graph."""

    def __init__(self, params, grads, exp_avgs, exp_avg_sqs, exp_avg_scales=None, exp_avg_sq_scales=None, copies=None,
                 weight_decay=0.0, lr_scale=1.0):
        k = len(params)
        lists = {"grads": grads, "exp_avgs": exp_avgs, "exp_avg_sqs": exp_avg_sqs, "exp_avg_scales": exp_avg_scales,
                 "exp_avg_sq_scales": exp_avg_sq_scales, "copies": copies}
        for name, v in lists.items():
            if v is not None and len(v) != k:
                raise ValueError(f"{name}: {len(v)} tensors for {k} parameters")
        if (exp_avg_scales is None) != (exp_avg_sq_scales is None):
            raise ValueError("8-bit moments need exp_avg_scales and exp_avg_sq_scales")
        self.bits8 = exp_avg_scales is not None
        self.param_dtype = params[0].dtype if k else torch.float32
        self._n = [p.numel() for p in params]
        self._c = (_AdamWTensorC * max(k, 1))()
        self._table, self._in_graph, self._of_graphs = None, False, []
        self._kept = [list(params), list(exp_avgs), list(exp_avg_sqs)] + [list(v) for v in (exp_avg_scales, exp_avg_sq_scales, copies) if v is not None]
        if self.param_dtype not in _ADAMW_DTYPE:
            raise ValueError(f"parameters must be float32 or bfloat16, not {self.param_dtype}")
        wd = weight_decay if isinstance(weight_decay, (list, tuple)) else [weight_decay] * k
        ls = lr_scale if isinstance(lr_scale, (list, tuple)) else [lr_scale] * k
        if len(wd) != k or len(ls) != k:
            raise ValueError("weight_decay and lr_scale: one number, or one per parameter")
        state = torch.uint8 if self.bits8 else torch.float32
        runs = [-(-n // 128) for n in self._n]
        self._pointers("param", params, "params", self._n, self.param_dtype)
        self._pointers("exp_avg", exp_avgs, "exp_avgs", self._n, state)
        self._pointers("exp_avg_sq", exp_avg_sqs, "exp_avg_sqs", self._n, state)
        if self.bits8:
            self._pointers("exp_avg_scales", exp_avg_scales, "exp_avg_scales", runs, torch.float32)
            self._pointers("exp_avg_sq_scales", exp_avg_sq_scales, "exp_avg_sq_scales", runs, torch.float32)
        if copies is not None:
            self._pointers("param_copy", copies, "copies", self._n, torch.bfloat16)
        for c, n, d, s in zip(self._c, self._n, wd, ls):
            c.n, c.weight_decay, c.lr_scale = n, d, s
        self.set_grads(grads)

    def _pointers(self, field, tensors, name, counts, dtype) -> None:
        """Checks one kind of tensors, then puts their addresses into the C array."""
        size = dtype.itemsize
        for i, (t, n) in enumerate(zip(tensors, counts)):
            _device(t, (name, i), n * size, dtype)
        for c, t in zip(self._c, tensors):
            setattr(c, field, t.data_ptr())

    def set_grads(self, grads) -> None:
        """Use these gradients from now on (all of one dtype)."""
        if len(grads) != len(self._n):
            raise ValueError(f"grads: {len(grads)} tensors for {len(self._n)} parameters")
        dtype = grads[0].dtype if grads else torch.float32
        if dtype not in _ADAMW_DTYPE:
            raise ValueError(f"gradients must be float32 or bfloat16, not {dtype}")
        self._pointers("grad", grads, "grads", self._n, dtype)
        if self._in_graph:
            self._of_graphs.append((self._table, self._grads))
            self._in_graph = False
        self.grad_dtype, self._grads = dtype, list(grads)
        nbytes, chunks = ctypes.c_size_t(0), ctypes.c_int64(0)
        args = (self._c, len(self._n), _ADAMW_DTYPE[self.param_dtype], _ADAMW_DTYPE[dtype], int(self.bits8))
        _check(lib.lp_adamw_plan(*args, None, ctypes.byref(nbytes), ctypes.byref(chunks)), "lp_adamw_plan")
        self._chunks, self._table = chunks.value, None
        if self._chunks:
            table = torch.empty(-(-nbytes.value // 8), dtype=torch.int64)
            _check(lib.lp_adamw_plan(*args, table.data_ptr(), ctypes.byref(nbytes), ctypes.byref(chunks)), "lp_adamw_plan")
            device = next(p.device for p, n in zip(self._kept[0], self._n) if n)
            self._table, self._home = table.to(device), _stream(None)


_ADAMW_DTYPE = {torch.float32: 0, torch.bfloat16: 1}


def lp_adamw(plan: AdamWPlan, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8, step: int = 1,
             grad_scale: Optional[torch.Tensor] = None, stream=None) -> None:
    """One AdamW step over the plan's tensors, in place.  step: 1 for the
    first; grad_scale: a float32 device scalar that multiplies every gradient."""
    if grad_scale is not None:
        _device(grad_scale, "grad_scale", 4, torch.float32)
    t, s = plan._table, _stream(stream)
    if t is not None and not plan._in_graph:
        plan._in_graph = _capturing(stream)
    if t is not None and s != plan._home:        # not to be reused before that stream is done with it
        t.record_stream(_torch_stream(s))
    _check(lib.lp_adamw(None if t is None else t.data_ptr(), len(plan._n), plan._chunks, _ADAMW_DTYPE[plan.param_dtype],
                        _ADAMW_DTYPE[plan.grad_dtype], int(plan.bits8), lr, beta1, beta2, eps, step,
                        None if grad_scale is None else grad_scale.data_ptr(), s), "lp_adamw")
