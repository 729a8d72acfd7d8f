"""FP8 linear layer with delayed scaling for B200 (sm_100a).

Thin ctypes binding of ``libfp8lin.so`` (declared in ``include/fp8lin.h``).
Every step of the path runs in the library's CUDA kernels; this module only
marshals tensors into pointers, sizes and the current CUDA stream.  PyTorch
supplies device memory and streams.  There is no CPU fallback: importing the
package without the built library raises.

Entry points carry the C names (``fp8_quantize``, ``fp8_mm``, ...).  A few
helpers (``ScaleRing``, ``quantize``, ``linear_forward``, ``linear_backward``)
allocate outputs with torch and call them.
"""
from __future__ import annotations

import ctypes
import os
import struct
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libfp8lin.so")

FP8_E4M3, FP8_E5M2 = 0, 1
FP8_DT_BF16, FP8_DT_FP16, FP8_DT_FP32, FP8_DT_E4M3, FP8_DT_E5M2 = 0, 1, 2, 3, 4
FP8_K_MAJOR, FP8_MN_MAJOR = 0, 1
FP8_TILE_AUTO, FP8_TILE_128x128, FP8_TILE_128x256, FP8_TILE_PAIR_256x256, FP8_TILE_SPLITK_128x128 = 0, 1, 2, 3, 4
FP8_TILE_STREAMK = 8
FP8_OK = 0
FP8_ERR_INVALID_ARG, FP8_ERR_UNSUPPORTED, FP8_ERR_MISALIGNED = -1, -2, -3
FP8_ERR_CUDA, FP8_ERR_DEVICE_TIMEOUT, FP8_ERR_WORKSPACE = -4, -5, -6
FP8_ERR_TOO_LARGE = -7
FP8_RAGGED_M, FP8_RAGGED_K = 0, 1
FP8_MAX_GROUPS, FP8_MAX_INT8_K = 1024, 131071
FP8_MAX = {FP8_E4M3: 448.0, FP8_E5M2: 57344.0}


class Fp8Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status} ({fp8_status_string(status)})")


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python fp8_delayed_scaling_03_b200/build.py` "
                      "(there is no CPU fallback)")

_lib = ctypes.CDLL(LIB_PATH)
_P, _I, _I64, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t


class MmArgs(ctypes.Structure):
    _fields_ = [("m", _I64), ("n", _I64), ("k", _I64),
                ("a", _P), ("fmt_a", _I), ("a_major", _I), ("lda", _I64),
                ("b", _P), ("fmt_b", _I), ("b_major", _I), ("ldb", _I64),
                ("scale_a", _P), ("scale_b", _P),
                ("bias", _P), ("bias_dtype", _I), ("bias_scale", _P),
                ("d", _P), ("ldd", _I64),
                ("tile_cfg", _I),
                ("workspace", _P), ("workspace_bytes", _SZ)]


class MmPlanInfo(ctypes.Structure):
    _fields_ = [("tile_cfg", _I), ("tiles", _I64), ("units", _I), ("est_us", ctypes.c_double),
                ("stream_k_ctas", _I), ("dp_tiles", _I64)]


class QuantizeArgs(ctypes.Structure):
    _fields_ = [("in_", _P), ("in_dtype", _I), ("rows", _I64), ("cols", _I64), ("ld_in", _I64),
                ("fmt", _I), ("ring", _P), ("hist_len", _I),
                ("out", _P), ("ld_out", _I64),
                ("amax_out", _P), ("scale_out", _P)]


class LinearFwdArgs(ctypes.Structure):
    _fields_ = [("M", _I64), ("N", _I64), ("K", _I64),
                ("x", _P), ("x_dtype", _I), ("ldx", _I64), ("x_scale_in", _P),
                ("w", _P), ("w_dtype", _I), ("ldw", _I64), ("w_scale_in", _P),
                ("bias", _P), ("bias_dtype", _I), ("bias_scale", _P),
                ("fmt_x", _I), ("fmt_w", _I), ("hist_len", _I),
                ("ring_x", _P), ("ring_w", _P),
                ("x8", _P), ("ldx8", _I64),
                ("w8", _P), ("ldw8", _I64),
                ("sx_out", _P), ("sw_out", _P), ("amax_x_out", _P), ("amax_w_out", _P),
                ("y", _P), ("ldy", _I64)]


class LinearBwdArgs(ctypes.Structure):
    _fields_ = [("M", _I64), ("N", _I64), ("K", _I64),
                ("g", _P), ("g_dtype", _I), ("ldg", _I64), ("g_scale_in", _P),
                ("fmt_g", _I), ("hist_len", _I), ("ring_g", _P),
                ("g8", _P), ("ldg8", _I64),
                ("sg_out", _P), ("amax_g_out", _P),
                ("x8", _P), ("ldx8", _I64), ("sx", _P), ("fmt_x", _I),
                ("w8", _P), ("ldw8", _I64), ("sw", _P), ("fmt_w", _I),
                ("need_dx", _I), ("need_dw", _I), ("need_dbias", _I),
                ("dx", _P), ("lddx", _I64),
                ("dw", _P), ("lddw", _I64),
                ("dbias", _P),
                ("workspace", _P), ("workspace_bytes", _SZ)]


class Groups(ctypes.Structure):
    _fields_ = [("groups", _I64), ("offsets", _P), ("offsets_64", _I),
                ("stride_b", _I64), ("stride_d", _I64), ("scale_b_step", _I)]


class GroupedPlanInfo(ctypes.Structure):
    _fields_ = [("tile_lanes", _I), ("tile_cols", _I), ("split", _I), ("max_tiles", _I64)]


class MmInt8Args(ctypes.Structure):
    _fields_ = [("m", _I64), ("n", _I64), ("k", _I64),
                ("a", _P), ("lda", _I64), ("b", _P), ("ldb", _I64),
                ("scale_a", _P), ("scale_b", _P),
                ("bias", _P), ("bias_dtype", _I),
                ("d", _P), ("d_dtype", _I), ("ldd", _I64)]


class LinearInt8Args(ctypes.Structure):
    _fields_ = [("M", _I64), ("N", _I64), ("K", _I64),
                ("x", _P), ("x_dtype", _I), ("ldx", _I64),
                ("w8", _P), ("ldw8", _I64), ("sw", _P),
                ("bias", _P), ("bias_dtype", _I),
                ("x8", _P), ("ldx8", _I64), ("sx_out", _P),
                ("y", _P), ("y_dtype", _I), ("ldy", _I64)]


_SIGS = {
    "fp8_ring_bytes": (_SZ, [_I]),
    "fp8_ring_init": (_I, [_P, _I, _P]),
    "fp8_ring_seed": (_I, [_P, _I, _I, _F, _P]),
    "fp8_quantize": (_I, [_P, _I, _I64, _I64, _I64, _I, _P, _I, _P, _I64, _P, _P, _P]),
    "fp8_quantize_dual": (_I, [ctypes.POINTER(QuantizeArgs), ctypes.POINTER(QuantizeArgs), _P]),
    "fp8_quantize_dbias": (_I, [ctypes.POINTER(QuantizeArgs), _P, _P, _SZ, _P]),
    "fp8_mm": (_I, [ctypes.POINTER(MmArgs), _P]),
    "fp8_mm_plan": (_I, [ctypes.POINTER(MmArgs), ctypes.POINTER(MmArgs), _I, ctypes.POINTER(MmPlanInfo)]),
    "fp8_mm_pair": (_I, [ctypes.POINTER(MmArgs), ctypes.POINTER(MmArgs), _P]),
    "fp8_mm_batched": (_I, [ctypes.POINTER(MmArgs), _I64, _I64, _I64, _I64, _P]),
    "fp8_mm_grouped": (_I, [ctypes.POINTER(MmArgs), _I, ctypes.POINTER(Groups), _P]),
    "fp8_mm_grouped_plan": (_I, [ctypes.POINTER(MmArgs), _I, ctypes.POINTER(Groups), _I, ctypes.POINTER(GroupedPlanInfo)]),
    "fp8_mm_int8_plan": (_I, [ctypes.POINTER(MmInt8Args), _I, ctypes.POINTER(GroupedPlanInfo)]),
    "fp8_quantize_int8": (_I, [_P, _I, _I64, _I64, _I64, _P, _I64, _P, _P]),
    "fp8_mm_int8": (_I, [ctypes.POINTER(MmInt8Args), _P]),
    "fp8_linear_grouped_forward": (_I, [ctypes.POINTER(LinearFwdArgs), ctypes.POINTER(Groups), _P]),
    "fp8_linear_grouped_backward": (_I, [ctypes.POINTER(LinearBwdArgs), ctypes.POINTER(Groups), _P]),
    "fp8_linear_int8_forward": (_I, [ctypes.POINTER(LinearInt8Args), _P]),
    "fp8_mm_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "fp8_quantize_ex": (_I, [ctypes.POINTER(QuantizeArgs), _I, _P]),
    "fp8_ring_finalize": (_I, [_P, _I, _I, _P, _P]),
    "fp8_dbias_workspace_bytes": (_SZ, [_I64, _I64]),
    "fp8_dbias": (_I, [_P, _I, _I64, _I64, _I64, _P, _P, _P, _SZ, _P]),
    "fp8_dbias_noalloc": (_I, [_P, _I, _I64, _I64, _I64, _P, _P, _P]),
    "fp8_linear_forward": (_I, [ctypes.POINTER(LinearFwdArgs), _P]),
    "fp8_linear_backward": (_I, [ctypes.POINTER(LinearBwdArgs), _P]),
    "fp8_linear_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "fp8_get_device_status": (_I, []),
    "fp8_wait_selftest": (_I, [_P, ctypes.c_uint64, _P, _P]),
    "fp8_status_string": (ctypes.c_char_p, [_I]),
    "fp8_version": (ctypes.c_char_p, []),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args

EXPORTED = tuple(_SIGS)

# --------------------------------------------------------------------------- helpers


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _stream(device=None):
    return torch.cuda.current_stream(device).cuda_stream


def _check(status: int, where: str):
    if status != FP8_OK:
        raise Fp8Error(status, where)


def _dtype_code(t: torch.Tensor, fp8_fmt: int | None = None) -> int:
    """torch dtype -> FP8_DT_*; uint8 tensors are fp8 codes of `fp8_fmt`."""
    if t.dtype == torch.bfloat16:
        return FP8_DT_BF16
    if t.dtype == torch.float16:
        return FP8_DT_FP16
    if t.dtype == torch.float32:
        return FP8_DT_FP32
    if t.dtype == torch.float8_e4m3fn:
        return FP8_DT_E4M3
    if t.dtype == torch.float8_e5m2:
        return FP8_DT_E5M2
    if t.dtype == torch.uint8 and fp8_fmt is not None:
        return FP8_DT_E4M3 + fp8_fmt
    raise TypeError(f"unsupported dtype {t.dtype}")


def _nbytes(t) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _ld(t: torch.Tensor) -> int:
    """Row stride (elements) of a 2-D tensor whose last dim is contiguous."""
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError("expected a 2-D tensor with a contiguous last dimension")
    return t.stride(0)


def fp8_alloc(rows: int, cols: int, device) -> torch.Tensor:
    """fp8 code buffer [rows, ld] with ld = cols rounded up to 16 (the TMA rule),
    returned as the [rows, cols] view."""
    ld = (cols + 15) // 16 * 16
    return torch.zeros((rows, ld), dtype=torch.uint8, device=device)[:, :cols]


# --------------------------------------------------------------------------- C names

def fp8_ring_bytes(hist_len: int) -> int:
    return _lib.fp8_ring_bytes(hist_len)


def fp8_ring_init(ring: torch.Tensor, hist_len: int) -> None:
    _check(_lib.fp8_ring_init(_ptr(ring), hist_len, _stream(ring.device)), "fp8_ring_init")


def fp8_ring_seed(ring: torch.Tensor, hist_len: int, fmt: int, amax: float) -> None:
    _check(_lib.fp8_ring_seed(_ptr(ring), hist_len, fmt, amax, _stream(ring.device)), "fp8_ring_seed")


def fp8_quantize(x: torch.Tensor, fmt: int, ring: torch.Tensor, hist_len: int, out: torch.Tensor,
                 amax_out: torch.Tensor | None = None, scale_out: torch.Tensor | None = None) -> None:
    rows, cols = x.shape
    _check(_lib.fp8_quantize(_ptr(x), _dtype_code(x), rows, cols, _ld(x), fmt, _ptr(ring), hist_len,
                             _ptr(out), _ld(out), _ptr(amax_out), _ptr(scale_out), _stream(x.device)),
           "fp8_quantize")


def quantize_args(x: torch.Tensor, fmt: int, ring: torch.Tensor, hist_len: int, out: torch.Tensor,
                  amax_out: torch.Tensor | None = None, scale_out: torch.Tensor | None = None) -> QuantizeArgs:
    rows, cols = x.shape
    return QuantizeArgs(_ptr(x), _dtype_code(x), rows, cols, _ld(x), fmt, _ptr(ring), hist_len, _ptr(out), _ld(out),
                        _ptr(amax_out), _ptr(scale_out))


FP8_QUANTIZE_DEFER_RING_STEP = 1


def fp8_quantize_ex(a: QuantizeArgs, flags: int, device=None) -> None:
    _check(_lib.fp8_quantize_ex(ctypes.byref(a), flags, _stream(device)), "fp8_quantize_ex")


def fp8_ring_finalize(ring: torch.Tensor, hist_len: int, fmt: int, amax_out: torch.Tensor | None = None) -> None:
    _check(_lib.fp8_ring_finalize(_ptr(ring), hist_len, fmt, _ptr(amax_out), _stream(ring.device)),
           "fp8_ring_finalize")


def fp8_quantize_dual(a: QuantizeArgs, b: QuantizeArgs, device=None) -> None:
    _check(_lib.fp8_quantize_dual(ctypes.byref(a), ctypes.byref(b), _stream(device)), "fp8_quantize_dual")


def fp8_quantize_dbias(g: QuantizeArgs, dbias: torch.Tensor, workspace: torch.Tensor) -> None:
    _check(_lib.fp8_quantize_dbias(ctypes.byref(g), _ptr(dbias), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _stream(dbias.device)),
           "fp8_quantize_dbias")


def fp8_mm_pair(a: MmArgs, b: MmArgs, device=None) -> None:
    _check(_lib.fp8_mm_pair(ctypes.byref(a), ctypes.byref(b), _stream(device)), "fp8_mm_pair")


def fp8_mm_batched(a: MmArgs, batch: int, stride_a: int, stride_b: int, stride_d: int, device=None) -> None:
    """batch GEMMs of a's shape; element strides between batches (0 shares an operand)."""
    _check(_lib.fp8_mm_batched(ctypes.byref(a), batch, stride_a, stride_b, stride_d, _stream(device)),
           "fp8_mm_batched")


def fp8_mm_grouped(a: MmArgs, ragged: int, groups: Groups, device=None) -> None:
    """Products grouped by expert: FP8_RAGGED_M (rows of A and D) or FP8_RAGGED_K (the contraction)."""
    _check(_lib.fp8_mm_grouped(ctypes.byref(a), ragged, ctypes.byref(groups), _stream(device)), "fp8_mm_grouped")


def fp8_mm_grouped_plan(a: MmArgs, ragged: int, groups: Groups, num_sms: int = 148) -> GroupedPlanInfo:
    """The tiles fp8_mm_grouped would take on a GPU with num_sms SMs; host arithmetic only (no device needed)."""
    info = GroupedPlanInfo()
    _check(_lib.fp8_mm_grouped_plan(ctypes.byref(a), ragged, ctypes.byref(groups), num_sms, ctypes.byref(info)),
           "fp8_mm_grouped_plan")
    return info


def fp8_mm_int8_plan(a: MmInt8Args, num_sms: int = 148) -> GroupedPlanInfo:
    """The tiles fp8_mm_int8 would take on a GPU with num_sms SMs; host arithmetic only (no device needed)."""
    info = GroupedPlanInfo()
    _check(_lib.fp8_mm_int8_plan(ctypes.byref(a), num_sms, ctypes.byref(info)), "fp8_mm_int8_plan")
    return info


def fp8_quantize_int8(x: torch.Tensor, out: torch.Tensor, scale: torch.Tensor) -> None:
    rows, cols = x.shape
    _check(_lib.fp8_quantize_int8(_ptr(x), _dtype_code(x), rows, cols, _ld(x), _ptr(out), _ld(out), _ptr(scale),
                                  _stream(x.device)), "fp8_quantize_int8")


def fp8_mm_int8(a: MmInt8Args, device=None) -> None:
    _check(_lib.fp8_mm_int8(ctypes.byref(a), _stream(device)), "fp8_mm_int8")


def fp8_linear_grouped_forward(args: LinearFwdArgs, groups: Groups, device=None) -> None:
    _check(_lib.fp8_linear_grouped_forward(ctypes.byref(args), ctypes.byref(groups), _stream(device)),
           "fp8_linear_grouped_forward")


def fp8_linear_grouped_backward(args: LinearBwdArgs, groups: Groups, device=None) -> None:
    _check(_lib.fp8_linear_grouped_backward(ctypes.byref(args), ctypes.byref(groups), _stream(device)),
           "fp8_linear_grouped_backward")


def fp8_linear_int8_forward(args: LinearInt8Args, device=None) -> None:
    _check(_lib.fp8_linear_int8_forward(ctypes.byref(args), _stream(device)), "fp8_linear_int8_forward")


def fp8_mm(m, n, k, a, fmt_a, a_major, lda, b, fmt_b, b_major, ldb, scale_a, scale_b, d, ldd,
           bias=None, bias_dtype=FP8_DT_BF16, bias_scale=None, stream=None, tile_cfg=FP8_TILE_AUTO,
           workspace=None) -> None:
    args = MmArgs(m, n, k, _ptr(a), fmt_a, a_major, lda, _ptr(b), fmt_b, b_major, ldb,
                  _ptr(scale_a), _ptr(scale_b), _ptr(bias), bias_dtype, _ptr(bias_scale), _ptr(d), ldd, tile_cfg,
                  _ptr(workspace), _nbytes(workspace))
    s = stream if stream is not None else _stream(d.device if isinstance(d, torch.Tensor) else None)
    _check(_lib.fp8_mm(ctypes.byref(args), s), "fp8_mm")


def fp8_mm_workspace_bytes(m: int, n: int, k: int) -> int:
    return _lib.fp8_mm_workspace_bytes(m, n, k)


def mm_workspace(m: int, n: int, k: int, device) -> torch.Tensor | None:
    """A zero-filled stream-K workspace for GEMMs of this size (None when empty)."""
    nb = fp8_mm_workspace_bytes(m, n, k)
    return torch.zeros(nb, dtype=torch.uint8, device=device) if nb else None


def fp8_mm_plan(a: MmArgs, b: MmArgs | None = None, num_sms: int = 148) -> MmPlanInfo:
    """The tile configuration fp8_mm (or fp8_mm_pair with b) would choose on a
    GPU with num_sms SMs; host arithmetic only (no device needed)."""
    info = MmPlanInfo()
    _check(_lib.fp8_mm_plan(ctypes.byref(a), ctypes.byref(b) if b is not None else None, num_sms,
                            ctypes.byref(info)), "fp8_mm_plan")
    return info


def fp8_dbias_workspace_bytes(M: int, N: int) -> int:
    return _lib.fp8_dbias_workspace_bytes(M, N)


def fp8_dbias(g: torch.Tensor, dbias: torch.Tensor, workspace: torch.Tensor,
              g_scale: torch.Tensor | None = None, g_fmt: int | None = None) -> None:
    M, N = g.shape
    _check(_lib.fp8_dbias(_ptr(g), _dtype_code(g, g_fmt), M, N, _ld(g), _ptr(g_scale), _ptr(dbias),
                          _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(g.device)),
           "fp8_dbias")


def fp8_dbias_noalloc(g: torch.Tensor, dbias: torch.Tensor, g_scale: torch.Tensor | None = None,
                      g_fmt: int | None = None) -> None:
    """fp8_dbias without a workspace: for callers that cannot allocate device
    memory; its scratch is a fixed 1 MiB array inside the library (calls that
    overlap on the GPU race; the first call on a device should come before any
    stream capture)."""
    M, N = g.shape
    _check(_lib.fp8_dbias_noalloc(_ptr(g), _dtype_code(g, g_fmt), M, N, _ld(g), _ptr(g_scale), _ptr(dbias),
                                  _stream(g.device)), "fp8_dbias_noalloc")


def fp8_linear_forward(args: LinearFwdArgs, device=None) -> None:
    _check(_lib.fp8_linear_forward(ctypes.byref(args), _stream(device)), "fp8_linear_forward")


def fp8_linear_backward(args: LinearBwdArgs, device=None) -> None:
    _check(_lib.fp8_linear_backward(ctypes.byref(args), _stream(device)), "fp8_linear_backward")


def fp8_linear_workspace_bytes(M: int, N: int, K: int) -> int:
    return _lib.fp8_linear_workspace_bytes(M, N, K)


def fp8_get_device_status() -> int:
    return _lib.fp8_get_device_status()


def fp8_wait_selftest(flag: torch.Tensor, limit_ns: int, results: torch.Tensor) -> None:
    """Runs the bounded-wait diagnostic kernel: results[0] / results[1] = 1
    where the flag wait / the mbarrier wait was satisfied, 0 where it ran out
    (which fp8_get_device_status then reports as FP8_ERR_DEVICE_TIMEOUT)."""
    _check(_lib.fp8_wait_selftest(_ptr(flag), limit_ns, _ptr(results), _stream(flag.device)), "fp8_wait_selftest")


def fp8_status_string(status: int) -> str:
    return _lib.fp8_status_string(status).decode()


def fp8_version() -> str:
    return _lib.fp8_version().decode()


# --------------------------------------------------------------------------- helpers

class ScaleRing:
    """Delayed-scaling state of one tensor: a device buffer laid out as
    [hist (H fp32) | scale | step | ticket | scratch]."""

    def __init__(self, hist_len: int = 16, device="cuda", seed_amax: float | None = None, fmt: int = FP8_E4M3,
                 buf: torch.Tensor | None = None):
        self.H = hist_len
        words = fp8_ring_bytes(hist_len) // 4
        if buf is not None:
            if buf.dtype != torch.float32 or buf.numel() != words or not buf.is_contiguous():
                raise ValueError(f"ring buffer must be {words} contiguous fp32 words")
            self.buf = buf
        else:
            self.buf = torch.empty(words, dtype=torch.float32, device=device)
        if seed_amax is None:
            fp8_ring_init(self.buf, hist_len)
        else:
            fp8_ring_seed(self.buf, hist_len, fmt, seed_amax)

    @property
    def hist(self):
        return self.buf[: self.H]

    @property
    def scale(self):
        return self.buf[self.H]

    @property
    def step(self):
        return int(self.buf[self.H + 1 : self.H + 2].view(torch.int32).item())

    def words(self):
        return self.buf.view(torch.int32)


def quantize(x: torch.Tensor, fmt: int, ring: ScaleRing | None, out: torch.Tensor | None = None):
    """Quantize x with its ring (ring None: current scaling from x's own amax);
    returns (codes [rows, cols] uint8 view with a 16-aligned row stride, amax
    (1-elem fp32), scale used (1-elem fp32))."""
    rows, cols = x.shape
    if out is None:
        out = fp8_alloc(rows, cols, x.device)
    amax = torch.empty(1, dtype=torch.float32, device=x.device)
    scale = torch.empty(1, dtype=torch.float32, device=x.device)
    fp8_quantize(x, fmt, ring.buf if ring is not None else None, ring.H if ring is not None else 0, out, amax, scale)
    return out, amax, scale


@dataclass
class ForwardResult:
    y: torch.Tensor
    x8: torch.Tensor
    w8: torch.Tensor
    sx: torch.Tensor
    sw: torch.Tensor
    amax_x: torch.Tensor
    amax_w: torch.Tensor


def _fp32_scale(scale: torch.Tensor | None, what: str) -> None:
    """The scale of an operand in fp8 codes, read as one fp32 word (a missing one is the library's to refuse)."""
    if scale is not None and (scale.dtype != torch.float32 or scale.numel() < 1):
        raise ValueError(f"{what}: expected an fp32 scale, got {scale.dtype} {tuple(scale.shape)}")


def linear_forward(x, w, ring_x: ScaleRing | None, ring_w: ScaleRing | None, bias=None, bias_scale=None,
                   fmt_x=FP8_E4M3, fmt_w=FP8_E4M3, x_scale_in=None, w_scale_in=None, hist_len=16,
                   y=None, x8=None, w8=None, scales=None) -> ForwardResult:
    """y = x w^T + bias through fp8_linear_forward.  x/w may be bf16/fp16/fp32
    or fp8 codes (torch.float8_* or uint8 with their fmt, plus *_scale_in).
    scales: optional 4-element fp32 device buffer receiving sx, sw, amax_x,
    amax_w (allocated here when None)."""
    M, K = x.shape
    N = w.shape[0]
    dev = x.device
    xq = x.dtype in (torch.uint8, torch.float8_e4m3fn, torch.float8_e5m2)
    wq = w.dtype in (torch.uint8, torch.float8_e4m3fn, torch.float8_e5m2)
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    # codes are used in place: the result holds the operand itself, not a buffer that stays unwritten
    if xq:
        x8 = x.view(torch.uint8)
        _fp32_scale(x_scale_in, "x_scale_in")
    elif x8 is None:
        x8 = fp8_alloc(M, K, dev)
    if wq:
        w8 = w.view(torch.uint8)
        _fp32_scale(w_scale_in, "w_scale_in")
    elif w8 is None:
        w8 = fp8_alloc(N, K, dev)
    sc = torch.empty(4, dtype=torch.float32, device=dev) if scales is None else scales
    H = ring_x.H if ring_x is not None else (ring_w.H if ring_w is not None else hist_len)
    bias_dtype = FP8_DT_BF16
    if bias is not None and bias.dtype != torch.bfloat16:
        bias_dtype = _dtype_code(bias, FP8_E4M3)
    args = LinearFwdArgs(
        M, N, K,
        _ptr(x), _dtype_code(x, fmt_x), _ld(x), _ptr(x_scale_in),
        _ptr(w), _dtype_code(w, fmt_w), _ld(w), _ptr(w_scale_in),
        _ptr(bias), bias_dtype, _ptr(bias_scale),
        fmt_x, fmt_w, H,
        _ptr(ring_x.buf) if ring_x is not None else None, _ptr(ring_w.buf) if ring_w is not None else None,
        _ptr(x8), _ld(x8), _ptr(w8), _ld(w8),
        _ptr(sc[0:1]), _ptr(sc[1:2]), _ptr(sc[2:3]), _ptr(sc[3:4]),
        _ptr(y), _ld(y))
    fp8_linear_forward(args, dev)
    return ForwardResult(y, x8, w8, sc[0:1], sc[1:2], sc[2:3], sc[3:4])


@dataclass
class BackwardResult:
    dx: torch.Tensor | None
    dw: torch.Tensor | None
    dbias: torch.Tensor | None
    g8: torch.Tensor
    sg: torch.Tensor
    amax_g: torch.Tensor


def linear_backward(g, fwd: ForwardResult, ring_g: ScaleRing | None, fmt_g=FP8_E5M2, fmt_x=FP8_E4M3,
                    fmt_w=FP8_E4M3, need_dx=True, need_dw=True, need_dbias=False, g_scale_in=None,
                    workspace=None, dx=None, dw=None, dbias=None, g8=None) -> BackwardResult:
    """dX, dW, dbias through fp8_linear_backward, reusing the forward's x8/w8
    and scale snapshots."""
    M, N = g.shape
    K = fwd.x8.shape[1]
    dev = g.device
    gq = g.dtype in (torch.uint8, torch.float8_e4m3fn, torch.float8_e5m2)
    if gq:
        g8 = g.view(torch.uint8)
        _fp32_scale(g_scale_in, "g_scale_in")
    elif g8 is None:
        g8 = fp8_alloc(M, N, dev)
    dx = torch.empty((M, K), dtype=torch.bfloat16, device=dev) if (need_dx and dx is None) else dx
    dw = torch.empty((N, K), dtype=torch.bfloat16, device=dev) if (need_dw and dw is None) else dw
    dbias = torch.empty(N, dtype=torch.bfloat16, device=dev) if (need_dbias and dbias is None) else dbias
    if need_dbias and workspace is None:
        workspace = torch.zeros(max(16, fp8_linear_workspace_bytes(M, N, K)), dtype=torch.uint8, device=dev)
    sc = torch.empty(2, dtype=torch.float32, device=dev)
    H = ring_g.H if ring_g is not None else 16
    args = LinearBwdArgs(
        M, N, K,
        _ptr(g), _dtype_code(g, fmt_g), _ld(g), _ptr(g_scale_in),
        fmt_g, H, _ptr(ring_g.buf) if ring_g is not None else None,
        _ptr(g8), _ld(g8), _ptr(sc[0:1]), _ptr(sc[1:2]),
        _ptr(fwd.x8), _ld(fwd.x8), _ptr(fwd.sx), fmt_x,
        _ptr(fwd.w8), _ld(fwd.w8), _ptr(fwd.sw), fmt_w,
        int(need_dx), int(need_dw), int(need_dbias),
        _ptr(dx), _ld(dx) if dx is not None else 0,
        _ptr(dw), _ld(dw) if dw is not None else 0,
        _ptr(dbias),
        _ptr(workspace), (workspace.numel() * workspace.element_size()) if workspace is not None else 0)
    fp8_linear_backward(args, dev)
    return BackwardResult(dx, dw, dbias, g8, sc[0:1], sc[1:2])


# --------------------------------------------------------------------------- grouped and int8
#
# These helpers run in the microseconds between two small launches, so they
# look each tensor property up once and hand the argument structs over as
# packed bytes (half the cost of a ctypes structure).

_CODE_TYPES = {torch.uint8: None, torch.float8_e4m3fn: FP8_E4M3, torch.float8_e5m2: FP8_E5M2}
_WIDE_TYPES = {torch.bfloat16: FP8_DT_BF16, torch.float16: FP8_DT_FP16, torch.float32: FP8_DT_FP32}


def _packer(structure) -> struct.Struct:
    """A struct.Struct that packs a ctypes structure's fields in order, in its C layout."""
    letters = {_I64: "q", _I: "i", _P: "P", _SZ: "N"}
    packer = struct.Struct("@" + "".join(letters[t] for _, t in structure._fields_) + "0q")
    assert packer.size == ctypes.sizeof(structure)
    return packer


def _packed_call(name: str, *args):
    """The entry point `name` with its structs as bytes."""
    fn = _lib[name]
    fn.restype, fn.argtypes = _I, args
    return fn


_pack_mm, _pack_groups = _packer(MmArgs).pack, _packer(Groups).pack
_pack_fwd, _pack_bwd, _pack_int8 = _packer(LinearFwdArgs).pack, _packer(LinearBwdArgs).pack, _packer(LinearInt8Args).pack
_B = ctypes.c_char_p
_call_mm_grouped = _packed_call("fp8_mm_grouped", _B, _I, _B, _P)
_call_grouped_forward = _packed_call("fp8_linear_grouped_forward", _B, _B, _P)
_call_grouped_backward = _packed_call("fp8_linear_grouped_backward", _B, _B, _P)
_call_linear_int8 = _packed_call("fp8_linear_int8_forward", _B, _P)


_current_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _call(where: str, dev: int, fn, *args) -> None:
    """fn on the current stream of device `dev`, which is made current for the call."""
    if _current_device() == dev:
        status = fn(*args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, _raw_stream(dev))
    if status != FP8_OK:
        raise Fp8Error(status, where)


def _one_device(first: torch.Tensor, *others: torch.Tensor | None) -> int:
    """The index of the GPU all the tensors live on."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError(f"expected CUDA tensors, got one on {first.device}")
    for t in others:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"tensors on different devices: {first.device} and {t.device}")
    return dev


_FP32 = torch.float32


def _address(t: torch.Tensor | None) -> int:
    return 0 if t is None else t.data_ptr()


def _matrix(t: torch.Tensor, what: str) -> tuple[int, int, int]:
    """(rows, columns, row stride) of a 2-D tensor with a contiguous last dimension."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or (stride[1] != 1 and shape[1] > 1):
        raise ValueError(f"{what}: expected a 2-D tensor with a contiguous last dimension, got {tuple(shape)}")
    return shape[0], shape[1], (stride[0] if shape[0] > 1 else max(stride[0], shape[1]))


def _experts(t: torch.Tensor, groups: int, what: str) -> tuple[int, int, int]:
    """(rows, columns, row stride) of each matrix of a [groups, rows, columns] tensor whose matrices follow one another."""
    shape, stride = t.shape, t.stride()
    if len(shape) != 3 or shape[0] != groups:
        raise ValueError(f"{what}: expected [groups, rows, columns] with {groups} groups, got {tuple(shape)}")
    if stride[2] != 1 and shape[2] > 1:
        raise ValueError(f"{what}: the last dimension has to be contiguous")
    if groups > 1 and stride[0] != shape[1] * stride[1]:
        raise ValueError(f"{what}: the groups' matrices have to follow one another (stride {shape[1] * stride[1]}, "
                         f"got {stride[0]})")
    return shape[1], shape[2], stride[1]


def _offsets(t: torch.Tensor) -> tuple[int, int]:
    """(groups, 1 for int64) of a row-offset vector."""
    shape, dtype = t.shape, t.dtype
    if len(shape) != 1 or shape[0] < 1 or (t.stride(0) != 1 and shape[0] > 1) or \
            (dtype != torch.int32 and dtype != torch.int64):
        raise ValueError("offsets: a contiguous int32 or int64 vector of groups + 1 row offsets")
    return shape[0] - 1, int(dtype == torch.int64)


def _one_scale(scale: torch.Tensor, what: str) -> None:
    if scale.numel() != 1 or scale.dtype is not _FP32:
        raise ValueError(f"{what}: one fp32 scale, got {scale.dtype} {tuple(scale.shape)}")


def _scale_step(scale: torch.Tensor, groups: int, what: str) -> int:
    n = scale.numel()
    if scale.dtype is not _FP32 or (n != 1 and n != groups) or not scale.is_contiguous():
        raise ValueError(f"{what}: a contiguous fp32 tensor of 1 or {groups} scales")
    return int(n != 1)


def _codes_fmt(t: torch.Tensor, fmt: int, what: str) -> None:
    """fp8 codes of format fmt: uint8, or the float8 type of that format."""
    if t.dtype is torch.uint8:
        return
    held = _CODE_TYPES.get(t.dtype, -1)
    if held != fmt:
        raise ValueError(f"{what}: expected fp8 codes of format {fmt}, got {t.dtype}")


def _own_codes(t: torch.Tensor, given: torch.Tensor | None, what: str) -> torch.Tensor:
    """The uint8 view of an operand that comes as fp8 codes.  The kernels read it in place: a caller's buffer for its
    codes would stay unwritten, so none but the operand itself is taken."""
    codes = t if t.dtype is torch.uint8 else t.view(torch.uint8)
    if given is not None and given is not t and (given.data_ptr() != codes.data_ptr() or given.shape != codes.shape or
                                                 given.stride() != codes.stride() or given.element_size() != 1):
        raise ValueError(f"{what}: the operand is already fp8 codes and used in place, a buffer for them would stay unwritten")
    return codes


def _operand_dtype(t: torch.Tensor, fmt: int) -> tuple[int, bool]:
    """(FP8_DT_*, whether it holds fp8 codes) of a linear's operand."""
    if t.dtype in _CODE_TYPES:
        return FP8_DT_E4M3 + (fmt if t.dtype == torch.uint8 else _CODE_TYPES[t.dtype]), True
    return _wide_dtype(t.dtype), False


def _wide_dtype(dtype: torch.dtype) -> int:
    code = _WIDE_TYPES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def _out(t: torch.Tensor | None, shape: tuple, dtype: torch.dtype, like: torch.Tensor, what: str) -> torch.Tensor:
    if t is None:  # (sizes as arguments: a quarter faster than a tuple)
        return like.new_empty(*shape, dtype=dtype)
    if tuple(t.shape) != shape or t.dtype != dtype:
        raise ValueError(f"{what}: expected {dtype} {shape}, got {t.dtype} {tuple(t.shape)}")
    return t


def fp8_alloc_experts(groups: int, rows: int, cols: int, device) -> torch.Tensor:
    """fp8 code buffer [groups, rows, ld] with ld = cols rounded up to 16, returned as the [groups, rows, cols] view."""
    ld = (cols + 15) // 16 * 16
    return torch.zeros((groups, rows, ld), dtype=torch.uint8, device=device)[:, :, :cols]


def grouped_mm(x8, w8, offsets, sx, sw, y=None, fmt_x=FP8_E4M3, fmt_w=FP8_E4M3, w_major=FP8_K_MAJOR) -> torch.Tensor:
    """y[r] = x8[r] w8[e]^T / (sx sw[e]) for the rows offsets[e] <= r < offsets[e + 1] (bf16; the other rows of y are
    left as they were, or not initialized).  x8 [rows, k] and w8 [groups, n, k] (w_major FP8_MN_MAJOR: [groups, k, n])
    are fp8 codes, sx one scale, sw one or one per group."""
    groups, off64 = _offsets(offsets)
    rows, k, ldx = _matrix(x8, "x8")
    n, kw, ldw = _experts(w8, groups, "w8")
    stride = n * ldw
    if w_major != FP8_K_MAJOR:
        n, kw = kw, n
    if kw != k:
        raise ValueError(f"x8 and w8 of one contraction length: {tuple(x8.shape)}, {tuple(w8.shape)}")
    _codes_fmt(x8, fmt_x, "x8")
    _codes_fmt(w8, fmt_w, "w8")
    _one_scale(sx, "sx")
    step = _scale_step(sw, groups, "sw")
    dev = _one_device(x8, w8, offsets, sx, sw, y)
    if y is None:
        y, ldy = x8.new_empty(rows, n, dtype=torch.bfloat16), n
    else:
        ldy = _matrix(_out(y, (rows, n), torch.bfloat16, x8, "y"), "y")[2]
    _call("fp8_mm_grouped", dev, _call_mm_grouped,
          _pack_mm(rows, n, k, x8.data_ptr(), fmt_x, FP8_K_MAJOR, ldx, w8.data_ptr(), fmt_w, w_major, ldw,
                   sx.data_ptr(), sw.data_ptr(), 0, 0, 0, y.data_ptr(), ldy, FP8_TILE_AUTO, 0, 0),
          FP8_RAGGED_M, _pack_groups(groups, offsets.data_ptr(), off64, stride, 0, step))
    return y


def grouped_linear_forward(x, w, offsets, ring_x: ScaleRing | None, ring_w: ScaleRing | None, fmt_x=FP8_E4M3,
                           fmt_w=FP8_E4M3, x_scale_in=None, w_scale_in=None, hist_len=16, y=None, x8=None,
                           w8=None) -> ForwardResult:
    """y = x w[e]^T for the rows of each group e, through fp8_linear_grouped_forward: the linear_forward of a mixture
    of experts.  x [rows, K] sorted by expert, w [groups, N, K]; either may be bf16/fp16/fp32 or fp8 codes with its
    *_scale_in (w's: one scale, or one per group).  x8 and w8 [groups, N, K] are buffers for the codes of a wide
    operand; one that is codes already is used in place and takes none."""
    groups, off64 = _offsets(offsets)
    M, K, ldx = _matrix(x, "x")
    N, kw, ldw = _experts(w, groups, "w")
    if kw != K:
        raise ValueError(f"x and w of one contraction length: {tuple(x.shape)}, {tuple(w.shape)}")
    (xd, xq), (wd, wq) = _operand_dtype(x, fmt_x), _operand_dtype(w, fmt_w)
    step = _scale_step(w_scale_in, groups, "w_scale_in") if wq and w_scale_in is not None else 0
    ring_x_buf, ring_w_buf = ring_x and ring_x.buf, ring_w and ring_w.buf
    if xq:
        x8 = _own_codes(x, x8, "x8")
        if x_scale_in is not None:
            _one_scale(x_scale_in, "x_scale_in")
    if wq:
        w8 = _own_codes(w, w8, "w8")
    dev = _one_device(x, w, offsets, x_scale_in, w_scale_in, x8, w8, y, ring_x_buf, ring_w_buf)
    if ring_x is not None and ring_w is not None and ring_x.H != ring_w.H:
        raise ValueError("ring_x and ring_w of one history length")
    H = ring_x.H if ring_x is not None else (ring_w.H if ring_w is not None else hist_len)
    y = _out(y, (M, N), torch.bfloat16, x, "y")
    if x8 is None:
        x8 = fp8_alloc(M, K, x.device)
    if w8 is None:
        w8 = fp8_alloc_experts(groups, N, K, x.device)
    if tuple(x8.shape) != (M, K) or tuple(w8.shape) != (groups, N, K) or x8.dtype != torch.uint8 or \
            w8.dtype != torch.uint8:
        raise ValueError("x8 [rows, K] and w8 [groups, N, K] as uint8 codes")
    sc = x.new_empty(3 + (groups if step else 1), dtype=torch.float32)
    at = sc.data_ptr()
    _call("fp8_linear_grouped_forward", dev, _call_grouped_forward,
          _pack_fwd(M, N, K, x.data_ptr(), xd, ldx, _address(x_scale_in), w.data_ptr(), wd, ldw, _address(w_scale_in),
                    0, 0, 0, fmt_x, fmt_w, H, _address(ring_x_buf), _address(ring_w_buf),
                    x8.data_ptr(), _matrix(x8, "x8")[2], w8.data_ptr(), _experts(w8, groups, "w8")[2],
                    at, at + 12, at + 4, at + 8, y.data_ptr(), _matrix(y, "y")[2]),
          _pack_groups(groups, offsets.data_ptr(), off64, 0, 0, step))
    return ForwardResult(y, x8, w8, sc[0:1], sc[3:], sc[1:2], sc[2:3])


def grouped_linear_backward(g, fwd: ForwardResult, offsets, ring_g: ScaleRing | None, fmt_g=FP8_E5M2, fmt_x=FP8_E4M3,
                            fmt_w=FP8_E4M3, need_dx=True, need_dw=True, g_scale_in=None, dx=None, dw=None,
                            g8=None) -> BackwardResult:
    """dx [rows, K] and dw [groups, N, K] through fp8_linear_grouped_backward, reusing the forward's x8, w8 and scale
    snapshots.  Rows of dx outside every group are left as they were (or not initialized).  For a g that comes as fp8
    codes the result's g8 is g itself (another g8 buffer is refused), its sg g_scale_in and its amax_g None."""
    groups, off64 = _offsets(offsets)
    M, N, ldg = _matrix(g, "g")
    x8, w8, sx, sw = fwd.x8, fwd.w8, fwd.sx, fwd.sw
    mx, K, ldx8 = _matrix(x8, "x8")
    nw, kw, ldw8 = _experts(w8, groups, "w8")
    if mx != M or nw != N or kw != K:
        raise ValueError(f"g {tuple(g.shape)}, x8 {tuple(x8.shape)} and w8 {tuple(w8.shape)} do not fit")
    _codes_fmt(x8, fmt_x, "x8")
    _codes_fmt(w8, fmt_w, "w8")
    _one_scale(sx, "sx")
    step = _scale_step(sw, groups, "sw")
    gd, gq = _operand_dtype(g, fmt_g)
    ring_buf = ring_g and ring_g.buf
    if gq:
        g8, ldg8 = _own_codes(g, g8, "g8"), ldg
        if g_scale_in is not None:
            _one_scale(g_scale_in, "g_scale_in")
    dev = _one_device(g, x8, w8, offsets, sx, sw, g_scale_in, dx, dw, g8, ring_buf)
    if not gq:
        g8 = fp8_alloc(M, N, g.device) if g8 is None else g8
        ldg8 = _matrix(_out(g8, (M, N), torch.uint8, g, "g8"), "g8")[2]
    lddx = lddw = K
    if not need_dx:
        dx = None
    elif dx is None:
        dx = g.new_empty(M, K, dtype=torch.bfloat16)
    else:
        lddx = _matrix(_out(dx, (M, K), torch.bfloat16, g, "dx"), "dx")[2]
    if not need_dw:
        dw = None
    elif dw is None:
        dw = g.new_empty(groups, N, K, dtype=torch.bfloat16)
    else:
        lddw = _experts(_out(dw, (groups, N, K), torch.bfloat16, g, "dw"), groups, "dw")[2]
    # a pre-quantized g comes with its scale; one quantized here gets snapshots
    sc = None if gq else g.new_empty(2, dtype=torch.float32)
    at = 0 if gq else sc.data_ptr()
    _call("fp8_linear_grouped_backward", dev, _call_grouped_backward,
          _pack_bwd(M, N, K, g.data_ptr(), gd, ldg, _address(g_scale_in), fmt_g, ring_g.H if ring_g is not None else 16,
                    _address(ring_buf), g8.data_ptr(), ldg8, at, at and at + 4,
                    x8.data_ptr(), ldx8, sx.data_ptr(), fmt_x, w8.data_ptr(), ldw8, sw.data_ptr(), fmt_w,
                    int(need_dx), int(need_dw), 0, _address(dx), lddx, _address(dw), lddw, 0, 0, 0),
          _pack_groups(groups, offsets.data_ptr(), off64, 0, 0, step))
    return BackwardResult(dx, dw, None, g8, g_scale_in, None) if gq else \
        BackwardResult(dx, dw, None, g8, sc[0:1], sc[1:2])


def quantize_int8(x: torch.Tensor, out: torch.Tensor | None = None, scale: torch.Tensor | None = None):
    """Rows of x to int8 by their own largest magnitude; returns (codes [rows, cols], scale [rows] fp32).  A weight
    [N, K] quantized so has one scale per output channel.  The row stride of out is a multiple of 16, and every row's
    bytes up to the next multiple of 16 columns are written (0), so they have to be out's own."""
    rows, cols, ldx = _matrix(x, "x")
    x_dtype = _wide_dtype(x.dtype)
    dev = _one_device(x, out, scale)
    if out is None:  # the kernel writes a row's padding too
        out = x.new_empty(rows, (cols + 15) // 16 * 16, dtype=torch.int8)[:, :cols]
    out = _out(out, (rows, cols), torch.int8, x, "out")
    scale = _out(scale, (rows,), torch.float32, x, "scale")
    if not scale.is_contiguous():
        raise ValueError("scale: contiguous")
    _call("fp8_quantize_int8", dev, _lib.fp8_quantize_int8, x.data_ptr(), x_dtype, rows, cols, ldx,
          out.data_ptr(), _matrix(out, "out")[2], scale.data_ptr())
    return out, scale


@dataclass
class Int8Result:
    y: torch.Tensor
    sx: torch.Tensor
    codes: torch.Tensor   # x8, or the buffer that holds sx and then x8's rows padded to 16
    cols: int

    @property
    def x8(self) -> torch.Tensor:
        if self.codes.dtype == torch.int8:
            return self.codes
        rows = self.sx.numel()
        return self.codes[(rows + 3) // 4 * 4:].view(torch.int8).view(rows, (self.cols + 15) // 16 * 16)[:, : self.cols]


def linear_int8(x, w8, sw, bias=None, y=None, x8=None, sx=None, out_dtype=None) -> Int8Result:
    """y = x w^T + bias in 8-bit integers through fp8_linear_int8_forward: x [rows, K] (bf16/fp16/fp32) is quantized
    row by row, w8 [N, K] int8 and sw [N] come from quantize_int8.  y has x's type unless out_dtype (or y) says
    otherwise."""
    M, K, ldx = _matrix(x, "x")
    N, kw, ldw = _matrix(w8, "w8")
    if kw != K or w8.dtype != torch.int8:
        raise ValueError(f"w8: int8 [N, {K}], got {w8.dtype} {tuple(w8.shape)}")
    if sw.dtype != torch.float32 or sw.numel() != N or not sw.is_contiguous():
        raise ValueError(f"sw: {N} contiguous fp32 scales")
    if bias is not None and (bias.numel() != N or not bias.is_contiguous()):
        raise ValueError(f"bias: {N} contiguous values")
    if out_dtype is None:
        out_dtype = x.dtype if y is None else y.dtype
    x_dtype, y_dtype = _wide_dtype(x.dtype), _wide_dtype(out_dtype)
    bias_dtype = 0 if bias is None else _wide_dtype(bias.dtype)
    dev = _one_device(x, w8, sw, bias, y, x8, sx)
    if y is None:
        y, ldy = x.new_empty(M, N, dtype=out_dtype), N
    else:
        ldy = _matrix(_out(y, (M, N), out_dtype, x, "y"), "y")[2]
    if x8 is None and sx is None:
        # one buffer for both: the scales, then the codes' rows
        ldx8, at = (K + 15) // 16 * 16, (M + 3) // 4 * 4
        codes = x.new_empty(at + M * ldx8 // 4, dtype=torch.float32)
        sx = codes.as_strided((M,), (1,))
        sx_ptr = codes.data_ptr()
        x8_ptr = sx_ptr + 4 * at
    else:
        codes = x8 if x8 is not None else x.new_empty(M, (K + 15) // 16 * 16, dtype=torch.int8)[:, :K]
        ldx8 = _matrix(_out(codes, (M, K), torch.int8, x, "x8"), "x8")[2]
        sx = _out(sx, (M,), torch.float32, x, "sx")
        if not sx.is_contiguous():
            raise ValueError("sx: contiguous")
        sx_ptr, x8_ptr = sx.data_ptr(), codes.data_ptr()
    _call("fp8_linear_int8_forward", dev, _call_linear_int8,
          _pack_int8(M, N, K, x.data_ptr(), x_dtype, ldx, w8.data_ptr(), ldw, sw.data_ptr(), _address(bias), bias_dtype,
                     x8_ptr, ldx8, sx_ptr, y.data_ptr(), y_dtype, ldy))
    return Int8Result(y, sx, codes, K)
