"""FP8 scaled quantization and scaled FP8 GEMM for AMD MI355X (gfx950).

Thin Python binding over the C ABI in include/fp8mi.h (libfp8mi.so).  torch
tensors serve only as device memory and streams: every step of the
computation runs in the library's HIP kernels.  There is no CPU path; every
call raises if the library is missing or the device is not gfx950.

    import fp8_precision_quantization_amd as fp8
    xq = fp8.quantize(x, "e4m3", "tensor")          # x: bf16/fp32 [rows, cols] on cuda
    wq = fp8.quantize(w, "e4m3", "tensor")
    y = fp8.scaled_gemm(xq.q, wq.q, xq.scale_inv, wq.scale_inv)   # y = x w^T, bf16
"""
from __future__ import annotations

import ctypes
import functools
import struct
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib
from ._lib import Fp8Error  # noqa: F401

__all__ = ["quantize", "quantize_dual", "quantize_tensors", "amax", "scaled_gemm", "blockscaled_gemm", "AmaxHistory", "Diag",
           "QuantResult", "Fp8Error", "FORMATS", "GRANULARITIES", "group_grid", "kv_store", "kv_load",
           "KVTensorCache", "KVCache", "grouped_gemm", "workspace", "kv_attention", "kv_evict", "kv_append",
           "lora_add"]

FORMATS = {"e4m3": _lib.FP8_E4M3, "e5m2": _lib.FP8_E5M2}
GRANULARITIES = {"tensor": _lib.FP8_GRAN_TENSOR, "row": _lib.FP8_GRAN_ROW,
                 "1x128": _lib.FP8_GRAN_BLOCK_1x128, "128x128": _lib.FP8_GRAN_BLOCK_128x128}
TORCH_FP8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def _fmt(f) -> int:
    if isinstance(f, str):
        return FORMATS[f]
    return int(f)


def _gran(g) -> int:
    if isinstance(g, str):
        return GRANULARITIES[g]
    return int(g)


# the handle of a device's current stream, without a Stream object around it
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device: torch.device) -> int:
    if _raw_stream is None or device.index is None:
        return torch.cuda.current_stream(device).cuda_stream
    return _raw_stream(device.index)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _same_device(t: torch.Tensor, device: torch.device, name: str) -> None:
    if t.device != device:
        raise ValueError("%s must be on %s, got %s" % (name, device, t.device))


def _matrix(x: torch.Tensor, name: str):
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("%s must be 2-D, got shape %s" % (name, tuple(shape)))
    if not x.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    rows, cols = shape
    stride = x.stride()
    if stride[1] != 1 and cols > 1:
        raise ValueError("%s must have a contiguous last dimension" % name)
    return rows, cols, max(stride[0], 1) if rows > 1 else max(cols, 1)


def _buf(t: torch.Tensor, n: int, dtype, device: torch.device, name: str) -> int:
    """Pointer of a buffer the library reads or writes as n packed elements
    of dtype on device; raises before any launch if t is not one."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.numel() == n and t.device == device
            and t.is_contiguous()):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError("%s must be a tensor on %s" % (name, device))
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    raise ValueError("%s must be a contiguous tensor of %d elements, got shape %s" % (name, n, tuple(t.shape)))


def _out_matrix(out: torch.Tensor, rows: int, cols: int, dtype, device: torch.device, name: str) -> int:
    """Leading dimension of an output matrix [rows, cols] of dtype on device
    with a contiguous last dimension; raises before any launch if out is not one."""
    if not isinstance(out, torch.Tensor) or out.device != device:
        raise ValueError("%s must be a tensor on %s" % (name, device))
    if out.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, out.dtype))
    if tuple(out.shape) != (rows, cols):
        raise ValueError("%s must have shape %s, got %s" % (name, (rows, cols), tuple(out.shape)))
    if cols > 1 and out.stride(1) != 1:
        raise ValueError("%s must have a contiguous last dimension" % name)
    return max(out.stride(0), 1) if rows > 1 else max(cols, 1)


def workspace(device="cuda") -> torch.Tensor:
    """A workspace for the calls that need one (fp8_workspace_size() bytes).
    Calls ordered on one stream may share it; calls running concurrently on
    different streams need one each."""
    return torch.empty(_lib.WORKSPACE_BYTES, dtype=torch.uint8, device=device)


def _workspace(ws: Optional[torch.Tensor], needed: bool, device: torch.device):
    """(tensor kept alive for the call, pointer, bytes).  Without one given, a
    needed workspace comes from torch's allocator, whose blocks are reused in
    the order of the current stream."""
    if not needed and ws is None:
        return None, None, 0
    if ws is None:
        ws = workspace(device)
    if not isinstance(ws, torch.Tensor) or ws.device != device or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on %s" % device)
    nbytes = ws.numel() * ws.element_size()
    if nbytes < _lib.WORKSPACE_BYTES:
        raise ValueError("workspace must hold %d bytes, got %d" % (_lib.WORKSPACE_BYTES, nbytes))
    return ws, ws.data_ptr(), nbytes


def _numel(shape) -> int:
    n = 1
    for d in shape:
        n *= d
    return n


def group_grid(granularity, rows: int, cols: int):
    g = _gran(granularity)
    if g == _lib.FP8_GRAN_TENSOR:
        return (1,)
    if g == _lib.FP8_GRAN_ROW:
        return (rows,)
    if g == _lib.FP8_GRAN_BLOCK_1x128:
        return (rows, (cols + 127) // 128)
    return ((rows + 127) // 128, (cols + 127) // 128)


class Diag:
    """Device counters (sat, nonfinite, underflow); the library adds to them."""

    def __init__(self, device="cuda"):
        self.buf = torch.zeros(4, dtype=torch.int32, device=device)

    def zero_(self):
        self.buf.zero_()
        return self

    def read(self) -> dict:
        v = self.buf.cpu().tolist()
        return {"sat": v[0], "nonfinite": v[1], "underflow": v[2]}


class AmaxHistory:
    """Delayed-scaling state: a 128-byte device struct (fp8_amax_history)."""

    def __init__(self, length: int = 16, device="cuda"):
        self.buf = torch.empty(_lib.HISTORY_BYTES // 4, dtype=torch.int32, device=device)
        self.length = length
        self.reset()

    def reset(self):
        dev = self.buf.device
        _lib.check(_lib.lib().fp8_history_init(self.buf.data_ptr(), self.length, _stream(dev)),
                   "fp8_history_init")

    def set_guard(self, threshold: float):
        """Spike threshold for quantize(..., spike_guard=True); <= 0 is off."""
        dev = self.buf.device
        _lib.check(_lib.lib().fp8_history_set_guard(self.buf.data_ptr(), float(threshold), _stream(dev)),
                   "fp8_history_set_guard")

    def state(self) -> dict:
        w = self.buf.cpu()
        f = w.view(torch.float32)
        return {"amax": f[:16].clone(), "len": int(w[16]), "pos": int(w[17]), "count": int(w[18]),
                "scale": float(f[21]), "scale_inv": float(f[22]), "steps": int(w[23]),
                "spike_threshold": float(f[24]), "spikes": int(w[25]), "last_spiked": int(w[19])}

    def save(self) -> torch.Tensor:
        return self.buf.clone()

    def load(self, saved: torch.Tensor):
        self.buf.copy_(saved)


@dataclass
class QuantResult:
    q: torch.Tensor            # uint8 codes
    scale_inv: torch.Tensor    # fp32, group grid
    amax: torch.Tensor         # fp32, group grid
    fmt: str

    def as_float8(self) -> torch.Tensor:
        return self.q.view(TORCH_FP8[self.fmt])


def quantize(x: torch.Tensor, fmt="e4m3", granularity="tensor", pow2: bool = False,
             history: Optional[AmaxHistory] = None, transpose: bool = False,
             diag: Optional[Diag] = None, out: Optional[torch.Tensor] = None,
             spike_guard: bool = False,
             scale_inv_out: Optional[torch.Tensor] = None,
             amax_out: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None) -> QuantResult:
    rows, cols, ld = _matrix(x, "x")
    if x.dtype == torch.bfloat16:
        in_dt = _lib.FP8_IN_BF16
    elif x.dtype == torch.float32:
        in_dt = _lib.FP8_IN_F32
    else:
        raise TypeError("x must be bfloat16 or float32, got %s" % x.dtype)
    fmt_name = fmt if isinstance(fmt, str) else ("e4m3" if fmt == 0 else "e5m2")
    grid = group_grid(granularity, rows, cols)
    dev = x.device
    oshape = (cols, rows) if transpose else (rows, cols)
    if out is None:
        out = torch.empty(oshape, dtype=torch.uint8, device=dev)
    ldq = _out_matrix(out, oshape[0], oshape[1], torch.uint8, dev, "out")
    if scale_inv_out is None:
        scale_inv_out = torch.empty(grid, dtype=torch.float32, device=dev)
    if amax_out is None:
        amax_out = torch.empty(grid, dtype=torch.float32, device=dev)
    _buf(scale_inv_out, _numel(grid), torch.float32, dev, "scale_inv_out")
    _buf(amax_out, _numel(grid), torch.float32, dev, "amax_out")
    flags = ((_lib.FP8_SCALE_POW2 if pow2 else 0) | (_lib.FP8_TRANSPOSE_OUT if transpose else 0)
             | (_lib.FP8_SPIKE_GUARD if spike_guard else 0))
    ws, ws_ptr, ws_bytes = _workspace(workspace, _gran(granularity) == _lib.FP8_GRAN_TENSOR, dev)
    st = _lib.lib().fp8_quantize(
        x.data_ptr(), in_dt, rows, cols, ld, _fmt(fmt), _gran(granularity), flags,
        _ptr(history.buf) if history is not None else None, out.data_ptr(), ldq,
        scale_inv_out.data_ptr(), amax_out.data_ptr(), _ptr(diag.buf) if diag is not None else None,
        ws_ptr, ws_bytes, _stream(dev))
    _lib.check(st, "fp8_quantize")
    return QuantResult(out, scale_inv_out, amax_out, fmt_name)


def quantize_dual(x: torch.Tensor, fmt="e5m2", pow2: bool = False, history: Optional[AmaxHistory] = None,
                  diag: Optional[Diag] = None, spike_guard: bool = False,
                  out: Optional[torch.Tensor] = None, out_t: Optional[torch.Tensor] = None,
                  scale_inv_out: Optional[torch.Tensor] = None,
                  amax_out: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None):
    """Per-tensor quantization into both layouts from one pass over x
    (fp8_quantize_dual).  Returns (QuantResult with q [rows x cols], qt [cols x rows])."""
    rows, cols, ld = _matrix(x, "x")
    if x.dtype == torch.bfloat16:
        in_dt = _lib.FP8_IN_BF16
    elif x.dtype == torch.float32:
        in_dt = _lib.FP8_IN_F32
    else:
        raise TypeError("x must be bfloat16 or float32, got %s" % x.dtype)
    fmt_name = fmt if isinstance(fmt, str) else ("e4m3" if fmt == 0 else "e5m2")
    dev = x.device
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
    if out_t is None:
        out_t = torch.empty((cols, rows), dtype=torch.uint8, device=dev)
    ldq = _out_matrix(out, rows, cols, torch.uint8, dev, "out")
    ldqt = _out_matrix(out_t, cols, rows, torch.uint8, dev, "out_t")
    if scale_inv_out is None:
        scale_inv_out = torch.empty((1, 1), dtype=torch.float32, device=dev)
    if amax_out is None:
        amax_out = torch.empty((1, 1), dtype=torch.float32, device=dev)
    _buf(scale_inv_out, 1, torch.float32, dev, "scale_inv_out")
    _buf(amax_out, 1, torch.float32, dev, "amax_out")
    flags = (_lib.FP8_SCALE_POW2 if pow2 else 0) | (_lib.FP8_SPIKE_GUARD if spike_guard else 0)
    ws, ws_ptr, ws_bytes = _workspace(workspace, True, dev)
    st = _lib.lib().fp8_quantize_dual(
        x.data_ptr(), in_dt, rows, cols, ld, _fmt(fmt), flags,
        _ptr(history.buf) if history is not None else None, out.data_ptr(), ldq, out_t.data_ptr(), ldqt,
        scale_inv_out.data_ptr(), amax_out.data_ptr(), _ptr(diag.buf) if diag is not None else None,
        ws_ptr, ws_bytes, _stream(dev))
    _lib.check(st, "fp8_quantize_dual")
    return QuantResult(out, scale_inv_out, amax_out, fmt_name), out_t


def quantize_tensors(xs, fmt="e4m3", pow2: bool = False, outs=None, diags=None, scale_inv_outs=None,
                     amax_outs=None, workspace: Optional[torch.Tensor] = None) -> list:
    """Just-in-time per-tensor quantization of up to 8 contiguous tensors in
    one amax launch and one cast launch (fp8_quantize_tensors).  xs: 2-D
    contiguous tensors of one dtype (bfloat16 or float32) on one device;
    outs: optional uint8 tensors of the same shapes; diags: optional Diag per
    tensor (None entries skip the counting); scale_inv_outs, amax_outs:
    optional one-element fp32 tensors per tensor.  Returns one QuantResult
    per tensor, each equal to quantize(x, fmt, "tensor", pow2)."""
    xs = list(xs)
    n = len(xs)
    if not 1 <= n <= _lib.MAX_TENSORS:
        raise ValueError("quantize_tensors takes 1..%d tensors, got %d" % (_lib.MAX_TENSORS, n))
    dev = xs[0].device
    if dev.type != "cuda":
        raise ValueError("tensors must be device tensors, got %s" % dev)
    dt = xs[0].dtype
    if dt == torch.bfloat16:
        in_dt = _lib.FP8_IN_BF16
    elif dt == torch.float32:
        in_dt = _lib.FP8_IN_F32
    else:
        raise TypeError("tensors must be bfloat16 or float32, got %s" % dt)
    fmt_name = fmt if isinstance(fmt, str) else ("e4m3" if fmt == 0 else "e5m2")
    outs = list(outs) if outs is not None else [None] * n
    diags = list(diags) if diags is not None else [None] * n
    sinvs = list(scale_inv_outs) if scale_inv_outs is not None else [None] * n
    amaxs = list(amax_outs) if amax_outs is not None else [None] * n
    if len(outs) != n or len(diags) != n or len(sinvs) != n or len(amaxs) != n:
        raise ValueError("outs, diags, scale_inv_outs and amax_outs must have one entry per tensor")
    descs = (_lib.Fp8Tensor * n)()
    results = []
    for i, x in enumerate(xs):
        if x.dtype != dt:
            raise TypeError("tensor %d is %s, tensor 0 is %s" % (i, x.dtype, dt))
        _same_device(x, dev, "tensor %d" % i)
        if x.dim() != 2:
            raise ValueError("tensor %d must be 2-D, got shape %s" % (i, tuple(x.shape)))
        rows, cols = x.shape
        if x.numel() > 0 and not x.is_contiguous():
            raise ValueError("tensor %d must be contiguous" % i)
        out = outs[i]
        if out is None:
            out = torch.empty((rows, cols), dtype=torch.uint8, device=dev)
        _out_matrix(out, rows, cols, torch.uint8, dev, "outs[%d]" % i)
        if not out.is_contiguous():
            raise ValueError("outs[%d] must be contiguous" % i)
        sinv = sinvs[i] if sinvs[i] is not None else torch.empty((1, 1), dtype=torch.float32, device=dev)
        am = amaxs[i] if amaxs[i] is not None else torch.empty((1, 1), dtype=torch.float32, device=dev)
        _buf(sinv, 1, torch.float32, dev, "scale_inv_outs[%d]" % i)
        _buf(am, 1, torch.float32, dev, "amax_outs[%d]" % i)
        descs[i] = _lib.Fp8Tensor(x.data_ptr(), rows, cols, out.data_ptr(), sinv.data_ptr(), am.data_ptr(),
                                  _ptr(diags[i].buf) if diags[i] is not None else None)
        results.append(QuantResult(out, sinv, am, fmt_name))
    ws, ws_ptr, ws_bytes = _workspace(workspace, True, dev)
    st = _lib.lib().fp8_quantize_tensors(ctypes.cast(descs, ctypes.c_void_p), n, in_dt, _fmt(fmt), _lib.FP8_SCALE_POW2 if pow2 else 0,
                                         ws_ptr, ws_bytes, _stream(dev))
    _lib.check(st, "fp8_quantize_tensors")
    return results


def amax(x: torch.Tensor, granularity="tensor", out: Optional[torch.Tensor] = None,
         workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    rows, cols, ld = _matrix(x, "x")
    in_dt = _lib.FP8_IN_BF16 if x.dtype == torch.bfloat16 else _lib.FP8_IN_F32
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("x must be bfloat16 or float32")
    grid = group_grid(granularity, rows, cols)
    if out is None:
        out = torch.empty(grid, dtype=torch.float32, device=x.device)
    _buf(out, _numel(grid), torch.float32, x.device, "out")
    ws, ws_ptr, ws_bytes = _workspace(workspace, _gran(granularity) == _lib.FP8_GRAN_TENSOR, x.device)
    st = _lib.lib().fp8_amax(x.data_ptr(), in_dt, rows, cols, ld, _gran(granularity), out.data_ptr(),
                             ws_ptr, ws_bytes, _stream(x.device))
    _lib.check(st, "fp8_amax")
    return out


def _out_dtype(dt) -> int:
    if dt == torch.bfloat16:
        return _lib.FP8_OUT_BF16
    if dt == torch.float32:
        return _lib.FP8_OUT_F32
    raise TypeError("out dtype must be bfloat16 or float32")


def scaled_gemm(a_q: torch.Tensor, b_q: torch.Tensor, a_scale_inv: torch.Tensor,
                b_scale_inv: torch.Tensor, fa="e4m3", fb="e4m3", out_dtype=torch.bfloat16,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """C = (A_q . B_q^T) * sa * sb with A_q [M, K], B_q [N, K] uint8 codes."""
    M, K, lda = _matrix(a_q, "a_q")
    N, K2, ldb = _matrix(b_q, "b_q")
    if K != K2:
        raise ValueError("K mismatch: %d vs %d" % (K, K2))
    dev = a_q.device
    _same_device(b_q, dev, "b_q")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    ldc = _out_matrix(out, M, N, out.dtype, dev, "out")
    a_row = 0 if a_scale_inv.numel() == 1 else 1
    b_row = 0 if b_scale_inv.numel() == 1 else 1
    if a_row and a_scale_inv.numel() != M:
        raise ValueError("a_scale_inv must hold 1 or M=%d values" % M)
    if b_row and b_scale_inv.numel() != N:
        raise ValueError("b_scale_inv must hold 1 or N=%d values" % N)
    _buf(a_scale_inv, M if a_row else 1, torch.float32, dev, "a_scale_inv")
    _buf(b_scale_inv, N if b_row else 1, torch.float32, dev, "b_scale_inv")
    st = _lib.lib().fp8_scaled_gemm(a_q.data_ptr(), _fmt(fa), lda, b_q.data_ptr(), _fmt(fb), ldb, M, N, K,
                                    a_scale_inv.data_ptr(), a_row, b_scale_inv.data_ptr(), b_row,
                                    out.data_ptr(), _out_dtype(out.dtype), ldc, _stream(a_q.device))
    _lib.check(st, "fp8_scaled_gemm")
    return out


def blockscaled_gemm(a_q: torch.Tensor, b_q: torch.Tensor, a_scale_inv: torch.Tensor,
                     b_scale_inv: torch.Tensor, out_dtype=torch.bfloat16,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """E4M3 block-scaled GEMM: a_scale_inv [M, K/128], b_scale_inv [N/128, K/128]."""
    M, K, lda = _matrix(a_q, "a_q")
    N, K2, ldb = _matrix(b_q, "b_q")
    if K != K2:
        raise ValueError("K mismatch: %d vs %d" % (K, K2))
    dev = a_q.device
    _same_device(b_q, dev, "b_q")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    ldc = _out_matrix(out, M, N, out.dtype, dev, "out")
    if K % 128 == 0 and N % 128 == 0:     # else the library reports the unsupported shape
        _buf(a_scale_inv, M * (K // 128), torch.float32, dev, "a_scale_inv")
        _buf(b_scale_inv, (N // 128) * (K // 128), torch.float32, dev, "b_scale_inv")
    st = _lib.lib().fp8_blockscaled_gemm(a_q.data_ptr(), lda, b_q.data_ptr(), ldb, M, N, K,
                                         a_scale_inv.data_ptr(), b_scale_inv.data_ptr(), out.data_ptr(),
                                         _out_dtype(out.dtype), ldc, _stream(a_q.device))
    _lib.check(st, "fp8_blockscaled_gemm")
    return out


# ------------------------------------------------------------ grouped GEMM --
def grouped_gemm(a_q: torch.Tensor, b_q: torch.Tensor, group_offsets: torch.Tensor, a_scale_inv: torch.Tensor,
                 b_scale_inv: torch.Tensor, fa="e4m3", fb="e4m3", out_dtype=torch.bfloat16,
                 out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """MoE grouped GEMM: rows [offs[g], offs[g+1]) of a_q [M, K] times expert
    g's b_q[g] ([G, N, K] uint8 codes): C[m] = (A_q[m] . B_q[g]^T) * sa * sb_g.
    group_offsets: int32 device tensor [G+1]; a_scale_inv: 1 or M values;
    b_scale_inv: G (one per expert) or G*N values.  Rows in no group are not
    written (out is allocated uninitialized when not given)."""
    M, K, lda = _matrix(a_q, "a_q")
    if b_q.dim() != 3 or not b_q.is_cuda or b_q.stride(2) != 1:
        raise ValueError("b_q must be a [G, N, K] device tensor with contiguous rows")
    G, N, K2 = b_q.shape
    if K != K2:
        raise ValueError("K mismatch: %d vs %d" % (K, K2))
    if (group_offsets.dtype != torch.int32 or not group_offsets.is_cuda or group_offsets.numel() != G + 1
            or not group_offsets.is_contiguous()):
        raise ValueError("group_offsets must be a contiguous int32 device tensor of G+1=%d entries" % (G + 1))
    ldb = b_q.stride(1) if N > 1 else K
    gstride = b_q.stride(0) if G > 1 else N * ldb
    dev = a_q.device
    _same_device(b_q, dev, "b_q")
    _same_device(group_offsets, dev, "group_offsets")
    if out is None:
        out = torch.empty((M, N), dtype=out_dtype, device=dev)
    ldc = _out_matrix(out, M, N, out.dtype, dev, "out")
    a_row = 0 if a_scale_inv.numel() == 1 else 1
    if a_row and a_scale_inv.numel() != M:
        raise ValueError("a_scale_inv must hold 1 or M=%d values" % M)
    if b_scale_inv.numel() == G:
        b_row = 0
    elif b_scale_inv.numel() == G * N:
        b_row = 1
    else:
        raise ValueError("b_scale_inv must hold G=%d or G*N=%d values" % (G, G * N))
    _buf(a_scale_inv, M if a_row else 1, torch.float32, dev, "a_scale_inv")
    _buf(b_scale_inv, G * N if b_row else G, torch.float32, dev, "b_scale_inv")
    ws, ws_ptr, ws_bytes = _workspace(workspace, True, dev)
    st = _lib.lib().fp8_grouped_gemm(a_q.data_ptr(), _fmt(fa), lda, b_q.data_ptr(), _fmt(fb), ldb, gstride, M, N, K,
                                     G, group_offsets.data_ptr(), a_scale_inv.data_ptr(), a_row,
                                     b_scale_inv.data_ptr(), b_row, out.data_ptr(), _out_dtype(out.dtype), ldc,
                                     ws_ptr, ws_bytes, _stream(a_q.device))
    _lib.check(st, "fp8_grouped_gemm")
    return out


# ------------------------------------------- adapters beside a projection --
@functools.lru_cache(maxsize=1024)
def _lora_workspace(rows, columns, inner, rank, adapters, slices) -> int:
    return _lib.lib().fp8_lora_workspace(rows, columns, inner, rank, adapters, slices)


def lora_add(y: torch.Tensor, x: torch.Tensor, a: torch.Tensor, b: torch.Tensor, ids: torch.Tensor,
             gain: Optional[torch.Tensor] = None, slices=None, out: Optional[torch.Tensor] = None,
             workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Add to every row of a projection's output y the product of the row's own
    low-rank adapter (fp8_lora_add): out[m] = y[m] + gain[l] * B_l (A_l x[m])
    with l = ids[m]; rows whose id is outside 0..adapters-1 stay as they are.

    y: bf16 or fp32 [rows, columns] (of scaled_gemm, say); x: bf16 [rows,
    inner], the projection's input before its cast; a: bf16 [adapters, rank,
    inner]; b: bf16 [adapters, columns, rank]; ids: int32 [rows], in any order
    (batches of more than 1024 rows are fastest with the rows of an adapter
    together); gain: fp32 [adapters], default 1.  slices: the columns of each
    part of a fused projection that has adapters of its own, (q, k, v) say;
    then a is [adapters, len(slices) * rank, inner].  rank: a multiple of 8 up
    to 128 (a smaller adapter is padded with zeros).

    out: where to write, y itself included (default: a new tensor).
    workspace: a uint8 device tensor for callers that may not allocate
    (fp8_lora_workspace bytes).  No gradient is formed.

    A x is summed and kept in fp32 and enters the second product with 16
    significant bits (bf16 out) or 24 (fp32 out); one rounding at the end.
    Infinities are the formula's, in their rows and columns alone."""
    rows, columns, ldy = _matrix(y, "y")
    rows_x, inner, ldx = _matrix(x, "x")
    dev = y.device
    _same_device(x, dev, "x")
    if x.dtype != torch.bfloat16:
        raise TypeError("x must be torch.bfloat16, got %s" % x.dtype)
    if rows_x != rows:
        raise ValueError("x has %d rows, y %d" % (rows_x, rows))
    dtype = _out_dtype(y.dtype)
    for t, name in ((a, "a"), (b, "b")):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError("%s must be a 3-D tensor" % name)
    parts = 1 if slices is None else len(slices)
    adapters, width, rank = a.shape[0], a.shape[1], b.shape[2]
    if slices is not None:
        if not 1 <= parts <= 4:
            raise ValueError("slices must name 1..4 parts, got %d" % parts)
        for n in slices:
            _int32(n, "slices")
    if a.shape[2] != inner or width != parts * rank:
        raise ValueError("a must be [adapters, %d, %d], got shape %s" % (parts * rank, inner, tuple(a.shape)))
    if tuple(b.shape[:2]) != (adapters, columns):
        raise ValueError("b must be [%d, %d, rank], got shape %s" % (adapters, columns, tuple(b.shape)))
    for value, name in ((adapters, "adapters"), (rank, "rank")):
        _int32(value, name)
    a_ptr = _buf(a, a.numel(), torch.bfloat16, dev, "a")
    b_ptr = _buf(b, b.numel(), torch.bfloat16, dev, "b")
    ids_ptr = _buf(ids, rows, torch.int32, dev, "ids")
    gain_ptr = None if gain is None else _buf(gain, adapters, torch.float32, dev, "gain")
    if out is None:
        out = torch.empty((rows, columns), dtype=y.dtype, device=dev)
    ldo = _out_matrix(out, rows, columns, y.dtype, dev, "out")
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.device != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on %s" % dev)
        ws_bytes = workspace.numel() * workspace.element_size()
    else:
        ws_bytes = _lora_workspace(rows, columns, inner, rank, adapters, parts)
        if ws_bytes > 0:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    cuts = None if slices is None else _INTS[parts](*slices)
    st = _call_on(dev, _lib.lib().fp8_lora_add, y.data_ptr(), ldy, x.data_ptr(), ldx, a_ptr, b_ptr, ids_ptr, gain_ptr,
                  out.data_ptr(), ldo, dtype, rows, columns, inner, rank, adapters, cuts, parts, _ptr(workspace),
                  ws_bytes)
    _lib.check(st, "fp8_lora_add")
    return out


# ------------------------------------------------------------ FP8 KV cache --
KV_STORAGE = {"e4m3": _lib.FP8_KV_E4M3, "e5m2": _lib.FP8_KV_E5M2, "bf16": _lib.FP8_KV_BF16}
KV_SCALING = {"token_head": _lib.FP8_KV_PER_TOKEN_HEAD, "head": _lib.FP8_KV_PER_HEAD}


def _kv_rows(x: torch.Tensor, heads: int, head_dim: int, name: str):
    """(n, ld) of a [n, heads*head_dim] or [n, heads, head_dim] device tensor
    whose heads are packed back to back within a token."""
    if not x.is_cuda:
        raise ValueError("%s must be a device tensor" % name)
    shape, stride = x.shape, x.stride()
    if len(shape) == 3:
        if shape[1] != heads or shape[2] != head_dim or stride[2] != 1 or (heads > 1 and stride[1] != head_dim):
            raise ValueError("%s [n, heads, head_dim] must have packed heads" % name)
    elif len(shape) == 2:
        if shape[1] != heads * head_dim or (shape[1] > 1 and stride[1] != 1):
            raise ValueError("%s must be [n, %d] with a contiguous last dimension" % (name, heads * head_dim))
    else:
        raise ValueError("%s must be 2-D or 3-D" % name)
    n = shape[0]
    return n, (stride[0] if n > 1 else heads * head_dim)


def _kv_scales(scale_inv: Optional[torch.Tensor], storage: str, scaling: str, capacity: int, heads: int,
               device: torch.device):
    """Pointer of a cache's scales: [capacity, heads] per (token, head), [heads]
    fixed per head; none for bf16 storage (the library reports a missing one)."""
    if scale_inv is None or storage == "bf16":
        return _ptr(scale_inv)
    n = capacity * heads if scaling == "token_head" else heads
    return _buf(scale_inv, n, torch.float32, device, "scale_inv")


def _slots(slots: Optional[torch.Tensor], n: int):
    if slots is None:
        return None
    if slots.dtype != torch.int64 or not slots.is_cuda or slots.shape != (n,) or not slots.is_contiguous():
        raise ValueError("slots must be a contiguous int64 device tensor of %d entries" % n)
    return slots.data_ptr()


def kv_store(x: torch.Tensor, cache: torch.Tensor, scale_inv: Optional[torch.Tensor], storage="e4m3",
             scaling="token_head", slots: Optional[torch.Tensor] = None, pow2: bool = False,
             diag: Optional[Diag] = None) -> None:
    """Store new tokens' vectors x [n, heads*head_dim] (bf16/fp32) into one
    layer's cache [capacity, heads, head_dim] (uint8 codes, bf16 for the
    "bf16" storage) at rows `slots` (None: rows 0..n-1; negative = padding)."""
    capacity, heads, head_dim = cache.shape
    n, ld = _kv_rows(x, heads, head_dim, "x")
    if x.dtype == torch.bfloat16:
        in_dt = _lib.FP8_IN_BF16
    elif x.dtype == torch.float32:
        in_dt = _lib.FP8_IN_F32
    else:
        raise TypeError("x must be bfloat16 or float32, got %s" % x.dtype)
    want = torch.bfloat16 if storage == "bf16" else torch.uint8
    if cache.dtype != want or not cache.is_contiguous():
        raise ValueError("cache must be a contiguous %s tensor" % want)
    _same_device(x, cache.device, "x")
    if slots is not None:
        _same_device(slots, cache.device, "slots")
    st = _lib.lib().fp8_kv_store(
        x.data_ptr(), in_dt, n, ld, heads, head_dim, _slots(slots, n), KV_STORAGE[storage],
        KV_SCALING[scaling], _lib.FP8_SCALE_POW2 if pow2 else 0, cache.data_ptr(),
        _kv_scales(scale_inv, storage, scaling, capacity, heads, cache.device), capacity,
        _ptr(diag.buf) if diag is not None else None, _stream(cache.device))
    _lib.check(st, "fp8_kv_store")


def kv_load(cache: torch.Tensor, scale_inv: Optional[torch.Tensor], n: Optional[int] = None, storage="e4m3",
            scaling="token_head", slots: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gather n cache rows (slots, or rows 0..n-1) as dequantized values
    out [n, heads*head_dim] (bf16 or fp32)."""
    capacity, heads, head_dim = cache.shape
    if n is None:
        n = slots.shape[0] if slots is not None else capacity
    if out is None:
        out = torch.empty((n, heads * head_dim), dtype=out_dtype, device=cache.device)
    n2, ld_out = _kv_rows(out, heads, head_dim, "out")
    if n2 != n:
        raise ValueError("out has %d rows, expected %d" % (n2, n))
    _same_device(out, cache.device, "out")
    if slots is not None:
        _same_device(slots, cache.device, "slots")
    st = _lib.lib().fp8_kv_load(
        cache.data_ptr(), KV_STORAGE[storage], KV_SCALING[scaling],
        _kv_scales(scale_inv, storage, scaling, capacity, heads, cache.device), capacity, heads, head_dim,
        _slots(slots, n), n, _out_dtype(out.dtype), out.data_ptr(), ld_out, _stream(cache.device))
    _lib.check(st, "fp8_kv_load")
    return out


# ---------------------------------------- attention over the cache, eviction --
_PAIR = struct.Struct("PPPPqPqPqiiiiiiii")     # fp8_kv_pair (_lib.Fp8KvPair) as the bytes a call passes


def _int32(value: int, name: str) -> None:
    """A number the library takes as int32: ctypes would pass its low 32 bits."""
    if not -(1 << 31) <= value < 1 << 31:
        raise ValueError("%s=%d does not fit in 32 bits" % (name, value))


# int32 arrays a call passes, by length
_INTS = [ctypes.c_int32 * n for n in range(5)]


_CACHE_DTYPE = {"e4m3": torch.uint8, "e5m2": torch.uint8, "bf16": torch.bfloat16}


def _caches(k_cache, v_cache, k_scale_inv, v_scale_inv, k_storage, v_storage, scaling):
    """A layer's K and V caches: (capacity, heads, head_dim, device, pointers of K's and V's scales).  Raises if one
    is not what the library would read."""
    shape = k_cache.shape
    if len(shape) != 3 or not k_cache.is_cuda:
        raise ValueError("k_cache must be a [capacity, heads, head_dim] device tensor")
    dev = k_cache.device
    if v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must have one shape, got %s and %s"
                         % (tuple(shape), tuple(v_cache.shape)))
    if k_cache.dtype is not _CACHE_DTYPE[k_storage] or not k_cache.is_contiguous():
        raise ValueError("k_cache must be a contiguous %s tensor on %s" % (_CACHE_DTYPE[k_storage], dev))
    if v_cache.dtype is not _CACHE_DTYPE[v_storage] or not v_cache.is_contiguous() or v_cache.device != dev:
        raise ValueError("v_cache must be a contiguous %s tensor on %s" % (_CACHE_DTYPE[v_storage], dev))
    capacity, heads, head_dim = shape
    return (capacity, heads, head_dim, dev,
            _kv_scales(k_scale_inv, k_storage, scaling, capacity, heads, dev) or 0,
            _kv_scales(v_scale_inv, v_storage, scaling, capacity, heads, dev) or 0)


def _kv_pair(k_cache, v_cache, page_table, lens, page_size, k_scale_inv, v_scale_inv, k_storage, v_storage, scaling,
             max_len):
    """The fp8_kv_pair (as bytes) of a layer's K and V caches and a batch's
    pages, and the sizes in it: (pair, heads, head_dim, batch, max_len).
    Raises before any launch if a buffer is not what the library would read."""
    _int32(page_size, "page_size")
    capacity, heads, head_dim, dev, k_scale, v_scale = _caches(k_cache, v_cache, k_scale_inv, v_scale_inv, k_storage,
                                                               v_storage, scaling)
    if page_table.dim() != 2 or page_table.dtype != torch.int32 or page_table.device != dev:
        raise ValueError("page_table must be an int32 [batch, pages] tensor on %s" % dev)
    batch, pages = page_table.shape
    page_ld, last = page_table.stride()
    if pages > 1 and last != 1:
        raise ValueError("page_table must have a contiguous last dimension")
    if batch <= 1:
        page_ld = pages
    elif page_ld < pages:
        raise ValueError("page_table must not overlap itself")
    if max_len is None:
        max_len = pages * page_size
    elif max_len > pages * page_size:
        raise ValueError("max_len=%d needs more than the %d pages of page_table" % (max_len, pages))
    pair = _PAIR.pack(
        k_cache.data_ptr(), v_cache.data_ptr(), k_scale, v_scale, capacity, page_table.data_ptr(),
        page_ld, _buf(lens, batch, torch.int32, dev, "lens"), max_len, KV_STORAGE[k_storage], KV_STORAGE[v_storage],
        KV_SCALING[scaling], heads, head_dim, page_size, batch, 0)
    return pair, heads, head_dim, batch, max_len


@functools.lru_cache(maxsize=1024)
def _attention_workspace(k_storage, heads, head_dim, page_size, batch, max_len, total_q, q_heads, ragged, window,
                         sinks, weighted, shared) -> int:
    """fp8_kv_attention_shared_workspace of these sizes (it reads nothing else)."""
    pair = _PAIR.pack(0, 0, 0, 0, 1, 0, max_len, 0, max_len, KV_STORAGE[k_storage], 0, 0, heads, head_dim, page_size,
                      batch, 0)
    return _lib.lib().fp8_kv_attention_shared_workspace(pair, total_q, q_heads, ragged, window, sinks, weighted, shared)


def _kv_weights(weights, batch: int, heads: int, least: int, device, name: str) -> int:
    """Leading dimension of fp32 weights [batch, heads, >= least]."""
    if not isinstance(weights, torch.Tensor) or weights.device != device:
        raise ValueError("%s must be a tensor on %s" % (name, device))
    if weights.dtype != torch.float32:
        raise TypeError("%s must be torch.float32, got %s" % (name, weights.dtype))
    if weights.dim() != 3 or tuple(weights.shape[:2]) != (batch, heads) or weights.shape[2] < least:
        raise ValueError("%s must be [%d, %d, >= %d], got shape %s" % (name, batch, heads, least,
                                                                       tuple(weights.shape)))
    ld = weights.shape[2]
    if heads > 1:
        ld = weights.stride(1)
    elif batch > 1:
        ld = weights.stride(0)
    if ((weights.shape[2] > 1 and weights.stride(2) != 1) or ld < weights.shape[2]
            or (batch > 1 and weights.stride(0) != heads * ld)):
        raise ValueError("%s must be rows of one pitch with a contiguous last dimension" % name)
    return max(ld, 1)


def _heads_matrix(x, head_dim: int, name: str):
    """(rows, heads, row pitch) of a [n, heads, head_dim] bf16 device tensor with packed heads."""
    if x.dtype != torch.bfloat16:
        raise TypeError("%s must be torch.bfloat16, got %s" % (name, x.dtype))
    if x.dim() != 3 or x.shape[2] != head_dim:
        raise ValueError("%s must be [n, heads, %d], got shape %s" % (name, head_dim, tuple(x.shape)))
    n, heads, _ = x.shape
    if x.stride(2) != 1 or (heads > 1 and x.stride(1) != head_dim):
        raise ValueError("%s must have packed heads" % name)
    return n, heads, x.stride(0) if n > 1 else heads * head_dim


# the current device's index, without the checks of a device that is in use already
_current = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call_on(device, func, *args):
    """func(*args, stream) on the device's current stream, whatever the current device is."""
    if device.index == _current():
        return func(*args, _stream(device))
    with torch.cuda.device(device):
        return func(*args, _stream(device))


def kv_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              slots: Optional[torch.Tensor] = None, q: Optional[torch.Tensor] = None,
              positions: Optional[torch.Tensor] = None, inv_freq: Optional[torch.Tensor] = None, sections=None,
              interleaved: bool = False, q_out: Optional[torch.Tensor] = None,
              k_scale_inv: Optional[torch.Tensor] = None, v_scale_inv: Optional[torch.Tensor] = None,
              k_storage="e4m3", v_storage=None, scaling="token_head", pow2: bool = False,
              diag: Optional[Diag] = None) -> Optional[torch.Tensor]:
    """Append new tokens to one layer's K and V caches in one launch, rotating
    q and k by their positions on the way (fp8_kv_append).

    k, v: [n, heads, head_dim] or [n, heads * head_dim], q (optional): [n,
    q_heads, head_dim] or 2-D, all bf16 or all fp32, heads packed within a
    token (slices of one projection's output are fine).  Caches, scales,
    storage and scaling as kv_store and kv_attention take them; slots: int64
    [n] cache rows (None: rows 0..n-1; outside the cache: not stored).

    inv_freq: fp32 [rotary_dim / 2], radians a position, of the pairs of the
    first rotary_dim channels (None: nothing turns): channels i and i +
    rotary_dim / 2, with interleaved 2i and 2i + 1.  positions: int64 [n], or
    [axes, n] with sections, the number of pairs that turn with each axis, in
    their order (time, height and width of a picture's patches, say); one row
    expanded over the axes will do (text beside pictures).  Angles are formed
    in 64 bits, the rotation in fp32; k is cast without a rounding between.

    Returns the rotated q in bf16, [n, q_heads, head_dim] (q_out where given,
    which may be q itself), or None without q."""
    if v_storage is None:
        v_storage = k_storage
    capacity, heads, head_dim, dev, k_scale, v_scale = _caches(k_cache, v_cache, k_scale_inv, v_scale_inv, k_storage,
                                                               v_storage, scaling)
    pair = _PAIR.pack(k_cache.data_ptr(), v_cache.data_ptr(), k_scale, v_scale, capacity, 0, 0, 0, 0,
                      KV_STORAGE[k_storage], KV_STORAGE[v_storage], KV_SCALING[scaling], heads, head_dim, 1, 0, 0)
    dtype = k.dtype
    if dtype is torch.bfloat16:
        in_dt = _lib.FP8_IN_BF16
    elif dtype is torch.float32:
        in_dt = _lib.FP8_IN_F32
    else:
        raise TypeError("k must be bfloat16 or float32, got %s" % dtype)
    if v.dtype is not dtype:
        raise TypeError("v must be %s as k, got %s" % (dtype, v.dtype))
    for t, name in ((k, "k"), (v, "v"), (q, "q"), (q_out, "q_out"), (slots, "slots")):
        if t is not None and t.device != dev:
            raise ValueError("%s must be on %s, got %s" % (name, dev, t.device))
    n, ldk = _kv_rows(k, heads, head_dim, "k")
    n2, ldv = _kv_rows(v, heads, head_dim, "v")
    if n2 != n:
        raise ValueError("v has %d tokens, k %d" % (n2, n))
    q_heads = ldq = ldqo = 0
    q_ptr = out_ptr = None
    if q is None:
        if q_out is not None:
            raise ValueError("q_out needs q")
    else:
        if q.dtype is not dtype:
            raise TypeError("q must be %s as k, got %s" % (dtype, q.dtype))
        shape = q.shape
        if len(shape) not in (2, 3) or (len(shape) == 2 and shape[1] % head_dim):
            raise ValueError("q must be [n, q_heads, %d] or [n, q_heads * %d], got shape %s"
                             % (head_dim, head_dim, tuple(shape)))
        q_heads = shape[1] if len(shape) == 3 else shape[1] // head_dim
        nq, ldq = _kv_rows(q, q_heads, head_dim, "q")
        if nq != n:
            raise ValueError("q has %d tokens, k %d" % (nq, n))
        if q_out is None:
            q_out = torch.empty((n, q_heads, head_dim), dtype=torch.bfloat16, device=dev)
            ldqo = q_heads * head_dim
        else:
            if q_out.dtype is not torch.bfloat16:
                raise TypeError("q_out must be torch.bfloat16, got %s" % q_out.dtype)
            no, ldqo = _kv_rows(q_out, q_heads, head_dim, "q_out")
            if no != n:
                raise ValueError("q_out has %d tokens, q %d" % (no, n))
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
    rotary, axes, pos_ld, cuts, flags = 0, 1, 0, None, _lib.FP8_SCALE_POW2 if pow2 else 0
    pos_ptr = freq_ptr = None
    if inv_freq is None:
        if positions is not None or sections is not None or interleaved:
            raise ValueError("positions, sections and interleaved need inv_freq")
    else:
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must be 1-D, got shape %s" % (tuple(inv_freq.shape),))
        rotary = 2 * inv_freq.shape[0]
        _int32(rotary, "rotary_dim")
        freq_ptr = _buf(inv_freq, rotary // 2, torch.float32, dev, "inv_freq")
        if not isinstance(positions, torch.Tensor):
            raise ValueError("inv_freq needs positions")
        if sections is None:
            want = (n,)
        else:
            axes = len(sections)
            if not 1 <= axes <= 4:
                raise ValueError("sections must name 1..4 axes, got %d" % axes)
            for pairs in sections:
                _int32(pairs, "sections")
            cuts = _INTS[axes](*sections)
            want = (axes, n)
        if positions.dtype is not torch.int64 or positions.device != dev:
            raise TypeError("positions must be torch.int64 on %s, got %s on %s" % (dev, positions.dtype, positions.device))
        if positions.shape != want:
            raise ValueError("positions must have shape %s, got %s" % (want, tuple(positions.shape)))
        stride = positions.stride()
        if n > 1 and stride[-1] != 1:
            raise ValueError("positions must have a contiguous last dimension")
        if axes > 1 and 0 < stride[0] < n:
            raise ValueError("positions of several axes must lie %d apart or more, or be one row for all (stride 0), "
                             "got stride %d" % (n, stride[0]))
        pos_ptr, pos_ld = positions.data_ptr(), stride[0] if axes > 1 else n
        if interleaved:
            flags |= _lib.FP8_ROTARY_INTERLEAVED
    st = _call_on(dev, _lib.lib().fp8_kv_append, pair, k.data_ptr(), ldk, v.data_ptr(), ldv, q_ptr, ldq, q_heads,
                  out_ptr, ldqo, in_dt, n, _slots(slots, n), pos_ptr, pos_ld, cuts, axes, freq_ptr, rotary, flags,
                  _ptr(diag.buf) if diag is not None else None)
    _lib.check(st, "fp8_kv_append")
    return q_out


def kv_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                 lens: torch.Tensor, page_size: int, k_scale_inv: Optional[torch.Tensor] = None,
                 v_scale_inv: Optional[torch.Tensor] = None, k_storage="e4m3", v_storage=None,
                 scaling="token_head", q_offsets: Optional[torch.Tensor] = None, max_len: Optional[int] = None,
                 window: int = 0, sinks: int = 0, scale: Optional[float] = None,
                 weights: Optional[torch.Tensor] = None, return_lse: bool = False,
                 out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, shared: int = 0):
    """Attention of a batch's newest tokens over one layer's paged cache,
    read in place (fp8_kv_attention).

    q: bf16 [total_q, q_heads, head_dim], the sequences' new tokens one after
    the other; their K and V are already stored.  Every sequence has
    total_q / batch of them (one: a decode step), or those q_offsets (int32
    device tensor [batch + 1]) gives.  k_cache, v_cache: [capacity, heads,
    head_dim] as kv_store fills them, with their scales; v_storage defaults to
    k_storage.  page_table: int32 [batch, pages]: token j of sequence b is in
    cache row page_table[b, j // page_size] * page_size + j % page_size (rows
    outside the cache are not there).  lens: int32 [batch], cached tokens
    including the new ones; max_len: an upper bound of them known on the host
    (default: what page_table holds).

    Causal; with window > 0 a token sees the last `window` tokens, itself
    included, and the first `sinks`.  scale: default head_dim ** -0.5.
    weights: fp32 [batch, heads, >= max_len], to which the call adds what each
    cached token receives (the input of kv_evict).  workspace: a uint8 device
    tensor for callers that may not allocate (fp8_kv_attention_workspace
    bytes; it follows max_len: with weights and one new token per sequence,
    batch * q_heads * max_len fp32 scores, so a max_len near the longest
    sequence saves memory where page_table holds more).  out must not overlap
    anything the call reads, q included.  No gradient is formed.

    shared: the number of first tokens that all sequences have in the same
    pages (a common instruction text or document), read once for the batch
    from the first row's pages, whatever that row's own length
    (fp8_kv_attention_shared; its workspace is
    fp8_kv_attention_shared_workspace bytes).  It pays for decode batches and
    drafted tokens; prompts (some 64 new tokens a sequence and more) are as
    fast or faster without it, and one new token with weights three times.

    Scores, softmax and sums are in fp32.  The weights of one new token per
    sequence enter the product with V with 16 significant bits, those of
    several, and of shared tokens with more than 32 rows (sequences * q_heads /
    heads), rounded once to bf16 (up to 2^-8 of sum p |v|, beside the output's
    own rounding).

    Returns out [total_q, q_heads, head_dim] bf16, with return_lse (or lse
    given) also the fp32 log-sum-exp of the scores [total_q, q_heads]."""
    if v_storage is None:
        v_storage = k_storage
    _int32(window, "window")
    _int32(sinks, "sinks")
    _int32(shared, "shared")
    pair, heads, head_dim, batch, max_len = _kv_pair(k_cache, v_cache, page_table, lens, page_size, k_scale_inv,
                                                     v_scale_inv, k_storage, v_storage, scaling, max_len)
    dev = k_cache.device
    _same_device(q, dev, "q")
    n, q_heads, ldq = _heads_matrix(q, head_dim, "q")
    if out is None:
        out = torch.empty((n, q_heads, head_dim), dtype=torch.bfloat16, device=dev)
        ldo = q_heads * head_dim
    else:
        _same_device(out, dev, "out")
        n2, h2, ldo = _heads_matrix(out, head_dim, "out")
        if (n2, h2) != (n, q_heads):
            raise ValueError("out must have shape %s, got %s" % (tuple(q.shape), tuple(out.shape)))
    want_lse = return_lse or lse is not None
    if lse is not None:
        _buf(lse, n * q_heads, torch.float32, dev, "lse")
    elif want_lse or weights is not None:
        lse = torch.empty((n, q_heads), dtype=torch.float32, device=dev)
    offsets = None
    if q_offsets is not None:
        offsets = _buf(q_offsets, batch + 1, torch.int32, dev, "q_offsets")
    ldw = 0
    if weights is not None:
        ldw = _kv_weights(weights, batch, heads, max_len, dev, "weights")
    ws_bytes = 0
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.device != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on %s" % dev)
        ws_bytes = workspace.numel() * workspace.element_size()
    else:
        ws_bytes = _attention_workspace(k_storage, heads, head_dim, page_size, batch, max_len, n, q_heads,
                                        offsets is not None, window, sinks, weights is not None, shared)
        if ws_bytes > 0:
            workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    st = _call_on(dev, _lib.lib().fp8_kv_attention_shared, pair, q.data_ptr(), ldq, n, q_heads, offsets,
                  head_dim ** -0.5 if scale is None else scale, window, sinks, shared, out.data_ptr(), ldo, _ptr(lse),
                  _ptr(weights), ldw, _ptr(workspace), ws_bytes)
    _lib.check(st, "fp8_kv_attention")
    return (out, lse) if want_lse else out


def kv_evict(k_cache: torch.Tensor, v_cache: torch.Tensor, weights: torch.Tensor, page_table: torch.Tensor,
             lens: torch.Tensor, page_size: int, budget: int, sinks: int = 0, recent: int = 0,
             k_scale_inv: Optional[torch.Tensor] = None, v_scale_inv: Optional[torch.Tensor] = None,
             k_storage="e4m3", v_storage=None, scaling="token_head", max_len: Optional[int] = None,
             dst_page_table: Optional[torch.Tensor] = None, weights_out: Optional[torch.Tensor] = None,
             kept: Optional[torch.Tensor] = None, new_lens: Optional[torch.Tensor] = None):
    """Cut every sequence of more than `budget` tokens to `budget`
    (fp8_kv_evict): each KV head keeps the first `sinks` tokens, the last
    `recent` and the heaviest of those between by weights [batch, heads, >=
    max_len] (the lower position among equals), moved together in their order.
    Without dst_page_table the cache, its scales and the weights are changed in
    place; with it (int32 [batch, pages] other pages of the same caches) the
    kept tokens are copied there.  Sequences of one call must not share pages
    that are written: with shared prefixes, evict into other pages.  A kept
    token without a page does not move, and its new row stays as it was.
    weights_out [batch, heads, >= budget]: the kept tokens' weights go there
    instead of into weights.

    Returns (kept, new_lens): int32 [batch, heads, budget] positions kept, -1
    behind the last, and int32 [batch] the new lengths.  lens is not changed:
    every layer of a model evicts with the same one."""
    if v_storage is None:
        v_storage = k_storage
    for value, name in ((budget, "budget"), (sinks, "sinks"), (recent, "recent")):
        _int32(value, name)
    pair, heads, _, batch, max_len = _kv_pair(k_cache, v_cache, page_table, lens, page_size, k_scale_inv, v_scale_inv,
                                              k_storage, v_storage, scaling, max_len)
    dev = k_cache.device
    if budget < 1:
        raise ValueError("budget must be >= 1, got %d" % budget)
    ldw = _kv_weights(weights, batch, heads, max_len, dev, "weights")
    ldwo = 0
    if weights_out is not None:
        ldwo = _kv_weights(weights_out, batch, heads, budget, dev, "weights_out")
    dst, dst_ld = None, 0
    if dst_page_table is not None:
        if (dst_page_table.dim() != 2 or dst_page_table.dtype != torch.int32 or dst_page_table.device != dev
                or dst_page_table.shape[0] != batch
                or (dst_page_table.shape[1] > 1 and dst_page_table.stride(1) != 1)):
            raise ValueError("dst_page_table must be an int32 [%d, pages] tensor on %s with a contiguous last "
                             "dimension" % (batch, dev))
        if dst_page_table.shape[1] * page_size < budget:
            raise ValueError("dst_page_table holds fewer than budget=%d tokens" % budget)
        dst = dst_page_table.data_ptr()
        dst_ld = dst_page_table.stride(0) if batch > 1 else dst_page_table.shape[1]
    if kept is None:
        kept = torch.empty((batch, heads, budget), dtype=torch.int32, device=dev)
    if new_lens is None:
        new_lens = torch.empty(batch, dtype=torch.int32, device=dev)
    st = _call_on(dev, _lib.lib().fp8_kv_evict, pair, weights.data_ptr(), ldw, budget, sinks, recent, dst, dst_ld,
                  _ptr(weights_out), ldwo, _buf(kept, batch * heads * budget, torch.int32, dev, "kept"),
                  _buf(new_lens, batch, torch.int32, dev, "new_lens"))
    _lib.check(st, "fp8_kv_evict")
    return kept, new_lens


class KVTensorCache:
    """One layer's K (or V) cache: `data` [capacity, heads, head_dim] (uint8
    codes; bf16 for the "bf16" storage) and `scale_inv` ([capacity, heads] for
    per-(token, head) scales, [heads] fixed scales for "head" scaling)."""

    def __init__(self, capacity: int, heads: int, head_dim: int, storage="e4m3", scaling="token_head",
                 head_scale_inv: Optional[torch.Tensor] = None, device="cuda"):
        if storage not in KV_STORAGE or scaling not in KV_SCALING:
            raise ValueError("storage %r / scaling %r" % (storage, scaling))
        self.storage, self.scaling = storage, scaling
        self.capacity, self.heads, self.head_dim = capacity, heads, head_dim
        dt = torch.bfloat16 if storage == "bf16" else torch.uint8
        self.data = torch.zeros((capacity, heads, head_dim), dtype=dt, device=device)
        if storage == "bf16":
            self.scale_inv = None
        elif scaling == "token_head":
            self.scale_inv = torch.zeros((capacity, heads), dtype=torch.float32, device=device)
        else:
            if head_scale_inv is None or head_scale_inv.numel() != heads:
                raise ValueError("'head' scaling needs head_scale_inv with %d entries" % heads)
            self.scale_inv = head_scale_inv.to(device=device, dtype=torch.float32).contiguous()

    @property
    def nbytes(self) -> int:
        n = self.data.numel() * self.data.element_size()
        return n + (self.scale_inv.numel() * 4 if self.scale_inv is not None else 0)

    def store(self, x: torch.Tensor, slots: Optional[torch.Tensor] = None, pow2: bool = False,
              diag: Optional[Diag] = None) -> None:
        kv_store(x, self.data, self.scale_inv, self.storage, self.scaling, slots, pow2, diag)

    def load(self, n: Optional[int] = None, slots: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
             out: Optional[torch.Tensor] = None) -> torch.Tensor:
        return kv_load(self.data, self.scale_inv, n, self.storage, self.scaling, slots, out_dtype, out)


class KVCache:
    """K and V caches of every layer of a model.  Layers listed in
    `bf16_k_layers` keep their K cache in bf16 (the per-layer fallback of a
    precision-sensitive layer); `bf16_v_layers` likewise for V."""

    def __init__(self, layers: int, capacity: int, kv_heads: int, head_dim: int, storage="e4m3",
                 scaling="token_head", bf16_k_layers=(), bf16_v_layers=(), head_scale_inv=None, device="cuda"):
        bk, bv = set(bf16_k_layers), set(bf16_v_layers)
        for s in (bk, bv):
            if any(not 0 <= i < layers for i in s):
                raise ValueError("fallback layer index out of range 0..%d" % (layers - 1))

        def make(i, fallback, which):
            st = "bf16" if i in fallback else storage
            hs = None if head_scale_inv is None else head_scale_inv[which][i]
            return KVTensorCache(capacity, kv_heads, head_dim, st, scaling, hs, device)

        self.k = [make(i, bk, 0) for i in range(layers)]
        self.v = [make(i, bv, 1) for i in range(layers)]

    @property
    def nbytes(self) -> int:
        return sum(c.nbytes for c in self.k + self.v)

    def store(self, layer: int, k: torch.Tensor, v: torch.Tensor, slots: Optional[torch.Tensor] = None,
              pow2: bool = False) -> None:
        self.k[layer].store(k, slots, pow2)
        self.v[layer].store(v, slots, pow2)

    def append(self, layer: int, k: torch.Tensor, v: torch.Tensor, slots: Optional[torch.Tensor] = None, **options):
        """kv_append of new tokens to a layer's caches (options: its keywords)."""
        return kv_append(k, v, self.k[layer].data, self.v[layer].data, slots, **self._layer(layer), **options)

    def load(self, layer: int, n: Optional[int] = None, slots: Optional[torch.Tensor] = None,
             out_dtype=torch.bfloat16):
        return (self.k[layer].load(n, slots, out_dtype), self.v[layer].load(n, slots, out_dtype))

    def _layer(self, layer: int) -> dict:
        k, v = self.k[layer], self.v[layer]
        return {"k_scale_inv": k.scale_inv, "v_scale_inv": v.scale_inv, "k_storage": k.storage,
                "v_storage": v.storage, "scaling": k.scaling}

    def attend(self, layer: int, q: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor, page_size: int,
               **options):
        """kv_attention of q over a layer's caches (options: its keywords)."""
        return kv_attention(q, self.k[layer].data, self.v[layer].data, page_table, lens, page_size,
                            **self._layer(layer), **options)

    def evict(self, layer: int, weights: torch.Tensor, page_table: torch.Tensor, lens: torch.Tensor, page_size: int,
              budget: int, sinks: int = 0, recent: int = 0, **options):
        """kv_evict of a layer's caches (options: its keywords)."""
        return kv_evict(self.k[layer].data, self.v[layer].data, weights, page_table, lens, page_size, budget, sinks,
                        recent, **self._layer(layer), **options)
