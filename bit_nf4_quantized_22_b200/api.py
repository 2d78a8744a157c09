"""Python binding of the QLoRA layer library.

Argument marshalling only: every function hands device pointers, sizes and
the current CUDA stream to the C ABI (include/qlora.h) and every step of the
computation runs in the library's CUDA kernels.  PyTorch provides device
memory (tensors, the workspace) and streams.
"""
from __future__ import annotations

import contextlib
import ctypes
from dataclasses import dataclass

import torch
from torch.autograd.function import once_differentiable

from . import _lib
from .codebook import nf4_codebook

BLOCK = 64
DQ_GROUP = 256
# double-quantization codes of the block scales (QLORA_DQ_* in qlora.h)
DQ_VARIANTS = {"u8": 1, "s8": 2, "mean": 3, "f8": 4}


def _at(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _raw_stream(t: torch.Tensor) -> int:
    """The current stream of t's device, without the Stream object (about 2 us of a call)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _cb_at(codebook: torch.Tensor | None):
    """The 16 host floats a call reads: the tensor's own where it has them in that form."""
    if codebook is not None and codebook.dtype == torch.float32 and codebook.shape == (16,) \
            and not codebook.is_cuda and codebook.is_contiguous():
        return codebook.data_ptr()
    return _cb_host(codebook)


def _cb_host(codebook: torch.Tensor | None) -> ctypes.Array:
    cb = nf4_codebook() if codebook is None else codebook.detach().to("cpu", torch.float32)
    arr = (ctypes.c_float * 16)(*cb.tolist())
    return arr


def _need(t: torch.Tensor, dtype, name: str, dims: int):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.dim() != dims:
        raise TypeError(f"{name}: expected a {dims}-D {dtype} tensor")
    if not t.is_cuda:
        raise TypeError(f"{name}: must be a CUDA tensor")
    if not t.is_contiguous():
        raise TypeError(f"{name}: must be contiguous")


@dataclass
class NF4Weight:
    """A quantized frozen weight Wt:[rows = Dout, cols = Din] (device buffers)."""
    rows: int
    cols: int
    double_quant: bool
    packed: torch.Tensor                   # uint8 [rows*cols/2]
    absmax: torch.Tensor | None = None     # fp32 [nb]
    codes: torch.Tensor | None = None      # uint8 [nb] (int8 two's complement for "mean")
    steps: torch.Tensor | None = None      # fp32 [ceil(nb/256)]
    block: int = BLOCK                     # weights per first-level scale (32, 64, 128, 256)
    dq_variant: str = "u8"                 # code of the scales: "u8", "s8", "mean" or "f8"
    means: torch.Tensor | None = None      # fp32 [ceil(nb/256)] group means ("mean")
    # the layer calls' 16-bit dtype (x, A, B, dY, y, dX, merged weight)
    compute_dtype: torch.dtype = torch.bfloat16

    @staticmethod
    def empty(rows: int, cols: int, double_quant: bool, device="cuda", block: int = BLOCK,
              dq_variant: str = "u8") -> "NF4Weight":
        nb = rows * cols // block
        packed = torch.empty(rows * cols // 2, dtype=torch.uint8, device=device)
        if double_quant:
            if dq_variant not in DQ_VARIANTS:
                raise ValueError(f"dq_variant: one of {sorted(DQ_VARIANTS)}")
            ng = (nb + DQ_GROUP - 1) // DQ_GROUP
            means = torch.empty(ng, dtype=torch.float32, device=device) if dq_variant == "mean" else None
            return NF4Weight(rows, cols, True, packed,
                             codes=torch.empty(nb, dtype=torch.uint8, device=device),
                             steps=torch.empty(ng, dtype=torch.float32, device=device), block=block,
                             dq_variant=dq_variant, means=means)
        return NF4Weight(rows, cols, False, packed,
                         absmax=torch.empty(nb, dtype=torch.float32, device=device), block=block)

    def c_struct(self) -> _lib.NF4WeightC:
        return _lib.NF4WeightC(
            self.rows, self.cols, self.block,
            DQ_VARIANTS[self.dq_variant] if self.double_quant else 0, DQ_GROUP,
            _DTYPE_CODES[self.compute_dtype],
            self.packed.data_ptr(),
            self.absmax.data_ptr() if self.absmax is not None else None,
            self.codes.data_ptr() if self.codes is not None else None,
            self.steps.data_ptr() if self.steps is not None else None,
            self.means.data_ptr() if self.means is not None else None)

    @property
    def nbytes(self) -> int:
        n = self.packed.numel()
        for t in (self.absmax, self.codes, self.steps, self.means):
            if t is not None:
                n += t.numel() * t.element_size()
        return n


def _pitch(cols: int) -> int:
    """Row pitch of new codes: whole 128-byte lines, which the products read fastest; short rows 16."""
    unit = 128 if cols >= 128 else 16
    return (cols + unit - 1) // unit * unit


@dataclass
class Int8Rows:
    """A matrix in 8-bit rows: row m stands for codes[m] * scales[m].  The rows are
    tokens for an activation, output channels for a weight Wt:[Dout, Din]."""
    codes: torch.Tensor    # int8 [rows, cols], unit column stride, row stride a multiple of 16
    scales: torch.Tensor   # fp32 [rows]

    @staticmethod
    def empty(rows: int, cols: int, device="cuda") -> "Int8Rows":
        codes = torch.empty_strided((rows, cols), (_pitch(cols), 1), dtype=torch.int8, device=device)
        return Int8Rows(codes, torch.empty(rows, dtype=torch.float32, device=device))

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    @property
    def cols(self) -> int:
        return self.codes.shape[1]

    @property
    def device(self) -> torch.device:
        return self.codes.device

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + 4 * self.scales.numel()

    def c_struct(self) -> _lib.Int8RowsC:
        c, s = self.codes, self.scales
        if c.dtype != torch.int8 or s.dtype != torch.float32 or c.dim() != 2 or s.dim() != 1:
            raise TypeError("Int8Rows: codes int8 [rows, cols] and scales fp32 [rows] are needed")
        if not c.is_cuda or s.get_device() != c.get_device():
            raise TypeError("Int8Rows: codes and scales must be CUDA tensors of one device")
        rows, cols = c.shape
        ld, unit = c.stride()
        if rows <= 1:
            ld = (cols + 15) // 16 * 16
        at = c.data_ptr()
        if s.shape[0] != rows or (rows > 1 and s.stride(0) != 1):
            raise ValueError("Int8Rows: one scale a row, contiguous")
        if cols < 1 or (unit != 1 and cols > 1) or ld < cols or ld % 16 or at % 16:
            raise ValueError("Int8Rows: codes need a unit column stride, and 16-byte aligned rows")
        return _lib.Int8RowsC(rows, cols, ld, at, s.data_ptr())


def load():
    """Load libqlora.so; raises if it is missing (no fallback exists)."""
    return _lib.load()


def check_codebook(codebook: torch.Tensor) -> int:
    return load().qlora_check_codebook(_cb_host(codebook))


def quantize(W: torch.Tensor, double_quant: bool = True, codebook: torch.Tensor | None = None,
             status: torch.Tensor | None = None, out: NF4Weight | None = None,
             block: int = BLOCK, dq_variant: str = "u8",
             compute_dtype: torch.dtype = torch.bfloat16) -> NF4Weight:
    """nf4_quantize on W (fp32 [Dout, Din], CUDA) in blocks of `block` weights
    (32, 64, 128 or 256; the layer calls need 64); with double quantization
    the block scales take the `dq_variant` code ("u8", "s8", "mean" or "f8").
    `compute_dtype` (bf16 or fp16) is the dtype the layer calls then use."""
    _need(W, torch.float32, "W", 2)
    if compute_dtype not in (torch.bfloat16, torch.float16):
        raise ValueError("compute_dtype: torch.bfloat16 or torch.float16")
    rows, cols = W.shape
    q = out if out is not None else NF4Weight.empty(rows, cols, double_quant, W.device, block,
                                                    dq_variant)
    if out is None:
        q.compute_dtype = compute_dtype
    qc = q.c_struct()
    rc = load().nf4_quantize(_ptr(W), ctypes.byref(qc), _cb_host(codebook), _ptr(status), _stream())
    _lib.check(rc, "nf4_quantize")
    return q


_DTYPE_CODES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def dequantize(q: NF4Weight, codebook: torch.Tensor | None = None,
               out: torch.Tensor | None = None, dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """The dequantized weight [rows, cols] in the compute dtype (bf16, fp16 or fp32)."""
    if dtype not in _DTYPE_CODES:
        raise TypeError(f"dtype: one of {list(_DTYPE_CODES)}")
    out = out if out is not None else torch.empty(q.rows, q.cols, dtype=dtype,
                                                  device=q.packed.device)
    if out.dtype != dtype:
        raise TypeError("out: dtype does not match")
    qc = q.c_struct()
    if dtype == torch.bfloat16:
        rc = load().nf4_dequantize(ctypes.byref(qc), _cb_host(codebook), _ptr(out), _stream())
    else:
        rc = load().nf4_dequantize_dtype(ctypes.byref(qc), _cb_host(codebook), _DTYPE_CODES[dtype],
                                         _ptr(out), _stream())
    _lib.check(rc, "nf4_dequantize")
    return out


def merge(q: NF4Weight, A: torch.Tensor, B: torch.Tensor, alpha: float, pool_group: int = 1,
          codebook: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """bf16 [Dout, Din] weight with the adapter folded in (qlora_merge)."""
    r = B.shape[0]
    out = out if out is not None else torch.empty(q.rows, q.cols, dtype=q.compute_dtype,
                                                  device=q.packed.device)
    qc = q.c_struct()
    rc = load().qlora_merge(ctypes.byref(qc), _cb_host(codebook), _ptr(A), _ptr(B), r,
                            float(alpha), pool_group, _ptr(out), _stream())
    _lib.check(rc, "qlora_merge")
    return out


def workspace_size(M: int, q: NF4Weight, r: int, pool_group: int = 1, which: int = 0) -> int:
    qc = q.c_struct()
    return int(load().qlora_workspace_size(M, ctypes.byref(qc), r, pool_group, which))


def _workspace(nbytes: int, device, ws: torch.Tensor | None):
    if nbytes == 0:
        return None, 0
    if ws is not None and ws.numel() >= nbytes:
        return ws, ws.numel()
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


def forward(x: torch.Tensor, q: NF4Weight, A: torch.Tensor, B: torch.Tensor, alpha: float,
            pool_group: int = 1, codebook: torch.Tensor | None = None, save_T: bool = True,
            workspace: torch.Tensor | None = None, status: torch.Tensor | None = None,
            out: torch.Tensor | None = None):
    """y = x dequant(W4) + (alpha/r) (u A) B.  Returns (y bf16 [M, Dout], T fp32 [M, r] or None)."""
    _need(x, q.compute_dtype, "x", 2)
    _need(A, q.compute_dtype, "A", 2)
    _need(B, q.compute_dtype, "B", 2)
    M = x.shape[0]
    r = A.shape[1]
    y = out if out is not None else torch.empty(M, q.rows, dtype=q.compute_dtype, device=x.device)
    T = torch.empty(M, r, dtype=torch.float32, device=x.device) if save_T else None
    ws, nbytes = _workspace(workspace_size(M, q, r, pool_group, 0), x.device, workspace)
    qc = q.c_struct()
    rc = load().qlora_forward(_ptr(x), M, ctypes.byref(qc), _cb_host(codebook), _ptr(A), _ptr(B),
                              r, float(alpha), pool_group, _ptr(y), _ptr(T), _ptr(ws), nbytes,
                              _ptr(status), _stream())
    _lib.check(rc, "qlora_forward")
    return y, T


def backward(x: torch.Tensor | Int8Rows | None, dy: torch.Tensor, q: NF4Weight, A: torch.Tensor,
             B: torch.Tensor, alpha: float, pool_group: int = 1, T: torch.Tensor | None = None,
             need_dx: bool = True, need_dA: bool = True, need_dB: bool = True,
             codebook: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
             status: torch.Tensor | None = None):
    """Returns (dX bf16 [M, Din] | None, dA fp32 | None, dB fp32 | None); W4 gets none.
    `x` may be the layer's input in 8 bits, int8_quantize(x) (qlora_backward_int8)."""
    if isinstance(x, Int8Rows):
        return _backward_int8(x, dy, q, A, B, alpha, pool_group, T, need_dx, need_dA, need_dB,
                              codebook, workspace, status)
    _need(dy, q.compute_dtype, "dy", 2)
    _need(A, q.compute_dtype, "A", 2)
    _need(B, q.compute_dtype, "B", 2)
    M = dy.shape[0]
    r = A.shape[1]
    dev = dy.device
    dX = torch.empty(M, q.cols, dtype=q.compute_dtype, device=dev) if need_dx else None
    dA = torch.empty(A.shape[0], r, dtype=torch.float32, device=dev) if need_dA else None
    dB = torch.empty(r, q.rows, dtype=torch.float32, device=dev) if need_dB else None
    ws, nbytes = _workspace(workspace_size(M, q, r, pool_group, 1), dev, workspace)
    qc = q.c_struct()
    rc = load().qlora_backward(_ptr(x), _ptr(dy), M, ctypes.byref(qc), _cb_host(codebook),
                               _ptr(A), _ptr(B), r, float(alpha), pool_group, _ptr(T), _ptr(dX),
                               _ptr(dA), _ptr(dB), _ptr(ws), nbytes, _ptr(status), _stream())
    _lib.check(rc, "qlora_backward")
    return dX, dA, dB


def _backward_int8(x: Int8Rows, dy, q: NF4Weight, A, B, alpha, pool_group, T, need_dx, need_dA, need_dB,
                   codebook, workspace, status):
    dt = q.compute_dtype
    _need(dy, dt, "dy", 2)
    _need(A, dt, "A", 2)
    _need(B, dt, "B", 2)
    xc, qc = x.c_struct(), q.c_struct()
    M, K, N = xc.rows, qc.cols, qc.rows
    Da, r = A.shape
    if tuple(dy.shape) != (M, N) or xc.cols != K:
        raise ValueError(f"dy [{M}, {N}] and x [{M}, {K}] are needed")
    if pool_group not in (1, 64) or Da != K // pool_group or tuple(B.shape) != (r, N):
        raise ValueError("A [Din/pool_group, r] and B [r, Dout] are needed")
    if T is not None:
        _need(T, torch.float32, "T", 2)
        if tuple(T.shape) != (M, r):
            raise ValueError(f"T [{M}, {r}] is needed")
    dev, lib = dy.device, load()
    with _on(dy, x.codes, A, B, T, workspace, status, q.packed):
        new = torch.empty if M else torch.zeros      # no token: the adapter gradients are zero
        dX = torch.empty((M, K), dtype=dt, device=dev) if need_dx else None
        dA = new((Da, r), dtype=torch.float32, device=dev) if need_dA else None
        dB = new((r, N), dtype=torch.float32, device=dev) if need_dB else None
        need = lib.qlora_backward_int8_workspace_size(M, ctypes.byref(qc), r, pool_group)
        ws, nbytes = _workspace(need, dev, workspace)
        cb = _cb_at(codebook)
        rc = lib.qlora_backward_int8(ctypes.byref(xc), dy.data_ptr(), M, ctypes.byref(qc), cb,
                                     A.data_ptr(), B.data_ptr(), r, alpha, pool_group, _at(T), _at(dX),
                                     _at(dA), _at(dB), _at(ws), nbytes, _at(status), _raw_stream(dy))
        _lib.check(rc, "qlora_backward_int8")
    return dX, dA, dB


def _on(t: torch.Tensor, *others):
    """A context in which t's device is the current one; the others must be on it too."""
    dev = t.get_device()
    for o in others:
        if o is not None and o.get_device() != dev:
            raise ValueError(f"tensors of one device are needed: {t.device} and {o.device} were given")
    return _HERE if dev == torch.cuda.current_device() else torch.cuda.device(dev)


_HERE = contextlib.nullcontext()


def int8_quantize(x: torch.Tensor, out: Int8Rows | None = None,
                  status: torch.Tensor | None = None) -> Int8Rows:
    """The rows of x (bf16, fp16 or fp32 [rows, cols], unit column stride) in 8 bits,
    one scale a row: a token's activation, or an output channel of a weight Wt."""
    dtype = _any_float(x, "x")
    rows, cols, ldx = _row_stride(x, "x")
    if out is None:
        q = Int8Rows.empty(rows, cols, x.device)
        qc = _lib.Int8RowsC(rows, cols, _pitch(cols), q.codes.data_ptr(), q.scales.data_ptr())
    else:
        q, qc = out, out.c_struct()
        if (q.rows, q.cols) != (rows, cols):
            raise ValueError(f"out: [{rows}, {cols}] is needed")
    with _on(x, q.codes, status):
        rc = load().int8_quantize(x.data_ptr(), dtype, ldx, ctypes.byref(qc), _at(status), _raw_stream(x))
        _lib.check(rc, "int8_quantize")
    return q


def _any_float(x, name: str) -> int:
    if isinstance(x, torch.Tensor) and x.is_cuda and x.dim() == 2:
        code = _DTYPE_CODES.get(x.dtype)
        if code is not None:
            return code
    raise TypeError(f"{name}: expected a 2-D bf16, fp16 or fp32 CUDA tensor")


def _row_stride(x: torch.Tensor, name: str):
    rows, cols = x.shape
    ldx = x.stride(0) if rows > 1 else max(cols, 1)
    if cols < 1 or (cols > 1 and x.stride(1) != 1) or ldx < cols:
        raise ValueError(f"{name}: at least one column, a unit column stride and rows that do not overlap are needed")
    return rows, cols, ldx


def int8_dequantize(q: Int8Rows, dtype: torch.dtype = torch.bfloat16,
                    out: torch.Tensor | None = None) -> torch.Tensor:
    """The values codes * scales [rows, cols] in bf16, fp16 or fp32."""
    if dtype not in _DTYPE_CODES:
        raise TypeError(f"dtype: one of {list(_DTYPE_CODES)}")
    out = out if out is not None else torch.empty(q.rows, q.cols, dtype=dtype, device=q.device)
    _need(out, dtype, "out", 2)
    if tuple(out.shape) != (q.rows, q.cols):
        raise ValueError(f"out: [{q.rows}, {q.cols}] is needed")
    with _on(out, q.codes):
        qc = q.c_struct()
        _lib.check(load().int8_dequantize(ctypes.byref(qc), _DTYPE_CODES[dtype], out.data_ptr(), _raw_stream(out)),
                   "int8_dequantize")
    return out


def int8_matmul(x: torch.Tensor | Int8Rows, w: Int8Rows, bias: torch.Tensor | None = None,
                dtype: torch.dtype | None = None, out: torch.Tensor | None = None,
                x8_out: Int8Rows | None = None, status: torch.Tensor | None = None) -> torch.Tensor:
    """y = x W^T (+ bias) with both operands in 8 bits: x [M, K] is a tensor (bf16, fp16 or
    fp32), quantized row by row in the call, or 8-bit rows already; w the weight's [N, K] rows
    (int8_quantize of an nn.Linear weight or of merge()'s).  y [M, N] has `dtype`: x's by
    default, bf16 for 8-bit rows.  `x8_out` receives a tensor x's rows, to be kept as the
    checkpoint of backward()."""
    given = isinstance(x, Int8Rows)
    xdt = 0 if given else _any_float(x, "x")
    if dtype is None:
        dtype = out.dtype if out is not None else (torch.bfloat16 if given else x.dtype)
    if dtype not in _DTYPE_CODES:
        raise TypeError(f"dtype: one of {list(_DTYPE_CODES)}")
    if given and x8_out is not None:
        raise ValueError("x8_out: only for a tensor x")
    wc = w.c_struct()
    N = wc.rows
    if given:
        xc, ldx, at = x.c_struct(), 0, None
        M, K = xc.rows, xc.cols
    else:
        M, K, ldx = _row_stride(x, "x")
        at = x.data_ptr()
        if x8_out is not None:
            xc = x8_out.c_struct()
            if (xc.rows, xc.cols) != (M, K):
                raise ValueError(f"x8_out: [{M}, {K}] is needed")
        else:   # codes and scales in one scratch tensor
            ld = _pitch(K)
            scratch = torch.empty(M * (ld + 4), dtype=torch.uint8, device=x.device)
            xc = _lib.Int8RowsC(M, K, ld, scratch.data_ptr(), scratch.data_ptr() + M * ld)
    if K != wc.cols:
        raise ValueError(f"x has {K} columns, w {wc.cols}")
    if out is None:
        y = torch.empty((M, N), dtype=dtype, device=w.codes.device)
    else:
        y = out
        _need(y, dtype, "out", 2)
        if tuple(y.shape) != (M, N):
            raise ValueError(f"out: [{M}, {N}] is needed")
    if bias is not None:
        _need(bias, dtype, "bias", 1)
        if bias.shape[0] != N:
            raise ValueError(f"bias: [{N}] is needed")
    with _on(y, w.codes, x.codes if given else x, None if x8_out is None else x8_out.codes, bias, status):
        rc = load().int8_matmul(at, xdt, ldx, ctypes.byref(xc), ctypes.byref(wc), _at(bias), y.data_ptr(),
                                _DTYPE_CODES[dtype], _at(status), _raw_stream(y))
        _lib.check(rc, "int8_matmul")
    return y


def int8_matmul_backward(dy: torch.Tensor, w: Int8Rows, out: torch.Tensor | None = None,
                         workspace: torch.Tensor | None = None,
                         status: torch.Tensor | None = None) -> torch.Tensor:
    """dX = dy dequant(w) [M, K] (bf16 or fp16): int8_matmul's gradient for its tokens."""
    if not isinstance(dy, torch.Tensor) or dy.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("dy: expected a 2-D bf16 or fp16 tensor")
    _need(dy, dy.dtype, "dy", 2)
    wc = w.c_struct()
    M, N = dy.shape
    if N != wc.rows:
        raise ValueError(f"dy has {N} columns, w {wc.rows} rows")
    if out is None:
        dX = torch.empty((M, wc.cols), dtype=dy.dtype, device=dy.device)
    else:
        dX = out
        _need(dX, dy.dtype, "out", 2)
        if tuple(dX.shape) != (M, wc.cols):
            raise ValueError(f"out: [{M}, {wc.cols}] is needed")
    with _on(dy, w.codes, dX, workspace, status):
        need = load().int8_matmul_backward_workspace_size(M, ctypes.byref(wc))
        ws, nbytes = _workspace(need, dy.device, workspace)
        rc = load().int8_matmul_backward(dy.data_ptr(), _DTYPE_CODES[dy.dtype], M, ctypes.byref(wc),
                                         dX.data_ptr(), _at(ws), nbytes, _at(status), _raw_stream(dy))
        _lib.check(rc, "int8_matmul_backward")
    return dX


def forward_noalloc(x: torch.Tensor, q: NF4Weight, A: torch.Tensor, B: torch.Tensor,
                    alpha: float, pool_group: int = 1, codebook: torch.Tensor | None = None,
                    out: torch.Tensor | None = None, T_out: torch.Tensor | None = None,
                    status: torch.Tensor | None = None):
    """qlora_forward_noalloc: the forward with the library's built-in scratch
    array instead of a workspace.  The caller passes the outputs (`out`,
    `T_out`); when omitted they are created here, which allocates."""
    _need(x, q.compute_dtype, "x", 2)
    _need(A, q.compute_dtype, "A", 2)
    _need(B, q.compute_dtype, "B", 2)
    M, r = x.shape[0], A.shape[1]
    y = out if out is not None else torch.empty(M, q.rows, dtype=q.compute_dtype, device=x.device)
    qc = q.c_struct()
    rc = load().qlora_forward_noalloc(_ptr(x), M, ctypes.byref(qc), _cb_host(codebook), _ptr(A),
                                      _ptr(B), r, float(alpha), pool_group, _ptr(y), _ptr(T_out),
                                      _ptr(status), _stream())
    _lib.check(rc, "qlora_forward_noalloc")
    return y, T_out


class QLoRALinearFn(torch.autograd.Function):
    """Autograd wrapper: gradients for x, A and B; none for the frozen W4."""

    @staticmethod
    def forward(ctx, x, A, B, q: NF4Weight, alpha: float, pool_group: int):
        y, T = forward(x, q, A, B, alpha, pool_group)
        ctx.save_for_backward(x, A, B, T)
        ctx.q, ctx.alpha, ctx.pool = q, alpha, pool_group
        return y

    @staticmethod
    def backward(ctx, dy):
        x, A, B, T = ctx.saved_tensors
        dX, dA, dB = backward(x, dy.contiguous(), ctx.q, A, B, ctx.alpha, ctx.pool, T=T,
                              need_dx=ctx.needs_input_grad[0], need_dA=ctx.needs_input_grad[1],
                              need_dB=ctx.needs_input_grad[2])
        return (dX, None if dA is None else dA.to(A.dtype), None if dB is None else dB.to(B.dtype),
                None, None, None)


class QLoRALinear8BitInputFn(torch.autograd.Function):
    """QLoRALinearFn with the input kept in 8 bits between forward and backward.  `x8` is
    int8_quantize(x), made here when None; layers that read the same x share one."""

    @staticmethod
    def forward(ctx, x, A, B, q: NF4Weight, alpha: float, pool_group: int = 1,
                x8: Int8Rows | None = None):
        y, T = forward(x, q, A, B, alpha, pool_group)
        x8 = int8_quantize(x) if x8 is None else x8
        if (x8.rows, x8.cols) != tuple(x.shape):
            raise ValueError("x8: int8_quantize(x) is needed")
        ctx.save_for_backward(x8.codes, x8.scales, A, B, T)
        ctx.q, ctx.alpha, ctx.pool = q, alpha, pool_group
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        codes, scales, A, B, T = ctx.saved_tensors
        dX, dA, dB = backward(Int8Rows(codes, scales), dy.contiguous(), ctx.q, A, B, ctx.alpha, ctx.pool, T=T,
                              need_dx=ctx.needs_input_grad[0], need_dA=ctx.needs_input_grad[1],
                              need_dB=ctx.needs_input_grad[2])
        return (dX, None if dA is None else dA.to(A.dtype), None if dB is None else dB.to(B.dtype),
                None, None, None, None)


class Int8LinearFn(torch.autograd.Function):
    """int8_matmul of a bf16 or fp16 x with a gradient for x (straight through its rounding);
    none for the frozen weight and bias: backward refuses a bias that requires one."""

    @staticmethod
    def forward(ctx, x, w: Int8Rows, bias=None):
        if x.dtype not in (torch.bfloat16, torch.float16):
            raise TypeError("x: expected bf16 or fp16")
        ctx.w = w
        return int8_matmul(x, w, bias)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        if any(ctx.needs_input_grad[2:]):
            raise RuntimeError("bias: frozen, it gets no gradient here; pass bias.detach()")
        return int8_matmul_backward(dy.contiguous(), ctx.w), None, None
