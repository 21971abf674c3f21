"""Thin Python binding of the C ABI in ``include/bq.h`` (``libbq.so``).

Argument marshalling only: every step of the quantizer and the linear layer
runs in the library's CUDA kernels.  Tensors are torch CUDA tensors used as
plain device buffers; outputs are allocated here with torch and their
pointers passed down.  There is no fallback: if the library is missing or a
call fails, an exception is raised.
"""
from __future__ import annotations

import ctypes
import os
import struct

import numpy as np
import torch

from . import build as _build

LIB_PATH = _build.LIB

# enums, mirrored from include/bq.h
BQ_OK, BQ_ERR_NULL, BQ_ERR_SHAPE, BQ_ERR_ALIGN, BQ_ERR_UNSUPPORTED = 0, 1, 2, 3, 4
BQ_ERR_WORKSPACE, BQ_ERR_NONFINITE, BQ_ERR_TIMEOUT, BQ_ERR_CUDA = 5, 6, 7, 8
BQ_F16, BQ_BF16, BQ_F32 = 0, 1, 2
BQ_LAYOUT_CANONICAL, BQ_LAYOUT_INTERLEAVED = 0, 1

LAYOUTS = {"canonical": BQ_LAYOUT_CANONICAL, "interleaved": BQ_LAYOUT_INTERLEAVED}
DTYPE_CODE = {torch.float16: BQ_F16, torch.bfloat16: BQ_BF16, torch.float32: BQ_F32}
CODE_DTYPE = {v: k for k, v in DTYPE_CODE.items()}
GROUP_OF_BITS = {4: 128, 2: 64}

#: every symbol include/bq.h declares
EXPORTS = (
    "bq_packed_bytes", "bq_group_count", "bq_mixed_offsets", "bq_quantize", "bq_quantize_symmetric",
    "bq_quantize_mixed",
    "bq_dequantize", "bq_fake_quantize", "bq_linear", "bq_linear_grad_input", "bq_check_division",
    "bq_check_const_division", "bq_quantize_f16s", "bq_linear_f16s", "bq_linear_workspace_bytes", "bq_linear_ws",
    "bq_dropout", "bq_lora", "bq_lora_grad", "bq_selftest_bounded_wait", "bq_set_option", "bq_get_option", "bq_device_status",
    "bq_status_string", "bq_version",
)
BQ_OPT_LINEAR_OVERLAP = 0


class BQError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)}")


_lib = None


def lib(path: str | None = None):
    """Load libbq.so (raises if it is missing; build it with build.build())."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise FileNotFoundError(f"{p} is missing: build the CUDA library first "
                                "(python -m quantized_gemm_group_b200.build)")
    L = ctypes.CDLL(p)
    i64, i32, vp, u8p = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p
    L.bq_packed_bytes.argtypes = [i64, i64, i32]
    L.bq_packed_bytes.restype = ctypes.c_size_t
    L.bq_group_count.argtypes = [i64, i64, i32]
    L.bq_group_count.restype = ctypes.c_size_t
    L.bq_mixed_offsets.argtypes = [u8p, i64, i64, vp, vp]
    L.bq_mixed_offsets.restype = i32
    L.bq_quantize.argtypes = [vp, i32, i64, i64, i32, i32, i32, vp, vp, vp, vp]
    L.bq_quantize.restype = i32
    L.bq_quantize_symmetric.argtypes = [vp, i32, i64, i64, i32, i32, i32, vp, vp, vp, vp]
    L.bq_quantize_symmetric.restype = i32
    L.bq_quantize_f16s.argtypes = [vp, i32, i64, i64, i32, i32, i32, vp, vp, vp, vp]
    L.bq_quantize_f16s.restype = i32
    L.bq_quantize_mixed.argtypes = [vp, i32, i64, i64, vp, i32, vp, vp, vp, vp]
    L.bq_quantize_mixed.restype = i32
    L.bq_dequantize.argtypes = [vp, vp, vp, vp, i32, i32, i64, i64, i32, vp, i32, vp]
    L.bq_dequantize.restype = i32
    L.bq_fake_quantize.argtypes = [vp, i32, i64, i64, i32, i32, vp, i32, vp]
    L.bq_fake_quantize.restype = i32
    L.bq_linear.argtypes = [vp, i32, i64, i64, vp, vp, vp, vp, i32, i32, i64, i32, vp, vp]
    L.bq_linear.restype = i32
    L.bq_linear_f16s.argtypes = [vp, i32, i64, i64, vp, vp, vp, i32, i32, i64, i32, vp, vp]
    L.bq_linear_f16s.restype = i32
    L.bq_linear_workspace_bytes.argtypes = [i64, i64, i64, i32, i32]
    L.bq_linear_workspace_bytes.restype = ctypes.c_size_t
    L.bq_linear_ws.argtypes = [vp, i32, i64, i64, vp, vp, vp, vp, i32, i32, i64, i32, vp, vp, ctypes.c_size_t, vp]
    L.bq_linear_ws.restype = i32
    L.bq_linear_grad_input.argtypes = [vp, i32, i64, i64, vp, vp, vp, vp, i32, i32, i64, i32, vp, vp]
    L.bq_linear_grad_input.restype = i32
    L.bq_dropout.argtypes = [vp, i32, i64, i64, i64, ctypes.c_double, vp, vp, i64, vp]
    L.bq_dropout.restype = i32
    L.bq_lora.argtypes = [ctypes.c_char_p, vp]
    L.bq_lora.restype = i32
    L.bq_lora_grad.argtypes = [ctypes.c_char_p, vp]
    L.bq_lora_grad.restype = i32
    L.bq_check_division.argtypes = [ctypes.c_uint32, ctypes.c_uint32, i32, vp, vp]
    L.bq_check_division.restype = i32
    L.bq_check_const_division.argtypes = [i32, ctypes.c_uint32, ctypes.c_uint32, vp, vp]
    L.bq_check_const_division.restype = i32
    L.bq_selftest_bounded_wait.argtypes = [ctypes.c_uint32, vp]
    L.bq_selftest_bounded_wait.restype = i32
    L.bq_set_option.argtypes = [i32, i32]
    L.bq_set_option.restype = i32
    L.bq_get_option.argtypes = [i32]
    L.bq_get_option.restype = i32
    L.bq_device_status.argtypes = [vp]
    L.bq_device_status.restype = i32
    L.bq_status_string.argtypes = [i32]
    L.bq_status_string.restype = ctypes.c_char_p
    L.bq_version.argtypes = []
    L.bq_version.restype = ctypes.c_char_p
    if path is None:
        _lib = L
    return L


def status_string(status: int) -> str:
    return lib().bq_status_string(int(status)).decode()


def _check(fn: str, status: int):
    if status != BQ_OK:
        raise BQError(fn, status)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


# ---------------------------------------------------------------------------
# size queries
# ---------------------------------------------------------------------------

def bq_packed_bytes(rows: int, cols: int, bits: int) -> int:
    return int(lib().bq_packed_bytes(rows, cols, bits))


def bq_group_count(rows: int, cols: int, group: int) -> int:
    return int(lib().bq_group_count(rows, cols, group))


def bq_mixed_offsets(bit_map, rows: int, cols: int):
    bm = np.ascontiguousarray(np.asarray(bit_map, dtype=np.uint8))
    nb = rows // 128
    co = np.zeros(nb + 1, dtype=np.int64)
    go = np.zeros(nb + 1, dtype=np.int64)
    _check("bq_mixed_offsets", lib().bq_mixed_offsets(bm.ctypes.data_as(ctypes.c_void_p), rows, cols,
                                                      co.ctypes.data_as(ctypes.c_void_p),
                                                      go.ctypes.data_as(ctypes.c_void_p)))
    return co, go


# ---------------------------------------------------------------------------
# quantize / dequantize / linear
# ---------------------------------------------------------------------------

def bq_quantize(W: torch.Tensor, bits: int, group: int | None = None, layout: str = "interleaved",
                out=None, stream=None, scheme: str = "asymmetric"):
    """Quantize W [N, K] (fp16/bf16, CUDA) with the asymmetric MinMax scheme (default), the
    symmetric abs-max one, or the MinMax scheme with binary16 scales ("asymmetric_f16_scale").
    Returns (packed u8, scales, zeros u8): scales f32 (f16 for the binary16 format) / zeros are
    [N, K/g] in the canonical layout and flat (128-row-block-major order) in the interleaved one."""
    group = group or GROUP_OF_BITS[bits]
    N, K = W.shape
    s16 = scheme == "asymmetric_f16_scale"
    if out is None:
        packed = torch.empty(max(1, bq_packed_bytes(N, K, bits)), dtype=torch.uint8, device=W.device)
        mshape = (N, K // group) if layout == "canonical" else (N * (K // group),)
        scales = torch.empty(mshape, dtype=torch.float16 if s16 else torch.float32, device=W.device)
        zeros = torch.empty(mshape, dtype=torch.uint8, device=W.device)
    else:
        packed, scales, zeros = out
    fn = {"symmetric": lib().bq_quantize_symmetric, "asymmetric_f16_scale": lib().bq_quantize_f16s,
          "asymmetric": lib().bq_quantize}[scheme]
    st = fn(_ptr(W), DTYPE_CODE[W.dtype], N, K, bits, group, LAYOUTS[layout],
            _ptr(packed), _ptr(scales), _ptr(zeros), _stream(stream))
    _check("bq_quantize", st)
    return packed, scales, zeros


def mixed_sizes(bit_map, rows: int, cols: int):
    co, go = bq_mixed_offsets(bit_map, rows, cols)
    return int(co[-1]), int(go[-1])


def bq_quantize_mixed(W: torch.Tensor, bit_map, layout: str = "interleaved", stream=None):
    """Per-128-row-block width (4 -> group 128, 2 -> group 64).  bit_map: host sequence.
    Returns (packed, scales, zeros, bit_map_dev)."""
    N, K = W.shape
    code_bytes, groups = mixed_sizes(bit_map, N, K)
    bm = torch.as_tensor(np.asarray(bit_map, dtype=np.uint8)).to(W.device)
    packed = torch.empty(max(1, code_bytes), dtype=torch.uint8, device=W.device)
    scales = torch.empty(max(1, groups), dtype=torch.float32, device=W.device)
    zeros = torch.empty(max(1, groups), dtype=torch.uint8, device=W.device)
    st = lib().bq_quantize_mixed(_ptr(W), DTYPE_CODE[W.dtype], N, K, _ptr(bm), LAYOUTS[layout],
                                 _ptr(packed), _ptr(scales), _ptr(zeros), _stream(stream))
    _check("bq_quantize_mixed", st)
    return packed, scales, zeros, bm


def bq_dequantize(packed, scales, zeros, rows: int, cols: int, bits: int = 4, group: int | None = None,
                  layout: str = "interleaved", out_dtype=torch.float32, bit_map_dev=None, stream=None):
    group = group or GROUP_OF_BITS.get(bits, 0)
    out = torch.empty((rows, cols), dtype=out_dtype, device=packed.device)
    st = lib().bq_dequantize(_ptr(packed), _ptr(scales), _ptr(zeros), _ptr(bit_map_dev), bits, group,
                             rows, cols, LAYOUTS[layout], _ptr(out), DTYPE_CODE[out_dtype], _stream(stream))
    _check("bq_dequantize", st)
    return out


def bq_fake_quantize(W: torch.Tensor, bits: int, group: int | None = None, out_dtype=None, out=None, stream=None):
    """dequant(quant(W)) in one pass (codes, scales, zeros not stored); out in W's dtype by default."""
    group = group or GROUP_OF_BITS[bits]
    N, K = W.shape
    o = out if out is not None else torch.empty((N, K), dtype=out_dtype or W.dtype, device=W.device)
    st = lib().bq_fake_quantize(_ptr(W), DTYPE_CODE[W.dtype], N, K, bits, group, _ptr(o), DTYPE_CODE[o.dtype],
                                _stream(stream))
    _check("bq_fake_quantize", st)
    return o


def bq_linear_workspace_bytes(M: int, N: int, K: int, bits: int = 4, mixed: bool = False) -> int:
    """Device workspace bytes that let bq_linear(..., workspace=...) split K (0: no split)."""
    return int(lib().bq_linear_workspace_bytes(M, N, K, bits, 1 if mixed else 0))


def bq_linear(x: torch.Tensor, packed, scales, zeros, N: int, bits: int = 4, group: int | None = None,
              bit_map_dev=None, layout: str = "interleaved", out=None, stream=None, workspace=None):
    """y [M, N] = x [M, K] . dequant(W)^T, y in x's dtype.  fp16 `scales` (from the binary16
    scale format) select bq_linear_f16s; a device `workspace` (uint8, from
    bq_linear_workspace_bytes) selects bq_linear_ws."""
    group = group or GROUP_OF_BITS.get(bits, 0)
    M, K = x.shape
    y = out if out is not None else torch.empty((M, N), dtype=x.dtype, device=x.device)
    if scales.dtype == torch.float16:
        if bit_map_dev is not None:
            raise ValueError("binary16 scales take no width map")
        st = lib().bq_linear_f16s(_ptr(x), DTYPE_CODE[x.dtype], M, K, _ptr(packed), _ptr(scales), _ptr(zeros),
                                  bits, group, N, LAYOUTS[layout], _ptr(y), _stream(stream))
        _check("bq_linear_f16s", st)
        return y
    if workspace is not None:
        st = lib().bq_linear_ws(_ptr(x), DTYPE_CODE[x.dtype], M, K, _ptr(packed), _ptr(scales), _ptr(zeros),
                                _ptr(bit_map_dev), bits, group, N, LAYOUTS[layout], _ptr(y), _ptr(workspace),
                                workspace.numel() * workspace.element_size(), _stream(stream))
        _check("bq_linear_ws", st)
        return y
    st = lib().bq_linear(_ptr(x), DTYPE_CODE[x.dtype], M, K, _ptr(packed), _ptr(scales), _ptr(zeros),
                         _ptr(bit_map_dev), bits, group, N, LAYOUTS[layout], _ptr(y), _stream(stream))
    _check("bq_linear", st)
    return y


def bq_linear_grad_input(dy: torch.Tensor, packed, scales, zeros, K: int, bits: int = 4, group: int | None = None,
                         layout: str = "interleaved", out=None, stream=None, bit_map_dev=None):
    """dx [M, K] = dy [M, N] . dequant(W), dx in dy's dtype (the input
    gradient of bq_linear); bit_map_dev: a width map's device copy, as for bq_linear."""
    group = group or GROUP_OF_BITS.get(bits, 0)
    M, N = dy.shape
    dx = out if out is not None else torch.empty((M, K), dtype=dy.dtype, device=dy.device)
    st = lib().bq_linear_grad_input(_ptr(dy), DTYPE_CODE[dy.dtype], M, N, _ptr(packed), _ptr(scales), _ptr(zeros),
                                    _ptr(bit_map_dev), bits, group, K, LAYOUTS[layout], _ptr(dx), _stream(stream))
    _check("bq_linear_grad_input", st)
    return dx


# ---------------------------------------------------------------------------
# dropout and low-rank adapters
# ---------------------------------------------------------------------------

# bq_lora_args and bq_lora_grad_args of include/bq.h: pointers, then int64 sizes, then p and the int32 fields
_LORA_ARGS = struct.Struct("=11Q6qd4i")
_LORA_GRAD_ARGS = struct.Struct("=15Q7qd4i")


def _bad(name: str, want: str, v):
    return ValueError(f"{name}: {want} expected, got {tuple(v.shape)} {v.dtype} on {v.device} with strides {v.stride()}")


def _matrix(name: str, v, rows: int, cols: int, dtype, dev: int) -> int:
    """The row stride of v [rows, cols] of dtype on CUDA device dev, columns contiguous."""
    if v.shape != (rows, cols) or v.dtype is not dtype or v.get_device() != dev:
        raise _bad(name, f"[{rows}, {cols}] {dtype} on cuda:{dev}", v)
    ld, unit = v.stride()
    if unit != 1 and cols > 1 and rows:
        raise _bad(name, "contiguous columns", v)
    return ld


def _dense(name: str, v, shape, dtype, dev: int) -> int:
    """The address of a contiguous tensor of this shape and dtype on CUDA device dev."""
    if v.shape != shape or v.dtype is not dtype or v.get_device() != dev or not v.is_contiguous():
        raise _bad(name, f"contiguous {shape} {dtype} on cuda:{dev}", v)
    return v.data_ptr()


def _rng_ptr(rng, dev: int) -> int:
    return 0 if rng is None else _dense("rng", rng, (2,), torch.int64, dev)


def _device(name: str, v) -> int:
    dev = v.get_device()
    if dev < 0:
        raise ValueError(f"{name}: a CUDA tensor expected")
    return dev


def _empty(shape, like, stream):
    """A result of like's type and device that belongs to the stream that the kernel runs on."""
    if stream is None:
        return torch.empty(shape, dtype=like.dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=like.dtype, device=like.device)


def _launch(name: str, fn, dev: int, stream, *args):
    """Call fn on the tensors' device, on its current stream or the one given."""
    if dev != torch._C._cuda_getDevice():
        with torch.cuda.device(dev):
            return _launch(name, fn, dev, stream, *args)
    st = fn(*args, stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(dev))
    if st != BQ_OK:
        raise BQError(name, st)


def bq_dropout(x: torch.Tensor, p: float, rng=None, out=None, stream=None):
    """mask * x / (1 - p) for x [rows, cols] (fp16 / bf16 / fp32, any row stride), the mask drawn
    from rng (int64 {seed, offset} on the device) and never stored.  The gradient is the same call on dy."""
    rows, cols = x.shape
    dev, dtype = _device("x", x), x.dtype
    if out is None:
        out = _empty((rows, cols), x, stream)
    _launch("bq_dropout", lib().bq_dropout, dev, stream, x.data_ptr(), DTYPE_CODE[dtype], rows, cols,
            _matrix("x", x, rows, cols, dtype, dev), p, _rng_ptr(rng, dev), out.data_ptr(),
            _matrix("out", out, rows, cols, dtype, dev))
    return out


def bq_lora(x: torch.Tensor, A, B, ranks, scales, seg_off, seg_adapter, base=None, out=None, p: float = 0.0, rng=None,
            t=None, stream=None):
    """y [M, N] = base + scales[a] (drop(x) A[a]^T) B[a]^T for the rows of each segment.

    x [M, K] and the pools A [L, R, K], B [L, N, R] in bf16 or fp16; segment i is rows
    seg_off[i] .. seg_off[i + 1] - 1 with adapter seg_adapter[i] (-1: none); rows behind the last segment keep what
    `out` holds.  base None: zeros; out may be base (in place) and is allocated when None.  t: fp32 [M, R] that
    receives drop(x) A[a]^T for bq_lora_grad."""
    M, K = x.shape
    L, N, R = B.shape
    S, = seg_adapter.shape
    dev, dtype = _device("x", x), x.dtype
    if out is None:
        out = _empty((M, N), x, stream)
    args = _LORA_ARGS.pack(
        x.data_ptr(), _dense("A", A, (L, R, K), dtype, dev), _dense("B", B, (L, N, R), dtype, dev),
        _dense("ranks", ranks, (L,), torch.int32, dev), _dense("scales", scales, (L,), torch.float32, dev),
        _dense("seg_off", seg_off, (S + 1,), torch.int32, dev),
        _dense("seg_adapter", seg_adapter, (S,), torch.int32, dev), _rng_ptr(rng, dev),
        0 if base is None else base.data_ptr(), out.data_ptr(),
        0 if t is None else _dense("t", t, (M, R), torch.float32, dev), M, K, N, _matrix("x", x, M, K, dtype, dev),
        0 if base is None else _matrix("base", base, M, N, dtype, dev), _matrix("out", out, M, N, dtype, dev), p, R, L, S,
        DTYPE_CODE[dtype])
    _launch("bq_lora", lib().bq_lora, dev, stream, args)
    return out


def bq_lora_grad(dy: torch.Tensor, x, t, A, B, ranks, scales, seg_off, seg_adapter, base=None, out=None,
                 p: float = 0.0, rng=None, dA=None, dB=None, workspace=None, need_dx: bool = True,
                 need_weights: bool = True, stream=None):
    """(dx, dA, dB) of bq_lora from dy [M, N], its input x, the t that it stored and the same p and rng.

    dx = base + mask / (1 - p) (scales[a] (dy B[a]) A[a]) in dy's dtype (base None: zeros; out may be base); dA [L, R, K]
    and dB [L, N, R] in fp32, written in full.  need_dx / need_weights False skip them (None is returned; x and t are
    not looked at without the weights).  workspace: fp32 [M, R] scratch, allocated when None."""
    M, N = dy.shape
    L, R, K = A.shape
    S, = seg_adapter.shape
    dev, dtype = _device("dy", dy), dy.dtype
    if stream is not None and (workspace is None or (need_dx and out is None) or (need_weights and (dA is None or dB is None))):
        # what is allocated here belongs to the stream that the kernels run on
        with torch.cuda.stream(stream):
            return bq_lora_grad(dy, x, t, A, B, ranks, scales, seg_off, seg_adapter, base, out, p, rng, dA, dB, workspace,
                                need_dx, need_weights)
    f32 = torch.float32
    if workspace is None:
        workspace = torch.empty((M, R), dtype=f32, device=dy.device)
    xp = tp = bp = op = ap = wp = ldx = ldb = ldo = 0
    if need_dx:
        if out is None:
            out = torch.empty((M, K), dtype=dtype, device=dy.device)
        op, ldo = out.data_ptr(), _matrix("out", out, M, K, dtype, dev)
        if base is not None:
            bp, ldb = base.data_ptr(), _matrix("base", base, M, K, dtype, dev)
    else:
        out = None
    if need_weights:
        if dA is None:
            dA = torch.empty((L, R, K), dtype=f32, device=dy.device)
        if dB is None:
            dB = torch.empty((L, N, R), dtype=f32, device=dy.device)
        ap, wp = _dense("dA", dA, (L, R, K), f32, dev), _dense("dB", dB, (L, N, R), f32, dev)
        xp, ldx, tp = x.data_ptr(), _matrix("x", x, M, K, dtype, dev), _dense("t", t, (M, R), f32, dev)
    else:
        dA = dB = None
    args = _LORA_GRAD_ARGS.pack(
        dy.data_ptr(), xp, tp, _dense("A", A, (L, R, K), dtype, dev), _dense("B", B, (L, N, R), dtype, dev),
        _dense("ranks", ranks, (L,), torch.int32, dev), _dense("scales", scales, (L,), f32, dev),
        _dense("seg_off", seg_off, (S + 1,), torch.int32, dev),
        _dense("seg_adapter", seg_adapter, (S,), torch.int32, dev), _rng_ptr(rng, dev), bp, op,
        _dense("workspace", workspace, (M, R), f32, dev), ap, wp, M, K, N, _matrix("dy", dy, M, N, dtype, dev), ldx, ldb,
        ldo, p, R, L, S, DTYPE_CODE[dtype])
    _launch("bq_lora_grad", lib().bq_lora_grad, dev, stream, args)
    return out, dA, dB


def bq_check_division(s_bits_begin: int, s_bits_end: int, refinements: int = 2, stream=None):
    """Returns (mismatches, pairs checked, first bad divisor bits, first bad fp16 numerator bits)."""
    res = torch.zeros(4, dtype=torch.int64, device="cuda")
    _check("bq_check_division", lib().bq_check_division(s_bits_begin, s_bits_end, refinements, _ptr(res),
                                                        _stream(stream)))
    torch.cuda.synchronize()
    return tuple(int(v) for v in res.cpu())


def bq_check_const_division(divisor: int, x_bits_begin: int, x_bits_end: int, stream=None):
    """Returns (mismatches, values checked, first bad x bits, its divisor)."""
    res = torch.zeros(4, dtype=torch.int64, device="cuda")
    _check("bq_check_const_division", lib().bq_check_const_division(divisor, x_bits_begin, x_bits_end, _ptr(res),
                                                                    _stream(stream)))
    torch.cuda.synchronize()
    return tuple(int(v) for v in res.cpu())


def bq_selftest_bounded_wait(limit: int, stream=None):
    _check("bq_selftest_bounded_wait", lib().bq_selftest_bounded_wait(limit, _stream(stream)))


def bq_set_option(option: int, value: int):
    _check("bq_set_option", lib().bq_set_option(option, value))


def bq_get_option(option: int) -> int:
    return int(lib().bq_get_option(option))


def bq_device_status(stream=None) -> int:
    return int(lib().bq_device_status(_stream(stream)))


def bq_version() -> str:
    return lib().bq_version().decode()


# ---------------------------------------------------------------------------
# host-buffer path (end-to-end: pinned host in, host out, through the C ABI)
# ---------------------------------------------------------------------------

def bq_linear_host(x_host: torch.Tensor, packed, scales, zeros, N: int, bits: int = 4, group=None,
                   bit_map_dev=None, x_dev=None, y_dev=None, y_host=None, stream=None):
    """Copy x from (pinned) host memory, run bq_linear, copy y back to host."""
    s = stream or torch.cuda.current_stream()
    if x_dev is None:
        x_dev = torch.empty(x_host.shape, dtype=x_host.dtype, device="cuda")
    x_dev.copy_(x_host, non_blocking=True)
    y_dev = bq_linear(x_dev, packed, scales, zeros, N, bits, group, bit_map_dev, out=y_dev, stream=s)
    if y_host is None:
        y_host = torch.empty(y_dev.shape, dtype=y_dev.dtype, pin_memory=True)
    y_host.copy_(y_dev, non_blocking=True)
    return y_host
