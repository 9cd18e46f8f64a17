"""Python binding of libmxq: the C entry points under the same names.

Argument marshalling only: every step of the computation runs in the HIP kernels
of libmxq.so. Inputs are torch tensors on the current GPU; outputs are allocated
here with torch (device memory only) unless passed in, and every call is enqueued
on torch's current stream. A missing library raises immediately: there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os
from typing import NamedTuple, Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmxq.so")

MXQ_OK, MXQ_EINVAL, MXQ_ESHAPE, MXQ_EALIGN, MXQ_EUNSUPPORTED, MXQ_EHIP = range(6)
BF16, F32 = 0, 1
MXFP4, NVFP4, NVFP4_2D = 0, 1, 2
RNE, SR, SR16 = 0, 1, 2
ROWWISE, COLWISE, BOTH = 1, 2, 3

_FMT = {"mxfp4": MXFP4, "nvfp4": NVFP4, "nvfp4_2d": NVFP4_2D}
_AXIS = {"row": ROWWISE, "col": COLWISE, "both": BOTH}
_RND = {"rne": RNE, "sr": SR, "sr16": SR16}
OPERAND_MXFP4, OPERAND_FP8 = 0, 1
_ACT = {"none": 0, "relu": 1, "gelu": 2, "silu": 3, "swiglu": 4}
SWIGLU = 4

_lib = None


def lib() -> ctypes.CDLL:
    """Load libmxq.so (built in-tree by mxfp4_microscaling_quantization_amd.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                           "`python -m mxfp4_microscaling_quantization_amd.build`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i32, i64, u16, u64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_uint16, ctypes.c_uint64
    L.mxq_quantize.argtypes = [vp, i32, i64, i64, i64, i32, i32, i32, u64, u64, vp, vp, vp, vp, vp, vp, vp]
    L.mxq_rht_quantize.argtypes = [vp, i32, i64, i64, i64, i32, i32, u64, i32, u64, u64, vp, vp, vp, vp,
                                   vp, vp, vp]
    L.mxq_rht_quantize_mask.argtypes = [vp, i32, i64, i64, i64, i32, i32, u16, i32, u64, u64, vp, vp, vp,
                                        vp, vp, vp, vp]
    L.mxq_dequantize.argtypes = [vp, vp, i32, i64, i64, vp, vp, i32, vp]
    L.mxq_fp8_to_mxfp4.argtypes = [vp, vp, i64, i64, vp, vp, vp]
    L.mxq_mxfp4_to_fp8.argtypes = [vp, vp, i64, i64, vp, vp, vp]
    L.mxq_fp4_row_to_fp8_col.argtypes = [vp, vp, i64, i64, vp, i64, vp, i64, vp, i64, vp]
    L.mxq_rht_apply.argtypes = [vp, i32, i64, i64, i64, u16, vp, vp]
    L.mxq_amax.argtypes = [vp, i32, i64, i64, i64, vp, vp]
    L.mxq_rht_amax.argtypes = [vp, i32, i64, i64, i64, i32, u16, vp, vp]
    L.mxq_rht_signs.argtypes = [u64]
    L.mxq_rht_signs.restype = u16
    L.mxq_status_string.argtypes = [i32]
    L.mxq_status_string.restype = ctypes.c_char_p
    L.mxq_gemm.argtypes = [vp, vp, i32, vp, vp, i32, i64, i64, i64, vp, i32, i32, vp, vp, i32, vp, vp]
    L.mxq_grouped_gemm.argtypes = [vp, vp, i32, vp, vp, i32, i64, i64, i64, vp, i64, vp, i32, i32, vp, vp, i32, vp, vp]
    L.mxq_grouped_wgrad.argtypes = [vp, vp, i64, i64, vp, vp, i64, i64, i64, i64, i64, vp, i64, vp, vp, i32, vp]
    L.mxq_act_grad.argtypes = [vp, vp, i32, i64, i64, i32, vp, i64, vp, vp, vp, vp]
    L.mxq_act_grad_workspace.argtypes = [i64, i64, i64]
    L.mxq_act_grad_workspace.restype = i64
    L.mxq_route.argtypes = [vp, i32, i64, i64, i64, i64, i32, vp, vp, vp]
    L.mxq_route_grad.argtypes = [vp, vp, vp, vp, i32, i64, i64, i64, i64, i32, vp, vp]
    L.mxq_expert_sort.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp]
    L.mxq_expert_sort_workspace.argtypes = [i64, i64]
    L.mxq_expert_sort_workspace.restype = i64
    L.mxq_dispatch.argtypes = [vp, i32, i64, i64, i64, vp, i64, i64, i32, vp, vp, vp]
    L.mxq_combine.argtypes = [vp, i32, i64, i64, vp, vp, i64, i64, vp, vp, i32, vp]
    L.mxq_combine_grad.argtypes = [vp, i32, vp, i32, i64, i64, vp, vp, i64, i64, vp, vp, vp]
    L.mxq_fp8_quantize.argtypes = [vp, i32, i64, i64, i64, vp, vp, vp]
    L.mxq_fp8_act_grad.argtypes = [vp, i32, vp, vp, i64, i64, i32, vp, i64, vp, vp, vp, vp, vp]
    for name in ("mxq_route", "mxq_route_grad", "mxq_expert_sort", "mxq_dispatch", "mxq_combine", "mxq_combine_grad",
                 "mxq_fp8_quantize", "mxq_fp8_act_grad", "mxq_gemm", "mxq_grouped_gemm", "mxq_grouped_wgrad", "mxq_act_grad", "mxq_quantize", "mxq_rht_quantize",
                 "mxq_rht_quantize_mask", "mxq_dequantize", "mxq_fp8_to_mxfp4", "mxq_mxfp4_to_fp8",
                 "mxq_fp4_row_to_fp8_col", "mxq_rht_apply", "mxq_amax", "mxq_rht_amax"):
        getattr(L, name).restype = i32
    _lib = L
    return L


class MxqError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        super().__init__(mxq_status_string(status))


def mxq_status_string(status: int) -> str:
    return lib().mxq_status_string(status).decode()


def mxq_rht_signs(seed: int) -> int:
    return int(lib().mxq_rht_signs(seed))


def _check(status: int) -> None:
    if status != MXQ_OK:
        raise MxqError(status)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream() -> int:
    # The current device's current stream by the functions under torch.cuda.current_stream(),
    # which builds a Stream object around it: 0.2 us instead of 2.8, where a small call takes 9.
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"unsupported input dtype {t.dtype}")


def _rows_view(x: torch.Tensor):
    if x.dim() != 2 or (x.shape[0] > 0 and x.stride(1) != 1):
        raise ValueError("expected a 2-D tensor with unit column stride")
    return x.shape[0], x.shape[1], (x.stride(0) if x.shape[0] > 0 else x.shape[1])


class Quantized(NamedTuple):
    codes_row: Optional[torch.Tensor]
    scales_row: Optional[torch.Tensor]
    codes_col: Optional[torch.Tensor]
    scales_col: Optional[torch.Tensor]
    tensor_scale: Optional[torch.Tensor]


def _alloc_outputs(x, rows, cols, fmt, axis):
    bs = 32 if fmt == MXFP4 else 16
    dev = x.device
    u8 = torch.uint8
    cr = sr = cc = sc = None
    if axis & ROWWISE:
        cr = torch.empty((rows, cols // 2), dtype=u8, device=dev)
        sr = torch.empty((rows, cols // bs), dtype=u8, device=dev)
    if axis & COLWISE:
        cc = torch.empty((cols, rows // 2), dtype=u8, device=dev)
        sc = torch.empty((cols, rows // bs), dtype=u8, device=dev)
    ts = torch.empty((1,), dtype=torch.float32, device=dev) if fmt != MXFP4 else None
    return cr, sr, cc, sc, ts


def mxq_quantize(x: torch.Tensor, fmt: str = "mxfp4", axis: str = "row", rnd: str = "rne",
                 sr_seed: int = 0, sr_offset: int = 0, amax: Optional[torch.Tensor] = None,
                 out: Optional[Quantized] = None) -> Quantized:
    """mxq_quantize: MXFP4/NVFP4 quantisation. NVFP4 takes the tensor amax (e.g. from
    mxq_amax), or computes it first when `amax` is None."""
    rows, cols, ldx = _rows_view(x)
    f, a, r = _FMT[fmt], _AXIS[axis], _RND[rnd]
    o = out if out is not None else Quantized(*_alloc_outputs(x, rows, cols, f, a))
    _check(lib().mxq_quantize(_ptr(x), _dtype_code(x), rows, cols, ldx, f, a, r, sr_seed, sr_offset,
                              _ptr(o.codes_row), _ptr(o.scales_row), _ptr(o.codes_col),
                              _ptr(o.scales_col), _ptr(amax), _ptr(o.tensor_scale), _stream()))
    return o


def mxq_rht_quantize(x: torch.Tensor, rht_seed: int, fmt: str = "mxfp4", axis: str = "row",
                     rnd: str = "rne", sr_seed: int = 0, sr_offset: int = 0,
                     amax: Optional[torch.Tensor] = None, out: Optional[Quantized] = None) -> Quantized:
    """mxq_rht_quantize: random-sign 16-point Hadamard (signs drawn from `rht_seed`,
    mxq_rht_signs) fused ahead of quantisation."""
    rows, cols, ldx = _rows_view(x)
    f, a, r = _FMT[fmt], _AXIS[axis], _RND[rnd]
    o = out if out is not None else Quantized(*_alloc_outputs(x, rows, cols, f, a))
    _check(lib().mxq_rht_quantize(_ptr(x), _dtype_code(x), rows, cols, ldx, f, a, rht_seed, r, sr_seed,
                                  sr_offset, _ptr(o.codes_row), _ptr(o.scales_row), _ptr(o.codes_col),
                                  _ptr(o.scales_col), _ptr(amax), _ptr(o.tensor_scale), _stream()))
    return o


def mxq_rht_quantize_mask(x: torch.Tensor, sign_mask: int, fmt: str = "mxfp4", axis: str = "row",
                          rnd: str = "rne", sr_seed: int = 0, sr_offset: int = 0,
                          amax: Optional[torch.Tensor] = None, out: Optional[Quantized] = None) -> Quantized:
    """mxq_rht_quantize_mask: as mxq_rht_quantize with the sign mask given directly
    (bit i -> s_i = -1; 0 = the deterministic H16)."""
    rows, cols, ldx = _rows_view(x)
    f, a, r = _FMT[fmt], _AXIS[axis], _RND[rnd]
    o = out if out is not None else Quantized(*_alloc_outputs(x, rows, cols, f, a))
    _check(lib().mxq_rht_quantize_mask(_ptr(x), _dtype_code(x), rows, cols, ldx, f, a, sign_mask, r, sr_seed,
                                       sr_offset, _ptr(o.codes_row), _ptr(o.scales_row), _ptr(o.codes_col),
                                       _ptr(o.scales_col), _ptr(amax), _ptr(o.tensor_scale), _stream()))
    return o


def mxq_dequantize(codes: torch.Tensor, scales: torch.Tensor, fmt: str = "mxfp4",
                   tensor_scale: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """mxq_dequantize: codes [R, C/2] + scales -> [R, C] in bf16 or fp32."""
    rows, cols = codes.shape[0], codes.shape[1] * 2
    y = out if out is not None else torch.empty((rows, cols), dtype=out_dtype, device=codes.device)
    _check(lib().mxq_dequantize(_ptr(codes), _ptr(scales), _FMT[fmt], rows, cols, _ptr(tensor_scale),
                                _ptr(y), _dtype_code(y), _stream()))
    return y


def mxq_fp8_to_mxfp4(q8: torch.Tensor, s128: torch.Tensor, out=None):
    """mxq_fp8_to_mxfp4: E4M3 [R, C] (uint8 view) + fp32 [R, C/128] -> (codes, e8m0)."""
    rows, cols = q8.shape
    if out is None:
        out = (torch.empty((rows, cols // 2), dtype=torch.uint8, device=q8.device),
               torch.empty((rows, cols // 32), dtype=torch.uint8, device=q8.device))
    _check(lib().mxq_fp8_to_mxfp4(_ptr(q8), _ptr(s128), rows, cols, _ptr(out[0]), _ptr(out[1]), _stream()))
    return out


def mxq_mxfp4_to_fp8(codes: torch.Tensor, e8m0: torch.Tensor, out=None):
    """mxq_mxfp4_to_fp8: (codes [R, C/2], e8m0 [R, C/32]) -> (E4M3 [R, C] uint8, fp32 [R, C/128])."""
    rows, cols = codes.shape[0], codes.shape[1] * 2
    if out is None:
        out = (torch.empty((rows, cols), dtype=torch.uint8, device=codes.device),
               torch.empty((rows, cols // 128), dtype=torch.float32, device=codes.device))
    _check(lib().mxq_mxfp4_to_fp8(_ptr(codes), _ptr(e8m0), rows, cols, _ptr(out[0]), _ptr(out[1]), _stream()))
    return out


def fp8_col_scale_slots(rows: int, n_experts: int) -> int:
    """Scale entries per output row that suffice for any split of `rows` into experts."""
    return (rows + 127 * n_experts) // 128


def mxq_fp4_row_to_fp8_col(codes: torch.Tensor, e8m0: torch.Tensor, offsets: torch.Tensor, out=None):
    """mxq_fp4_row_to_fp8_col: MXFP4 rows of tokens grouped by expert (device int64
    offsets [E+1]) -> (E4M3 of X^T [C, R] uint8, fp32 scales [C, S]), one scale per
    128-token group of an expert; `out` = (q8 [C, ld_q8], scales [C, ld_s])."""
    rows, cols = codes.shape[0], codes.shape[1] * 2
    n_experts = offsets.numel() - 1
    if out is None:
        ld_q8 = (rows + 15) // 16 * 16
        out = (torch.empty((cols, ld_q8), dtype=torch.uint8, device=codes.device),
               torch.empty((cols, fp8_col_scale_slots(rows, n_experts)), dtype=torch.float32,
                           device=codes.device))
    q8, s = out
    _check(lib().mxq_fp4_row_to_fp8_col(_ptr(codes), _ptr(e8m0), rows, cols, _ptr(offsets), n_experts,
                                        _ptr(q8), q8.stride(0), _ptr(s), s.stride(0), _stream()))
    return q8[:, :rows], s


def mxq_rht_apply(x: torch.Tensor, sign_mask: int, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """mxq_rht_apply: y = (1/4) H16 (s * x) on every 16-chunk of each row, fp32."""
    rows, cols, ldx = _rows_view(x)
    y = out if out is not None else torch.empty((rows, cols), dtype=torch.float32, device=x.device)
    _check(lib().mxq_rht_apply(_ptr(x), _dtype_code(x), rows, cols, ldx, sign_mask, _ptr(y), _stream()))
    return y


def mxq_amax(x: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """mxq_amax: max |x| over the tensor as a device fp32[1] (NaN/Inf propagate)."""
    rows, cols, ldx = _rows_view(x)
    a = out if out is not None else torch.empty((1,), dtype=torch.float32, device=x.device)
    _check(lib().mxq_amax(_ptr(x), _dtype_code(x), rows, cols, ldx, _ptr(a), _stream()))
    return a


def mxq_rht_amax(x: torch.Tensor, sign_mask: int, axis: str = "row",
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """mxq_rht_amax: max |(1/4) H16 (s * x)| with the transform along rows ("row") or
    columns ("col"), as a device fp32[1]."""
    rows, cols, ldx = _rows_view(x)
    a = out if out is not None else torch.empty((1,), dtype=torch.float32, device=x.device)
    _check(lib().mxq_rht_amax(_ptr(x), _dtype_code(x), rows, cols, ldx, _AXIS[axis], sign_mask, _ptr(a),
                              _stream()))
    return a


# ---------------------------------------------------------------------------
# Matrix products (include/mxq_gemm.h). An operand is a pair (codes, scales): MXFP4 is
# uint8 codes [R, K/2] with uint8 E8M0 bytes [R, K/32], FP8 is E4M3 bytes [R, K] with
# fp32 scales [R, K/128]; for experts' weights [E, N, ...].

# scale dtype -> (format, elements of a code byte, elements of a scale)
_OPERANDS = {torch.uint8: (OPERAND_MXFP4, 2, 32), torch.float32: (OPERAND_FP8, 1, 128)}
_DTYPES = {torch.bfloat16: BF16, torch.float32: F32}


def _operand(op, dims: int):
    """(code pointer, scale pointer, format, k, shape of the codes) of an operand of `dims`
    dimensions, checked."""
    codes, scales = op
    kind = _OPERANDS.get(scales.dtype)
    if kind is None:
        raise TypeError(f"unsupported scale dtype {scales.dtype}")
    if codes.dtype != torch.uint8:
        raise TypeError(f"unsupported code dtype {codes.dtype}")
    fmt, per_code, per_scale = kind
    shape, sshape = codes.shape, scales.shape
    k = shape[-1] * per_code
    if len(shape) != dims or sshape[:-1] != shape[:-1] or sshape[-1] != k // per_scale:
        raise ValueError(f"operand of {dims} dimensions expected, got codes {tuple(shape)} and scales "
                         f"{tuple(sshape)}")
    if not (codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError("operands must be dense")
    return codes.data_ptr(), scales.data_ptr(), fmt, k, shape


def _dense(t: torch.Tensor, shape, dtype, what: str) -> int:
    """Pointer of a dense tensor of this shape and type, checked."""
    if t.shape != shape or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{what}: dense {dtype} {tuple(shape)} expected, got {t.dtype} {tuple(t.shape)}")
    return t.data_ptr()


def _float_code(dtype) -> int:
    code = _DTYPES.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def _offsets(offsets: torch.Tensor) -> int:
    if offsets.dtype != torch.int64 or offsets.dim() != 1 or offsets.numel() < 2 or not offsets.is_contiguous():
        raise ValueError("offsets: dense int64 [experts + 1] expected")
    return offsets.numel() - 1


def _on_gpu(first: torch.Tensor, *others: Optional[torch.Tensor]) -> int:
    """The current stream of the current GPU, on which all of these tensors must be: a kernel
    that follows a host pointer, or another GPU's, ends the process."""
    device = first.get_device()  # -1: host memory
    elsewhere = device < 0
    for t in others:
        if t is not None and t.get_device() != device:
            elsewhere = True
    if elsewhere or device != torch._C._cuda_getDevice():
        where = sorted({str(t.device) for t in (first, *others) if t is not None})
        raise ValueError(f"tensors on the current GPU expected, got some on {', '.join(where)}")
    return torch._C._cuda_getCurrentRawStream(device)


def _product(a, b, offsets, bias, act, residual, preact, out_dtype, out):
    ap, asp, afmt, k, ashape = _operand(a, 2)
    bp, bsp, bfmt, bk, bshape = _operand(b, 2 if offsets is None else 3)
    if bk != k:
        raise ValueError(f"contracted dimensions differ: {k} and {bk}")
    m, n, code = ashape[0], bshape[-2], _ACT[act]
    shape = (m, n // 2 if code == SWIGLU else n)
    d = z = None
    if out is not None:
        d, z = out
        out_dtype = d.dtype
    dt = _float_code(out_dtype)
    if d is None:
        d = a[0].new_empty(shape, dtype=out_dtype)
    else:
        _dense(d, shape, out_dtype, "out")
    if preact and z is None:
        z = a[0].new_empty((m, n), dtype=out_dtype)
    zp = None if z is None else _dense(z, (m, n), out_dtype, "z")
    rp = None if residual is None else _dense(residual, shape, out_dtype, "residual")
    bias_p, bdt = None, F32
    if bias is not None:
        bdt = _float_code(bias.dtype)
        bias_p = _dense(bias, bshape[:-1], bias.dtype, "bias")
    given = () if out is None else (d, z)
    stream = _on_gpu(*a, *b, offsets, bias, residual, *given)
    if offsets is None:
        status = lib().mxq_gemm(ap, asp, afmt, bp, bsp, bfmt, m, n, k, bias_p, bdt, code, rp, d.data_ptr(), dt, zp,
                                stream)
    else:
        experts = _offsets(offsets)
        if bshape[0] != experts:
            raise ValueError(f"{bshape[0]} weights for {experts} experts")
        status = lib().mxq_grouped_gemm(ap, asp, afmt, bp, bsp, bfmt, m, n, k, offsets.data_ptr(), experts, bias_p,
                                        bdt, code, rp, d.data_ptr(), dt, zp, stream)
    _check(status)
    return (d, z) if preact else d


def mxq_gemm(a, b, bias: Optional[torch.Tensor] = None, act: str = "none", residual: Optional[torch.Tensor] = None,
             preact: bool = False, out_dtype=torch.bfloat16, out=None):
    """mxq_gemm: d = act(A B^T + bias) + residual for operands a [M, K] and b [N, K] of
    (codes, scales); act is "none", "relu", "gelu", "silu" or "swiglu" (rows of B in
    gate/up pairs, d [M, N/2]). With `preact` the result is (d, z), z = A B^T + bias,
    which mxq_act_grad takes. `out` = (d, z or None); residual may be d itself."""
    return _product(a, b, None, bias, act, residual, preact, out_dtype, out)


def mxq_grouped_gemm(a, b, offsets: torch.Tensor, bias: Optional[torch.Tensor] = None, act: str = "none",
                     residual: Optional[torch.Tensor] = None, preact: bool = False, out_dtype=torch.bfloat16,
                     out=None):
    """mxq_grouped_gemm: mxq_gemm with the rows of a [R, K] grouped by expert (device
    int64 offsets [E+1]), one weight b [E, N, K] and bias [E, N] per expert."""
    return _product(a, b, offsets, bias, act, residual, preact, out_dtype, out)


def mxq_grouped_wgrad(y, x, offsets: torch.Tensor, rows: int, add: Optional[torch.Tensor] = None,
                      out_dtype=torch.bfloat16, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """mxq_grouped_wgrad: per expert dW = dY^T X (+ add) over its tokens, from the FP8
    columns that mxq_fp4_row_to_fp8_col returns: y = (q8 [N, >= rows], scales [N, S]),
    x likewise [K, ...]; d [E, N, K]. `rows` tokens in all; add may be `out`."""
    experts = _offsets(offsets)
    slots = fp8_col_scale_slots(rows, experts)
    for q8, s in (y, x):
        if q8.dtype != torch.uint8 or s.dtype != torch.float32:
            raise TypeError("FP8 columns are uint8 with fp32 scales")
        if q8.dim() != 2 or s.dim() != 2 or s.shape[0] != q8.shape[0] or q8.shape[1] < rows or s.shape[1] < slots:
            raise ValueError(f"columns of {rows} tokens and {slots} scales expected, got {tuple(q8.shape)} and "
                             f"{tuple(s.shape)}")
        if (q8.numel() and q8.stride(1) != 1) or (s.numel() and s.stride(1) != 1):
            raise ValueError("columns must have unit token stride")
    (yq, ys), (xq, xs) = y, x
    n, k = yq.shape[0], xq.shape[0]
    shape = (experts, n, k)
    if out is None:
        d = yq.new_empty(shape, dtype=out_dtype)
    else:
        d, out_dtype = out, out.dtype
    dt, dp = _float_code(out_dtype), _dense(d, shape, out_dtype, "out")
    addp = None if add is None else _dense(add, shape, out_dtype, "add")
    stream = _on_gpu(yq, ys, xq, xs, d, offsets, add)
    _check(lib().mxq_grouped_wgrad(yq.data_ptr(), ys.data_ptr(), yq.stride(0), ys.stride(0), xq.data_ptr(),
                                   xs.data_ptr(), xq.stride(0), xs.stride(0), rows, n, k, offsets.data_ptr(), experts,
                                   addp, dp, dt, stream))
    return d


def mxq_act_grad(dy: torch.Tensor, z: torch.Tensor, act: str = "none", offsets: Optional[torch.Tensor] = None,
                 bias_grad: bool = False, out: Optional[torch.Tensor] = None, db: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None):
    """mxq_act_grad: dz = act'(z) dy for the z that a product kept, and with `bias_grad`
    also the bias gradient: (dz, db), db fp32 [N], or [E, N] with expert offsets. `out`
    may be z; `workspace` (uint8, mxq_act_grad_workspace bytes) is allocated if absent."""
    rows, n = shape = z.shape
    code, dtype = _ACT[act], z.dtype
    dt = _float_code(dtype)
    zp = _dense(z, shape, dtype, "z")
    dyp = _dense(dy, (rows, n // 2 if code == SWIGLU else n), dtype, "dy")
    groups, offp = (1, None) if offsets is None else (_offsets(offsets), offsets.data_ptr())
    dz = torch.empty_like(z) if out is None else out
    dzp = _dense(dz, shape, dtype, "out")
    dbp = wsp = None
    if bias_grad:
        db_shape = (n,) if offsets is None else (groups, n)
        if db is None:
            db = z.new_empty(db_shape, dtype=torch.float32)
        dbp = _dense(db, db_shape, torch.float32, "db")
        need = lib().mxq_act_grad_workspace(rows, n, groups)
        if workspace is None:
            workspace = z.new_empty((need,), dtype=torch.uint8)
        elif workspace.numel() * workspace.element_size() < need:
            raise ValueError(f"workspace of {need} bytes expected")
        wsp = workspace.data_ptr()
    stream = _on_gpu(dy, z, dz, offsets, *((db, workspace) if bias_grad else ()))
    _check(lib().mxq_act_grad(dyp, zp, dt, rows, n, code, offp, groups, dzp, dbp, wsp, stream))
    return (dz, db) if bias_grad else dz


# ---------------------------------------------------------------------------
# Around the experts' products (include/mxq_moe.h). Assignment t k + j is token t's choice
# j of top k; `positions` [T, k] holds the rows of the assignments (-1: none).

_ROWS = {None: 0, "mxfp4": 1, "fp8": 2}


def _strided_rows(t: torch.Tensor, what: str):
    """(rows, columns, row stride) of a matrix whose columns lie side by side."""
    shape = t.shape
    if len(shape) != 2 or (shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{what}: a matrix with unit column stride expected")
    rows, cols = shape
    # (a stride means nothing where there are fewer than two rows)
    return rows, cols, t.stride(0) if rows > 1 else cols


def _positions(positions: torch.Tensor):
    if positions.dtype != torch.int32 or positions.dim() != 2 or not positions.is_contiguous():
        raise ValueError("positions: dense int32 [tokens, top_k] expected")
    return positions.shape


def mxq_route(logits: torch.Tensor, top_k: int, renorm: bool = False, out=None):
    """mxq_route: (weights fp32 [T, k], experts int32 [T, k]) of the top_k largest logits
    [T, E] of every token, in falling order; weights by the softmax over all experts or,
    with `renorm`, over the chosen ones. -Inf is never chosen: expert -1, weight 0."""
    tokens, n_experts, ld = _strided_rows(logits, "logits")
    dt = _float_code(logits.dtype)
    shape = (tokens, top_k)
    if out is None:  # (what is made here needs no checks: 0.4 us each, where a small call takes 8)
        stream = _on_gpu(logits)
        out = logits.new_empty(shape, dtype=torch.float32), logits.new_empty(shape, dtype=torch.int32)
        wp, ep = out[0].data_ptr(), out[1].data_ptr()
    else:
        wp, ep = _dense(out[0], shape, torch.float32, "weights"), _dense(out[1], shape, torch.int32, "experts")
        stream = _on_gpu(logits, *out)
    _check(lib().mxq_route(logits.data_ptr(), dt, tokens, n_experts, ld, top_k, int(renorm), wp, ep, stream))
    return out


def mxq_route_grad(dw: torch.Tensor, weights: torch.Tensor, experts: torch.Tensor, logits: torch.Tensor,
                   renorm: bool = False, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """mxq_route_grad: the gradient of the logits [T, E] (their type, dense) from the
    gradient `dw` of the weights that mxq_route gave for them."""
    tokens, n_experts, ld = _strided_rows(logits, "logits")
    dt, shape = _float_code(logits.dtype), dw.shape
    if len(shape) != 2 or shape[0] != tokens:
        raise ValueError(f"dw: [{tokens}, top_k] expected, got {tuple(shape)}")
    dwp = _dense(dw, shape, torch.float32, "dw")
    wp, ep = _dense(weights, shape, torch.float32, "weights"), _dense(experts, shape, torch.int32, "experts")
    if out is None:
        stream = _on_gpu(logits, dw, weights, experts)
        out = logits.new_empty((tokens, n_experts))
        op = out.data_ptr()
    else:
        op = _dense(out, (tokens, n_experts), logits.dtype, "out")
        stream = _on_gpu(logits, dw, weights, experts, out)
    _check(lib().mxq_route_grad(dwp, wp, ep, logits.data_ptr(), dt, tokens, n_experts, ld, shape[1], int(renorm), op,
                                stream))
    return out


class ExpertRows(NamedTuple):
    offsets: torch.Tensor    # int64 [E + 1]: rows of every expert
    positions: torch.Tensor  # int32, as the experts: the row of every assignment, or -1
    order: torch.Tensor      # int32 [assignments]: the assignment of every row, -1 behind the last one


def mxq_expert_sort(experts: torch.Tensor, n_experts: int, out: Optional[ExpertRows] = None,
                    workspace: Optional[torch.Tensor] = None) -> ExpertRows:
    """mxq_expert_sort: the rows of every expert from the choices `experts` (int32 [T, k];
    values outside [0, n_experts) have no row), those of one expert in the tokens' order.
    `workspace` (uint8, mxq_expert_sort_workspace bytes) is allocated if absent."""
    ep, count = _dense(experts, experts.shape, torch.int32, "experts"), experts.numel()
    need = lib().mxq_expert_sort_workspace(count, n_experts)
    if workspace is not None and (workspace.numel() * workspace.element_size() < need or not workspace.is_contiguous()):
        raise ValueError(f"dense workspace of {need} bytes expected")
    if out is None:
        stream = _on_gpu(experts, workspace)
        out = ExpertRows(experts.new_empty((n_experts + 1,), dtype=torch.int64), torch.empty_like(experts),
                         experts.new_empty((count,)))
        offp, pp, op = out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr()
    else:
        offp = _dense(out[0], (n_experts + 1,), torch.int64, "offsets")
        pp = _dense(out[1], experts.shape, torch.int32, "positions")
        op = _dense(out[2], (count,), torch.int32, "order")
        stream = _on_gpu(experts, *out, workspace)
    if need and workspace is None:
        workspace = experts.new_empty((need,), dtype=torch.uint8)
    _check(lib().mxq_expert_sort(ep, count, n_experts, offp, pp, op, _ptr(workspace), stream))
    return out


def mxq_dispatch(x: torch.Tensor, positions: torch.Tensor, rows: Optional[int] = None, fmt: Optional[str] = None,
                 out=None):
    """mxq_dispatch: every token's row x [T, H] copied to the rows of its assignments; the
    result has `rows` rows (T k if absent), of which those of no assignment are left as
    they are. fmt None: rows as x; "mxfp4": (codes, e8m0), the bits of mxq_quantize;
    "fp8": (E4M3, scales), the bits of mxq_fp8_quantize. The gradient is mxq_combine
    without weights."""
    tokens, width, ldx = _strided_rows(x, "x")
    dt, code = _float_code(x.dtype), _ROWS[fmt]
    if _positions(positions)[0] != tokens:
        raise ValueError(f"positions of {positions.shape[0]} tokens for {tokens}")
    if rows is None:
        rows = positions.numel() if out is None else (out if code == 0 else out[0]).shape[0]
    sp = None
    if code == 0:
        if out is None:
            stream = _on_gpu(x, positions)
            out = x.new_empty((rows, width))
            op = out.data_ptr()
        else:
            op = _dense(out, (rows, width), x.dtype, "out")
            stream = _on_gpu(x, positions, out)
    else:
        per, block, kind = (2, 32, torch.uint8) if code == 1 else (1, 128, torch.float32)
        if out is None:
            stream = _on_gpu(x, positions)
            out = (x.new_empty((rows, width // per), dtype=torch.uint8),
                   x.new_empty((rows, width // block), dtype=kind))
            op, sp = out[0].data_ptr(), out[1].data_ptr()
        else:
            op = _dense(out[0], (rows, width // per), torch.uint8, "codes")
            sp = _dense(out[1], (rows, width // block), kind, "scales")
            stream = _on_gpu(x, positions, *out)
    _check(lib().mxq_dispatch(x.data_ptr(), dt, tokens, width, ldx, positions.data_ptr(), positions.shape[1], rows,
                              code, op, sp, stream))
    return out


def mxq_combine(y: torch.Tensor, positions: torch.Tensor, weights: Optional[torch.Tensor] = None,
                residual: Optional[torch.Tensor] = None, out_dtype=torch.bfloat16,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """mxq_combine: out [T, H] = residual + sum over j of weights[:, j] times the rows
    y[positions[:, j]] (weights fp32 [T, k], 1 if absent; residual of the result's type, may
    be `out` itself). Assignments without a row add nothing."""
    tokens, _ = shape = _positions(positions)
    rows, width = y.shape
    if out is not None:
        out_dtype = out.dtype
    ydt, dt = _float_code(y.dtype), _float_code(out_dtype)
    yp = _dense(y, (rows, width), y.dtype, "y")
    wp = None if weights is None else _dense(weights, shape, torch.float32, "weights")
    rp = None if residual is None else _dense(residual, (tokens, width), out_dtype, "residual")
    if out is None:
        stream = _on_gpu(y, positions, weights, residual)
        out = y.new_empty((tokens, width), dtype=out_dtype)
        op = out.data_ptr()
    else:
        op = _dense(out, (tokens, width), out_dtype, "out")
        stream = _on_gpu(y, positions, weights, residual, out)
    _check(lib().mxq_combine(yp, ydt, rows, width, positions.data_ptr(), wp, tokens, shape[1], rp, op, dt, stream))
    return out


def mxq_combine_grad(grad: torch.Tensor, y: torch.Tensor, positions: torch.Tensor,
                     weights: Optional[torch.Tensor] = None, weight_grad: bool = True,
                     out: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None):
    """mxq_combine_grad: from the gradient `grad` [T, H] of mxq_combine's result the
    gradient dy of its rows y [R, H] (y's type; rows of no assignment are left as they are)
    and, with `weight_grad`, (dy, dw), dw fp32 [T, k] that of its weights. `out` may be y."""
    tokens, _ = shape = _positions(positions)
    rows, width = y.shape
    gdt, ydt = _float_code(grad.dtype), _float_code(y.dtype)
    gp, yp = _dense(grad, (tokens, width), grad.dtype, "grad"), _dense(y, (rows, width), y.dtype, "y")
    wp = None if weights is None else _dense(weights, shape, torch.float32, "weights")
    given = []
    if out is not None:
        _dense(out, (rows, width), y.dtype, "out")
        given.append(out)
    if weight_grad and dw is not None:
        _dense(dw, shape, torch.float32, "dw")
        given.append(dw)
    stream = _on_gpu(grad, y, positions, weights, *given)
    if out is None:
        out = torch.empty_like(y)
    if weight_grad and dw is None:
        dw = grad.new_empty(shape, dtype=torch.float32)
    dwp = dw.data_ptr() if weight_grad else None
    _check(lib().mxq_combine_grad(gp, gdt, yp, ydt, rows, width, positions.data_ptr(), wp, tokens, shape[1],
                                  out.data_ptr(), dwp, stream))
    return (out, dw) if weight_grad else out


def mxq_fp8_quantize(x: torch.Tensor, out=None):
    """mxq_fp8_quantize: (E4M3 uint8 [R, C], power-of-two fp32 scales [R, ceil(C / 128)]) of
    x [R, C]: an operand of the products (C a multiple of 128), or z kept for
    mxq_fp8_act_grad (any C)."""
    rows, cols, ldx = _strided_rows(x, "x")
    dt, groups = _float_code(x.dtype), (cols + 127) // 128
    if out is None:
        stream = _on_gpu(x)
        out = x.new_empty((rows, cols), dtype=torch.uint8), x.new_empty((rows, groups), dtype=torch.float32)
        qp, sp = out[0].data_ptr(), out[1].data_ptr()
    else:
        qp = _dense(out[0], (rows, cols), torch.uint8, "codes")
        sp = _dense(out[1], (rows, groups), torch.float32, "scales")
        stream = _on_gpu(x, *out)
    _check(lib().mxq_fp8_quantize(x.data_ptr(), dt, rows, cols, ldx, qp, sp, stream))
    return out


def mxq_fp8_act_grad(dy: torch.Tensor, z8, act: str = "none", offsets: Optional[torch.Tensor] = None,
                     bias_grad: bool = False, recompute: bool = False, out: Optional[torch.Tensor] = None,
                     db: Optional[torch.Tensor] = None, h: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None):
    """mxq_fp8_act_grad: mxq_act_grad for a z that was kept as z8 = (E4M3 [R, N], scales
    [R, ceil(N / 128)]) by mxq_fp8_quantize. Gives dz (dy's type), then db with `bias_grad`,
    then h = act(z) with `recompute` (dy's type and shape; may be dy): a tuple where there
    is more than dz."""
    q8, scales = z8
    if q8.dim() != 2:
        raise ValueError("z8: a matrix of codes expected")
    rows, n = shape = q8.shape
    code, dtype = _ACT[act], dy.dtype
    dt = _float_code(dtype)
    qp = _dense(q8, shape, torch.uint8, "z8")
    sp = _dense(scales, (rows, (n + 127) // 128), torch.float32, "z8's scales")
    dy_shape = (rows, n // 2 if code == SWIGLU else n)
    dyp = _dense(dy, dy_shape, dtype, "dy")
    groups, offp = (1, None) if offsets is None else (_offsets(offsets), offsets.data_ptr())
    given = []
    if out is not None:
        _dense(out, shape, dtype, "out")
        given.append(out)
    need = 0
    if bias_grad:
        db_shape = (n,) if offsets is None else (groups, n)
        if db is not None:
            _dense(db, db_shape, torch.float32, "db")
            given.append(db)
        need = lib().mxq_act_grad_workspace(rows, n, groups)
        if workspace is not None:
            if workspace.numel() * workspace.element_size() < need or not workspace.is_contiguous():
                raise ValueError(f"dense workspace of {need} bytes expected")
            given.append(workspace)
    if recompute and h is not None:
        _dense(h, dy_shape, dtype, "h")
        given.append(h)
    stream = _on_gpu(dy, q8, scales, offsets, *given)
    if out is None:
        out = dy.new_empty(shape)
    got = [out]
    dbp = wsp = hp = None
    if bias_grad:
        if db is None:
            db = dy.new_empty(db_shape, dtype=torch.float32)
        if workspace is None:
            workspace = dy.new_empty((need,), dtype=torch.uint8)
        dbp, wsp = db.data_ptr(), workspace.data_ptr()
        got.append(db)
    if recompute:
        if h is None:
            h = torch.empty_like(dy)
        hp = h.data_ptr()
        got.append(h)
    _check(lib().mxq_fp8_act_grad(dyp, dt, qp, sp, rows, n, code, offp, groups, out.data_ptr(), dbp, hp, wsp, stream))
    return tuple(got) if len(got) > 1 else out
