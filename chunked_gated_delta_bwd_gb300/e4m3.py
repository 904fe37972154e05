"""Python binding of the 8-bit products (argument marshalling only, as ``api``): e4m3 operands with
a scale for each block of 128, and the quantisation that makes them.  ``rmsnorm_fwd`` with
``quant="block"`` or ``"token"`` gives the product's first operand too, and so does, with
``"token"`` on rows of 128 channels, the norm of each head.
"""
import ctypes

import torch

from .api import _check, lib
from .block import _TYPES, _need, _ptr, _rows, _stream

E4M3 = torch.float8_e4m3fn
_LIB = None


def _lib():
    global _LIB
    if _LIB is None:
        L = lib()
        vp, i32, i64, st = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_int
        L.gdr_quant_e4m3.restype, L.gdr_quant_e4m3.argtypes = st, [i64, i32, vp, i64, i32, i32] + [vp] * 5
        L.gdr_linear_e4m3.restype, L.gdr_linear_e4m3.argtypes = st, [i64, i32, i32, vp, vp, i32] + [vp] * 5
        _LIB = L
    return _LIB


def quant_e4m3(x, tiles=False, transposed=False):
    """e4m3 codes of x (bf16 or float32 [..., C]; rows of one stride) with a float32 scale for each 128 channels of
    a row, or with ``tiles`` (x [R, C], a weight) for each 128 x 128 tile.  Returns dict(y, scale): scale
    [rows, ceil(C / 128)] or [ceil(R / 128), ceil(C / 128)]; with ``transposed`` (and ``tiles``) also y_t [C, R] and
    scale_t, the same codes as the product's backward reads them."""
    if x is None or x.dim() < 1 or x.dtype not in _TYPES:
        raise ValueError("x must be a bfloat16 or float32 tensor [..., C]")
    if transposed and not tiles:
        raise ValueError("transposed goes with tiles")
    if tiles and x.dim() != 2:
        raise ValueError("tiles take x [R, C]")
    shape, C = x.shape, x.shape[-1]
    if x.dim() != 2:
        x = x.reshape(-1, C) if x.numel() else x.reshape(shape[:-1].numel(), C)
    R = x.shape[0]
    ldx = _rows(x, tuple(_TYPES), (R, C), "x")
    nb = (C + 127) // 128
    nr = (R + 127) // 128 if tiles else R
    f32 = dict(dtype=torch.float32, device=x.device)
    out = {"y": torch.empty(shape, dtype=E4M3, device=x.device), "scale": torch.empty((nr, nb), **f32)}
    if transposed:
        out["y_t"], out["scale_t"] = torch.empty((C, R), dtype=E4M3, device=x.device), torch.empty((nb, nr), **f32)
    rc = _lib().gdr_quant_e4m3(R, C, x.data_ptr(), ldx, _TYPES[x.dtype], bool(tiles), out["y"].data_ptr(),
                               out["scale"].data_ptr(), _ptr(out.get("y_t")), _ptr(out.get("scale_t")), _stream(x))
    if rc:
        _check(rc, "gdr_quant_e4m3")
    return out


def linear_e4m3(x, x_scale, weight, weight_scale, bias=None, out=None):
    """y = x weight^T (+ bias) of e4m3 operands: x [..., K] with x_scale float32 [rows, ceil(K / 128)] (or [rows, 1],
    one for the whole row), weight [N, K] with weight_scale float32 [ceil(N / 128), ceil(K / 128)], bias float32 [N].
    Returns y bf16 [..., N]."""
    if x is None or x.dim() < 1 or weight is None or weight.dim() != 2:
        raise ValueError("x must be [..., K] and weight [N, K]")
    xshape, (N, K) = x.shape, weight.shape
    rows, nb = xshape[0] if len(xshape) == 2 else xshape[:-1].numel(), (K + 127) // 128
    _need(x, E4M3, xshape[:-1] + (K,) if xshape[-1] != K else xshape, "x")
    _need(weight, E4M3, (N, K), "weight")
    blocks = 1 if x_scale is not None and x_scale.dim() == 2 and x_scale.shape[1] == 1 else nb
    _need(x_scale, torch.float32, (rows, blocks), "x_scale")
    _need(weight_scale, torch.float32, ((N + 127) // 128, nb), "weight_scale")
    if bias is not None:
        _need(bias, torch.float32, (N,), "bias")
    shape = (rows, N) if len(xshape) == 2 else xshape[:-1] + (N,)
    y = torch.empty(shape, dtype=torch.bfloat16, device=x.device) if out is None else _need(out, torch.bfloat16, shape, "out")
    rc = _lib().gdr_linear_e4m3(rows, K, N, x.data_ptr(), x_scale.data_ptr(), blocks, weight.data_ptr(),
                                weight_scale.data_ptr(), _ptr(bias), y.data_ptr(),
                                _stream(x, x_scale, weight, weight_scale, bias, y))
    if rc:
        _check(rc, "gdr_linear_e4m3")
    return y
