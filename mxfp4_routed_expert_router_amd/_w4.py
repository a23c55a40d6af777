"""ctypes binding of the dense product with 4-bit weights and group scales
(include/moe_fp4.h).  Argument marshalling only, as in _block.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._block import (_ANY, _HALF, _I32, _I64, _INT, _P, _TYPES, ACT_NONE, _call, _given, _opt, _out_type, _refuse, _rows,
                     _vector)
from ._lib import ACCUMULATE, _lib

W4_MX, W4_INT4 = 0, 1


class W4Dims(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("M", "N", "K", "code", "group", "type", "out_type", "bias_type", "scale_type", "act")] +
                [(n, _I64) for n in ("ldx", "ldy", "ldr", "ldw")])


_f = _lib.moe_fp4_linear_w4
_f.argtypes, _f.restype = [ctypes.POINTER(W4Dims), _P, _P, _P, _P, _P, _P, _P, _INT, _P], ctypes.c_int


class W4Weights:
    """4-bit weights [N, K] as they are stored: codes [N, K/2] uint8, the low nibble of a
    byte holding the even input, and scales [N, ceil(K / group)].  uint8 scales are
    UE8M0 (group 32) and the codes E2M1, the experts' checkpoint format; fp32, bf16 or
    fp16 scales (group 32, 64, 128 or 256) go with int4 codes: weight = (code - zero)
    * scale, zeros [N, ceil(K / group)] uint8, 8 where None."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, zeros: Optional[torch.Tensor] = None, group: int = 32):
        self.ldw = _rows(codes, "codes", (torch.uint8,))
        dev = codes.device
        self.N, self.K = codes.shape[0], 2 * codes.shape[1]
        if group not in (32, 64, 128, 256):
            raise ValueError("group must be 32, 64, 128 or 256")
        shape = (self.N, (self.K + group - 1) // group)
        if not (isinstance(scales, torch.Tensor) and scales.dtype in _ANY + (torch.uint8,) and scales.device == dev and
                scales.shape == shape and scales.is_contiguous()):
            _refuse(scales, "scales", _ANY + (torch.uint8,), dev, shape, 2)
        self.code = W4_MX if scales.dtype == torch.uint8 else W4_INT4
        if self.code == W4_MX and (group != 32 or zeros is not None):
            raise ValueError("UE8M0 scales go with groups of 32 and without zeros")
        if zeros is not None and not (isinstance(zeros, torch.Tensor) and zeros.dtype == torch.uint8 and
                                      zeros.device == dev and zeros.shape == shape and zeros.is_contiguous()):
            _refuse(zeros, "zeros", (torch.uint8,), dev, shape, 2)
        self.codes, self.scales, self.zeros, self.group = codes, scales, zeros, group


def moe_fp4_linear_w4(x: torch.Tensor, w: W4Weights, bias: Optional[torch.Tensor] = None, act: int = ACT_NONE,
                      residual: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None, out_dtype=None,
                      accumulate: bool = False) -> torch.Tensor:
    """y [M, N] = act(x [M, K] . W [N, K]^T + bias [N]) + residual [M, N]; y may be the
    residual.  Made for up to 64 rows."""
    ldx = _rows(x, "x", _HALF)
    dev = x.device
    if not isinstance(w, W4Weights):
        raise TypeError("w must be W4Weights")
    if w.codes.device != dev:
        raise ValueError(f"w is on {w.codes.device}, expected {dev}")
    M, K = x.shape
    N = w.N
    if w.K != K:
        raise ValueError("x and w disagree on the number of inputs")
    if y is None:
        if accumulate:
            raise ValueError("accumulate needs y")
        y, ldy = torch.empty((M, N), dtype=_out_type(out_dtype, x.dtype), device=dev), 0
    else:
        ldy = _given(y, "y", out_dtype, x.dtype, dev, (M, N))
    ldr = _rows(residual, "residual", (y.dtype,), dev, (M, N)) if residual is not None else 0
    if bias is not None:
        _vector(bias, "bias", N, _ANY, dev)
    t = _TYPES[x.dtype]
    d = W4Dims(M, N, K, w.code, w.group, t, _TYPES[y.dtype], t if bias is None else _TYPES[bias.dtype],
               _TYPES.get(w.scales.dtype, 0), act, ldx, ldy, ldr, w.ldw)
    _call(_lib.moe_fp4_linear_w4, dev, d, x.data_ptr(), w.codes.data_ptr(), w.scales.data_ptr(), _opt(w.zeros),
          _opt(bias), _opt(residual), y.data_ptr(), ACCUMULATE if accumulate else 0)
    return y
