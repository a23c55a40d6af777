"""ctypes binding of the router's losses and of the gradients' norm and clipping
(include/moe_fp4.h).

Argument marshalling only, as in _block: the work is done by the HIP kernels of
libmoe_fp4.so on the current stream of the tensors' device.
"""
from __future__ import annotations

import ctypes
import operator
from array import array
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

from ._block import (_ANY, _FP32, _I32, _I64, _INT, _P, _SZ, _TYPES, _call, _index, _opt, _refuse, _rows, _vector,
                     _workspace)
from ._lib import ACCUMULATE, _check, _lib

SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1


class RouterLossDims(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("T", "E", "k", "S", "score", "type", "out_type")] +
                [(n, _I64) for n in ("ld", "ldd")])


class GradTensor(ctypes.Structure):
    """moe_fp4_grad_tensor."""
    _fields_ = [("data", _P), ("out", _P), ("n", _I64), ("type", _I32), ("out_type", _I32)]


_R = ctypes.POINTER(RouterLossDims)
for _name, _args in (
        ("router_loss_workspace_size", [_R, ctypes.POINTER(_SZ)]),
        ("router_loss", [_R, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
        ("router_loss_backward", [_R, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _P, _INT, _P]),
        ("grad_sumsq_workspace_size", [_P, _INT, ctypes.POINTER(_SZ)]),
        ("grad_sumsq", [_P, _INT, _P, _INT, _P, _SZ, _P]),
        ("grad_clip", [_P, _INT, _P, ctypes.c_float, ctypes.c_float, _P, _P])):
    _f = getattr(_lib, "moe_fp4_" + _name)
    _f.argtypes, _f.restype = _args, ctypes.c_int


# ---------------------------------------------------------------- the router's losses
@dataclass
class RouterLoss:
    """What moe_fp4_router_loss returns, one row a sequence: counts [S, E] int32,
    tokens [S] int32, probs [S, E], balance [S] and z [S] fp32."""
    counts: torch.Tensor
    tokens: torch.Tensor
    probs: torch.Tensor
    balance: torch.Tensor
    z: torch.Tensor


def _table(t, name: str, shape, dtype, device):
    """Checks a dense matrix."""
    if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == device and t.shape == shape and
            t.is_contiguous()):
        _refuse(t, name, (dtype,), device, shape, len(shape))


def _batch(logits, topk_idx, seqs, mask):
    """The logits' row stride, the choices of a token and the sequences' number, after the checks."""
    ld = _rows(logits, "logits", _ANY)
    dev, T, S = logits.device, logits.shape[0], 1
    if seqs is not None:
        _index(seqs, "seqs", None, dev)
        S = seqs.numel() - 1
    if mask is not None:
        _vector(mask, "mask", T, (torch.bool, torch.uint8), dev)
    if not (isinstance(topk_idx, torch.Tensor) and topk_idx.dim() == 2):
        raise TypeError("topk_idx must be a 2-d tensor")
    _table(topk_idx, "topk_idx", (T, topk_idx.shape[1]), torch.int32, dev)
    return ld, topk_idx.shape[1], S


def moe_fp4_router_loss_workspace_size(T: int, E: int, S: int = 1, dtype=torch.float32) -> int:
    """Bytes of workspace of moe_fp4_router_loss."""
    n = _SZ()
    _check(_lib.moe_fp4_router_loss_workspace_size(RouterLossDims(T, E, 1, S, 0, _TYPES[dtype], 0), n),
           "moe_fp4_router_loss_workspace_size")
    return n.value


def moe_fp4_router_loss(logits: torch.Tensor, topk_idx: torch.Tensor, score: int = SCORE_SOFTMAX,
                        seqs: Optional[torch.Tensor] = None, mask: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None) -> RouterLoss:
    """Per-expert counts, the balance loss and the z loss of each sequence: logits
    [T, E], topk_idx [T, k] int32 (a Route's), seqs [S+1] int32 (sequence s is the
    tokens seqs[s] .. seqs[s+1]-1; None: one of all tokens), mask [T] bool or uint8
    (0 leaves a token out)."""
    ld, k, S = _batch(logits, topk_idx, seqs, mask)
    dev = logits.device
    T, E = logits.shape
    d = RouterLossDims(T, E, k, S, score, _TYPES[logits.dtype], 0, ld)
    ws, nws, keep = _workspace(_lib.moe_fp4_router_loss_workspace_size, d, workspace=workspace, device=dev)
    # one allocation for the five results
    counts, tokens, probs, balance, z = torch.empty(S * (2 * E + 3), dtype=torch.float32, device=dev).split(
        (S * E, S, S * E, S, S))
    counts, tokens, probs = counts.view(torch.int32).view(-1, E), tokens.view(torch.int32), probs.view(-1, E)
    _call(_lib.moe_fp4_router_loss, dev, d, logits.data_ptr(), topk_idx.data_ptr(), _opt(seqs), _opt(mask),
          counts.data_ptr(), tokens.data_ptr(), probs.data_ptr(), balance.data_ptr(), z.data_ptr(), ws, nws)
    return RouterLoss(counts, tokens, probs, balance, z)


def moe_fp4_router_loss_backward(logits: torch.Tensor, topk_idx: torch.Tensor, loss: Optional[RouterLoss] = None,
                                 dbalance: Optional[torch.Tensor] = None, dz: Optional[torch.Tensor] = None,
                                 gates: Optional[torch.Tensor] = None, dgates: Optional[torch.Tensor] = None,
                                 score: int = SCORE_SOFTMAX, seqs: Optional[torch.Tensor] = None,
                                 mask: Optional[torch.Tensor] = None, dlogits: Optional[torch.Tensor] = None,
                                 out_dtype=None, accumulate: bool = False) -> torch.Tensor:
    """dlogits [T, E]: the gradient of sum_s dbalance[s] balance[s] + dz[s] z[s] (fp32
    [S] each; `loss` gives counts and tokens, summed over ranks where they balance
    together), and of the gates [T, k] (a Route's) where dgates is given.  Rows of
    masked tokens are zeros; rows of no sequence are left as they were (in a new
    dlogits: undefined).  dlogits of the logits' type or fp32, any of the three for
    fp32 logits."""
    ld, k, S = _batch(logits, topk_idx, seqs, mask)
    dev = logits.device
    T, E = logits.shape
    if dbalance is None and dz is None and dgates is None:
        raise ValueError("nothing to compute")
    if (gates is None) != (dgates is None):
        raise ValueError("gates and dgates go together")
    counts = tokens = None
    if dbalance is not None or dz is not None:
        if loss is None:
            raise ValueError("the losses' gradients need the forward pass's loss")
        tokens = loss.tokens
        _vector(tokens, "loss.tokens", S, (torch.int32,), dev)
    if dbalance is not None:
        counts = loss.counts
        _table(counts, "loss.counts", (S, E), torch.int32, dev)
        _vector(dbalance, "dbalance", S, _FP32, dev)
    if dz is not None:
        _vector(dz, "dz", S, _FP32, dev)
    if gates is not None:
        _table(gates, "gates", (T, k), torch.float32, dev)
        _table(dgates, "dgates", (T, k), torch.float32, dev)
    allowed = _ANY if logits.dtype == torch.float32 else (logits.dtype, torch.float32)
    if dlogits is None:
        if accumulate:
            raise ValueError("accumulate needs dlogits")
        dt = logits.dtype if out_dtype is None else out_dtype
        if dt not in allowed:
            raise TypeError(f"out_dtype must be one of {allowed}")
        dlogits, ldd = torch.empty((T, E), dtype=dt, device=dev), 0
    else:
        if out_dtype is not None and dlogits.dtype != out_dtype:
            raise TypeError("dlogits and out_dtype disagree")
        ldd = _rows(dlogits, "dlogits", allowed, dev, (T, E))
    d = RouterLossDims(T, E, k, S, score, _TYPES[logits.dtype], _TYPES[dlogits.dtype], ld, ldd)
    _call(_lib.moe_fp4_router_loss_backward, dev, d, logits.data_ptr(), topk_idx.data_ptr(), _opt(seqs), _opt(mask),
          _opt(counts), _opt(tokens), _opt(dbalance), _opt(dz), _opt(gates), _opt(dgates), dlogits.data_ptr(),
          ACCUMULATE if accumulate else 0)
    return dlogits


# ---------------------------------------------------------------- the gradients' norm
def _dense(t) -> bool:
    """Whether a tensor's elements fill its storage range without gaps or repeats."""
    if t.is_contiguous():
        return True
    n = 1
    for st, sz in sorted(zip(t.stride(), t.shape)):
        if sz != 1:
            if st != n:
                return False
            n *= sz
    return True


_ptr, _numel, _device_of, _dtype = (torch.Tensor.data_ptr, torch.Tensor.numel, torch.Tensor.get_device,
                                    operator.attrgetter("dtype"))
_SAME = {t: c | c << 32 for t, c in _TYPES.items()}  # type and out_type


def _refuse_grads(tensors, out):
    """Says what is wrong with the tensors of a list (nothing: returns)."""
    dev = None
    for i, t in enumerate(tensors):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"tensors[{i}] must be a tensor")
        if not t.is_cuda:
            raise ValueError(f"tensors[{i}] must be on a GPU")
        dev = t.device if dev is None else dev
        if t.device != dev:
            raise ValueError(f"tensors[{i}] is on {t.device}, expected {dev}")
        if t.dtype not in _TYPES:
            raise TypeError(f"tensors[{i}] has dtype {t.dtype}, expected one of {_ANY}")
        if not _dense(t):
            raise ValueError(f"tensors[{i}] must fill its memory without gaps")
        if out is None:
            continue
        o, allowed = out[i], _ANY if t.dtype == torch.float32 else (t.dtype,)
        if not isinstance(o, torch.Tensor):
            raise TypeError(f"out[{i}] must be a tensor")
        if o.dtype not in allowed:
            raise TypeError(f"out[{i}] has dtype {o.dtype}, expected one of {allowed}")
        if o.device != dev or o.numel() != t.numel():
            raise ValueError(f"out[{i}] must have its gradient's device and number of elements")
        if not (o.is_contiguous() and t.is_contiguous()) and (o.shape != t.shape or o.stride() != t.stride()):
            raise ValueError(f"out[{i}] must have its gradient's shape and strides where one is not contiguous")


def _grads(tensors, out):
    """The library's list of tensors (GradTensor's layout, as 64-bit words: data, out, n, type and
    out_type), its address, and the tensors' device (None without tensors).  A list is
    gone through by built-in calls alone: a third of a microsecond a tensor."""
    if out is not None and len(out) != len(tensors):
        raise ValueError("out must have a tensor for each of the gradients")
    n = len(tensors)
    table = array("q", bytes(32 * n))
    if n == 0:
        return table, None, None
    try:
        where, types, sizes = set(map(_device_of, tensors)), list(map(_dtype, tensors)), list(map(_numel, tensors))
        ok = len(where) == 1 and -1 not in where and all(map(torch.Tensor.is_contiguous, tensors))
        table[0::4] = array("q", map(_ptr, tensors))
        table[2::4] = array("q", sizes)
        codes = map(_SAME.__getitem__, types)
        if out is not None:
            to = list(map(_dtype, out))
            ok = ok and set(map(_device_of, out)) == where and all(map(torch.Tensor.is_contiguous, out)) and \
                list(map(_numel, out)) == sizes
            table[1::4] = array("q", map(_ptr, out))
            if to != types:
                ok = ok and all(a == b or a == torch.float32 for a, b in zip(types, to))
                codes = [_TYPES[a] | _TYPES[b] << 32 for a, b in zip(types, to)]
        table[3::4] = array("q", codes)
    except (TypeError, KeyError, AttributeError) as e:
        _refuse_grads(tensors, out)
        raise TypeError("tensors and out must be lists of tensors") from e
    if not ok:
        _refuse_grads(tensors, out)
    return table, table.buffer_info()[0], tensors[0].device


def moe_fp4_grad_sumsq_workspace_size(tensors: Sequence[torch.Tensor]) -> int:
    """Bytes of workspace of moe_fp4_grad_sumsq for these tensors."""
    n = _SZ()
    table, at, _ = _grads(tensors, None)
    _check(_lib.moe_fp4_grad_sumsq_workspace_size(at, len(tensors), n), "moe_fp4_grad_sumsq_workspace_size")
    return n.value


def moe_fp4_grad_sumsq(tensors: Sequence[torch.Tensor], sumsq: Optional[torch.Tensor] = None, accumulate: bool = False,
                       workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """sumsq [1] fp64: the sum of the squares of all elements of the tensors (fp32,
    bf16 and fp16, mixed), in place of sumsq or added to it.  Ranks that hold
    different gradients add theirs up before moe_fp4_grad_clip."""
    table, at, dev = _grads(tensors, None)
    if sumsq is None:
        if accumulate:
            raise ValueError("accumulate needs sumsq")
        if dev is None:
            raise ValueError("without tensors sumsq must be given")
        sumsq = torch.empty(1, dtype=torch.float64, device=dev)
    else:
        dev = sumsq.device if dev is None else dev
        _vector(sumsq, "sumsq", 1, (torch.float64,), dev)
        if not sumsq.is_cuda:
            raise ValueError("sumsq must be on a GPU")
    n = _SZ()
    _check(_lib.moe_fp4_grad_sumsq_workspace_size(at, len(tensors), n), "moe_fp4_grad_sumsq_workspace_size")
    ws = None
    if workspace is not None:
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError(f"workspace must be contiguous and on {dev}")
        ws = workspace
    elif n.value:
        ws = torch.empty(n.value, dtype=torch.uint8, device=dev)
    _call(_lib.moe_fp4_grad_sumsq, dev, at, len(tensors), sumsq.data_ptr(), ACCUMULATE if accumulate else 0, _opt(ws),
          0 if ws is None else ws.numel() * ws.element_size())
    return sumsq


def moe_fp4_grad_clip(tensors: Sequence[torch.Tensor], sumsq: torch.Tensor, max_norm: float, eps: float = 1e-6,
                      out: Optional[Sequence[torch.Tensor]] = None) -> torch.Tensor:
    """Multiplies the tensors by min(1, max_norm / (sqrt(sumsq) + eps)), in place or into
    `out` (each as large as its gradient and of its type, any of the three for an fp32
    one).
    Returns the norm sqrt(sumsq), [1] fp32."""
    table, at, dev = _grads(tensors, out)
    if dev is None:
        dev = getattr(sumsq, "device", None)
    _vector(sumsq, "sumsq", 1, (torch.float64,), dev)
    if not sumsq.is_cuda:
        raise ValueError("sumsq must be on a GPU")
    norm = torch.empty(1, dtype=torch.float32, device=dev)
    _call(_lib.moe_fp4_grad_clip, dev, at, len(tensors), sumsq.data_ptr(), max_norm, eps, norm.data_ptr())
    return norm
