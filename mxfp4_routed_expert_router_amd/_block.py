"""ctypes binding of the operators around the routed experts: products grouped
by expert, the dense product with its epilogue, norms with weights, and their
backward passes (include/moe_fp4.h).

Argument marshalling only, as in _lib: the work is done by the HIP kernels of
libmoe_fp4.so on the current stream of the tensors' device.  Tensors may have
any row stride that keeps rows apart; the last dimension is contiguous.
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from ._lib import ACCUMULATE, _check, _lib

F32, BF16, F16 = 0, 1, 2
ACT_NONE, ACT_RELU, ACT_GELU, ACT_GELU_TANH, ACT_SILU = range(5)
NORM_LAYER, NORM_RMS = 0, 1
GROUPED_FORWARD, GROUPED_DGRAD, GROUPED_WGRAD = range(3)
TILES_256X256, TILES_128X128, TILES_64X128, TILES_ANY = range(1, 5)

_TYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}
_HALF = (torch.bfloat16, torch.float16)
_ANY = (torch.float32, torch.bfloat16, torch.float16)
_FP32 = (torch.float32,)

_I32, _I64, _P, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t


class GroupedDims(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("E", "P", "N", "K", "R", "row_div", "type", "out_type")] +
                [(n, _I64) for n in ("ldx", "ldw", "ldy", "expert_stride")])


class LinearDims(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("M", "N", "K", "type", "out_type", "bias_type", "dw_type", "act")] +
                [(n, _I64) for n in ("ldx", "ldw", "ldy", "ldr", "ldz", "lddx", "lddw")])


class NormDims(ctypes.Structure):
    _fields_ = ([(n, _I32) for n in ("T", "H", "x_type", "y_type", "w_type", "kind")] +
                [("eps", ctypes.c_float)] + [(n, _I64) for n in ("ldx", "ldy", "lddx")])


class ProductPlan(ctypes.Structure):
    """Which kernels a product takes (moe_fp4_product_plan)."""
    _fields_ = [(n, _I32) for n in ("rows", "tiles", "splits", "columns", "rest_tiles", "rest_splits")]

    def __repr__(self):
        return "ProductPlan(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


_G, _L, _N = ctypes.POINTER(GroupedDims), ctypes.POINTER(LinearDims), ctypes.POINTER(NormDims)
_INT = ctypes.c_int
for _name, _args in (
        ("grouped_workspace_size", [_G, _INT, ctypes.POINTER(_SZ)]),
        ("grouped_plan", [_G, _INT, ctypes.POINTER(ProductPlan)]),
        ("grouped_forward", [_G, _P, _P, _P, _P, _P, _INT, _P, _SZ, _P]),
        ("grouped_dgrad", [_G, _P, _P, _P, _P, _INT, _P, _SZ, _P]),
        ("grouped_wgrad", [_G, _P, _P, _P, _P, _P, _INT, _P, _SZ, _P]),
        ("linear_workspace_size", [_L, _INT, ctypes.POINTER(_SZ)]),
        ("linear_plan", [_L, _INT, ctypes.POINTER(ProductPlan)]),
        ("linear", [_L, _P, _P, _P, _P, _P, _P, _INT, _P, _SZ, _P]),
        ("linear_backward", [_L, _P, _P, _P, _P, _P, _P, _P, _INT, _P, _SZ, _P]),
        ("norm", [_N, _P, _P, _P, _P, _P, _P, _P]),
        ("norm_backward_workspace_size", [_N, ctypes.POINTER(_SZ)]),
        ("norm_backward", [_N, _P, _P, _P, _P, _P, _P, _P, _P, _INT, _P, _SZ, _P])):
    _f = getattr(_lib, "moe_fp4_" + _name)
    _f.argtypes, _f.restype = _args, ctypes.c_int


def _rows(t, name: str, dtypes, device=None, shape=None, ndim: int = 2) -> int:
    """Checks a tensor of rows and returns its row stride in elements (0: dense)."""
    try:
        ok = (t.dtype in dtypes and t.is_cuda and t.dim() == ndim and (device is None or t.device == device) and
              (shape is None or t.shape == shape))
    except AttributeError:
        raise TypeError(f"{name} must be a tensor") from None
    if not ok:
        _refuse(t, name, dtypes, device, shape, ndim)
    if t.is_contiguous():
        return 0
    st, sz = t.stride(), t.shape
    if sz[-1] > 1 and st[-1] != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    if sz[-2] <= 1:
        return 0
    if st[-2] < sz[-1]:
        raise ValueError(f"{name} has rows that overlap (stride {st[-2]} of {sz[-1]} elements)")
    return st[-2]


def _refuse(t, name, dtypes, device, shape, ndim):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must be a {ndim}-d tensor")
    if tuple(t.shape) == tuple(shape):
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _vector(t, name: str, n: int, dtypes, device):
    """Checks a contiguous vector of n elements."""
    if not (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.device == device and t.shape == (n,) and
            t.is_contiguous()):
        _refuse(t, name, dtypes, device, (n,), 1)


def _experts(t: torch.Tensor, name: str, dtypes, device=None, shape=None):
    """As _rows for weights [E, N, K]: the row stride and the experts' distance."""
    ld = _rows(t, name, dtypes, device, shape, 3)
    if ld == 0 and t.is_contiguous():
        return 0, 0
    E, N, K = t.shape
    row = ld or K
    if E <= 1:
        return ld, 0
    if t.stride(0) < (N - 1) * row + K:
        raise ValueError(f"{name} has experts that overlap")
    return ld, t.stride(0)


def _index(t, name: str, n: Optional[int], device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != torch.int32:
        raise TypeError(f"{name} has dtype {t.dtype}, expected torch.int32")
    if t.device != device or t.dim() != 1 or not t.is_contiguous() or (n is not None and t.numel() != n):
        raise ValueError(f"{name} must be a contiguous int32 vector" +
                         (f" of {n}" if n is not None else "") + f" on {device}")


def _out_type(dtype, like, name: str = "out_dtype"):
    if dtype is None:
        return like
    if dtype not in (like, torch.float32):
        raise TypeError(f"{name} must be {like} or torch.float32")
    return dtype


def _allowed(dtype, like):
    """The types of a given result: as asked, or `like` and fp32."""
    return (like, torch.float32) if dtype is None else (dtype,)


def _given(t, name: str, dtype, like, device, shape, asked: str = "out_dtype") -> int:
    """The row stride of a result that the caller gave."""
    _out_type(dtype, like, asked)
    return _rows(t, name, _allowed(dtype, like), device, shape)


def _workspace(fn, d, *args, workspace, device):
    """The call's workspace: the given one (checked by the library), or a new one."""
    n = _SZ()
    rc = fn(d, *args, n)
    if rc:
        _check(rc, fn.__name__)
    if workspace is None:
        if n.value == 0:
            return None, 0, None
        workspace = torch.empty(n.value, dtype=torch.uint8, device=device)
    elif workspace.device != device:
        raise ValueError(f"workspace must be on {device}")
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


# The current device and stream as torch's own wrappers get them (1.1 us a call less than
# through those), or through those where this torch has no such names.
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)


def _call(fn, device, *args):
    """Calls the library for tensors on `device`, on its current stream, whatever
    the current device is."""
    i = device.index
    if _device() == i:
        rc = fn(*args, _raw_stream(i))
    else:
        with torch.cuda.device(i):
            rc = fn(*args, _raw_stream(i))
    if rc:
        _check(rc, fn.__name__)


def _opt(t):
    return None if t is None else t.data_ptr()


# ---------------------------------------------------------------- products grouped by expert
def moe_fp4_grouped_workspace_size(E: int, P: int, N: int, K: int, op: int, dtype=torch.bfloat16,
                                   out_dtype=None) -> int:
    """Bytes of workspace of a grouped product; `op` is one of GROUPED_*."""
    d = GroupedDims(E, P, N, K, P, 1, _TYPES[dtype], _TYPES[_out_type(out_dtype, dtype)])
    n = _SZ()
    _check(_lib.moe_fp4_grouped_workspace_size(d, op, n),
           "moe_fp4_grouped_workspace_size")
    return n.value


def moe_fp4_grouped_plan(E: int, P: int, N: int, K: int, op: int, dtype=torch.bfloat16, out_dtype=None) -> ProductPlan:
    """The kernels of a grouped product of dense, aligned tensors; `op` is one of GROUPED_*."""
    d = GroupedDims(E, P, N, K, P, 1, _TYPES[dtype], _TYPES[_out_type(out_dtype, dtype)])
    p = ProductPlan()
    _check(_lib.moe_fp4_grouped_plan(d, op, p), "moe_fp4_grouped_plan")
    return p


def moe_fp4_grouped_forward(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
                            rows: Optional[torch.Tensor] = None, row_div: int = 1,
                            y: Optional[torch.Tensor] = None, out_dtype=None,
                            accumulate: bool = False, workspace: Optional[torch.Tensor] = None):
    """y [P, N] = each row times its expert's weight: x [P, K] in expert order, or
    with `rows` [P] (int32) x[rows[s] // row_div] (a Route's sorted_pairs and
    row_div = k take a token's row for each of its pairs).  w [E, N, K];
    offsets [E+1] int32 (a Route's).  Rows of y outside
    [offsets[0], offsets[E]) are left as they were."""
    ldx = _rows(x, "x", _HALF)
    dev = x.device
    ldw, es = _experts(w, "w", (x.dtype,), dev)
    E, N, K = w.shape
    if x.shape[1] != K:
        raise ValueError("x and w disagree on the number of inputs")
    _index(offsets, "offsets", E + 1, dev)
    P = x.shape[0]
    if rows is not None:
        _index(rows, "rows", None, dev)
        P = rows.numel()
    if y is None:
        if accumulate:
            raise ValueError("accumulate needs y")
        y, ldy = torch.empty((P, N), dtype=_out_type(out_dtype, x.dtype), device=dev), 0
    else:
        ldy = _given(y, "y", out_dtype, x.dtype, dev, (P, N))
    d = GroupedDims(E, P, N, K, x.shape[0], row_div, _TYPES[x.dtype], _TYPES[y.dtype], ldx, ldw, ldy, es)
    ws, nws, keep = _workspace(_lib.moe_fp4_grouped_workspace_size, d, GROUPED_FORWARD, workspace=workspace,
                               device=dev)
    _call(_lib.moe_fp4_grouped_forward, dev, d, x.data_ptr(), w.data_ptr(), offsets.data_ptr(), _opt(rows),
          y.data_ptr(), ACCUMULATE if accumulate else 0, ws, nws)
    return y


def moe_fp4_grouped_dgrad(dy: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor,
                          dx: Optional[torch.Tensor] = None, out_dtype=None,
                          accumulate: bool = False, workspace: Optional[torch.Tensor] = None):
    """dx [P, K] = dy [P, N] times each row's expert's weight w [E, N, K] (rows in
    expert order; a gathered x's gradient is the sum of its rows of dx)."""
    ldy = _rows(dy, "dy", _HALF)
    dev = dy.device
    ldw, es = _experts(w, "w", (dy.dtype,), dev)
    E, N, K = w.shape
    if dy.shape[1] != N:
        raise ValueError("dy and w disagree on the number of outputs")
    _index(offsets, "offsets", E + 1, dev)
    P = dy.shape[0]
    if dx is None:
        if accumulate:
            raise ValueError("accumulate needs dx")
        dx, ldx = torch.empty((P, K), dtype=_out_type(out_dtype, dy.dtype), device=dev), 0
    else:
        ldx = _given(dx, "dx", out_dtype, dy.dtype, dev, (P, K))
    d = GroupedDims(E, P, N, K, P, 1, _TYPES[dy.dtype], _TYPES[dx.dtype], ldx, ldw, ldy, es)
    ws, nws, keep = _workspace(_lib.moe_fp4_grouped_workspace_size, d, GROUPED_DGRAD, workspace=workspace, device=dev)
    _call(_lib.moe_fp4_grouped_dgrad, dev, d, dy.data_ptr(), w.data_ptr(), offsets.data_ptr(), dx.data_ptr(),
          ACCUMULATE if accumulate else 0, ws, nws)
    return dx


def moe_fp4_grouped_wgrad(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor,
                          rows: Optional[torch.Tensor] = None, row_div: int = 1,
                          dw: Optional[torch.Tensor] = None, out_dtype=None,
                          accumulate: bool = False, workspace: Optional[torch.Tensor] = None):
    """dw [E, N, K] = each expert's rows of dy [P, N] against its rows of x (see
    moe_fp4_grouped_forward); zeros for an expert without rows."""
    ldy = _rows(dy, "dy", _HALF)
    dev = dy.device
    ldx = _rows(x, "x", (dy.dtype,), dev)
    P, N = dy.shape
    K = x.shape[1]
    _index(offsets, "offsets", None, dev)
    E = offsets.numel() - 1
    if rows is not None:
        _index(rows, "rows", P, dev)
    elif x.shape[0] != P:
        raise ValueError("x and dy disagree on the number of rows")
    if dw is None:
        if accumulate:
            raise ValueError("accumulate needs dw")
        dw, ldw, es = torch.empty((E, N, K), dtype=_out_type(out_dtype, dy.dtype), device=dev), 0, 0
    else:
        ldw, es = _experts(dw, "dw", _allowed(out_dtype, dy.dtype), dev, (E, N, K))
    d = GroupedDims(E, P, N, K, x.shape[0], row_div, _TYPES[dy.dtype], _TYPES[dw.dtype], ldx, ldw, ldy, es)
    ws, nws, keep = _workspace(_lib.moe_fp4_grouped_workspace_size, d, GROUPED_WGRAD, workspace=workspace, device=dev)
    _call(_lib.moe_fp4_grouped_wgrad, dev, d, dy.data_ptr(), x.data_ptr(), offsets.data_ptr(), _opt(rows),
          dw.data_ptr(), ACCUMULATE if accumulate else 0, ws, nws)
    return dw


# ---------------------------------------------------------------- dense product
def moe_fp4_linear_workspace_size(M: int, N: int, K: int, backward: bool = False, dtype=torch.bfloat16,
                                  out_dtype=None, dw_dtype=None, act: int = ACT_NONE) -> int:
    """Bytes of workspace of moe_fp4_linear or moe_fp4_linear_backward."""
    t = _TYPES[dtype]
    d = LinearDims(M, N, K, t, _TYPES[_out_type(out_dtype, dtype)], t,
                   _TYPES[_out_type(dw_dtype, dtype, "dw_dtype")], act)
    n = _SZ()
    _check(_lib.moe_fp4_linear_workspace_size(d, int(backward), n),
           "moe_fp4_linear_workspace_size")
    return n.value


def moe_fp4_linear_plan(M: int, N: int, K: int, op: int, dtype=torch.bfloat16, out_dtype=None, dw_dtype=None,
                        act: int = ACT_NONE) -> ProductPlan:
    """The kernels of a product of moe_fp4_linear (GROUPED_FORWARD) or of its backward
    pass (GROUPED_DGRAD: dx, GROUPED_WGRAD: dw), dense, aligned tensors."""
    t = _TYPES[dtype]
    d = LinearDims(M, N, K, t, _TYPES[_out_type(out_dtype, dtype)], t,
                   _TYPES[_out_type(dw_dtype, dtype, "dw_dtype")], act)
    p = ProductPlan()
    _check(_lib.moe_fp4_linear_plan(d, op, p), "moe_fp4_linear_plan")
    return p


def moe_fp4_linear(x: torch.Tensor, w: torch.Tensor, bias: Optional[torch.Tensor] = None,
                   act: int = ACT_NONE, residual: Optional[torch.Tensor] = None,
                   y: Optional[torch.Tensor] = None, out_dtype=None, save_z: bool = False,
                   accumulate: bool = False, workspace: Optional[torch.Tensor] = None):
    """y [M, N] = act(x [M, K] . w [N, K]^T + bias [N]) + residual [M, N]; y may be
    the residual.  With save_z returns (y, z), z the pre-activation in x's type."""
    ldx = _rows(x, "x", _HALF)
    dev = x.device
    ldw = _rows(w, "w", (x.dtype,), dev)
    M, K = x.shape
    N = w.shape[0]
    if w.shape[1] != K:
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
    z = torch.empty((M, N), dtype=x.dtype, device=dev) if save_z else None
    t = _TYPES[x.dtype]
    d = LinearDims(M, N, K, t, _TYPES[y.dtype], t if bias is None else _TYPES[bias.dtype], t, act, ldx, ldw, ldy, ldr)
    ws, nws, keep = _workspace(_lib.moe_fp4_linear_workspace_size, d, 0, workspace=workspace, device=dev)
    _call(_lib.moe_fp4_linear, dev, d, x.data_ptr(), w.data_ptr(), _opt(bias), _opt(residual), y.data_ptr(), _opt(z),
          ACCUMULATE if accumulate else 0, ws, nws)
    return (y, z) if save_z else y


def moe_fp4_linear_backward(dy: torch.Tensor, x: Optional[torch.Tensor], w: Optional[torch.Tensor],
                            z: Optional[torch.Tensor] = None, act: int = ACT_NONE, need_dx: bool = True,
                            need_dw: bool = True, need_db: bool = True, dw_dtype=None,
                            dx: Optional[torch.Tensor] = None, dw: Optional[torch.Tensor] = None,
                            db: Optional[torch.Tensor] = None, accumulate: bool = False,
                            workspace: Optional[torch.Tensor] = None):
    """(dx [M, K], dw [N, K], db [N] fp32) of moe_fp4_linear, None where not
    needed; the residual's gradient is dy.  z as moe_fp4_linear kept it (act not
    NONE); x is needed for dw, w for dx.  accumulate adds to the given dw and db."""
    if (need_dx and w is None) or (need_dw and x is None):
        raise ValueError("x is needed for dw and w for dx")
    if act != ACT_NONE and z is None:
        raise ValueError("the activation's backward pass needs z")
    if not (need_dx or need_dw or need_db):
        raise ValueError("nothing to compute")
    some = next((t for t in (x, w, z) if t is not None), None)
    if some is not None:
        dt = some.dtype
        if dt not in _HALF:
            raise TypeError(f"x, w and z have dtype {dt}, expected one of {_HALF}")
    else:  # db alone: dy's type, or with an fp32 dy either of the two
        dt = getattr(dy, "dtype", None)
        dt = dt if dt in _HALF else torch.bfloat16
    ldy = _rows(dy, "dy", (dt, torch.float32))
    dev = dy.device
    M, N = dy.shape
    K = x.shape[1] if x is not None else w.shape[1] if w is not None else 1
    ldx = _rows(x, "x", (dt,), dev, (M, K)) if x is not None else 0
    ldw = _rows(w, "w", (dt,), dev, (N, K)) if w is not None else 0
    ldz = _rows(z, "z", (dt,), dev, (M, N)) if z is not None else 0
    lddx = lddw = 0
    if accumulate and ((need_dw and dw is None) or (need_db and db is None)):
        raise ValueError("accumulate needs dw and db")
    if need_dx:
        if dx is None:
            dx = torch.empty((M, K), dtype=dt, device=dev)
        else:
            lddx = _rows(dx, "dx", (dt,), dev, (M, K))
    if need_dw:
        if dw is None:
            dw = torch.empty((N, K), dtype=_out_type(dw_dtype, dt, "dw_dtype"), device=dev)
        else:
            lddw = _given(dw, "dw", dw_dtype, dt, dev, (N, K), "dw_dtype")
    if need_db:
        if db is None:
            db = torch.empty(N, dtype=torch.float32, device=dev)
        else:
            _vector(db, "db", N, _FP32, dev)
    dx, dw, db = dx if need_dx else None, dw if need_dw else None, db if need_db else None
    t = _TYPES[dt]
    d = LinearDims(M, N, K, t, _TYPES[dy.dtype], t, t if dw is None else _TYPES[dw.dtype], act, ldx, ldw, ldy, 0, ldz,
                   lddx, lddw)
    ws, nws, keep = _workspace(_lib.moe_fp4_linear_workspace_size, d, 1, workspace=workspace, device=dev)
    _call(_lib.moe_fp4_linear_backward, dev, d, dy.data_ptr(), _opt(x), _opt(w), _opt(z), _opt(dx), _opt(dw), _opt(db),
          ACCUMULATE if accumulate else 0, ws, nws)
    return dx, dw, db


# ---------------------------------------------------------------- norms
def _norm_y_types(x):
    return _ANY if x.dtype == torch.float32 else (x.dtype,)


def _norm_weight(w, name, H, dev, other=None):
    if w is None:
        return other
    _vector(w, name, H, _ANY if other is None else (other,), dev)
    return w.dtype


def moe_fp4_norm(x: torch.Tensor, gamma: Optional[torch.Tensor] = None, beta: Optional[torch.Tensor] = None,
                 eps: float = 1e-6, kind: int = NORM_LAYER, y: Optional[torch.Tensor] = None, out_dtype=None,
                 save_stats: bool = False):
    """y [T, H] = (x - mean) * rstd * gamma + beta (NORM_LAYER), or with mean 0
    (NORM_RMS).  x fp32, bf16 or fp16; y of x's type, or any of the three for
    fp32 x.  With save_stats returns (y, mean, rstd), both [T] fp32, mean None
    for the RMS kind."""
    ldx = _rows(x, "x", _ANY)
    dev = x.device
    T, H = x.shape
    if y is None:
        dt = x.dtype if out_dtype is None else out_dtype
        if dt not in _norm_y_types(x):
            raise TypeError(f"out_dtype must be one of {_norm_y_types(x)}")
        y, ldy = torch.empty((T, H), dtype=dt, device=dev), 0
    else:
        if out_dtype is not None and y.dtype != out_dtype:
            raise TypeError("y and out_dtype disagree")
        ldy = _rows(y, "y", _norm_y_types(x), dev, (T, H))
    wt = _norm_weight(beta, "beta", H, dev, _norm_weight(gamma, "gamma", H, dev)) or x.dtype
    mean = rstd = None
    if save_stats:
        rstd = torch.empty(T, dtype=torch.float32, device=dev)
        if kind == NORM_LAYER:
            mean = torch.empty_like(rstd)
    d = NormDims(T, H, _TYPES[x.dtype], _TYPES[y.dtype], _TYPES[wt], kind, eps, ldx, ldy)
    _call(_lib.moe_fp4_norm, dev, d, x.data_ptr(), _opt(gamma), _opt(beta), y.data_ptr(), _opt(mean), _opt(rstd))
    return (y, mean, rstd) if save_stats else y


def moe_fp4_norm_backward_workspace_size(T: int, H: int, dtype=torch.bfloat16) -> int:
    """Bytes of workspace of moe_fp4_norm_backward for x of type `dtype`."""
    n = _SZ()
    _check(_lib.moe_fp4_norm_backward_workspace_size(NormDims(T, H, _TYPES[dtype], _TYPES[dtype], F32), n),
           "moe_fp4_norm_backward_workspace_size")
    return n.value


def moe_fp4_norm_backward(dy: torch.Tensor, x: torch.Tensor, gamma: Optional[torch.Tensor],
                          mean: Optional[torch.Tensor], rstd: torch.Tensor, kind: int = NORM_LAYER,
                          need_dx: bool = True, need_dgamma: Optional[bool] = None,
                          need_dbeta: Optional[bool] = None, dx: Optional[torch.Tensor] = None,
                          dgamma: Optional[torch.Tensor] = None, dbeta: Optional[torch.Tensor] = None,
                          accumulate: bool = False, workspace: Optional[torch.Tensor] = None):
    """(dx, dgamma [H] fp32, dbeta [H] fp32) of moe_fp4_norm, None where not
    needed; by default dgamma where gamma is given and dbeta with it for the
    layer kind.  dx may be dy.  accumulate adds to the given dgamma and dbeta."""
    ldx = _rows(x, "x", _ANY)
    dev = x.device
    T, H = x.shape
    ldy = _rows(dy, "dy", _norm_y_types(x), dev, (T, H))
    wt = _norm_weight(gamma, "gamma", H, dev) or x.dtype
    if need_dgamma is None:
        need_dgamma = gamma is not None
    if need_dbeta is None:
        need_dbeta = gamma is not None and kind == NORM_LAYER
    if not (need_dx or need_dgamma or need_dbeta):
        raise ValueError("nothing to compute")
    _vector(rstd, "rstd", T, _FP32, dev)
    if kind == NORM_LAYER:
        _vector(mean, "mean", T, _FP32, dev)
    else:
        mean = None
    if accumulate and ((need_dgamma and dgamma is None) or (need_dbeta and dbeta is None)):
        raise ValueError("accumulate needs dgamma and dbeta")
    lddx = 0
    if need_dx:
        if dx is None:
            dx = torch.empty((T, H), dtype=x.dtype, device=dev)
        else:
            lddx = _rows(dx, "dx", (x.dtype,), dev, (T, H))
    if need_dgamma:
        if dgamma is None:
            dgamma = torch.empty(H, dtype=torch.float32, device=dev)
        else:
            _vector(dgamma, "dgamma", H, _FP32, dev)
    if need_dbeta:
        if dbeta is None:
            dbeta = torch.empty(H, dtype=torch.float32, device=dev)
        else:
            _vector(dbeta, "dbeta", H, _FP32, dev)
    dx, dgamma, dbeta = dx if need_dx else None, dgamma if need_dgamma else None, dbeta if need_dbeta else None
    d = NormDims(T, H, _TYPES[x.dtype], _TYPES[dy.dtype], _TYPES[wt], kind, 0.0, ldx, ldy, lddx)
    ws, nws, keep = None, 0, None
    if need_dgamma or need_dbeta:
        ws, nws, keep = _workspace(_lib.moe_fp4_norm_backward_workspace_size, d, workspace=workspace, device=dev)
    _call(_lib.moe_fp4_norm_backward, dev, d, dy.data_ptr(), x.data_ptr(), _opt(gamma), _opt(mean), rstd.data_ptr(),
          _opt(dx), _opt(dgamma), _opt(dbeta), ACCUMULATE if accumulate else 0, ws, nws)
    return dx, dgamma, dbeta
