"""Refusals of the operators around the routed experts, without a GPU: every call
below fails validation, which happens on the host before any HIP call; the fake
device addresses are never dereferenced."""
import ctypes

import pytest

FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def b():
    from mxfp4_routed_expert_router_amd import _block
    return _block


@pytest.fixture(scope="module")
def lib():
    from mxfp4_routed_expert_router_amd import _lib
    return _lib


def grouped(b, **over):
    d = dict(E=4, P=100, N=64, K=128, R=50, row_div=2, type=b.BF16, out_type=b.BF16, ldx=0, ldw=0, ldy=0, expert_stride=0)
    d.update(over)
    return b.GroupedDims(**d)


def linear(b, **over):
    d = dict(M=10, N=64, K=128, type=b.BF16, out_type=b.BF16, bias_type=b.BF16, dw_type=b.BF16, act=0)
    d.update(over)
    return b.LinearDims(**d)


def norm(b, **over):
    d = dict(T=10, H=64, x_type=b.BF16, y_type=b.BF16, w_type=b.BF16, kind=0, eps=1e-6)
    d.update(over)
    return b.NormDims(**d)


def call_grouped(b, lib, op, d, a=FAKE, w=FAKE, off=FAKE, rows=FAKE, c=FAKE, flags=2):
    """flags=2 is never valid, so that a call that passes every earlier check still stops there."""
    L, r = lib._lib, ctypes.byref(d) if d is not None else None
    if op == 1:
        return L.moe_fp4_grouped_dgrad(r, a, w, off, c, flags, None, 0, None)
    f = L.moe_fp4_grouped_forward if op == 0 else L.moe_fp4_grouped_wgrad
    return f(r, a, w, off, rows, c, flags, None, 0, None)


@pytest.mark.parametrize("op", [0, 1, 2])
@pytest.mark.parametrize("over,code", [
    (dict(E=0), "EINVAL"), (dict(P=-1), "EINVAL"), (dict(N=0), "EINVAL"), (dict(K=-5), "EINVAL"),
    (dict(E=1025), "EUNSUPPORTED"), (dict(P=1048577), "EUNSUPPORTED"), (dict(N=65537), "EUNSUPPORTED"),
    (dict(K=65537), "EUNSUPPORTED"), (dict(type=0), "EUNSUPPORTED"), (dict(type=3), "EUNSUPPORTED"),
    (dict(out_type=2), "EUNSUPPORTED"), (dict(ldx=127), "EINVAL"), (dict(ldw=100), "EINVAL"), (dict(ldy=63), "EINVAL"),
    (dict(ldx=-128), "EINVAL"), (dict(expert_stride=64 * 128 - 1), "EINVAL"), (dict(expert_stride=-1), "EINVAL"),
    (dict(ldw=256, expert_stride=63 * 256 + 127), "EINVAL"), (dict(ldw=2**41), "EINVAL")])
def test_grouped_dims(b, lib, op, over, code):
    assert call_grouped(b, lib, op, grouped(b, **over), flags=0) == getattr(lib, code)
    n = ctypes.c_size_t()
    assert lib._lib.moe_fp4_grouped_workspace_size(ctypes.byref(grouped(b, **over)), op, ctypes.byref(n)) == getattr(lib, code)


@pytest.mark.parametrize("op", [0, 2])
def test_grouped_gather(b, lib, op):
    for over in (dict(row_div=0), dict(row_div=-3), dict(R=-1)):
        assert call_grouped(b, lib, op, grouped(b, **over), flags=0) == lib.EINVAL
    assert call_grouped(b, lib, op, grouped(b, R=1048577), flags=0) == lib.EUNSUPPORTED
    # not read without a row index
    assert call_grouped(b, lib, op, grouped(b, row_div=0, R=-1), rows=None) == lib.EUNSUPPORTED


@pytest.mark.parametrize("op", [0, 1, 2])
def test_grouped_pointers_and_flags(b, lib, op):
    d = grouped(b)
    assert call_grouped(b, lib, op, None, flags=0) == lib.EINVAL
    for null in ("a", "w", "off", "c"):
        assert call_grouped(b, lib, op, d, flags=0, **{null: None}) == lib.EINVAL
    for odd in ("a", "w", "c"):
        assert call_grouped(b, lib, op, d, flags=0, **{odd: FAKE + 1}) == lib.EALIGN
    assert call_grouped(b, lib, op, d, flags=0, off=FAKE + 2) == lib.EALIGN
    if op != 1:
        assert call_grouped(b, lib, op, d, flags=0, rows=FAKE + 2) == lib.EALIGN
    assert call_grouped(b, lib, op, grouped(b, out_type=0), flags=0, c=FAKE + 2) == lib.EALIGN
    assert call_grouped(b, lib, op, d, flags=2) == lib.EUNSUPPORTED


def test_grouped_workspace_arguments(b, lib):
    n = ctypes.c_size_t()
    f = lib._lib.moe_fp4_grouped_workspace_size
    assert f(None, 0, ctypes.byref(n)) == lib.EINVAL
    assert f(ctypes.byref(grouped(b)), 0, None) == lib.EINVAL
    for op in (-1, 3):
        assert f(ctypes.byref(grouped(b)), op, ctypes.byref(n)) == lib.EUNSUPPORTED


def call_linear(lib, d, x=FAKE, w=FAKE, bias=FAKE, r=FAKE, y=FAKE, z=FAKE, flags=2):
    return lib._lib.moe_fp4_linear(ctypes.byref(d) if d is not None else None, x, w, bias, r, y, z, flags, None, 0, None)


def call_back(lib, d, dy=FAKE, x=FAKE, w=FAKE, z=FAKE, dx=FAKE, dw=FAKE, db=FAKE, flags=2, ws=FAKE, n=0):
    return lib._lib.moe_fp4_linear_backward(ctypes.byref(d) if d is not None else None, dy, x, w, z, dx, dw, db, flags,
                                            ws, n, None)


@pytest.mark.parametrize("over,code", [
    (dict(M=-1), "EINVAL"), (dict(N=0), "EINVAL"), (dict(K=0), "EINVAL"), (dict(M=1048577), "EUNSUPPORTED"),
    (dict(N=65537), "EUNSUPPORTED"), (dict(K=65537), "EUNSUPPORTED"), (dict(type=0), "EUNSUPPORTED"),
    (dict(out_type=2), "EUNSUPPORTED"), (dict(act=-1), "EUNSUPPORTED"), (dict(act=5), "EUNSUPPORTED"),
    (dict(ldx=127), "EINVAL"), (dict(ldw=1), "EINVAL"), (dict(ldy=63), "EINVAL"), (dict(ldr=63), "EINVAL"),
    (dict(ldz=-1), "EINVAL"), (dict(lddx=127), "EINVAL"), (dict(lddw=127), "EINVAL")])
def test_linear_dims(b, lib, over, code):
    d = linear(b, **over)
    n = ctypes.c_size_t()
    assert call_linear(lib, d, flags=0) == getattr(lib, code)
    assert call_back(lib, d, flags=0) == getattr(lib, code)
    for back in (0, 1):
        assert lib._lib.moe_fp4_linear_workspace_size(ctypes.byref(d), back, ctypes.byref(n)) == getattr(lib, code)


def test_linear_types_of_one_direction(b, lib):
    assert call_linear(lib, linear(b, bias_type=3), flags=0) == lib.EUNSUPPORTED
    assert call_back(lib, linear(b, dw_type=2), flags=0) == lib.EUNSUPPORTED


def test_linear_pointers(b, lib):
    d = linear(b, act=2)
    assert call_linear(lib, None) == lib.EINVAL and call_back(lib, None) == lib.EINVAL
    for null in ("x", "w", "y"):
        assert call_linear(lib, d, flags=0, **{null: None}) == lib.EINVAL
    for odd in ("x", "w", "y", "z", "r", "bias"):
        assert call_linear(lib, d, flags=0, **{odd: FAKE + 1}) == lib.EALIGN
    assert call_linear(lib, d) == lib.EUNSUPPORTED
    for null in ("dy", "x", "w", "z"):
        assert call_back(lib, d, flags=0, **{null: None}) == lib.EINVAL
    assert call_back(lib, d, flags=0, dx=None, dw=None, db=None) == lib.EINVAL
    for odd in ("dy", "x", "w", "z", "dx", "dw", "db"):
        assert call_back(lib, d, flags=0, **{odd: FAKE + 1}) == lib.EALIGN
    assert call_back(lib, d) == lib.EUNSUPPORTED
    n = ctypes.c_size_t()
    assert lib._lib.moe_fp4_linear_workspace_size(ctypes.byref(d), 1, ctypes.byref(n)) == 0 and n.value > 0
    assert call_back(lib, d, flags=0, n=n.value - 1) == lib.EWORKSPACE
    assert call_back(lib, d, flags=0, ws=None, n=n.value) == lib.EINVAL
    assert call_back(lib, d, flags=0, ws=FAKE + 128, n=n.value) == lib.EALIGN


def call_norm(lib, d, x=FAKE, g=FAKE, bt=FAKE, y=FAKE, m=FAKE, r=FAKE):
    return lib._lib.moe_fp4_norm(ctypes.byref(d) if d is not None else None, x, g, bt, y, m, r, None)


def call_norm_back(lib, d, dy=FAKE, x=FAKE, g=FAKE, m=FAKE, r=FAKE, dx=FAKE, dg=FAKE, db=FAKE, flags=2, ws=FAKE, n=0):
    return lib._lib.moe_fp4_norm_backward(ctypes.byref(d) if d is not None else None, dy, x, g, m, r, dx, dg, db, flags,
                                          ws, n, None)


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), "EINVAL"), (dict(H=0), "EINVAL"), (dict(eps=-1e-6), "EINVAL"), (dict(eps=float("nan")), "EINVAL"),
    (dict(T=1048577), "EUNSUPPORTED"), (dict(H=16385), "EUNSUPPORTED"), (dict(x_type=3), "EUNSUPPORTED"),
    (dict(y_type=0), "EUNSUPPORTED"), (dict(y_type=2), "EUNSUPPORTED"), (dict(w_type=-1), "EUNSUPPORTED"),
    (dict(kind=2), "EUNSUPPORTED"), (dict(ldx=63), "EINVAL"), (dict(ldy=63), "EINVAL"), (dict(lddx=-64), "EINVAL")])
def test_norm_dims(b, lib, over, code):
    d = norm(b, **over)
    n = ctypes.c_size_t()
    assert call_norm(lib, d) == getattr(lib, code)
    assert call_norm_back(lib, d, flags=0) == getattr(lib, code)
    assert lib._lib.moe_fp4_norm_backward_workspace_size(ctypes.byref(d), ctypes.byref(n)) == getattr(lib, code)


def test_norm_pointers(b, lib):
    d = norm(b)
    assert call_norm(lib, None) == lib.EINVAL and call_norm_back(lib, None) == lib.EINVAL
    for null in ("x", "y"):
        assert call_norm(lib, d, **{null: None}) == lib.EINVAL
    for odd in ("x", "g", "bt", "y", "m", "r"):
        assert call_norm(lib, d, **{odd: FAKE + 1}) == lib.EALIGN
    for null in ("dy", "x", "r", "m"):
        assert call_norm_back(lib, d, flags=0, **{null: None}) == lib.EINVAL
    assert call_norm_back(lib, d, flags=0, dx=None, dg=None, db=None) == lib.EINVAL
    for odd in ("dy", "x", "g", "m", "r", "dx", "dg", "db"):
        assert call_norm_back(lib, d, flags=0, **{odd: FAKE + 1}) == lib.EALIGN
    assert call_norm_back(lib, d) == lib.EUNSUPPORTED
    n = ctypes.c_size_t()
    assert lib._lib.moe_fp4_norm_backward_workspace_size(ctypes.byref(d), ctypes.byref(n)) == 0
    assert call_norm_back(lib, d, flags=0, n=n.value - 1) == lib.EWORKSPACE
    assert call_norm_back(lib, d, flags=0, ws=None, n=n.value) == lib.EINVAL
    assert lib._lib.moe_fp4_norm_backward_workspace_size(ctypes.byref(d), None) == lib.EINVAL


def test_binding_wants_gpu_tensors(b):
    import torch
    x, w = torch.zeros(2, 8, dtype=torch.bfloat16), torch.zeros(1, 4, 8, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        b.moe_fp4_grouped_forward(x, w, torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        b.moe_fp4_linear(x, w[0])
    with pytest.raises(ValueError):
        b.moe_fp4_norm(x)
    with pytest.raises(TypeError):
        b.moe_fp4_norm([1.0])
