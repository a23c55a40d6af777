"""Refusals of the router's losses, the gradients' norm and the 4-bit product,
without a GPU: every call below fails validation, which happens on the host before any
HIP call; the fake device addresses are never dereferenced."""
import ctypes

import pytest

FAKE = 0x7F0000000000


@pytest.fixture(scope="module")
def b():
    from mxfp4_routed_expert_router_amd import _block, _train, _w4  # noqa: F401
    return _train


@pytest.fixture(scope="module")
def lib():
    from mxfp4_routed_expert_router_amd import _lib
    return _lib


def loss_dims(b, **over):
    d = dict(T=1000, E=16, k=4, S=3, score=0, type=1, out_type=1, ld=0, ldd=0)
    d.update(over)
    return b.RouterLossDims(**d)


def forward(lib, d, logits=FAKE, idx=FAKE, seqs=FAKE, mask=FAKE, outs=(FAKE,) * 5, ws=FAKE, n=0):
    return lib._lib.moe_fp4_router_loss(ctypes.byref(d) if d is not None else None, logits, idx, seqs, mask, *outs, ws, n, None)


def backward(lib, d, logits=FAKE, idx=FAKE, seqs=FAKE, mask=FAKE, counts=FAKE, tokens=FAKE, db=FAKE, dz=FAKE, gates=FAKE,
             dgates=FAKE, out=FAKE, flags=2):
    """flags=2 is never valid, so that a call that passes the checks of sizes still stops there."""
    return lib._lib.moe_fp4_router_loss_backward(ctypes.byref(d) if d is not None else None, logits, idx, seqs, mask, counts,
                                                 tokens, db, dz, gates, dgates, out, flags, None)


@pytest.mark.parametrize("over,code", [
    (dict(T=-1), "EINVAL"), (dict(E=0), "EINVAL"), (dict(k=0), "EINVAL"), (dict(S=0), "EINVAL"), (dict(k=17), "EINVAL"),
    (dict(ld=15), "EINVAL"), (dict(ld=-16), "EINVAL"), (dict(T=1048577), "EUNSUPPORTED"), (dict(E=1025), "EUNSUPPORTED"),
    (dict(E=32, k=17), "EUNSUPPORTED"), (dict(S=65537), "EUNSUPPORTED"), (dict(score=2), "EUNSUPPORTED"),
    (dict(score=-1), "EUNSUPPORTED"), (dict(type=3), "EUNSUPPORTED")])
def test_loss_dims(b, lib, over, code):
    d, n = loss_dims(b, **over), ctypes.c_size_t()
    assert forward(lib, d) == getattr(lib, code)
    assert backward(lib, d, flags=0) == getattr(lib, code)
    assert lib._lib.moe_fp4_router_loss_workspace_size(ctypes.byref(d), ctypes.byref(n)) == getattr(lib, code)


def test_loss_of_one_direction(b, lib):
    for over, code in ((dict(ldd=15), lib.EINVAL), (dict(out_type=2), lib.EUNSUPPORTED), (dict(out_type=3), lib.EUNSUPPORTED)):
        assert backward(lib, loss_dims(b, **over), flags=0) == code
        assert forward(lib, loss_dims(b, **over)) == lib.EWORKSPACE  # not read there
    assert backward(lib, loss_dims(b)) == lib.EUNSUPPORTED


def test_loss_pointers(b, lib):
    d, n = loss_dims(b), ctypes.c_size_t()
    assert forward(lib, None) == lib.EINVAL and backward(lib, None) == lib.EINVAL
    assert lib._lib.moe_fp4_router_loss_workspace_size(ctypes.byref(d), None) == lib.EINVAL
    assert lib._lib.moe_fp4_router_loss_workspace_size(ctypes.byref(d), ctypes.byref(n)) == 0 and n.value > 0
    for null in ("logits", "idx", "seqs"):
        assert forward(lib, d, **{null: None}) == lib.EINVAL
    for i in range(5):
        outs = [FAKE] * 5
        outs[i] = None
        assert forward(lib, d, outs=outs) == lib.EINVAL
        outs[i] = FAKE + 2
        assert forward(lib, d, outs=outs) == lib.EALIGN
    assert forward(lib, d, logits=FAKE + 1) == lib.EALIGN
    for odd in ("idx", "seqs"):
        assert forward(lib, d, **{odd: FAKE + 2}) == lib.EALIGN
    assert forward(lib, d, n=n.value - 1) == lib.EWORKSPACE
    assert forward(lib, d, ws=None, n=n.value) == lib.EINVAL
    assert forward(lib, d, ws=FAKE + 64, n=n.value) == lib.EALIGN
    assert forward(lib, loss_dims(b, S=1), seqs=None) == lib.EWORKSPACE  # one sequence needs no offsets
    assert lib._lib.moe_fp4_router_loss_workspace_size(ctypes.byref(loss_dims(b, T=100)), ctypes.byref(n)) == 0 and n.value == 0
    for null in ("logits", "tokens", "counts", "seqs", "out", "idx", "gates", "dgates"):
        assert backward(lib, d, flags=0, **{null: None}) == lib.EINVAL
    assert backward(lib, d, flags=0, db=None, dz=None, gates=None, dgates=None) == lib.EINVAL
    for odd in ("idx", "seqs", "counts", "tokens", "db", "dz", "gates", "dgates"):
        assert backward(lib, d, flags=0, **{odd: FAKE + 2}) == lib.EALIGN
    for odd in ("logits", "out"):
        assert backward(lib, d, flags=0, **{odd: FAKE + 1}) == lib.EALIGN


def table(b, *rows):
    """rows of (data, out, n, type, out_type)"""
    return (b.GradTensor * len(rows))(*[b.GradTensor(*r) for r in rows])


def sumsq(lib, t, n, out=FAKE, flags=2, ws=FAKE, nws=0):
    return lib._lib.moe_fp4_grad_sumsq(t, n, out, flags, ws, nws, None)


def clip(lib, t, n, ss=FAKE, max_norm=1.0, eps=1e-6, norm=FAKE):
    return lib._lib.moe_fp4_grad_clip(t, n, ss, max_norm, eps, norm, None)


def test_gradients(b, lib):
    size = ctypes.c_size_t()
    good = table(b, (FAKE, None, 100, 0, 0), (FAKE + 4096, None, 7, 1, 0))
    f = lib._lib.moe_fp4_grad_sumsq_workspace_size
    assert f(good, 2, ctypes.byref(size)) == 0 and size.value == 16
    assert f(None, 0, ctypes.byref(size)) == 0 and size.value == 0
    assert f(good, 2, None) == lib.EINVAL and f(None, 1, ctypes.byref(size)) == lib.EINVAL
    assert f(good, -1, ctypes.byref(size)) == lib.EINVAL
    many = (b.GradTensor * 4097)()
    for rows, n, code in ((table(b, (FAKE, None, -1, 0, 0)), 1, lib.EINVAL), (table(b, (FAKE, None, 1, 3, 0)), 1, lib.EUNSUPPORTED),
                          (table(b, (FAKE, None, 2**40 + 1, 0, 0)), 1, lib.EUNSUPPORTED), (many, 4097, lib.EUNSUPPORTED)):
        assert f(rows, n, ctypes.byref(size)) == code
        assert sumsq(lib, rows, n, flags=0) == code and clip(lib, rows, n) == code
    assert sumsq(lib, good, 2) == lib.EUNSUPPORTED
    assert sumsq(lib, good, 2, out=None, flags=0) == lib.EINVAL and sumsq(lib, good, 2, out=FAKE + 4, flags=0) == lib.EALIGN
    assert sumsq(lib, good, 2, flags=0, nws=15) == lib.EWORKSPACE and sumsq(lib, good, 2, flags=0, ws=None, nws=16) == lib.EINVAL
    for rows, code in ((table(b, (None, None, 5, 0, 0)), lib.EINVAL), (table(b, (FAKE + 2, None, 5, 0, 0)), lib.EALIGN),
                       (table(b, (FAKE + 1, None, 5, 1, 0)), lib.EALIGN)):
        assert sumsq(lib, rows, 1, flags=0) == code and clip(lib, rows, 1) == code


def test_clip_arguments(b, lib):
    good = table(b, (FAKE, None, 100, 0, 0))
    assert clip(lib, good, 1, ss=None) == lib.EINVAL
    for v in (-1.0, float("nan")):
        assert clip(lib, good, 1, max_norm=v) == lib.EINVAL and clip(lib, good, 1, eps=v) == lib.EINVAL
    assert clip(lib, good, 1, ss=FAKE + 4) == lib.EALIGN and clip(lib, good, 1, norm=FAKE + 2) == lib.EALIGN
    assert clip(lib, table(b, (FAKE, FAKE + 4096, 5, 1, 0)), 1) == lib.EUNSUPPORTED  # bf16 into fp32
    assert clip(lib, table(b, (FAKE, FAKE + 4096, 5, 0, 3)), 1) == lib.EUNSUPPORTED
    assert clip(lib, table(b, (FAKE, FAKE + 4097, 5, 0, 1)), 1) == lib.EALIGN


def test_clip_overlaps(b, lib):
    """A written range meets another tensor's: the calls that a race would follow."""
    A, far = FAKE, FAKE + (1 << 20)
    for rows in ([(A, None, 100, 0, 0), (A, None, 100, 0, 0)],                   # a tensor twice, in place
                 [(A, None, 100, 0, 0), (A + 396, None, 100, 0, 0)],              # the last element
                 [(A + 396, None, 100, 0, 0), (far, None, 5, 0, 0), (A, None, 100, 0, 0)],
                 [(A, far, 100, 0, 0), (far + 64, None, 2, 0, 0)],                # a result over an input
                 [(A, far, 100, 0, 1), (far + 8192, far + 198, 4, 0, 1)],         # results over one another
                 [(A, A + 4, 100, 0, 0)],                                         # moved by an element
                 [(A, A, 100, 0, 1)],                                             # narrower, over its own input
                 [(A, far, 1000, 0, 0), (far + 3996, far + 8192, 1, 0, 0)]):
        assert clip(lib, table(b, *rows), len(rows)) == lib.EINVAL, rows


def w4(b, **over):
    from mxfp4_routed_expert_router_amd import _w4
    d = dict(M=3, N=10, K=64, code=1, group=64, type=1, out_type=1, bias_type=1, scale_type=1, act=0)
    d.update(over)
    return _w4.W4Dims(**d)


def call_w4(lib, d, x=FAKE, codes=FAKE, scales=FAKE, zeros=FAKE, bias=FAKE, r=FAKE, y=FAKE, flags=0):
    return lib._lib.moe_fp4_linear_w4(ctypes.byref(d) if d is not None else None, x, codes, scales, zeros, bias, r, y, flags, None)


@pytest.mark.parametrize("over,code", [
    (dict(M=-1), "EINVAL"), (dict(N=0), "EINVAL"), (dict(K=0), "EINVAL"), (dict(group=0), "EINVAL"), (dict(ldx=63), "EINVAL"),
    (dict(ldy=9), "EINVAL"), (dict(ldr=9), "EINVAL"), (dict(ldw=31), "EINVAL"), (dict(ldw=2**23), "EINVAL"),
    (dict(ldw=40), "EALIGN"), (dict(M=1048577), "EUNSUPPORTED"), (dict(N=65537), "EUNSUPPORTED"),
    (dict(K=65568), "EUNSUPPORTED"), (dict(K=48), "EUNSUPPORTED"), (dict(code=2), "EUNSUPPORTED"),
    (dict(code=0, group=64), "EUNSUPPORTED"), (dict(group=16), "EUNSUPPORTED"), (dict(group=512), "EUNSUPPORTED"),
    (dict(group=96), "EUNSUPPORTED"), (dict(type=0), "EUNSUPPORTED"), (dict(out_type=2), "EUNSUPPORTED"),
    (dict(bias_type=3), "EUNSUPPORTED"), (dict(scale_type=3), "EUNSUPPORTED"), (dict(act=5), "EUNSUPPORTED"),
    (dict(act=-1), "EUNSUPPORTED")])
def test_w4_dims(b, lib, over, code):
    assert call_w4(lib, w4(b, **over)) == getattr(lib, code)


def test_w4_pointers(b, lib):
    d = w4(b)
    assert call_w4(lib, None) == lib.EINVAL and call_w4(lib, d, flags=2) == lib.EUNSUPPORTED
    for null in ("x", "codes", "scales", "y"):
        assert call_w4(lib, d, **{null: None}) == lib.EINVAL
    assert call_w4(lib, w4(b, code=0, group=32)) == lib.EINVAL  # zeros with MX
    for odd in ("x", "scales", "bias", "r", "y"):
        assert call_w4(lib, d, **{odd: FAKE + 1}) == lib.EALIGN
    assert call_w4(lib, d, codes=FAKE + 8) == lib.EALIGN
    assert call_w4(lib, w4(b, M=0), x=None, y=None) == lib.OK  # nothing to do


def test_binding_wants_gpu_tensors(b):
    import torch
    import mxfp4_routed_expert_router_amd as moe
    with pytest.raises(ValueError):
        moe.moe_fp4_router_loss(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        moe.moe_fp4_grad_sumsq([torch.zeros(4)])
    with pytest.raises(ValueError):
        moe.moe_fp4_grad_sumsq([])
    with pytest.raises(TypeError):
        moe.moe_fp4_grad_sumsq([None])
    with pytest.raises(ValueError):
        moe.W4Weights(torch.zeros(4, 16, dtype=torch.uint8), torch.zeros(4, 1, dtype=torch.uint8))
    with pytest.raises(ValueError):
        moe.moe_fp4_linear_w4(torch.zeros(1, 32, dtype=torch.bfloat16), None)
