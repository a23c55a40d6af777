"""The dense product with bias, activation and residual, and its backward pass,
against 64-bit references: one row to many, odd sizes, strides, both types and
result types, and the gradients against differences."""
import pytest
import torch

from block_common import U32, act64, bounded, gen, half_step, padded, randn, slope64

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
# |act'| and |act''| of every activation here stay below these (gelu' <= 1.13, gelu'' <= 0.8;
# relu's slope jumps, but its argument z is the same number on both sides of the backward pass)
SLOPE = 1.15


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_routed_expert_router_amd as m
    return m


def act_id(moe, name):
    return {"none": moe.ACT_NONE, "relu": moe.ACT_RELU, "gelu": moe.ACT_GELU, "gelu_tanh": moe.ACT_GELU_TANH,
            "silu": moe.ACT_SILU}[name]


def forward64(x, w, bias, act, residual):
    """y, z and bounds of both before their rounding."""
    K = x.shape[1]
    z = x @ w.t()
    e_z = K * U32 * (x.abs() @ w.abs().t())
    if bias is not None:
        z = z + bias
        e_z = e_z + U32 * (z.abs() + bias.abs())
    a = act64(z, act)
    # the activation's own evaluation: a few operations, exp and erfc within 4 steps, on
    # arguments of rounded products (|z| steps of the exponent)
    e_y = SLOPE * e_z if act != "none" else e_z
    if act not in ("none", "relu"):
        e_y = e_y + (16 + 4 * z.abs()) * U32 * (a.abs() + SUBN)
    y = a
    if residual is not None:
        y = a + residual
        e_y = e_y + U32 * (a.abs() + residual.abs())
    return y, z, e_y, e_z


SUBN = 2.0 ** -100

SHAPES = [(1, 16, 32), (1, 1, 1), (1, 5120, 512), (1, 640, 5120), (2, 288, 320), (6, 512, 1024), (16, 100, 96),
          (17, 72, 2304), (33, 130, 77), (64, 256, 512), (100, 1001, 515), (129, 127, 130), (257, 264, 264),
          (300, 512, 256), (5, 33, 1001), (1, 1001, 515), (700, 64, 64), (4, 999, 2051), (31, 257, 1029), (1300, 2064, 72),
          (2000, 4104, 136), (48, 72, 5120), (40, 67, 4099)]


@pytest.mark.parametrize("dt", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward(moe, M, N, K, dt):
    g = gen(M * 7 + N + K)
    x, w = randn(g, M, K, dtype=dt), randn(g, N, K, dtype=dt, scale=K ** -0.5)
    combos = [("none", None, False, dt), ("none", F32, True, F32), ("gelu", dt, True, dt), ("silu", dt, False, F32),
              ("gelu_tanh", BF if dt == HF else HF, False, dt), ("relu", None, True, dt)]
    for act, bt, res, out in combos:
        bias = randn(g, N, dtype=bt) if bt else None
        r = randn(g, M, N, dtype=out) if res else None
        y, z = moe.moe_fp4_linear(x, w, bias=bias, act=act_id(moe, act), residual=r, out_dtype=out, save_z=True)
        wy, wz, ey, ez = forward64(x.double(), w.double(), bias.double() if bt else None, act, r.double() if res else None)
        assert y.dtype == out and z.dtype == dt
        bounded(y, wy, ey, out, f"y {act} {out}")
        bounded(z, wz, ez, dt, "z")
        y2 = moe.moe_fp4_linear(x, w, bias=bias, act=act_id(moe, act), residual=r, out_dtype=out)
        assert torch.equal(y, y2)


@pytest.mark.parametrize("M,N,K", [(1, 256, 128), (50, 130, 96), (3, 33, 47)])
def test_residual_in_place_and_accumulate(moe, M, N, K):
    g = gen(M + N)
    x, w, b = randn(g, M, K, dtype=BF), randn(g, N, K, dtype=BF), randn(g, N, dtype=BF)
    r = randn(g, M, N)
    want = moe.moe_fp4_linear(x, w, bias=b, residual=r, out_dtype=F32)
    y = r.clone()
    moe.moe_fp4_linear(x, w, bias=b, residual=y, y=y)
    assert torch.equal(y, want)
    y = r.clone()
    moe.moe_fp4_linear(x, w, bias=b, y=y, accumulate=True)
    wy, _, ey, _ = forward64(x.double(), w.double(), b.double(), "none", r.double())
    bounded(y, wy, ey, F32, "y +=")


@pytest.mark.parametrize("M", [1, 9, 70])
@pytest.mark.parametrize("pad,offset", [(8, 8), (1, 0), (3, 5)])
def test_strides_and_alignment(moe, M, pad, offset):
    g = gen(M + pad)
    N, K = 136, 200
    x, _ = padded(randn(g, M, K, dtype=BF), pad, offset)
    w, _ = padded(randn(g, N, K, dtype=BF), pad, offset)
    r, _ = padded(randn(g, M, N, dtype=BF), pad, offset)
    y, buf = padded(torch.zeros(M, N, dtype=BF, device="cuda"), pad, offset, fill=7.0)
    moe.moe_fp4_linear(x, w, residual=r, y=y, act=moe.ACT_SILU)
    wy, _, ey, _ = forward64(x.double(), w.double(), None, "silu", r.double())
    bounded(y, wy, ey, BF, "y")
    left = buf.clone()
    left.as_strided(y.shape, y.stride(), offset).fill_(7.0)
    assert bool((left == 7.0).all())
    dy, _ = padded(randn(g, M, N, dtype=BF), pad, offset)
    z, _ = padded(randn(g, M, N, dtype=BF), pad, offset)
    dx, bufx = padded(torch.zeros(M, K, dtype=BF, device="cuda"), pad, offset, fill=7.0)
    dw, bufw = padded(torch.zeros(N, K, dtype=F32, device="cuda"), pad, offset, fill=7.0)
    for act in ("none", "silu"):
        moe.moe_fp4_linear_backward(dy, x, w, z=z, act=act_id(moe, act), dx=dx, dw=dw)
        (wx, ww, wb), (ex, ew, eb) = backward64(dy.double(), x.double(), w.double(), z.double(), act, BF)
        bounded(dx, wx, ex, BF, "dx")
        bounded(dw, ww, ew, F32, "dw")
        for out, b in ((dx, bufx), (dw, bufw)):
            left = b.clone()
            left.as_strided(out.shape, out.stride(), offset).fill_(7.0)
            assert bool((left == 7.0).all())


def backward64(dy, x, w, z, act, dt):
    M, N = dy.shape
    if act == "none":
        dz, e = dy, torch.zeros_like(dy)
    else:
        s = slope64(z, act)
        dz = dy * s
        # the slope's evaluation; its terms cancel where it is small, so relative to 1 + |z|
        e = dy.abs() * (16 + 8 * z.abs()) * U32 * 1.2
        if act == "relu":
            e = torch.zeros_like(dy)
    e_db = e.sum(0) + (M + 1) * U32 * (dz.abs() + e).sum(0)
    # dz rounded to the products' type (never where it is dy itself)
    e16 = e + (half_step(dt) * (dz.abs() + e) if act != "none" else 0)
    mag = dz.abs() + e16
    e_dx = e16 @ w.abs() + N * U32 * (mag @ w.abs())
    e_dw = e16.t() @ x.abs() + M * U32 * (mag.t() @ x.abs())
    return (dz @ w, dz.t() @ x, dz.sum(0)), (e_dx, e_dw, e_db)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dt", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(1, 16, 32), (1, 1, 1), (3, 288, 320), (64, 256, 512), (100, 101, 115),
                                   (300, 520, 264), (1030, 64, 96), (4100, 40, 24), (4100, 33, 25), (600, 2056, 1544),
                                   (5, 4096, 64)])
def test_backward(moe, M, N, K, dt, act):
    g = gen(M * 11 + N + K)
    x, w = randn(g, M, K, dtype=dt), randn(g, N, K, dtype=dt, scale=K ** -0.5)
    z, dy = randn(g, M, N, dtype=dt, scale=2.0), randn(g, M, N, dtype=dt)
    (wx, ww, wb), (ex, ew, eb) = backward64(dy.double(), x.double(), w.double(), z.double(), act, dt)
    for dwt in (dt, F32):
        dx, dw, db = moe.moe_fp4_linear_backward(dy, x, w, z=None if act == "none" else z, act=act_id(moe, act),
                                                 dw_dtype=dwt)
        assert dx.dtype == dt and dw.dtype == dwt and db.dtype == F32
        bounded(dx, wx, ex, dt, "dx")
        bounded(dw, ww, ew, dwt, "dw")
        bounded(db, wb, eb, F32, "db")
    # one at a time, and on top of given gradients
    one, none, no = moe.moe_fp4_linear_backward(dy, None, w, z=z, act=act_id(moe, act), need_dw=False, need_db=False)
    assert torch.equal(one, dx) and none is None and no is None
    w0, b0 = randn(g, N, K), randn(g, N)
    a, b = w0.clone(), b0.clone()
    moe.moe_fp4_linear_backward(dy, x, None, z=z, act=act_id(moe, act), need_dx=False, dw=a, db=b, accumulate=True)
    bounded(a, ww + w0.double(), ew + U32 * (ww.abs() + w0.double().abs()), F32, "dw +=")
    bounded(b, wb + b0.double(), eb + U32 * (wb.abs() + b0.double().abs()), F32, "db +=")


@pytest.mark.parametrize("act", ["none", "silu"])
def test_backward_of_fp32_gradients(moe, act):
    """dy in fp32 (the residual stream's type): rounded to the products' type once, as dz."""
    g = gen(2)
    M, N, K = 70, 96, 128
    x, w, z = randn(g, M, K, dtype=BF), randn(g, N, K, dtype=BF), randn(g, M, N, dtype=BF)
    dy = randn(g, M, N)
    dx, dw, db = moe.moe_fp4_linear_backward(dy, x, w, z=z, act=act_id(moe, act), dw_dtype=F32)
    (wx, ww, wb), (ex, ew, eb) = backward64(dy.double(), x.double(), w.double(), z.double(), act, BF)
    if act == "none":  # rounded here too
        e16 = half_step(BF) * dy.double().abs()
        ex, ew = ex + 1.01 * (e16 @ w.double().abs()), ew + 1.01 * (e16.t() @ x.double().abs())
    bounded(dx, wx, ex, BF, "dx")
    bounded(dw, ww, ew, F32, "dw")
    bounded(db, wb, eb, F32, "db")


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(moe, act):
    """f = sum(act(x w^T + b) c) in 64 bits, differences along random directions, against the
    kernels' gradients (z away from relu's kink)."""
    g = gen(77)
    M, N, K = 24, 40, 56
    x, w, b = randn(g, M, K, dtype=BF), randn(g, N, K, dtype=BF, scale=K ** -0.5), randn(g, N, dtype=BF)
    c = randn(g, M, N, dtype=BF)
    _, z = moe.moe_fp4_linear(x, w, bias=b, act=act_id(moe, act), save_z=True)
    if act == "relu":
        c = torch.where(z.abs() < 0.05, torch.zeros_like(c), c)
    dx, dw, db = moe.moe_fp4_linear_backward(c, x, w, z=z, act=act_id(moe, act), dw_dtype=F32)
    f = lambda x, w, b: (act64(x @ w.t() + b, act) * c.double()).sum()
    args = [x.double(), w.double(), b.double()]
    h = 2.0 ** -14
    for i, grad in enumerate((dx, dw, db)):
        v = randn(g, *grad.shape).double()
        plus, minus = list(args), list(args)
        plus[i], minus[i] = args[i] + h * v, args[i] - h * v
        diff = ((f(*plus) - f(*minus)) / (2 * h)).item()
        got = (grad.double() * v).sum().item()
        # each gradient's relative roundings: z and dz to bf16 (z's moves the slope by at most
        # 0.8 |z| eps/2, |z| < 6), the result's own; bounded by the sums of magnitudes
        zz = z.double()
        terms = c.double().abs() * (1.13 + 0.8 * zz.abs())
        reach = (lambda: terms @ w.double().abs(), lambda: terms.t() @ x.double().abs(), lambda: terms.sum(0))[i]()
        pos = (reach * v.abs()).sum().item()
        assert abs(diff - got) <= (3 * half_step(BF) + 64 * h * h) * pos, (i, diff, got)


def test_no_rows(moe):
    x, w = torch.empty(0, 64, dtype=BF, device="cuda"), torch.ones(32, 64, dtype=BF, device="cuda")
    assert moe.moe_fp4_linear(x, w).shape == (0, 32)
    dx, dw, db = moe.moe_fp4_linear_backward(torch.empty(0, 32, dtype=BF, device="cuda"), x, w)
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())


def test_nan_and_inf_stay_in_their_rows(moe):
    g = gen(41)
    for M in (4, 80):
        x, w = randn(g, M, 96, dtype=BF), randn(g, 64, 96, dtype=BF)
        x[1, 5], x[3, 0] = float("nan"), float("-inf")
        y = moe.moe_fp4_linear(x, w, act=moe.ACT_RELU, out_dtype=F32)
        bad = ~torch.isfinite(y).all(1)
        assert bad.nonzero().flatten().tolist() == [1, 3]


def test_same_bits_twice(moe):
    g = gen(43)
    for M, N, K in ((1, 640, 2304), (40, 96, 4096), (200, 100, 130)):
        x, w, dy = randn(g, M, K, dtype=BF), randn(g, N, K, dtype=BF), randn(g, M, N, dtype=BF)
        assert torch.equal(moe.moe_fp4_linear(x, w), moe.moe_fp4_linear(x, w))
        one, two = (moe.moe_fp4_linear_backward(dy, x, w, z=dy, act=moe.ACT_GELU) for _ in range(2))
        assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_binding_refusals(moe):
    x, w = torch.zeros(4, 32, dtype=BF, device="cuda"), torch.zeros(16, 32, dtype=BF, device="cuda")
    dy = torch.zeros(4, 16, dtype=BF, device="cuda")
    with pytest.raises(TypeError):
        moe.moe_fp4_linear(x.float(), w.float())
    with pytest.raises(ValueError):
        moe.moe_fp4_linear(x, w[:, :31])
    with pytest.raises(ValueError):
        moe.moe_fp4_linear(x, w, bias=torch.zeros(15, device="cuda"))
    with pytest.raises(TypeError):
        moe.moe_fp4_linear(x, w, residual=dy.float())
    with pytest.raises(moe.MoeFp4Error):
        moe.moe_fp4_linear(x, w, act=9)
    with pytest.raises(ValueError):
        moe.moe_fp4_linear(x, w, accumulate=True)
    with pytest.raises(ValueError):
        moe.moe_fp4_linear_backward(dy, x, w, act=moe.ACT_GELU)
    with pytest.raises(ValueError):
        moe.moe_fp4_linear_backward(dy, None, w)
    with pytest.raises(ValueError):
        moe.moe_fp4_linear_backward(dy, x, w, need_dx=False, need_dw=False, need_db=False)
    with pytest.raises(ValueError):
        moe.moe_fp4_linear_backward(dy, x, w, accumulate=True)
    ws = torch.empty(moe.moe_fp4_linear_workspace_size(4, 16, 32, backward=True) - 1, dtype=torch.uint8, device="cuda")
    with pytest.raises(moe.MoeFp4Error):
        moe.moe_fp4_linear_backward(dy, x, w, workspace=ws)
