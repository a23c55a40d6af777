"""Layer norm and RMS norm with weights, forward and backward, against 64-bit
references: every type, widths from one element to the widest, rows from one,
strides and alignments, accumulation, and the gradients against differences."""
import pytest
import torch

from block_common import U32, bounded, gen, padded, randn

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6
TYPES = [(F32, F32, F32), (F32, BF, F32), (F32, HF, BF), (BF, BF, BF), (BF, BF, F32), (HF, HF, HF)]
TIDS = ["f32", "f32_bf16", "f32_f16_wbf16", "bf16", "bf16_wf32", "f16"]
SHAPES = [(1, 1), (1, 5120), (3, 8), (5, 64), (7, 33), (2, 1000), (9, 1025), (300, 256), (1100, 40), (33, 2048),
          (6, 2056), (5, 4097), (4, 8192), (3, 8200), (2, 16384), (2, 16383), (600, 2304)]


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_routed_expert_router_amd as m
    return m


def forward64(x, gamma, beta, layer):
    mean = x.mean(1, keepdim=True) if layer else torch.zeros_like(x[:, :1])
    d = x - mean
    rstd = 1 / torch.sqrt(d.square().mean(1, keepdim=True) + EPS)
    y = d * rstd
    if gamma is not None:
        y = y * gamma
    if beta is not None:
        y = y + beta
    return y, mean, rstd


def forward_bounds(x, gamma, beta, layer):
    """Bounds of mean, of rstd (relative) and of y before its rounding."""
    H = x.shape[1]
    y, mean, rstd = forward64(x, gamma, beta, layer)
    e_mean = (H * U32 * x.abs().mean(1, keepdim=True) + U32 * mean.abs()) if layer else torch.zeros_like(mean)
    d = (x - mean).abs()
    e_d = e_mean + U32 * (d + e_mean)                       # x - mean, one rounding
    # the sum of squares: H additions and squares, and the errors of x - mean
    e_var = ((2 * d * e_d + e_d * e_d).mean(1, keepdim=True) + (H + 2) * U32 * (d * d).mean(1, keepdim=True))
    rel = 0.5 * e_var * rstd * rstd * 1.1 + 4 * U32          # d(rstd)/rstd = -dvar / (2 (var + eps)); root, division
    g = gamma.abs() if gamma is not None else 1.0
    e_y = (e_d * rstd * (1 + rel) + d * rstd * (rel + 2 * U32)) * g + 2 * U32 * y.abs()
    if beta is not None:
        e_y = e_y + U32 * beta.abs()
    return (y, mean, rstd), (e_y, e_mean, rel * rstd)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("types", TYPES, ids=TIDS)
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward(moe, T, H, types, kind):
    xt, yt, wt = types
    layer = kind == "layer"
    g = gen(T * 31 + H)
    x = (randn(g, T, H) * 2 + 0.5).to(xt)
    for affine in (True, False):
        gamma = randn(g, H, dtype=wt) if affine else None
        beta = randn(g, H, dtype=wt) if affine and layer else None
        y, mean, rstd = moe.moe_fp4_norm(x, gamma, beta, eps=EPS, kind=moe.NORM_LAYER if layer else moe.NORM_RMS,
                                         out_dtype=yt, save_stats=True)
        dbl = lambda t: None if t is None else t.double()
        (wy, wm, wr), (ey, em, er) = forward_bounds(x.double(), dbl(gamma), dbl(beta), layer)
        assert y.dtype == yt
        bounded(y, wy, ey, yt, "y")
        bounded(rstd[:, None], wr, er, F32, "rstd")
        if layer:
            bounded(mean[:, None], wm, em, F32, "mean")
        else:
            assert mean is None


def backward64(dy, x, gamma, mean, rstd, layer):
    """dx, dgamma, dbeta and the bounds of each before its rounding."""
    H, T = x.shape[1], x.shape[0]
    d = x - mean
    xh = d * rstd
    e_xh = U32 * (2 * xh.abs())
    g = dy * gamma if gamma is not None else dy
    e_g = U32 * g.abs()
    a = (g * xh).mean(1, keepdim=True)
    e_a = ((H + 3) * U32 * (g * xh).abs().mean(1, keepdim=True) + (e_g * xh.abs() + g.abs() * e_xh).mean(1, keepdim=True))
    b = g.mean(1, keepdim=True) if layer else torch.zeros_like(a)
    e_b = ((H + 2) * U32 * g.abs().mean(1, keepdim=True) + e_g.mean(1, keepdim=True)) if layer else torch.zeros_like(a)
    dx = rstd * (g - b - xh * a)
    e_dx = rstd * (e_g + e_b + xh.abs() * e_a + e_xh * a.abs() + 3 * U32 * (g.abs() + b.abs() + (xh * a).abs())) + U32 * dx.abs()
    dgamma, dbeta = (dy * xh).sum(0), dy.sum(0)
    e_dg = (T + 2) * U32 * (dy * xh).abs().sum(0) + (dy.abs() * e_xh).sum(0)
    e_db = (T + 2) * U32 * dy.abs().sum(0)
    return (dx, dgamma, dbeta), (e_dx, e_dg, e_db)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("types", TYPES, ids=TIDS)
@pytest.mark.parametrize("T,H", SHAPES)
def test_backward(moe, T, H, types, kind):
    xt, yt, wt = types
    layer = kind == "layer"
    k = moe.NORM_LAYER if layer else moe.NORM_RMS
    g = gen(T * 37 + H)
    x = (randn(g, T, H) * 2 + 0.5).to(xt)
    dy = randn(g, T, H, dtype=yt)
    gamma = randn(g, H, dtype=wt)
    _, m, r = forward64(x.double(), None, None, layer)
    mean, rstd = (m[:, 0].float() if layer else None), r[:, 0].float()
    m64 = mean.double()[:, None] if layer else torch.zeros_like(m)
    (dx, dg, db), (ex, eg, eb) = backward64(dy.double(), x.double(), gamma.double(), m64, rstd.double()[:, None], layer)
    gx, gg, gb = moe.moe_fp4_norm_backward(dy, x, gamma, mean, rstd, kind=k)
    bounded(gx, dx, ex, xt, "dx")
    bounded(gg, dg, eg, F32, "dgamma")
    if layer:
        bounded(gb, db, eb, F32, "dbeta")
    else:
        assert gb is None
    # on top of given gradients
    a0, b0 = randn(g, H), randn(g, H)
    a, b = a0.clone(), b0.clone()
    moe.moe_fp4_norm_backward(dy, x, gamma, mean, rstd, kind=k, need_dx=False, need_dbeta=True, dgamma=a, dbeta=b,
                              accumulate=True)
    bounded(a, dg + a0.double(), eg + U32 * (dg + a0.double()).abs(), F32, "dgamma +=")
    bounded(b, db + b0.double(), eb + U32 * (db + b0.double()).abs(), F32, "dbeta +=")
    # without weights
    (dx, _, _), (ex, _, _) = backward64(dy.double(), x.double(), None, m64, rstd.double()[:, None], layer)
    gx, gg, gb = moe.moe_fp4_norm_backward(dy, x, None, mean, rstd, kind=k)
    assert gg is None and gb is None
    bounded(gx, dx, ex, xt, "dx without weights")


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("H", [64, 33, 2304])
def test_gradients_against_differences(moe, H, kind):
    """f(x, gamma, beta) = sum(y c) in 64 bits: central differences along a random
    direction against the kernels' gradients."""
    layer = kind == "layer"
    k = moe.NORM_LAYER if layer else moe.NORM_RMS
    T = 13
    g = gen(H)
    x, c, gamma, beta = randn(g, T, H), randn(g, T, H), randn(g, H), randn(g, H)
    _, mean, rstd = moe.moe_fp4_norm(x, gamma, beta, eps=EPS, kind=k, save_stats=True)
    dx, dg, db = moe.moe_fp4_norm_backward(c, x, gamma, mean, rstd, kind=k, need_dbeta=True)
    f = lambda a, b, d: (forward64(a, b, d, layer)[0] * c.double()).sum()
    x64, g64, b64 = x.double(), gamma.double(), beta.double()
    h = 2.0 ** -13
    for what, grad, args in (("x", dx, 0), ("gamma", dg, 1), ("beta", db, 2)):
        v = randn(g, *grad.shape).double()
        plus, minus = [x64, g64, b64], [x64, g64, b64]
        plus[args], minus[args] = plus[args] + h * v, minus[args] - h * v
        diff = ((f(*plus) - f(*minus)) / (2 * h)).item()
        got = (grad.double() * v).sum().item()
        # differences: h^2/6 of the third derivative (of order 1 a term here) and 2^-52 / h of f's
        # terms; gradients: H fp32 additions of each term
        scale = (grad.double().abs() * v.abs()).sum().item() + c.double().abs().sum().item()
        assert abs(diff - got) <= (8 * h * h + (H + 16) * U32) * scale, (what, diff, got)


@pytest.mark.parametrize("H", [40, 2304, 1001])
@pytest.mark.parametrize("pad,offset", [(8, 8), (1, 0), (3, 1)])
def test_strides_and_alignment(moe, H, pad, offset):
    g = gen(H + pad)
    T = 21
    x, _ = padded(randn(g, T, H, dtype=BF), pad, offset)
    dy, _ = padded(randn(g, T, H, dtype=BF), pad, offset)
    gamma, beta = randn(g, H, dtype=BF), randn(g, H, dtype=BF)
    y, buf = padded(torch.zeros(T, H, dtype=BF, device="cuda"), pad, offset, fill=7.0)
    moe.moe_fp4_norm(x, gamma, beta, eps=EPS, y=y)
    (wy, m, r), (ey, _, _) = forward_bounds(x.double(), gamma.double(), beta.double(), True)
    bounded(y, wy, ey, BF, "y")
    mean, rstd = m[:, 0].float(), r[:, 0].float()
    dx, buf2 = padded(torch.zeros(T, H, dtype=BF, device="cuda"), pad, offset, fill=7.0)
    _, dg, db = moe.moe_fp4_norm_backward(dy, x, gamma, mean, rstd, dx=dx)
    (wx, wg, wb), (ex, eg, eb) = backward64(dy.double(), x.double(), gamma.double(), mean.double()[:, None],
                                            rstd.double()[:, None], True)
    bounded(dx, wx, ex, BF, "dx")
    bounded(dg, wg, eg, F32, "dgamma")
    bounded(db, wb, eb, F32, "dbeta")
    for out, b in ((y, buf), (dx, buf2)):
        left = b.clone()
        left.as_strided(out.shape, out.stride(), offset).fill_(7.0)
        assert bool((left == 7.0).all())


def test_in_place(moe):
    g = gen(3)
    x, gamma, beta = randn(g, 50, 2304, dtype=BF), randn(g, 2304), randn(g, 2304)
    y, mean, rstd = moe.moe_fp4_norm(x, gamma, beta, save_stats=True)
    x2 = x.clone()
    moe.moe_fp4_norm(x2, gamma, beta, y=x2)
    assert torch.equal(x2, y)
    dy = randn(g, 50, 2304, dtype=BF)
    dx, dg, db = moe.moe_fp4_norm_backward(dy, x, gamma, mean, rstd)
    d2 = dy.clone()
    _, dg2, db2 = moe.moe_fp4_norm_backward(d2, x, gamma, mean, rstd, dx=d2)
    assert torch.equal(d2, dx) and torch.equal(dg, dg2) and torch.equal(db, db2)


def test_rms_without_weights_is_the_pre_norm(moe):
    """The stack's own pre-norm of an fp32 stream: the same numbers but for fp32 roundings."""
    g = gen(4)
    x = randn(g, 17, 5120)
    a = moe.moe_fp4_prenorm_bf16(x, eps=1e-6).double()
    b = moe.moe_fp4_norm(x, kind=moe.NORM_RMS, out_dtype=BF).double()
    # both round values that agree to fp32 accuracy: at most one step apart
    assert bool(((a - b).abs() <= 2.0 ** -7 * a.abs()).all())
    assert (a != b).double().mean().item() < 0.01


def test_large_mean_keeps_its_digits(moe):
    """Values around 1000 with deviations around 1: the variance is that of the deviations."""
    g = gen(6)
    x = randn(g, 8, 4096) + 1000.0
    y, mean, rstd = moe.moe_fp4_norm(x, eps=EPS, save_stats=True)
    (wy, wm, wr), (ey, em, er) = forward_bounds(x.double(), None, None, True)
    assert ((rstd.double() - wr[:, 0]).abs() / wr[:, 0]).max().item() < 1e-5
    bounded(y, wy, ey, F32, "y")


def test_rows_with_nan_or_inf_stay_alone(moe):
    g = gen(8)
    x = randn(g, 40, 300, dtype=BF)
    x[3, 7], x[20, 0] = float("nan"), float("inf")
    y = moe.moe_fp4_norm(x)
    assert (~torch.isfinite(y).all(1)).nonzero().flatten().tolist() == [3, 20]


def test_constant_and_zero_rows(moe):
    x = torch.zeros(4, 512, device="cuda")
    x[1] = 3.0
    y, mean, rstd = moe.moe_fp4_norm(x, eps=1e-6, save_stats=True)
    assert bool((y == 0).all()) and mean.tolist()[:2] == [0.0, 3.0]
    assert torch.allclose(rstd, torch.full_like(rstd, 1e3), rtol=1e-6)


def test_no_rows(moe):
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    gamma = torch.ones(64, dtype=BF, device="cuda")
    y, mean, rstd = moe.moe_fp4_norm(x, gamma, gamma, save_stats=True)
    assert y.shape == (0, 64) and mean.shape == (0,)
    dx, dg, db = moe.moe_fp4_norm_backward(x, x, gamma, mean, rstd)
    assert dx.shape == (0, 64) and bool((dg == 0).all()) and bool((db == 0).all())


def test_same_bits_twice(moe):
    g = gen(9)
    x, dy, gamma = randn(g, 3000, 1280, dtype=BF), randn(g, 3000, 1280, dtype=BF), randn(g, 1280)
    _, mean, rstd = moe.moe_fp4_norm(x, save_stats=True)
    one = moe.moe_fp4_norm_backward(dy, x, gamma, mean, rstd)
    two = moe.moe_fp4_norm_backward(dy, x, gamma, mean, rstd)
    assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_binding_refusals(moe):
    x = torch.zeros(4, 64, dtype=BF, device="cuda")
    with pytest.raises(TypeError):
        moe.moe_fp4_norm(x, out_dtype=F32)
    with pytest.raises(TypeError):
        moe.moe_fp4_norm(x.double())
    with pytest.raises(ValueError):
        moe.moe_fp4_norm(x, torch.ones(63, dtype=BF, device="cuda"))
    with pytest.raises(TypeError):
        moe.moe_fp4_norm(x, torch.ones(64, dtype=BF, device="cuda"), torch.ones(64, device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_fp4_norm(x.t())
    with pytest.raises(moe.MoeFp4Error):
        moe.moe_fp4_norm(x, eps=-1.0)
    with pytest.raises(moe.MoeFp4Error):
        moe.moe_fp4_norm(x, kind=2)
    with pytest.raises(moe.MoeFp4Error):
        moe.moe_fp4_norm(torch.zeros(2, 16385, device="cuda"))
    r = torch.ones(4, device="cuda")
    with pytest.raises(TypeError):
        moe.moe_fp4_norm_backward(x, x, None, None, r)
    with pytest.raises(ValueError):
        moe.moe_fp4_norm_backward(x, x, None, r, r, need_dx=False)
    with pytest.raises(ValueError):
        moe.moe_fp4_norm_backward(x, x, x[0].contiguous(), r, r, accumulate=True)
