"""The operators around the routed experts at the ends of their types' ranges."""
import pytest
import torch

from block_common import U32, bounded, gen, half_step, randn, slope64

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_routed_expert_router_amd as m
    return m


@pytest.mark.parametrize("dyt", ["same", "f32"])
@pytest.mark.parametrize("dt", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_slopes_far_from_zero(moe, act, dt, dyt):
    """The slope is 1 far above zero and 0 far below, also where z^2 or z^3 passes fp32
    and where the kept z is infinite (a pre-activation of -7e4 is -inf in fp16, and its
    activation -0).  At |z| >= 200 both are exact: what is left out is below e^-199.  dy
    and w are small whole numbers, so every product and sum is exact too."""
    far = [200.0, -200.0, 6e4, -6e4, float("inf"), float("-inf")]
    if dt == BF:
        far += [1e13, -1e13, 1.9e19, -1.9e19, 3e38, -3e38]
    z = torch.tensor([far, far[::-1], [-v for v in far]], device="cuda").to(dt)
    M, N = z.shape
    K = 24
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    ints = lambda *s: torch.randint(-4, 5, s, generator=g, device="cuda")
    dy, x, w = ints(M, N).to(dt if dyt == "same" else F32), ints(M, K).to(dt), ints(N, K).to(dt)
    a = {"gelu": moe.ACT_GELU, "gelu_tanh": moe.ACT_GELU_TANH, "silu": moe.ACT_SILU}[act]
    dx, dw, db = moe.moe_fp4_linear_backward(dy, x, w, z=z, act=a, dw_dtype=F32)
    dz = torch.where(z > 0, dy.double(), torch.zeros_like(dy.double()))
    assert torch.equal(db.double(), dz.sum(0))
    assert torch.equal(dx.double(), dz @ w.double())
    assert torch.equal(dw.double(), dz.t() @ x.double())


@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_slope_of_nan_is_nan(moe, act):
    z = torch.zeros(2, 8, dtype=BF, device="cuda")
    z[1, 3] = float("nan")
    a = {"gelu": moe.ACT_GELU, "gelu_tanh": moe.ACT_GELU_TANH, "silu": moe.ACT_SILU}[act]
    dy, w = torch.ones(2, 8, dtype=BF, device="cuda"), torch.ones(8, 8, dtype=BF, device="cuda")
    dx, _, db = moe.moe_fp4_linear_backward(dy, None, w, z=z, act=a, need_dw=False)
    assert torch.isnan(db).tolist() == [False] * 3 + [True] + [False] * 4
    assert torch.isnan(dx).all(1).tolist() == [False, True]


def backward64(dy, x, w, z, act, top=None):
    """dx, dw, db of fp16 operands in 64 bits, and bounds of each before its rounding.

    dz = dy act'(z) is rounded to fp16 after a power of two that brings its largest
    finite magnitude `top` into [2^14, 2^15): off by half a step of the value, or of the
    smallest numbers of the type, 2^-25 after that power, at most 2^-39 top before it.
    The products' additions keep steps of 2^-14 below it (terms are aligned by exponent
    field): of 2^-28 top at most on the side of dz."""
    M, N = dy.shape
    if act == "none":
        dz, e = dy, torch.zeros_like(dy)
    else:
        # the slope's evaluation; its terms cancel where it is small, so relative to 1 + |z|
        dz = dy * slope64(z, act)
        e = dy.abs() * (16 + 8 * z.abs()) * U32 * 1.2
    e_db = e.sum(0) + (M + 1) * U32 * (dz.abs() + e).sum(0)
    top = dz.abs().max() if top is None else top
    e16 = e + torch.maximum(half_step(HF) * (dz.abs() + e), 2.0 ** -39 * top)
    mag = torch.maximum(dz.abs() + e16, 2.0 ** -28 * top)
    up = lambda v: v.abs().clamp(min=2.0 ** -14)
    e_dx = e16 @ w.abs() + N * U32 * (mag @ up(w))
    e_dw = e16.t() @ x.abs() + M * U32 * (mag.t() @ up(x))
    return (dz @ w, dz.t() @ x, dz.sum(0)), (e_dx, e_dw, e_db)


DZ_SHAPES = [(1, 16, 32), (3, 7, 5), (70, 96, 128), (100, 101, 115), (300, 520, 264), (4100, 33, 25), (5, 4096, 64),
             (600, 2056, 1544)]


@pytest.mark.parametrize("power", [-60, -30, -18, 0, 18, 60, "mixed"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu"])
@pytest.mark.parametrize("M,N,K", DZ_SHAPES)
def test_fp32_gradients_into_fp16_products(moe, M, N, K, act, power):
    """dy in fp32 passes fp16's range at both ends; dw and db are fp32 and hold the answer."""
    g = gen(M + N + K)
    x, w, z = randn(g, M, K, dtype=HF), randn(g, N, K, dtype=HF, scale=2.0 ** -12), randn(g, M, N, dtype=HF)
    dy = randn(g, M, N)
    if power == "mixed":  # gradients of very different size next to each other
        dy *= torch.exp2(torch.randint(-30, 19, (M, N), generator=g, device="cuda").float())
    else:
        dy *= 2.0 ** power
    a = {"none": moe.ACT_NONE, "silu": moe.ACT_SILU, "gelu": moe.ACT_GELU}[act]
    (wx, ww, wb), (ex, ew, eb) = backward64(dy.double(), x.double(), w.double(), z.double(), act)
    holds = wx.abs().max().item() < 60000  # dx is fp16
    dx, dw, db = moe.moe_fp4_linear_backward(dy, x, w, z=z, act=a, dw_dtype=F32, need_dx=holds)
    if holds:
        bounded(dx, wx, ex, HF, "dx")
    bounded(dw, ww, ew, F32, "dw")
    bounded(db, wb, eb, F32, "db")
    more = dw.clone()
    moe.moe_fp4_linear_backward(dy, x, w, z=z, act=a, dw=more, need_dx=False, need_db=False, accumulate=True)
    bounded(more, ww + dw.double(), ew + U32 * ww.abs(), F32, "dw +=")


@pytest.mark.parametrize("power", [-22, 0])
@pytest.mark.parametrize("M,N,K", DZ_SHAPES)
def test_small_fp16_gradients(moe, M, N, K, power):
    """dy in fp16 near its smallest numbers: the slope's digits are not lost."""
    g = gen(M + N + K + 1)
    x, w, z = randn(g, M, K, dtype=HF), randn(g, N, K, dtype=HF), randn(g, M, N, dtype=HF)
    dy = (randn(g, M, N) * 2.0 ** power).to(HF)
    (wx, ww, wb), (ex, ew, eb) = backward64(dy.double(), x.double(), w.double(), z.double(), "silu")
    dx, dw, db = moe.moe_fp4_linear_backward(dy, x, w, z=z, act=moe.ACT_SILU, dw_dtype=F32)
    bounded(dx, wx, ex, HF, "dx")
    bounded(dw, ww, ew, F32, "dw")
    bounded(db, wb, eb, F32, "db")


@pytest.mark.parametrize("dyt", [HF, F32], ids=["f16", "f32"])
def test_an_infinite_gradient_stays_in_its_row(moe, dyt):
    """The power of two goes by the finite values: the other rows keep theirs."""
    g = gen(11)
    M, N, K = 70, 96, 128
    x, w, z = randn(g, M, K, dtype=HF), randn(g, N, K, dtype=HF), randn(g, M, N, dtype=HF)
    dy = randn(g, M, N, dtype=dyt)
    dy[7, 5], dy[20, 3], dy[21, 90] = float("inf"), float("nan"), float("-inf")
    dx, _, db = moe.moe_fp4_linear_backward(dy, x, w, z=z, act=moe.ACT_SILU)
    ok = torch.isfinite(dy).all(1)
    assert (~torch.isfinite(dx).all(1)).nonzero().flatten().tolist() == [7, 20, 21]
    dz = dy.double() * slope64(z.double(), "silu")
    top = dz[torch.isfinite(dz)].abs().max()
    (wx, _, _), (ex, _, _) = backward64(dy[ok].double(), x[ok].double(), w.double(), z[ok].double(), "silu", top)
    bounded(dx[ok], wx, ex, HF, "dx")
    assert (~torch.isfinite(db)).nonzero().flatten().tolist() == [3, 5, 90]


@pytest.mark.parametrize("value", [0.0, 1e-45, 3.4e38])
def test_gradients_at_the_ends_of_fp32(moe, value):
    g = gen(12)
    M, N, K = 9, 8, 16
    x, w = torch.ones(M, K, dtype=HF, device="cuda"), torch.ones(N, K, dtype=HF, device="cuda")
    dy = torch.zeros(M, N, device="cuda")
    dy[4, 2] = value
    _, dw, db = moe.moe_fp4_linear_backward(dy, x, w, need_dx=False, dw_dtype=F32)
    # one term each: 2^126 is the largest power, so the smallest fp32 numbers lie 2^-23
    # below 1 there and fp16 keeps them to 2^-25
    want = torch.zeros(N, K, dtype=torch.float64, device="cuda")
    want[2] = dy[4, 2].double()
    lim = half_step(HF) * want.abs() + 2.0 ** -151
    assert bool(((dw.double() - want).abs() <= lim).all())
    assert torch.equal(db, dy.sum(0))


@pytest.mark.parametrize("types", [(F32, F32), (F32, BF), (BF, BF), (HF, HF)], ids=["f32", "f32_bf16", "bf16", "f16"])
@pytest.mark.parametrize("H", [1, 7, 33, 200, 1000, 1024, 2304, 4095, 5120, 8192, 16383, 16384])
def test_constant_rows_far_from_zero(moe, H, types):
    """Rows of one value have no deviations, whatever the rounding of their sum: y = 0.

    A row's sum passes at most n = 48 additions one after another (24 or fewer of a
    thread, 6 of a wave, 16 waves, the product by 1 / H), so the first mean is off by
    n U |c| and what the second step leaves of that by n U of it; the deviations are
    divided by sqrt(eps) at least."""
    xt, yt = types
    values = [1000.1, -3.3, 123456.7, 1000000.3, -0.1, 7e-4]
    if xt == HF:
        values = [1000.1, -3.3, 65504.0, -0.1, 7e-4]
    c = torch.tensor(values, device="cuda").to(xt)
    x = c[:, None].expand(-1, H).contiguous()
    y, mean, rstd = moe.moe_fp4_norm(x, eps=EPS, out_dtype=yt, save_stats=True)
    c = c.double()
    left = (48 * U32) ** 2 * c.abs()
    assert bool((y.double().abs() <= 1.02 * left[:, None] / EPS ** 0.5 + 2.0 ** -25).all()), y.abs().max(1)
    assert bool(((mean.double() - c).abs() <= U32 * c.abs() + left).all())
    # the variance: the squares of the first deviations, n U |c| at most, cancel to n U of them
    var = 50 * U32 * (48 * U32 * c) ** 2
    want = EPS ** -0.5
    near = var < 1e-3 * EPS
    assert bool(((rstd.double() - want).abs() <= (0.51 * var / EPS + 8 * U32) * want)[near].all())


@pytest.mark.parametrize("H", [1000, 5120])
def test_one_element_apart_from_a_constant_row(moe, H):
    """One element a step off the others: its own deviation is what is left."""
    c = 1000.1
    x = torch.full((1, H), c, device="cuda")
    x[0, 17] += 0.25
    y, mean, rstd = moe.moe_fp4_norm(x, eps=EPS, save_stats=True)
    x64 = x.double()
    d = x64 - x64.mean(1, keepdim=True)
    r = 1 / torch.sqrt(d.square().mean(1, keepdim=True) + EPS)
    # deviations off by (48 U)^2 of the mean and a step of themselves, the variance by 52 U
    # of it and by 50 U of the first deviations' square, (48 U c)^2
    ed = (48 * U32) ** 2 * c + 2 * U32 * d.abs()
    ev = 52 * U32 * d.square().mean() + 50 * U32 * (48 * U32 * c) ** 2 + 2 * (d.abs() * ed).mean()
    rel = 0.51 * ev * r * r + 8 * U32
    assert bool(((y.double() - d * r).abs() <= 1.02 * (ed * r + (d * r).abs() * (rel + 4 * U32))).all())


def test_fp16_gradients_in_a_captured_graph(moe):
    """The power of two is found on the device: a replay goes by the gradients of that
    replay.  Two graphs with workspaces of their own, eager calls between."""
    g = gen(13)
    M, N, K = 300, 520, 264
    x, w, z = randn(g, M, K, dtype=HF), randn(g, N, K, dtype=HF, scale=2.0 ** -12), randn(g, M, N, dtype=HF)
    dys = [torch.zeros(M, N, device="cuda") for _ in range(2)]
    call = lambda dy: moe.moe_fp4_linear_backward(dy, x, w, z=z, act=moe.ACT_SILU, dw_dtype=F32)
    call(dys[0])
    torch.cuda.synchronize()
    graphs, outs = [], []
    for dy in dys:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(call(dy))
        graphs.append(graph)
    for power in (0, 17, -40, 12, -12):
        for i, dy in enumerate(dys):
            dy.copy_(randn(g, M, N) * 2.0 ** (power + 3 * i))
        want = [call(dy) for dy in dys]
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for got, ref in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(got, ref)), power
            assert all(bool(torch.isfinite(a).all()) for a in got)


@pytest.mark.parametrize("dyt", [HF, F32], ids=["f16", "f32"])
def test_no_rows_of_fp16_gradients(moe, dyt):
    x, w = torch.empty(0, 64, dtype=HF, device="cuda"), torch.ones(32, 64, dtype=HF, device="cuda")
    dy, z = torch.empty(0, 32, dtype=dyt, device="cuda"), torch.empty(0, 32, dtype=HF, device="cuda")
    dx, dw, db = moe.moe_fp4_linear_backward(dy, x, w, z=z, act=moe.ACT_SILU)
    assert dx.shape == (0, 64) and bool((dw == 0).all()) and bool((db == 0).all())


@pytest.mark.parametrize("dt", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("dyt", ["same", "f32"])
@pytest.mark.parametrize("act", ["none", "silu", "gelu", "gelu_tanh", "relu"])
def test_dz_is_rounded_once(moe, act, dyt, dt):
    """What dx and dw add to the roundings of their sums and results is dz's one rounding,
    of half a step: a product with the identity brings out the rounded dz, and dx and dw
    are its products."""
    g = gen(17)
    M, N, K = 260, 136, 328
    a = {"none": moe.ACT_NONE, "silu": moe.ACT_SILU, "gelu": moe.ACT_GELU, "gelu_tanh": moe.ACT_GELU_TANH,
         "relu": moe.ACT_RELU}[act]
    x, w, z = randn(g, M, K, dtype=dt), randn(g, N, K, dtype=dt), randn(g, M, N, dtype=dt)
    dy = randn(g, M, N, dtype=dt if dyt == "same" else F32)
    one = torch.eye(N, device="cuda").to(dt)
    dz, _, _ = moe.moe_fp4_linear_backward(dy, None, one, z=z, act=a, need_dw=False, need_db=False)
    s = torch.ones_like(z.double()) if act == "none" else slope64(z.double(), act)
    e = 0 if act in ("none", "relu") else dy.double().abs() * (16 + 8 * z.double().abs()) * U32 * 1.2  # the slope's own
    bounded(dz, dy.double() * s, torch.zeros_like(s) + e, dt, "dz")
    dx, dw, _ = moe.moe_fp4_linear_backward(dy, x, w, z=z, act=a, dw_dtype=F32, need_db=False)
    dz, x, w = dz.double(), x.double(), w.double()
    # fp16 takes steps of 2^-14 of a value below it, and dz has been 2^12 and more times itself there
    low = 2.0 ** -14 if dt == HF else 0.0
    bounded(dx, dz @ w, N * U32 * (dz.abs().clamp(min=low) @ w.abs().clamp(min=low)), dt, "dx")
    bounded(dw, dz.t() @ x, M * U32 * (dz.t().abs().clamp(min=low) @ x.abs().clamp(min=low)), F32, "dw")
