"""The dense product with 4-bit weights against 64 bits: both codes, every scale type
and group, one row to many, odd outputs, short sums and groups cut by the row's end,
strides, zero points, scales at the ends of their range."""
import pytest
import torch

from block_common import U32, act64, bounded, gen, padded, randn

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
SLOPE, SUBN = 1.15, 2.0 ** -100
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
KINDS = [("mx", 32, None), ("int4", 32, BF), ("int4", 64, HF), ("int4", 128, F32), ("int4", 256, BF)]
IDS = [f"{c}_{n}" for c, n, _ in KINDS]


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_routed_expert_router_amd as m
    return m


def weights(moe, g, N, K, kind, zeros=False):
    """W4Weights, and in 64 bits the weights and the magnitudes whose sums are rounded."""
    code, group, st = kind
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    G = (K + group - 1) // group
    z = None
    if code == "mx":
        scales = torch.randint(110, 130, (N, G), generator=g, device="cuda", dtype=torch.uint8)
    else:
        scales = (0.02 + torch.rand(N, G, generator=g, device="cuda")).to(st)
        z = torch.randint(0, 256 if zeros == "any" else 16, (N, G), generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    w = moe.W4Weights(codes, scales, z, group)
    return (w,) + weights64(w)


def weights64(w):
    c = torch.stack([w.codes & 15, w.codes >> 4], dim=2).reshape(w.N, w.K).long()
    up = lambda t: t.double().repeat_interleave(w.group, 1)[:, :w.K]
    if w.scales.dtype == torch.uint8:
        v = torch.tensor(E2M1 + [-a for a in E2M1], dtype=torch.float64, device="cuda")[c]
        s = torch.exp2(up(w.scales) - 127)
        return v * s, (v * s).abs()
    z = up(w.zeros) if w.zeros is not None else 8.0
    return (c.double() - z) * up(w.scales), (c.double() + z) * up(w.scales).abs()


def check(moe, x, w, w64, mag, out, act="none", bias=None, residual=None, y=None):
    K = x.shape[1]
    got = moe.moe_fp4_linear_w4(x, w, bias=bias, act=getattr(moe, "ACT_" + act.upper()), residual=residual, out_dtype=out, y=y)
    z = x.double() @ w64.t()
    # K terms, and for every group of 32 at most a scale's product and two additions
    e = (K + K // 8 + 8) * U32 * (x.double().abs() @ mag.t())
    if bias is not None:
        z = z + bias.double()
        e = e + U32 * (z.abs() + bias.double().abs())
    a = act64(z, act)
    if act != "none":
        e = SLOPE * e
    if act not in ("none", "relu"):
        e = e + (16 + 4 * z.abs()) * U32 * (a.abs() + SUBN)
    if residual is not None:
        a, e = a + residual.double(), e + U32 * (a.abs() + residual.double().abs())
    bounded(got, a, e, out or x.dtype, f"{act} {out}")
    return got


SHAPES = [(1, 1, 32), (1, 16, 5120), (1, 288, 5120), (2, 33, 64), (3, 100, 96), (5, 17, 2304), (15, 130, 160), (16, 64, 1024),
          (17, 40, 288), (33, 31, 640), (48, 129, 544), (64, 512, 256), (65, 20, 416), (130, 72, 1184), (1, 2304, 4640),
          (8, 5120, 512), (300, 16, 64), (1, 70, 16384)]


@pytest.mark.parametrize("dt", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(moe, M, N, K, kind, dt):
    g = gen(M + N + K)
    x = randn(g, M, K, dtype=dt)
    w, w64, mag = weights(moe, g, N, K, kind)
    check(moe, x, w, w64, mag, F32)
    if kind[0] == "int4":
        w, w64, mag = weights(moe, g, N, K, kind, zeros=True)
    check(moe, x, w, w64, mag, dt if kind[0] == "mx" else F32, act="gelu", bias=randn(g, N, dtype=BF))
    check(moe, x, w, w64, mag, F32, act="silu", bias=randn(g, N), residual=randn(g, M, N))


@pytest.mark.parametrize("dt", [BF, HF], ids=["bf16", "f16"])
def test_every_code_exactly(moe, dt):
    """Whole-number x of one element at a time: each weight comes back exactly."""
    K = 256
    x = torch.eye(K, dtype=dt, device="cuda")[:, :]
    codes = torch.arange(256, device="cuda", dtype=torch.uint8).repeat(16, 1)[:, :K // 2].contiguous()
    codes[1::2] = 255 - codes[1::2]
    for kind in KINDS:
        code, group, st = kind
        G = (K + group - 1) // group
        if code == "mx":
            w = moe.W4Weights(codes, torch.arange(120, 120 + 16 * G, device="cuda").remainder(16).add(120).to(torch.uint8).view(16, G))
        else:
            z = torch.arange(16 * G, device="cuda").remainder(16).to(torch.uint8).view(16, G)
            w = moe.W4Weights(codes, (2.0 ** (torch.arange(16 * G, device="cuda") % 5 - 2)).view(16, G).to(st), z, group)
        w64, _ = weights64(w)
        for rows in (slice(0, 1), slice(100, 116), slice(0, 256)):
            y = moe.moe_fp4_linear_w4(x[rows], w, out_dtype=F32)
            assert torch.equal(y.double(), w64.t()[rows]), (kind, rows)


@pytest.mark.parametrize("dt", [BF, HF], ids=["bf16", "f16"])
def test_scales_at_their_ends(moe, dt):
    """UE8M0 bytes 2 and 252 beside others: products and sums stay in fp32's range."""
    g = gen(4)
    codes = torch.randint(0, 256, (3, 64), generator=g, device="cuda", dtype=torch.uint8)
    x = randn(g, 4, 128, dtype=dt)
    for lo, hi in ((2, 3), (200, 245), (2, 100)):
        scales = torch.randint(lo, hi, (3, 4), generator=g, device="cuda", dtype=torch.uint8)
        w = moe.W4Weights(codes, scales)
        check(moe, x, w, *weights64(w), F32)
    scales = torch.full((3, 4), 252, dtype=torch.uint8, device="cuda")
    w = moe.W4Weights(codes, scales)
    small = (x * 2.0 ** -9).to(dt)
    check(moe, small, w, *weights64(w), F32)


@pytest.mark.parametrize("dt", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(3, 16384, 32), (16, 16385, 96), (7, 16400, 1184), (16, 20001, 2080), (5, 65536, 160),
                                   (11, 16384, 4992), (4, 16389, 5152), (16, 16384, 10336), (40, 20500, 96),
                                   (64, 20485, 5120), (70, 20480, 1184), (33, 20481, 640), (20, 32769, 160), (32, 32800, 2336),
                                   (16, 49153, 416), (3, 49160, 1024), (9, 8193, 288), (16, 9216, 5120), (100, 20480, 32)])
def test_many_columns(moe, M, N, K, kind, dt):
    """Wide weights, whose short last tile overlaps the one before; sums of one to three
    chunks; rows shared through LDS."""
    g = gen(M + N + K)
    x = randn(g, M, K, dtype=dt)
    w, w64, mag = weights(moe, g, N, K, kind, zeros=kind[0] == "int4" and M % 2 == 1)
    check(moe, x, w, w64, mag, dt if kind[0] == "mx" else F32, act="silu", bias=randn(g, N, dtype=BF))
    r = randn(g, M, N)
    y, buf = padded(r, 3, 1, fill=7.0)
    check(moe, x, w, w64, mag, F32, residual=r, y=y)
    left = buf.clone()
    left.as_strided(y.shape, y.stride(), 1).fill_(7.0)
    assert bool((left == 7.0).all())


def test_zero_points_of_any_byte(moe):
    g = gen(5)
    for kind in KINDS[1:]:
        w, w64, mag = weights(moe, g, 40, 416, kind, zeros="any")
        for M in (1, 20):
            check(moe, randn(g, M, 416, dtype=BF), w, w64, mag, F32)


@pytest.mark.parametrize("M", [1, 9, 40])
@pytest.mark.parametrize("pad,offset", [(8, 8), (1, 0), (3, 5)])
@pytest.mark.parametrize("kind", [KINDS[0], KINDS[2]], ids=["mx", "int4"])
def test_strides_and_alignment(moe, M, pad, offset, kind):
    g = gen(M + pad)
    N, K = 70, 352
    w, w64, mag = weights(moe, g, N, K, kind)
    wide = torch.full((N, 256), 0xFF, dtype=torch.uint8, device="cuda")
    wide[:, :K // 2] = w.codes
    w = moe.W4Weights(wide[:, :K // 2], w.scales, w.zeros, w.group)
    x, _ = padded(randn(g, M, K, dtype=BF), pad, offset)
    r, _ = padded(randn(g, M, N, dtype=BF), pad, offset)
    y, buf = padded(torch.zeros(M, N, dtype=BF, device="cuda"), pad, offset, fill=7.0)
    check(moe, x, w, w64, mag, None, act="silu", residual=r, y=y)
    left = buf.clone()
    left.as_strided(y.shape, y.stride(), offset).fill_(7.0)
    assert bool((left == 7.0).all())


def test_residual_in_place_and_accumulate(moe):
    g = gen(6)
    for kind in KINDS[:2]:
        for M in (1, 30):
            w, w64, mag = weights(moe, g, 48, 320, kind)
            x, r = randn(g, M, 320, dtype=BF), randn(g, M, 48)
            want = moe.moe_fp4_linear_w4(x, w, residual=r, out_dtype=F32)
            y = r.clone()
            moe.moe_fp4_linear_w4(x, w, residual=y, y=y)
            assert torch.equal(y, want)
            y = r.clone()
            moe.moe_fp4_linear_w4(x, w, y=y, accumulate=True)
            assert torch.equal(y, want)


def test_rows_do_not_meet(moe):
    """A row's result is its own: NaN and infinities in other rows of x do not show."""
    g = gen(7)
    for kind in KINDS:
        w, _, _ = weights(moe, g, 40, 288, kind)
        x = randn(g, 37, 288, dtype=BF)
        want = moe.moe_fp4_linear_w4(x, w, out_dtype=F32)
        bad = x.clone()
        bad[5], bad[30, 7] = float("nan"), float("inf")
        got = moe.moe_fp4_linear_w4(bad, w, out_dtype=F32)
        keep = [i for i in range(37) if i not in (5, 30)]
        assert torch.equal(got[keep], want[keep]) and not bool(torch.isfinite(got[5]).any())


def test_experts_weights_are_dense_ones(moe):
    """An expert's w1 of the layer, as it is stored: h of the layer's definition from two products."""
    g = gen(8)
    H, I = 256, 96
    codes = torch.randint(0, 256, (3, I, H // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(118, 124, (3, I, H // 32), generator=g, device="cuda", dtype=torch.uint8)
    x = randn(g, 4, H, dtype=BF)
    w = moe.W4Weights(codes[1], scales[1])
    check(moe, x, w, *weights64(w), BF)


def test_no_rows_and_refusals(moe):
    g = gen(9)
    w, _, _ = weights(moe, g, 24, 64, KINDS[0])
    assert moe.moe_fp4_linear_w4(torch.empty(0, 64, dtype=BF, device="cuda"), w).shape == (0, 24)
    x = torch.zeros(2, 64, dtype=BF, device="cuda")
    with pytest.raises(TypeError):
        moe.moe_fp4_linear_w4(x.float(), w)
    with pytest.raises(ValueError):
        moe.moe_fp4_linear_w4(x[:, :32], w)
    with pytest.raises(TypeError):
        moe.moe_fp4_linear_w4(x, w.codes)
    with pytest.raises(TypeError):
        moe.moe_fp4_linear_w4(x, w, out_dtype=HF)
    with pytest.raises(ValueError):
        moe.moe_fp4_linear_w4(x, w, accumulate=True)
    with pytest.raises(ValueError):
        moe.W4Weights(w.codes, w.scales, group=64)
    with pytest.raises(ValueError):
        moe.W4Weights(w.codes, w.scales, zeros=w.scales)
    with pytest.raises(ValueError):
        moe.W4Weights(w.codes, torch.ones(24, 1, device="cuda"), group=48)
    with pytest.raises(moe.MoeFp4Error):
        moe.moe_fp4_linear_w4(torch.zeros(2, 40, dtype=BF, device="cuda"),
                              moe.W4Weights(torch.zeros(4, 20, dtype=torch.uint8, device="cuda"), torch.ones(4, 2, device="cuda")))
    with pytest.raises(moe.MoeFp4Error):
        odd = torch.zeros(24 * 32 + 8, dtype=torch.uint8, device="cuda")[8:].view(24, 32)
        moe.moe_fp4_linear_w4(x, moe.W4Weights(odd, w.scales))


def test_most_rows(moe):
    """2^20 rows: more than a grid's second dimension holds of single tiles."""
    g = gen(11)
    M, N, K = 1 << 20, 17, 64
    w, w64, mag = weights(moe, g, N, K, KINDS[0])
    x = randn(g, M, K, dtype=BF)
    y = moe.moe_fp4_linear_w4(x, w, out_dtype=F32)
    tail = slice(M - 200, M)
    bounded(y[tail], x[tail].double() @ w64.t(), (K + 16) * U32 * (x[tail].double().abs() @ mag.t()), F32, "last rows")
    assert torch.equal(y[:40], moe.moe_fp4_linear_w4(x[:40], w, out_dtype=F32))


def test_codes_past_32_bits(moe):
    """65536 rows 128 KB apart: byte offsets past 2^32."""
    N, K = 65536, 64
    free, _ = torch.cuda.mem_get_info()
    if free < 12 << 30:
        pytest.skip("needs 12 GB")
    g = gen(10)
    buf = torch.zeros(N, 131072, dtype=torch.uint8, device="cuda")
    buf[:, :K // 2] = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    w = moe.W4Weights(buf[:, :K // 2], torch.randint(118, 124, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8))
    for M in (1, 20):
        check(moe, randn(g, M, K, dtype=BF), w, *weights64(w), F32)


# one and two rows, tiles, rows held in registers, rows shared through LDS
EACH_KERNEL = [(1, 70, 1024), (2, 300, 1056), (4, 70, 160), (30, 530, 160), (3, 16390, 160), (20, 32769, 160), (40, 20485, 160)]


@pytest.mark.parametrize("dt", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("M,N,K", EACH_KERNEL)
def test_scales_at_their_ends_in_each_kernel(moe, M, N, K, dt):
    """UE8M0 bytes 2 and 252, alone and beside others.  252: |x| below 2^-10 keeps a sum of 1056
    terms up to 6 * 2^125 in fp32's range."""
    g = gen(M + N)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    x = randn(g, M, K, dtype=dt)
    for lo, hi in ((2, 3), (200, 245), (2, 100)):
        w = moe.W4Weights(codes, torch.randint(lo, hi, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8))
        check(moe, x, w, *weights64(w), F32)
    w = moe.W4Weights(codes, torch.full((N, K // 32), 252, dtype=torch.uint8, device="cuda"))
    check(moe, (x.float() * 2.0 ** -13).to(dt), w, *weights64(w), F32)


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("M,N,K", EACH_KERNEL)
def test_fp16_below_its_normal_numbers(moe, M, N, K, kind):
    """x of subnormal fp16 alone: its products with the codes are exact in fp32 all the same."""
    g = gen(M + N + 1)
    x = (randn(g, M, K) * 2.0 ** -18).to(HF)
    w, w64, mag = weights(moe, g, N, K, kind, zeros=kind[0] == "int4")
    check(moe, x, w, w64, mag, F32)


@pytest.mark.parametrize("kind", KINDS, ids=IDS)
@pytest.mark.parametrize("M,N,K", [(1, 40, 65536), (2, 33, 40000), (5, 40, 65536), (20, 50, 32800), (4, 16390, 15392), (18, 32770, 10240)])
def test_long_sums(moe, M, N, K, kind):
    """The most inputs, more than a workgroup's threads or chunks take at once."""
    g = gen(M + N)
    w, w64, mag = weights(moe, g, N, K, kind, zeros=kind[0] == "int4")
    check(moe, randn(g, M, K, dtype=BF), w, w64, mag, F32)
