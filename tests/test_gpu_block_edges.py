"""The products at their edges: sums and rows a few elements off the widths of
the kernels' chunks and tiles, results off the 16-byte grid from operands on it,
fp16 values below the normal range, and the largest row strides."""
import pytest
import torch

from block_common import U32, bounded, gen, offsets_of, padded, randn

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_routed_expert_router_amd as m
    return m


def mm(a, b):
    """A product in 64 bits and the sum of its terms' magnitudes."""
    a, b = a.double(), b.double()
    return a @ b, a.abs() @ b.abs()


def untouched(buf, view, offset):
    left = buf.clone()
    left.as_strided(view.shape, view.stride(), offset).fill_(7.0)
    return bool((left == 7.0).all())


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 63, 64, 65, 71, 129])
@pytest.mark.parametrize("m", [1, 4, 20, 70])
def test_sums_and_widths_near_a_chunk(moe, m, n):
    """Each of the three sizes near a chunk's, NaN behind every row's end."""
    g = gen(100 * m + n)
    for N, K in ((n, 130), (130, n), (n, n), (n, 7), (5, n)):
        x, _ = padded(randn(g, m, K, dtype=BF), 3, 1)
        w, _ = padded(randn(g, N, K, dtype=BF), 5, 3)
        dy, _ = padded(randn(g, m, N, dtype=BF), 1, 5)
        y = moe.moe_fp4_linear(x, w, out_dtype=F32)
        dx, dw, db = moe.moe_fp4_linear_backward(dy, x, w, dw_dtype=F32)
        want, s = mm(x, w.t())
        bounded(y, want, K * U32 * s, F32, "y")
        want, s = mm(dy, w)
        bounded(dx, want, N * U32 * s, BF, "dx")
        want, s = mm(dy.t(), x)
        bounded(dw, want, m * U32 * s, F32, "dw")
        bounded(db, dy.double().sum(0), (m + 1) * U32 * dy.double().abs().sum(0), F32, "db")


@pytest.mark.parametrize("offset,pad", [(1, 0), (4, 3), (0, 4), (2, 8)])
@pytest.mark.parametrize("rows", [40, 300, 2100])
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
def test_results_off_the_grid(moe, rows, offset, pad, out):
    """Aligned operands, so the tiles that load into LDS directly, and results of any alignment."""
    g = gen(rows + offset)
    N, K = 512, 264
    counts = [rows // 3, 0, rows - rows // 3]
    off = offsets_of(counts)
    x, dy, w = randn(g, rows, K, dtype=BF), randn(g, rows, N, dtype=BF), randn(g, 3, N, K, dtype=BF)
    y, by = padded(torch.zeros(rows, N, dtype=out, device="cuda"), pad, offset, fill=7.0)
    dx, bx = padded(torch.zeros(rows, K, dtype=out, device="cuda"), pad, offset, fill=7.0)
    dw, bw = padded(torch.zeros(3, N, K, dtype=out, device="cuda"), pad, offset, fill=7.0)
    moe.moe_fp4_grouped_forward(x, w, off, y=y)
    moe.moe_fp4_grouped_dgrad(dy, w, off, dx=dx)
    moe.moe_fp4_grouped_wgrad(dy, x, off, dw=dw)
    lo = 0
    for e, c in enumerate(counts):
        r = slice(lo, lo + c)
        lo += c
        want, s = mm(x[r], w[e].t())
        bounded(y[r], want, K * U32 * s, out, "y")
        want, s = mm(dy[r], w[e])
        bounded(dx[r], want, N * U32 * s, out, "dx")
        want, s = mm(dy[r].t(), x[r])
        bounded(dw[e], want, max(c, 1) * U32 * s, out, "dw")
    for b, v in ((by, y), (bx, dx), (bw, dw)):
        assert untouched(b, v, offset)
    # and dense, with every part of the epilogue off the grid
    res, _ = padded(randn(g, rows, N, dtype=out), pad, offset)
    y, by = padded(torch.zeros(rows, N, dtype=out, device="cuda"), pad, offset, fill=7.0)
    bias = randn(g, N + 1, dtype=BF)[1:]
    moe.moe_fp4_linear(x, w[0], bias=bias, residual=res, y=y)
    want, s = mm(x, w[0].t())
    mag = want.abs() + bias.double().abs() + res.double().abs()
    bounded(y, want + bias.double() + res.double(), K * U32 * s + 2 * U32 * mag, out, "dense y")
    assert untouched(by, y, offset)


def test_fp16_steps_below_the_normal_range(moe):
    """The matrix instruction aligns its terms by their exponent fields, and a value
    below 2^-14 has the field of 2^-14: of a term a b it keeps what lies within 24
    bits of max(|a|, 2^-14) max(|b|, 2^-14).  2^-24 * 1 + 2^-24 * 2^-k is exact as
    long as 2^(-24 - k) >= 2^(-14 - 24)."""
    k = torch.arange(15, device="cuda")
    dy = torch.full((2, 8), 2.0 ** -24, device="cuda").to(HF)
    x = torch.ones(2, 16, device="cuda")
    x[1, :15] = torch.exp2(-k.float())
    dw = moe.moe_fp4_grouped_wgrad(dy, x.to(HF), offsets_of([2]), out_dtype=F32)[0]
    assert torch.equal(dw.double(), dy.double().t() @ x.double())


@pytest.mark.parametrize("M", [1, 3, 9, 40, 300])
def test_fp16_below_the_normal_range(moe, M):
    """Values of 2^-24 to 2^-14 are not taken as zero on the way through a product.
    By the alignment above each addition is off by at most one step, 2^-23, of the
    largest of the partial sum and the terms with |a| and |b| raised to 2^-14: n 2^-23
    times the sum of those bounds n additions."""
    def raised(a, b):
        a, b = a.double(), b.double()
        return a @ b, a.abs().clamp(min=2.0 ** -14) @ b.abs().clamp(min=2.0 ** -14)

    g = gen(M)
    N, K = 136, 512
    x = (randn(g, M, K) * 2.0 ** -17).to(HF)
    w = randn(g, N, K, dtype=HF)
    y = moe.moe_fp4_linear(x, w, out_dtype=F32)
    want, s = raised(x, w.t())
    bounded(y, want, K * U32 * s, F32, "y")
    off = offsets_of([M])
    dy = (randn(g, M, N) * 2.0 ** -17).to(HF)
    want, s = raised(dy, w)
    bounded(moe.moe_fp4_grouped_dgrad(dy, w[None], off, out_dtype=F32), want, N * U32 * s, F32, "dx")
    z = randn(g, M, K, dtype=HF)
    want, s = raised(dy.t(), z)
    bounded(moe.moe_fp4_grouped_wgrad(dy, z, off, out_dtype=F32)[0], want, M * U32 * s, F32, "dw")


@pytest.mark.parametrize("ld", [1 << 22, (1 << 22) - 1])
@pytest.mark.parametrize("rows", [4, 300])
def test_largest_row_strides(moe, ld, rows):
    """Rows 8 MB apart: a tile's byte offsets reach 2^31."""
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GB")
    g = gen(rows)
    N, K = 264, 72

    def apart(t):
        v = torch.empty(t.shape[0] * ld, dtype=t.dtype, device="cuda").as_strided(t.shape, (ld, 1))
        return v.copy_(t)

    x, w, dy = (apart(randn(g, *s, dtype=BF)) for s in ((rows, K), (N, K), (rows, N)))
    y = apart(torch.zeros(rows, N, dtype=BF, device="cuda"))
    moe.moe_fp4_linear(x, w, y=y)
    want, s = mm(x, w.t())
    bounded(y, want, K * U32 * s, BF, "y")
    del y
    dx, dw, _ = moe.moe_fp4_linear_backward(dy, x, w, dw=apart(torch.zeros(N, K, device="cuda", dtype=BF)))
    want, s = mm(dy, w)
    bounded(dx, want, N * U32 * s, BF, "dx")
    want, s = mm(dy.t(), x)
    bounded(dw, want, rows * U32 * s, BF, "dw")
