"""16-bit products grouped by expert against 64-bit references: ragged and empty
experts, gathered rows, odd sizes, strides and alignments, rows that belong to no
expert, accumulation, both types and both result types."""
import numpy as np
import pytest
import torch

from block_common import U32, bounded, gen, offsets_of, padded, randn

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_routed_expert_router_amd as m
    return m


def src_rows(x, rows, div, P):
    """The rows of x that the ragged side reads, in 64 bits; zeros where out of range."""
    if rows is None:
        return x[:P].double()
    r = rows.long()
    s = torch.div(r, div, rounding_mode="floor")
    ok = (r >= 0) & (s < x.shape[0])
    out = torch.zeros(P, x.shape[1], dtype=torch.float64, device=x.device)
    out[ok] = x[s[ok]].double()
    return out


def reference(op, a, b, counts, lo=0):
    """(value, sum of magnitudes, terms) by expert; a: xs or dy, b: w, or (wgrad) xs."""
    outs, mags = [], []
    for e, c in enumerate(counts):
        r = slice(lo, lo + c)
        lo += c
        if op == "fwd":
            m = (a[r], b[e].double().t())
        elif op == "dgrad":
            m = (a[r], b[e].double())
        else:
            m = (a[r].t(), b[r])
        outs.append(m[0] @ m[1])
        mags.append(m[0].abs() @ m[1].abs())
    if op == "wgrad":
        return torch.stack(outs), torch.stack(mags)
    return torch.cat(outs), torch.cat(mags)


SHAPES = [  # counts, N, K
    ([1], 16, 32),
    ([1], 1, 1),
    ([0, 1, 0], 64, 64),
    ([3, 0, 1, 2], 288, 512),
    ([5, 64, 0, 65, 63], 96, 160),
    ([129, 0, 127, 128, 1], 256, 288),
    ([255, 256, 257], 128, 96),
    ([300, 2, 0, 0, 41], 320, 256),
    ([7, 9], 33, 47),
    ([70, 0, 13], 130, 1001),
    ([2] * 70, 72, 40),
    ([0] * 100 + [17] + [0] * 100, 64, 128),
    ([1, 0, 2, 0, 1, 1, 0, 1], 576, 1280),
    ([513, 700], 264, 520),
    # each tile shape at its own sizes: the largest, ragged; the middle one; and long sums in parts
    ([700, 0, 1300, 257, 900, 64, 33, 1], 1032, 136),
    ([130] * 9, 1032, 1160),
    ([40, 0, 90], 64, 2048),
    ([40, 33], 65, 2051),
    ([3000, 5, 0, 2900], 72, 80),
    ([2500, 1700], 35, 51),
]
IDS = [f"E{len(c)}_P{sum(c)}_N{n}_K{k}" for c, n, k in SHAPES]


@pytest.mark.parametrize("dt", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("op", ["fwd", "dgrad", "wgrad"])
@pytest.mark.parametrize("counts,N,K", SHAPES, ids=IDS)
def test_products(moe, counts, N, K, op, dt):
    g = gen(len(counts) * 1000 + N + K)
    E, P = len(counts), sum(counts)
    off = offsets_of(counts)
    x, dy = randn(g, P, K, dtype=dt), randn(g, P, N, dtype=dt)
    w = randn(g, E, N, K, dtype=dt)
    for out in (dt, F32):
        if op == "fwd":
            got = moe.moe_fp4_grouped_forward(x, w, off, out_dtype=out)
            want, mag = reference(op, x.double(), w, counts)
            n = K
        elif op == "dgrad":
            got = moe.moe_fp4_grouped_dgrad(dy, w, off, out_dtype=out)
            want, mag = reference(op, dy.double(), w, counts)
            n = N
        else:
            got = moe.moe_fp4_grouped_wgrad(dy, x, off, out_dtype=out)
            want, mag = reference(op, dy.double(), x.double(), counts)
            n = max(counts)
        assert got.dtype == out
        bounded(got, want, n * U32 * mag, out, f"{op} {out}")


@pytest.mark.parametrize("op", ["fwd", "wgrad"])
@pytest.mark.parametrize("k", [1, 2, 6])
def test_gathered_rows(moe, op, k):
    """Pair ids of a routing as the row index: every token's row k times, in expert order."""
    T, E, N, K = 53, 11, 160, 224
    g = gen(7 + k)
    lg = randn(g, T, E)
    r = moe.moe_fp4_route(lg, k)
    counts = r.counts.tolist()
    x, dy, w = randn(g, T, K, dtype=BF), randn(g, T * k, N, dtype=BF), randn(g, E, N, K, dtype=BF)
    xs = src_rows(x, r.sorted_pairs, k, T * k)
    if op == "fwd":
        got = moe.moe_fp4_grouped_forward(x, w, r.offsets, rows=r.sorted_pairs, row_div=k, out_dtype=F32)
        want, mag = reference(op, xs, w, counts)
        n = K
    else:
        got = moe.moe_fp4_grouped_wgrad(dy, x, r.offsets, rows=r.sorted_pairs, row_div=k, out_dtype=F32)
        want, mag = reference(op, dy.double(), xs, counts)
        n = max(counts)
    bounded(got, want, n * U32 * mag, F32, op)


@pytest.mark.parametrize("N,K", [(128, 256), (33, 47)])
@pytest.mark.parametrize("op", ["fwd", "wgrad"])
def test_row_index_outside_x_reads_zeros(moe, op, N, K):
    """Entries below 0, at and past the last row, and the same row twice."""
    g = gen(5)
    counts, R = [3, 0, 6], 4
    P = sum(counts)
    rows = torch.tensor([0, -1, 3, 4, 3, 2**31 - 1, -2**31, 1, 0], dtype=torch.int32, device="cuda")
    x, dy, w = randn(g, R, K, dtype=BF), randn(g, P, N, dtype=BF), randn(g, 3, N, K, dtype=BF)
    xs = src_rows(x, rows, 1, P)
    off = offsets_of(counts)
    if op == "fwd":
        got = moe.moe_fp4_grouped_forward(x, w, off, rows=rows, out_dtype=F32)
        want, mag = reference(op, xs, w, counts)
    else:
        got = moe.moe_fp4_grouped_wgrad(dy, x, off, rows=rows, out_dtype=F32)
        want, mag = reference(op, dy.double(), xs, counts)
    bounded(got, want, max(K, P) * U32 * mag, F32, op)


@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 8), (24, 0), (1, 0), (0, 1), (3, 5)])
@pytest.mark.parametrize("op", ["fwd", "dgrad", "wgrad"])
def test_strides_and_alignment(moe, op, pad, offset):
    """Rows apart from each other, off the 16-byte grid, and NaN in between: none of it reaches a result."""
    g = gen(31 + pad)
    counts, N, K = [70, 0, 5, 130], 136, 200
    P, E = sum(counts), 4
    off = offsets_of(counts)
    x, _ = padded(randn(g, P, K, dtype=BF), pad, offset)
    dy, _ = padded(randn(g, P, N, dtype=BF), pad, offset)
    w, _ = padded(randn(g, E, N, K, dtype=BF), pad, offset)
    if op == "fwd":
        out, buf = padded(torch.zeros(P, N, dtype=BF, device="cuda"), pad, offset, fill=7.0)
        moe.moe_fp4_grouped_forward(x, w, off, y=out)
        want, mag = reference(op, x.double(), w, counts)
        n = K
    elif op == "dgrad":
        out, buf = padded(torch.zeros(P, K, dtype=BF, device="cuda"), pad, offset, fill=7.0)
        moe.moe_fp4_grouped_dgrad(dy, w, off, dx=out)
        want, mag = reference(op, dy.double(), w, counts)
        n = N
    else:
        out, buf = padded(torch.zeros(E, N, K, dtype=BF, device="cuda"), pad, offset, fill=7.0)
        moe.moe_fp4_grouped_wgrad(dy, x, off, dw=out)
        want, mag = reference(op, dy.double(), x.double(), counts)
        n = max(counts)
    bounded(out, want, n * U32 * mag, BF, op)
    # what lies between the rows was not written
    left = buf.clone()
    left.as_strided(out.shape, out.stride(), offset).fill_(7.0)
    assert bool((left == 7.0).all())


@pytest.mark.parametrize("N,K", [(128, 256), (33, 47)])
def test_rows_without_an_expert(moe, N, K):
    """Rows before the first and behind the last expert's keep what they held, and their
    inputs (NaN) reach nothing; so do the weights of experts without rows."""
    g = gen(11)
    counts, before, behind = [20, 0, 70], 3, 40
    P = before + sum(counts) + behind
    off = (offsets_of(counts) + before).to(torch.int32)
    x, dy, w = randn(g, P, K, dtype=BF), randn(g, P, N, dtype=BF), randn(g, 3, N, K, dtype=BF)
    for t in (x, dy):
        t[:before] = float("nan")
        t[P - behind:] = float("inf")
    w[1] = float("nan")
    mid = slice(before, P - behind)
    y = torch.full((P, N), 5.0, dtype=BF, device="cuda")
    moe.moe_fp4_grouped_forward(x, w, off, y=y)
    want, mag = reference("fwd", x.double(), w, counts, before)
    bounded(y[mid], want, K * U32 * mag, BF, "fwd")
    assert bool((y[:before] == 5).all()) and bool((y[P - behind:] == 5).all())
    dx = torch.full((P, K), 5.0, dtype=F32, device="cuda")
    moe.moe_fp4_grouped_dgrad(dy, w, off, dx=dx)
    want, mag = reference("dgrad", dy.double(), w, counts, before)
    bounded(dx[mid], want, N * U32 * mag, F32, "dgrad")
    assert bool((dx[:before] == 5).all()) and bool((dx[P - behind:] == 5).all())
    dw = moe.moe_fp4_grouped_wgrad(dy, x, off, out_dtype=F32)
    want, mag = reference("wgrad", dy.double(), x.double(), counts, before)
    bounded(dw, want, 70 * U32 * mag, F32, "wgrad")
    assert bool((dw[1] == 0).all())


@pytest.mark.parametrize("N,K", [(128, 256), (33, 47)])
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
def test_accumulate(moe, N, K, out):
    g = gen(13)
    counts = [40, 0, 9]
    P, off = 49, offsets_of([40, 0, 9])
    x, dy, w = randn(g, P, K, dtype=BF), randn(g, P, N, dtype=BF), randn(g, 3, N, K, dtype=BF)
    for op in ("fwd", "dgrad", "wgrad"):
        shape = {"fwd": (P, N), "dgrad": (P, K), "wgrad": (3, N, K)}[op]
        c0 = randn(g, *shape, dtype=out, scale=4.0)
        c = c0.clone()
        if op == "fwd":
            moe.moe_fp4_grouped_forward(x, w, off, y=c, accumulate=True)
            want, mag = reference(op, x.double(), w, counts)
        elif op == "dgrad":
            moe.moe_fp4_grouped_dgrad(dy, w, off, dx=c, accumulate=True)
            want, mag = reference(op, dy.double(), w, counts)
        else:
            moe.moe_fp4_grouped_wgrad(dy, x, off, dw=c, accumulate=True)
            want, mag = reference(op, dy.double(), x.double(), counts)
        mag = mag + c0.double().abs()
        bounded(c, want + c0.double(), (max(N, K, P) + 1) * U32 * mag, out, op)
        if op == "wgrad":
            assert bool((c[1] == c0[1]).all())  # an expert without rows: unchanged


def test_no_rows(moe):
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    dy = torch.empty(0, 32, dtype=BF, device="cuda")
    w = torch.ones(3, 32, 64, dtype=BF, device="cuda")
    assert moe.moe_fp4_grouped_forward(x, w, off).shape == (0, 32)
    assert moe.moe_fp4_grouped_dgrad(dy, w, off).shape == (0, 64)
    dw = torch.full((3, 32, 64), 3.0, dtype=F32, device="cuda")
    moe.moe_fp4_grouped_wgrad(dy, x, off, dw=dw, accumulate=True)
    assert bool((dw == 3).all())
    moe.moe_fp4_grouped_wgrad(dy, x, off, dw=dw)
    assert bool((dw == 0).all())


def test_offsets_that_are_not_ascending_stay_in_bounds(moe):
    """No defined values, and no access outside the arrays (guard elements around them)."""
    g = gen(17)
    N, K, P = 72, 104, 40
    off = torch.tensor([50, -7, 30, 10, 2**31 - 1, 5], dtype=torch.int32, device="cuda")
    x, dy, w = randn(g, P, K, dtype=BF), randn(g, P, N, dtype=BF), randn(g, 5, N, K, dtype=BF)
    buf = torch.full((P * N + 2048,), 3.0, dtype=BF, device="cuda")
    y = buf[1024:1024 + P * N].view(P, N)
    moe.moe_fp4_grouped_forward(x, w, off, y=y)
    assert bool((buf[:1024] == 3).all()) and bool((buf[1024 + P * N:] == 3).all())
    buf = torch.full((P * K + 2048,), 3.0, dtype=BF, device="cuda")
    moe.moe_fp4_grouped_dgrad(dy, w, off, dx=buf[1024:1024 + P * K].view(P, K))
    assert bool((buf[:1024] == 3).all()) and bool((buf[1024 + P * K:] == 3).all())
    moe.moe_fp4_grouped_wgrad(dy, x, off)
    torch.cuda.synchronize()


@pytest.mark.parametrize("N,K", [(256, 512), (65, 130)])
def test_same_bits_twice(moe, N, K):
    g = gen(19)
    counts = [100, 3, 0, 300]
    off = offsets_of(counts)
    x, dy, w = randn(g, 403, K, dtype=BF), randn(g, 403, N, dtype=BF), randn(g, 4, N, K, dtype=BF)
    for f in (lambda: moe.moe_fp4_grouped_forward(x, w, off), lambda: moe.moe_fp4_grouped_dgrad(dy, w, off),
              lambda: moe.moe_fp4_grouped_wgrad(dy, x, off)):
        assert torch.equal(f().view(torch.int16), f().view(torch.int16))


def test_infinities_and_nan_stay_in_their_rows(moe):
    g = gen(23)
    x, w = randn(g, 90, 128, dtype=BF), randn(g, 2, 64, 128, dtype=BF)
    x[7, 3], x[50, 9] = float("nan"), float("inf")
    y = moe.moe_fp4_grouped_forward(x, w, offsets_of([40, 50]), out_dtype=F32)
    bad = ~torch.isfinite(y).all(1)
    assert bad.nonzero().flatten().tolist() == [7, 50]


def test_binding_refusals(moe):
    x = torch.zeros(4, 32, dtype=BF, device="cuda")
    w = torch.zeros(2, 16, 32, dtype=BF, device="cuda")
    off = offsets_of([2, 2])
    dy = torch.zeros(4, 16, dtype=BF, device="cuda")
    with pytest.raises(TypeError):
        moe.moe_fp4_grouped_forward(x.float(), w, off)
    with pytest.raises(TypeError):
        moe.moe_fp4_grouped_forward(x, w.half(), off)
    with pytest.raises(TypeError):
        moe.moe_fp4_grouped_forward(x, w, off.long())
    with pytest.raises(ValueError):
        moe.moe_fp4_grouped_forward(x, w, off[:2])
    with pytest.raises(ValueError):
        moe.moe_fp4_grouped_forward(x.cpu(), w, off)
    with pytest.raises(ValueError):
        moe.moe_fp4_grouped_forward(x[:, :16], w, off)
    with pytest.raises(ValueError):
        moe.moe_fp4_grouped_forward(x[:1].expand(4, 32), w, off)
    with pytest.raises(ValueError):
        moe.moe_fp4_grouped_forward(x, w, off, accumulate=True)
    with pytest.raises(ValueError):
        moe.moe_fp4_grouped_forward(x, w.transpose(1, 2).contiguous().transpose(1, 2), off)
    with pytest.raises(TypeError):
        moe.moe_fp4_grouped_forward(x, w, off, out_dtype=HF)
    with pytest.raises(ValueError):
        moe.moe_fp4_grouped_wgrad(dy, x[:3], off)
    with pytest.raises(ValueError):
        moe.moe_fp4_grouped_dgrad(x, w, off)
    with pytest.raises(moe.MoeFp4Error):
        moe.moe_fp4_grouped_forward(x, w, off, rows=torch.zeros(4, dtype=torch.int32, device="cuda"), row_div=0)
