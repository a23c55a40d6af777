"""The products through each of their kernels (tiles of every shape, split sums, the launch
of the columns behind whole rounds of tiles, one row to sixteen), at sizes that end inside
tiles and steps, in both types, gathered and with the whole epilogue, against 64 bits.

Twice: with normal values, held to the bounds of fp32 sums, and with whole numbers of -4 to
4, whose products and sums are exact in fp32 in any order, so that one wrong term of
thousands shows: the results have to be equal."""
import pytest
import torch

from block_common import U32, bounded, gen, offsets_of, padded, randn
from block_paths import ANY, DENSE, DGRAD, FWD, GROUPED, LONG_SUMS, WGRAD, counts_of, names
from test_gpu_grouped import reference, src_rows
from test_gpu_linear import forward64

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_routed_expert_router_amd as m
    return m


def whole(g, *shape, dtype):
    return torch.randint(-4, 5, shape, generator=g, device="cuda").to(dtype)


def exactly(got, want, what=""):
    assert want.abs().max().item() < 2 ** 24
    assert torch.equal(got, want.to(got.dtype)), (what, (got.double() - want).abs().max().item())


def untouched(buf, view, offset):
    buf.as_strided(view.shape, view.stride(), offset).fill_(7.0)
    return bool((buf == 7.0).all())


@pytest.mark.parametrize("dt", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("case,path", DENSE, ids=names(DENSE))
def test_dense(moe, case, path, dt):
    op, M, N, K = case
    g = gen(M + N + K)
    if op == FWD:
        x, w = randn(g, M, K, dtype=dt), randn(g, N, K, dtype=dt, scale=K ** -0.5)
        bias = randn(g, N, dtype=F32)
        z64 = forward64(x.double(), w.double(), None, "none", None)
        for out in (dt, F32):  # the plain epilogue
            bounded(moe.moe_fp4_linear(x, w, out_dtype=out), z64[0], z64[2], out, f"plain {out}")
        # all of it, the result and the residual in strided rows off the 16-byte grid
        r, _ = padded(randn(g, M, N, dtype=dt), 3, 1)
        y, buf = padded(torch.zeros(M, N, dtype=dt, device="cuda"), 5, 3, fill=7.0)
        _, z = moe.moe_fp4_linear(x, w, bias=bias, act=moe.ACT_GELU, residual=r, y=y, save_z=True)
        wy, wz, ey, ez = forward64(x.double(), w.double(), bias.double(), "gelu", r.double())
        bounded(y, wy, ey, dt, "y")
        bounded(z, wz, ez, dt, "z")
        assert untouched(buf, y, 3)
    elif op == DGRAD:
        dy, w = randn(g, M, N, dtype=dt), randn(g, N, K, dtype=dt, scale=N ** -0.5)
        dx, buf = padded(torch.zeros(M, K, dtype=dt, device="cuda"), 5, 3, fill=7.0)
        one, _, _ = moe.moe_fp4_linear_backward(dy, None, w, need_dw=False, need_db=False)
        moe.moe_fp4_linear_backward(dy, None, w, need_dw=False, need_db=False, dx=dx)
        want, mag = dy.double() @ w.double(), dy.double().abs() @ w.double().abs()
        bounded(one, want, N * U32 * mag, dt, "dx")
        assert torch.equal(dx, one) and untouched(buf, dx, 3)
    else:
        dy, x = randn(g, M, N, dtype=dt, scale=M ** -0.5), randn(g, M, K, dtype=dt)
        want, mag = dy.double().t() @ x.double(), dy.double().t().abs() @ x.double().abs()
        for out in (dt, F32):
            _, dw, _ = moe.moe_fp4_linear_backward(dy, x, None, need_dx=False, need_db=False, dw_dtype=out)
            bounded(dw, want, M * U32 * mag, out, f"dw {out}")
        old = randn(g, N, K)
        dw, buf = padded(old, 5, 3, fill=7.0)
        moe.moe_fp4_linear_backward(dy, x, None, need_dx=False, need_db=False, dw=dw, accumulate=True)
        old = old.double()
        bounded(dw, want + old, M * U32 * mag + U32 * (want.abs() + old.abs()), F32, "dw +=")
        assert untouched(buf, dw, 3)


@pytest.mark.parametrize("dt", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("case,path", DENSE, ids=names(DENSE))
def test_dense_exactly(moe, case, path, dt):
    op, M, N, K = case
    g = gen(M + N + K + 1)
    x, w, dy = whole(g, M, K, dtype=dt), whole(g, N, K, dtype=dt), whole(g, M, N, dtype=dt)
    if op == FWD:
        z64 = x.double() @ w.double().t()
        for out in (dt, F32):
            exactly(moe.moe_fp4_linear(x, w, out_dtype=out), z64, "plain")
            bias, r = whole(g, N, dtype=dt), whole(g, M, N, dtype=out)
            y, z = moe.moe_fp4_linear(x, w, bias=bias, act=moe.ACT_RELU, residual=r, out_dtype=out, save_z=True)
            exactly(z, z64 + bias.double(), "z")
            exactly(y, (z64 + bias.double()).clamp(min=0) + r.double(), "y")
    elif op == DGRAD:
        dx, _, _ = moe.moe_fp4_linear_backward(dy, None, w, need_dw=False, need_db=False)
        exactly(dx, dy.double() @ w.double())
    else:
        for out in (dt, F32):
            old = whole(g, N, K, dtype=out)
            dw = old.clone()
            moe.moe_fp4_linear_backward(dy, x, None, need_dx=False, need_db=False, dw=dw, accumulate=True)
            exactly(dw, dy.double().t() @ x.double() + old.double())


# with the rows in expert order, and gathered (the rows' gradient takes them in order only)
ROWS = [(c, p, False) for c, p in GROUPED] + [(c, p, True) for c, p in GROUPED if c[0] != DGRAD]
ROW_IDS = names(GROUPED) + [n + "_gathered" for n in names([g for g in GROUPED if g[0][0] != DGRAD])]


@pytest.mark.parametrize("exact", [False, True], ids=["normal", "whole"])
@pytest.mark.parametrize("dt", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("case,path,gathered", ROWS, ids=ROW_IDS)
def test_grouped(moe, case, path, dt, gathered, exact):
    op, E, P, N, K = case
    g = gen(E + P + N + K)
    counts = counts_of(E, P)
    assert sum(counts) == P
    # three rows before the first expert's and two behind the last's stay as they are
    off = offsets_of(counts)
    lead = 0 if path[0] else 3
    off, Q = off + lead, P + lead + (2 if lead else 0)
    div, R = (3, (Q + 2) // 3) if gathered else (1, Q)
    make = whole if exact else randn
    x, dy = make(g, R, K, dtype=dt), make(g, Q, N, dtype=dt)
    rows = None
    if gathered:
        rows = torch.randint(0, R * div, (Q,), generator=g, device="cuda", dtype=torch.int32)
        rows[::37], rows[5::41] = -1, R * div
    xs = src_rows(x, rows, div, Q)
    plan = moe.moe_fp4_grouped_plan(E, Q, N, K, op)
    assert (plan.rows, plan.tiles, int(plan.splits > 1)) == path, plan
    if op == WGRAD:
        want, mag = reference("wgrad", dy.double(), xs, counts, lead)
        for out in (dt, F32):
            got = moe.moe_fp4_grouped_wgrad(dy, x, off, rows=rows, row_div=div, out_dtype=out)
            if exact:
                exactly(got, want, "dw")
            else:
                bounded(got, want, max(counts) * U32 * mag, out, f"dw {out}")
        return
    w = make(g, E, N, K, dtype=dt)
    width, n = (N, K) if op == FWD else (K, N)
    want, mag = reference("fwd" if op == FWD else "dgrad", xs if op == FWD else dy.double(), w, counts, lead)
    for out in (dt, F32):
        y, buf = padded(torch.zeros(Q, width, dtype=out, device="cuda"), 8, 16, fill=7.0)
        y.fill_(7.0)
        if op == FWD:
            moe.moe_fp4_grouped_forward(x, w, off, rows=rows, row_div=div, y=y)
        else:
            moe.moe_fp4_grouped_dgrad(dy, w, off, dx=y)
        if exact:
            exactly(y[lead:lead + P], want)
        else:
            bounded(y[lead:lead + P], want, n * U32 * mag, out, f"{out}")
        assert untouched(buf, y[lead:lead + P], 16 + lead * y.stride(0))


@pytest.mark.parametrize("dt", [BF, HF], ids=["bf16", "f16"])
@pytest.mark.parametrize("case,path", LONG_SUMS, ids=[f"{c[1]}x{c[2]}_{sum(c[0])}" for c, _ in LONG_SUMS])
def test_long_gathered_sums(moe, case, path, dt):
    """The weights' gradient holds 1024 row indexes at a time: sums of one less, one more and
    several times as many, a row taken several times, some indexes outside x."""
    counts, N, K = case
    P, div = sum(counts), 3
    g = gen(P + N)
    R = P // div
    x, dy = whole(g, R, K, dtype=dt), whole(g, P, N, dtype=dt)
    rows = torch.randint(0, R * div, (P,), generator=g, device="cuda", dtype=torch.int32)
    rows[11::97], rows[1023::1024], rows[1024::1024] = -5, R * div, 2 ** 31 - 1
    off = offsets_of(counts)
    want, _ = reference("wgrad", dy.double(), src_rows(x, rows, div, P), counts)
    exactly(moe.moe_fp4_grouped_wgrad(dy, x, off, rows=rows, row_div=div, out_dtype=F32), want, "f32")
    exactly(moe.moe_fp4_grouped_wgrad(dy, x, off, rows=rows, row_div=div), want, "16 bits")
    old = whole(g, *want.shape, dtype=F32)
    more = old.clone()
    moe.moe_fp4_grouped_wgrad(dy, x, off, rows=rows, row_div=div, dw=more, accumulate=True)
    exactly(more, want + old.double(), "dw +=")


def test_unaligned_pointers_take_the_tiles_of_any_alignment(moe):
    """A plan is for pointers on 16-byte boundaries; rows off them give the same sums to rounding."""
    g = gen(1)
    M, N, K = 203, 1584, 1168
    assert moe.moe_fp4_linear_plan(M, N, K, FWD).tiles != ANY
    x, _ = padded(randn(g, M, K, dtype=BF), 8, 4)
    w = randn(g, N, K, dtype=BF)
    want, mag = x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t()
    bounded(moe.moe_fp4_linear(x, w, out_dtype=F32), want, K * U32 * mag, F32, "y")
