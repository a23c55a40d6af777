"""The gradients' global norm and clipping against 64 bits: types and their mixes,
sizes around the chunks, none and many tensors, alignment, values that fp32 squares
lose, results of other types, infinities."""
import pytest
import torch

from block_common import U32, bounded, gen, randn

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_routed_expert_router_amd as m
    return m


def sumsq64(tensors):
    return sum((t.double().square().sum() for t in tensors), torch.zeros((), dtype=torch.float64, device="cuda"))


def check(moe, tensors, max_norm, eps=1e-6, out=None):
    """sumsq to fp64 accuracy (n additions of positive terms in some order), the factor
    rounded to fp32 once, the product once, and once more to the result's type."""
    before = [t.clone() for t in tensors]
    ss = moe.moe_fp4_grad_sumsq(tensors)
    want = sumsq64(tensors)
    n = sum(t.numel() for t in tensors)
    assert abs(ss.item() - want.item()) <= (n + 8) * 2.0 ** -52 * want.item()
    norm = moe.moe_fp4_grad_clip(tensors, ss, max_norm, eps=eps, out=out)
    root = want.sqrt()
    assert abs(norm.item() - root.item()) <= U32 * root.item()
    factor = min(1.0, max_norm / (root.item() + eps))
    for b, t, o in zip(before, tensors, out if out is not None else tensors):
        bounded(o.reshape(1, -1), b.double().reshape(1, -1) * factor, 1.1 * U32 * b.double().abs().reshape(1, -1) * factor, o.dtype,
                f"{t.dtype} -> {o.dtype}, {t.numel()}")
        if out is not None:
            assert torch.equal(b, t)
        elif factor == 1:
            assert torch.equal(b, t)


SIZES = [[1], [0], [3, 0, 5], [8191, 8192, 8193], [16383, 16384, 16385, 24577], [100000, 7, 131072], [5120] * 9,
         [1000003], [17] * 300, [2304 * 512, 40, 9999]]


@pytest.mark.parametrize("max_norm", [0.5, 1e9, 0.0])
@pytest.mark.parametrize("types", [[F32], [BF], [HF], [F32, BF, HF]], ids=["f32", "bf16", "f16", "mixed"])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{s[0]}")
def test_norm_and_clip(moe, sizes, types, max_norm):
    g = gen(sum(sizes))
    make = lambda: [randn(g, n, dtype=types[i % len(types)], scale=10.0 ** -(i % 3)) for i, n in enumerate(sizes)]
    check(moe, make(), max_norm)
    tensors = make()
    check(moe, tensors, max_norm, out=[torch.full_like(t, 7.0) for t in tensors])
    if F32 in types:
        kinds = [HF, F32, BF]
        check(moe, tensors, max_norm, out=[torch.full_like(t, 7.0, dtype=kinds[i % 3] if t.dtype == F32 else t.dtype)
                                           for i, t in enumerate(tensors)])


def test_any_alignment_leaves_the_neighbours(moe):
    g = gen(2)
    for dt in (F32, BF, HF):
        buf = randn(g, 200000, dtype=dt)
        keep = buf.clone()
        spans = [(1, 40001), (40002, 40003), (40007, 90001), (90001, 199998)]
        views = [buf[a:b] for a, b in spans]
        ss = moe.moe_fp4_grad_sumsq(views)
        moe.moe_fp4_grad_clip(views, ss, 1.0)
        outside = torch.ones(200000, dtype=torch.bool, device="cuda")
        for a, b in spans:
            outside[a:b] = False
        assert torch.equal(buf[outside], keep[outside])
        f = 1.0 / (sumsq64([keep[a:b] for a, b in spans]).sqrt().item() + 1e-6)
        bounded(buf[~outside], keep[~outside].double() * f, 1.1 * U32 * keep[~outside].double().abs() * f, dt, "clipped")


def test_layouts(moe):
    """A transposed and a channels-last gradient fill their memory; a strided view does not."""
    g = gen(3)
    a = randn(g, 30, 50).t()
    b = randn(g, 2, 3, 4, 5).to(memory_format=torch.channels_last)
    check(moe, [a, b], 1.0)
    check(moe, [a, b], 1.0, out=[torch.empty_like(a), torch.empty_like(b)])
    for bad in (randn(g, 10, 10)[:, :5], randn(g, 10)[::2], randn(g, 1, 5).expand(3, 5)):
        with pytest.raises(ValueError):
            moe.moe_fp4_grad_sumsq([bad])
    with pytest.raises(ValueError):
        moe.moe_fp4_grad_clip([a], moe.moe_fp4_grad_sumsq([a]), 1.0, out=[torch.empty(50, 30, device="cuda")])


def test_values_that_fp32_squares_lose(moe):
    for v in (1e-30, 1e-40, 3e38, 1e25):
        t = torch.full((5000,), v, device="cuda")
        ss = moe.moe_fp4_grad_sumsq([t])
        want = t.double().square().sum().item()
        assert abs(ss.item() - want) <= 1e-12 * want
        norm = moe.moe_fp4_grad_clip([t], ss, 1e9)
        assert abs(norm.item() - want ** 0.5) <= U32 * want ** 0.5 + 2.0 ** -149 or norm.item() == float("inf") and want ** 0.5 > 3.4e38


def test_inf_and_nan(moe):
    t = torch.ones(100, device="cuda")
    t[5] = float("inf")
    ss = moe.moe_fp4_grad_sumsq([t])
    norm = moe.moe_fp4_grad_clip([t], ss, 1.0)
    assert norm.item() == float("inf") and torch.isnan(t).nonzero()[:, 0].tolist() == [5] and bool((t[:5] == 0).all())
    t = torch.ones(100, device="cuda")
    t[5] = float("nan")
    ss = moe.moe_fp4_grad_sumsq([t])
    assert torch.isnan(moe.moe_fp4_grad_clip([t], ss, 1.0)).item() and bool(torch.isnan(t).all())


def test_accumulate_and_no_tensors(moe):
    g = gen(4)
    a, b = randn(g, 9000, dtype=BF), randn(g, 50)
    ss = moe.moe_fp4_grad_sumsq([a])
    moe.moe_fp4_grad_sumsq([b], sumsq=ss, accumulate=True)
    want = sumsq64([a, b]).item()
    assert abs(ss.item() - want) <= 1e-11 * want
    moe.moe_fp4_grad_sumsq([], sumsq=ss, accumulate=True)
    assert abs(ss.item() - want) <= 1e-11 * want
    assert moe.moe_fp4_grad_clip([], ss, 1.0).item() == pytest.approx(want ** 0.5, rel=1e-6)
    moe.moe_fp4_grad_sumsq([], sumsq=ss)
    assert ss.item() == 0
    # a norm of zero divides by eps, or by nothing
    z = torch.zeros(10, device="cuda")
    for eps in (1e-6, 0.0):
        for max_norm in (1.0, 0.0):
            assert moe.moe_fp4_grad_clip([z], ss, max_norm, eps=eps).item() == 0 and bool((z == 0).all())


def test_more_than_2_to_32_bytes(moe):
    """One tensor of 2^31 + 12345 elements: byte offsets past 2^32."""
    n = (1 << 31) + 12345
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GB")
    t = torch.full((n,), 0.5, dtype=BF, device="cuda")
    t[-1] = 3.0
    ss = moe.moe_fp4_grad_sumsq([t])
    want = 0.25 * (n - 1) + 9
    assert abs(ss.item() - want) <= 1e-9 * want
    moe.moe_fp4_grad_clip([t], ss, want ** 0.5 / 2, eps=0.0)
    assert t[:100].unique().item() == 0.25 and t[n // 2] == 0.25 and t[-2] == 0.25 and t[-1] == 1.5


def test_same_bits_twice_and_any_workspace(moe):
    g = gen(5)
    ts = [randn(g, n, dtype=BF) for n in (3000001, 500, 70000)]
    n = moe.moe_fp4_grad_sumsq_workspace_size(ts)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(moe.moe_fp4_grad_sumsq(ts), moe.moe_fp4_grad_sumsq(ts, workspace=ws))
    with pytest.raises(moe.MoeFp4Error):
        moe.moe_fp4_grad_sumsq(ts, workspace=ws[:n - 8])


def test_binding_refusals(moe):
    t = torch.ones(8, device="cuda")
    ss = moe.moe_fp4_grad_sumsq([t])
    with pytest.raises(moe.MoeFp4Error):
        moe.moe_fp4_grad_clip([t, t], ss, 1.0)
    with pytest.raises(moe.MoeFp4Error):
        moe.moe_fp4_grad_clip([t], ss, -1.0)
    with pytest.raises(TypeError):
        moe.moe_fp4_grad_sumsq([t.double()])
    with pytest.raises(TypeError):
        moe.moe_fp4_grad_clip([t], ss.float(), 1.0)
    with pytest.raises(TypeError):
        moe.moe_fp4_grad_clip([t.to(BF)], ss, 1.0, out=[t])
    with pytest.raises(ValueError):
        moe.moe_fp4_grad_clip([t], ss, 1.0, out=[])
    with pytest.raises(ValueError):
        moe.moe_fp4_grad_sumsq([t], accumulate=True)
    with pytest.raises(ValueError):
        moe.moe_fp4_grad_sumsq([t, t.cpu()])


@pytest.mark.parametrize("out_type", [1, 2, 3, -1, 1 << 20])
def test_a_type_of_no_result_is_not_read(moe, out_type):
    """The C call in place, out_type anything: fp32 tensors are clipped in fp32."""
    from mxfp4_routed_expert_router_amd import _lib, _train
    g = gen(6)
    tensors = [randn(g, 20000), randn(g, 33, dtype=BF), randn(g, 9000)]
    keep = [t.clone() for t in tensors]
    ss = moe.moe_fp4_grad_sumsq(tensors)
    rows = [_train.GradTensor(t.data_ptr(), None, t.numel(), _train._TYPES[t.dtype], out_type) for t in tensors]
    table = (_train.GradTensor * 3)(*rows)
    norm = torch.zeros(1, device="cuda")
    assert _lib._lib.moe_fp4_grad_clip(table, 3, ss.data_ptr(), 1.0, 0.0, norm.data_ptr(),
                                       torch.cuda.current_stream().cuda_stream) == _lib.OK
    factor = 1.0 / sumsq64(keep).sqrt().item()
    for t, k in zip(tensors, keep):
        bounded(t, k.double() * factor, 1.1 * U32 * k.double().abs() * factor, t.dtype, "clipped")


def test_a_norm_of_inf_without_a_limit(moe):
    """max_norm inf: nothing is clipped; an infinite norm still gives a factor of 0."""
    inf = float("inf")
    t = torch.ones(100, device="cuda")
    assert moe.moe_fp4_grad_clip([t], moe.moe_fp4_grad_sumsq([t]), inf).item() == 10.0 and bool((t == 1).all())
    t[5] = inf
    norm = moe.moe_fp4_grad_clip([t], moe.moe_fp4_grad_sumsq([t]), inf)
    assert norm.item() == inf and torch.isnan(t).nonzero()[:, 0].tolist() == [5] and bool((t[:5] == 0).all())


@pytest.mark.parametrize("max_norm", [0.5, 1e9])
@pytest.mark.parametrize("out", [False, True], ids=["in_place", "out"])
def test_lists_of_more_chunks_than_workgroups(moe, out, max_norm):
    """Some 200 MB in one launch: a workgroup goes from tensor to tensor, of other types and of sizes
    from one element to many times all workgroups' chunks."""
    g = gen(8)
    sizes = [20000003, 1, 16385, 70000, 9, 40000001, 8191, 500001, 3000000, 17, 1000003, 16384] + [5000 + 977 * i for i in range(60)]
    types = [F32, BF, HF]
    tensors = [randn(g, n, dtype=types[i % 3], scale=10.0 ** -(i % 3)) for i, n in enumerate(sizes)]
    kinds = [HF, F32, BF]
    check(moe, tensors, max_norm, out=[torch.full_like(t, 7.0, dtype=kinds[i // 3 % 3] if t.dtype == F32 else t.dtype)
                                       for i, t in enumerate(tensors)] if out else None)
