"""The plans of the products, without a GPU: the sizes of the kernel-path tests take the
kernels they are meant for, and a split sum is what a workspace is asked for."""
import ctypes

import pytest

from block_paths import DENSE, GROUPED, LONG_SUMS, WGRAD, names


@pytest.fixture(scope="module")
def moe():
    import mxfp4_routed_expert_router_amd as m
    return m


def of(plan, columns):
    assert (plan.tiles == 0) == (plan.rows > 0)
    if plan.tiles:
        assert 0 < plan.columns <= columns and (plan.columns < columns) == (plan.rest_tiles > 0)
    return plan.rows, plan.tiles, int(plan.splits > 1), plan.rest_tiles, int(plan.rest_splits > 1)


@pytest.mark.parametrize("case,path", DENSE, ids=names(DENSE))
def test_dense(moe, case, path):
    op, M, N, K = case
    p = moe.moe_fp4_linear_plan(M, N, K, op)
    assert of(p, N if op == 0 else K) == path, p
    if op == 0:
        assert (moe.moe_fp4_linear_workspace_size(M, N, K) > 0) == (p.splits > 1 or p.rest_splits > 1)


@pytest.mark.parametrize("case,path", GROUPED, ids=names(GROUPED))
def test_grouped(moe, case, path):
    op, E, P, N, K = case
    p = moe.moe_fp4_grouped_plan(E, P, N, K, op)
    assert of(p, N if op == 0 else K) == path + (0, 0), p
    assert (moe.moe_fp4_grouped_workspace_size(E, P, N, K, op) > 0) == (p.splits > 1)


@pytest.mark.parametrize("case,path", LONG_SUMS, ids=[f"{c[1]}x{c[2]}_{sum(c[0])}" for c, _ in LONG_SUMS])
def test_long_sums(moe, case, path):
    counts, N, K = case
    p = moe.moe_fp4_grouped_plan(len(counts), sum(counts), N, K, WGRAD)
    assert of(p, K) == (0,) + path + (0, 0), p


def test_no_rows(moe):
    p = moe.moe_fp4_linear_plan(0, 64, 64, 0)
    assert (p.rows, p.tiles) == (0, 0)
    assert moe.moe_fp4_grouped_plan(4, 0, 64, 64, 1).tiles == 0
    assert moe.moe_fp4_grouped_plan(4, 0, 64, 64, 2).tiles > 0  # zeros are written


def test_refusals(moe):
    from mxfp4_routed_expert_router_amd import _block, _lib
    L, p = _lib._lib, _block.ProductPlan()
    g = _block.GroupedDims(4, 100, 64, 128, 100, 1, _block.BF16, _block.BF16)
    d = _block.LinearDims(10, 64, 128, _block.BF16, _block.BF16, _block.BF16, _block.BF16, 0)
    for f, dims in ((L.moe_fp4_grouped_plan, g), (L.moe_fp4_linear_plan, d)):
        assert f(None, 0, ctypes.byref(p)) == _lib.EINVAL
        assert f(ctypes.byref(dims), 0, None) == _lib.EINVAL
        for op in (-1, 3):
            assert f(ctypes.byref(dims), op, ctypes.byref(p)) == _lib.EUNSUPPORTED
        assert f(ctypes.byref(dims), 0, ctypes.byref(p)) == _lib.OK
    with pytest.raises(moe.MoeFp4Error):
        moe.moe_fp4_linear_plan(5, 0, 8, 0)
    with pytest.raises(moe.MoeFp4Error):
        moe.moe_fp4_grouped_plan(1025, 5, 8, 8, 0)
