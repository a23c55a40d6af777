"""The binding of the operators around the routed experts: calls that take only some
of their tensors."""
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


@pytest.mark.parametrize("dyt", [BF, HF, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,N", [(0, 5), (1, 1), (70, 33), (3000, 264)])
def test_bias_gradient_alone(moe, M, N, dyt):
    """Without an activation db needs dy only: no x, no w, no z."""
    dy = randn(gen(M + N), M, N, dtype=dyt)
    dx, dw, db = moe.moe_fp4_linear_backward(dy, None, None, need_dx=False, need_dw=False)
    assert dx is None and dw is None and db.dtype == F32
    bounded(db, dy.double().sum(0), (M + 1) * U32 * dy.double().abs().sum(0), F32, "db")
    more = db.clone()
    moe.moe_fp4_linear_backward(dy, None, None, need_dx=False, need_dw=False, db=more, accumulate=True)
    bounded(more, dy.double().sum(0) + db.double(), (M + 2) * U32 * dy.double().abs().sum(0) + U32 * db.double().abs(),
            F32, "db +=")


def test_public_calls_for_device_and_stream(moe, monkeypatch):
    """What a torch without the private names uses: the current stream all the same."""
    from mxfp4_routed_expert_router_amd import _block
    g = gen(2)
    x, w = randn(g, 40, 256, dtype=BF), randn(g, 96, 256, dtype=BF)
    want = moe.moe_fp4_linear(x, w)
    s = torch.cuda.Stream()
    monkeypatch.setattr(_block, "_device", torch.cuda.current_device)
    seen = []
    monkeypatch.setattr(_block, "_raw_stream", lambda i: seen.append(torch.cuda.current_stream(i).cuda_stream) or seen[-1])
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = moe.moe_fp4_linear(x, w)
    s.synchronize()
    assert seen == [s.cuda_stream] and torch.equal(got, want)
