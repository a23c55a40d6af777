"""The operators around the routed experts at the ends of their types' ranges."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


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
