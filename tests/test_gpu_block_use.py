"""The operators around the routed experts as a program uses them: one after the
other through a whole block and its backward pass, replayed from HIP graphs,
on several streams and host threads, and on arrays past 32 bits."""
import threading

import pytest
import torch

from block_common import U32, act64, bounded, gen, half_step, offsets_of, randn

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_routed_expert_router_amd as m
    return m


def block_forward(moe, p, x, k):
    """norm -> router -> experts' two products with silu between -> combine; a dense
    product beside; both added to the stream.  x [T, H] fp32."""
    u, mean, rstd = moe.moe_fp4_norm(x, p["gamma"], p["beta"], out_dtype=BF, save_stats=True)
    logits = moe.moe_fp4_router_logits(u, p["router"])
    r = moe.moe_fp4_route(logits, k)
    a = moe.moe_fp4_grouped_forward(u, p["up"], r.offsets, rows=r.sorted_pairs, row_div=k)
    h = torch.nn.functional.silu(a.float()).to(BF)
    yp = moe.moe_fp4_grouped_forward(h, p["down"], r.offsets, out_dtype=F32)
    slot = r.pair_slot.long()
    moe_out = (yp[slot].view(x.shape[0], k, -1) * r.gates[..., None]).sum(1)
    y, z = moe.moe_fp4_linear(u, p["w"], bias=p["b"], act=moe.ACT_GELU, residual=x, out_dtype=F32, save_z=True)
    return y + moe_out, dict(u=u, mean=mean, rstd=rstd, r=r, a=a, h=h, yp=yp, z=z)


def block_backward(moe, p, x, dy, s, k):
    """Gradients of the experts, the dense product, the norm and x (the gates' own
    gradient left out: they are constants here)."""
    T, r = x.shape[0], s["r"]
    gates = r.gates.reshape(-1)[r.sorted_pairs.long()]
    dyp = (dy[r.sorted_pairs.long() // k] * gates[:, None]).to(BF)
    ddown = moe.moe_fp4_grouped_wgrad(dyp, s["h"], r.offsets, out_dtype=F32)
    dh = moe.moe_fp4_grouped_dgrad(dyp, p["down"], r.offsets, out_dtype=F32)
    a = s["a"].float()
    sg = torch.sigmoid(a)
    da = (dh * sg * (1 + a * (1 - sg))).to(BF)
    dup = moe.moe_fp4_grouped_wgrad(da, s["u"], r.offsets, rows=r.sorted_pairs, row_div=k, out_dtype=F32)
    dup_rows = moe.moe_fp4_grouped_dgrad(da, p["up"], r.offsets, out_dtype=F32)
    du = dup_rows[r.pair_slot.long()].view(T, k, -1).sum(1)
    dlin, dw, db = moe.moe_fp4_linear_backward(dy, s["u"], p["w"], z=s["z"], act=moe.ACT_GELU, dw_dtype=F32)
    du = (du + dlin.float()).to(BF)
    dx, dgamma, dbeta = moe.moe_fp4_norm_backward(du, x, p["gamma"], s["mean"], s["rstd"])
    return dict(down=ddown, up=dup, w=dw, b=db, gamma=dgamma, beta=dbeta, x=dx + dy)


@pytest.mark.parametrize("T,E,k,H,N", [(70, 9, 3, 128, 96), (1, 5, 2, 256, 64), (33, 4, 4, 64, 160)])
def test_block_and_its_backward_pass(moe, T, E, k, H, N):
    """Against autograd of the same block in 64 bits, with this run's routing.  Each of
    about six roundings to bf16 on a path (u, a, h, dyp, da, du) is 2^-8 relative at
    most; norms of the differences, which add over the paths, stay within 2^-4."""
    g = gen(T + E)
    p = dict(gamma=1 + 0.1 * randn(g, H), beta=0.1 * randn(g, H), router=randn(g, E, H, dtype=BF, scale=H ** -0.5),
             up=randn(g, E, N, H, dtype=BF, scale=H ** -0.5), down=randn(g, E, H, N, dtype=BF, scale=N ** -0.5),
             w=randn(g, H, H, dtype=BF, scale=H ** -0.5), b=randn(g, H, dtype=BF))
    x, dy = randn(g, T, H), randn(g, T, H)
    y, s = block_forward(moe, p, x, k)
    got = block_backward(moe, p, x, dy, s, k)
    q = {n: t.double().requires_grad_(True) for n, t in p.items()}
    x64 = x.double().requires_grad_(True)
    with torch.enable_grad():
        m = x64.mean(1, keepdim=True)
        u = (x64 - m) / torch.sqrt((x64 - m).square().mean(1, keepdim=True) + 1e-6) * q["gamma"] + q["beta"]
        idx, gates = s["r"].topk_idx.long(), s["r"].gates.double()
        out = x64 + act64(u @ q["w"].t() + q["b"], "gelu")
        for j in range(k):
            up, down = q["up"][idx[:, j]], q["down"][idx[:, j]]
            h = act64(torch.matmul(up, u[:, :, None])[:, :, 0], "silu")
            out = out + gates[:, j:j + 1] * torch.matmul(down, h[:, :, None])[:, :, 0]
        out.backward(dy.double())
    want = {n: q[n].grad for n in ("down", "up", "w", "b", "gamma", "beta")}
    want["x"] = x64.grad
    for n, a, b in [("y", y, out.detach())] + [(n, got[n], want[n]) for n in want]:
        rel = ((a.double() - b).norm() / b.norm()).item()
        print(f"  {n}: rel {rel:.2e}", flush=True)
        assert rel <= 2.0 ** -4, (n, rel)


def calls(moe, x, dy, w, off, rows, k, lw, b, gamma):
    """Every operator once, all results."""
    y = moe.moe_fp4_grouped_forward(x, w, off, rows=rows, row_div=k)
    dx = moe.moe_fp4_grouped_dgrad(dy, w, off)
    dw = moe.moe_fp4_grouped_wgrad(dy, x, off, rows=rows, row_div=k, out_dtype=F32)
    l, z = moe.moe_fp4_linear(x, lw, bias=b, act=moe.ACT_SILU, residual=None, save_z=True)
    ldx, ldw, ldb = moe.moe_fp4_linear_backward(l, x, lw, z=z, act=moe.ACT_SILU)
    n, mean, rstd = moe.moe_fp4_norm(x, gamma, gamma, save_stats=True)
    ndx, dg, db = moe.moe_fp4_norm_backward(n, x, gamma, mean, rstd)
    return [y, dx, dw, l, z, ldx, ldw, ldb, n, mean, rstd, ndx, dg, db]


def inputs(g, T, E, k, N, K):
    x, lw, b = randn(g, T, K, dtype=BF), randn(g, N, K, dtype=BF, scale=K ** -0.5), randn(g, N, dtype=BF)
    w, dy, gamma = randn(g, E, N, K, dtype=BF), randn(g, T * k, N, dtype=BF), randn(g, K, dtype=BF)
    e = torch.randint(0, E, (T * k,), generator=g, device="cuda")
    rows = torch.argsort(e, stable=True).to(torch.int32)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.cumsum(torch.bincount(e, minlength=E), 0)
    return [x, dy, w, off, rows, k, lw, b, gamma]


SIZES = [(1, 8, 3, 96, 256), (5, 3, 2, 72, 2048), (150, 6, 2, 264, 136), (40, 5, 2, 33, 47)]


@pytest.mark.parametrize("size", SIZES)
def test_graph_replays_equal_eager(moe, size):
    """Captured once, replayed with new inputs in the captured buffers and eager work
    between the replays: the same bits as eager calls.  (Split sums and the weight
    gradients' parts take their workspaces inside the capture.)"""
    bufs = inputs(gen(1), *size)
    calls(moe, *bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls(moe, *bufs)
    for turn in range(4):
        new = inputs(gen(10 + turn), *size)
        for a, b in zip(bufs, new):
            if isinstance(a, torch.Tensor):
                a.copy_(b)
        graph.replay()
        want = calls(moe, *new)
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), (turn, i)


@pytest.mark.parametrize("size", SIZES)
def test_streams_and_threads(moe, size):
    """Four streams at once, then four host threads with a stream each, every one with
    its own data: the results of calls made alone."""
    sets = [inputs(gen(100 + i), *size) for i in range(4)]
    want = [calls(moe, *s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None] * 4
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = calls(moe, *sets[i])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))
    errors = []

    def work(i):
        try:
            with torch.cuda.stream(streams[i]):
                for _ in range(5):
                    got[i] = calls(moe, *sets[i])
        except Exception as e:  # noqa: BLE001 -- reported by the test
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_given_workspace_is_used_and_may_hold_anything(moe):
    g = gen(3)
    M, N, K = 40, 72, 5120
    x, w, dy = randn(g, M, K, dtype=BF), randn(g, N, K, dtype=BF), randn(g, M, N, dtype=BF)
    n = moe.moe_fp4_linear_workspace_size(M, N, K)
    assert n > 0  # a split sum
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")  # NaN in every type
    assert torch.equal(moe.moe_fp4_linear(x, w, workspace=ws), moe.moe_fp4_linear(x, w))
    n = moe.moe_fp4_linear_workspace_size(M, N, K, backward=True, act=moe.ACT_GELU)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    for a, b in zip(moe.moe_fp4_linear_backward(dy, x, w, z=dy, act=moe.ACT_GELU, workspace=ws),
                    moe.moe_fp4_linear_backward(dy, x, w, z=dy, act=moe.ACT_GELU)):
        assert torch.equal(a, b)
    n = moe.moe_fp4_norm_backward_workspace_size(M, K)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    r = torch.ones(M, device="cuda")
    for a, b in zip(moe.moe_fp4_norm_backward(x, x, x[0].contiguous(), r, r, workspace=ws),
                    moe.moe_fp4_norm_backward(x, x, x[0].contiguous(), r, r)):
        assert torch.equal(a, b)
    P, E = 4200, 2
    off = offsets_of([2500, 1700])
    x, dy = randn(g, P, 64, dtype=BF), randn(g, P, 32, dtype=BF)
    n = moe.moe_fp4_grouped_workspace_size(E, P, 32, 64, moe.GROUPED_WGRAD)
    assert n > 0
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(moe.moe_fp4_grouped_wgrad(dy, x, off, workspace=ws), moe.moe_fp4_grouped_wgrad(dy, x, off))
    with pytest.raises(moe.MoeFp4Error):
        moe.moe_fp4_grouped_wgrad(dy, x, off, workspace=ws[:n - 256])


def test_weights_past_32_bits(moe):
    """All 384 experts of a layer's w1 in 16 bits: 9 GB, element offsets past 2^32."""
    E, N, K = 384, 2304, 5120
    free, _ = torch.cuda.mem_get_info()
    if free < 24 << 30:
        pytest.skip("needs 24 GB")
    g = gen(5)
    w = torch.empty(E, N, K, dtype=BF, device="cuda").normal_(generator=g)
    for counts in ({0: 1, 200: 2, 383: 3}, {0: 300, 383: 290}):
        c = [counts.get(e, 0) for e in range(E)]
        P = sum(c)
        off = offsets_of(c)
        x, dy = randn(g, P, K, dtype=BF), randn(g, P, N, dtype=BF)
        y = moe.moe_fp4_grouped_forward(x, w, off, out_dtype=F32)
        dx = moe.moe_fp4_grouped_dgrad(dy, w, off, out_dtype=F32)
        for e in counts:
            r = slice(sum(c[:e]), sum(c[:e + 1]))
            w64, x64, d64 = w[e].double(), x[r].double(), dy[r].double()
            bounded(y[r], x64 @ w64.t(), K * U32 * (x64.abs() @ w64.abs().t()), F32, "y")
            bounded(dx[r], d64 @ w64, N * U32 * (d64.abs() @ w64.abs()), F32, "dx")
    dw = moe.moe_fp4_grouped_wgrad(dy, x, off)
    for e in (0, 383):
        r = slice(0, 300) if e == 0 else slice(300, 590)
        d64, x64 = dy[r].double(), x[r].double()
        bounded(dw[e], d64.t() @ x64, 300 * U32 * (d64.abs().t() @ x64.abs()), BF, "dw")
    assert bool((dw[100] == 0).all())


def test_rows_past_32_bits(moe):
    """2^20 rows of 4104 elements: row offsets past 2^32 elements."""
    T, H = 1 << 20, 4104
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    g = gen(6)
    x = torch.empty(T, H, dtype=BF, device="cuda").normal_(generator=g)
    w = randn(g, 16, H, dtype=BF)
    tail = slice(T - 70, T)
    y = moe.moe_fp4_linear(x, w, out_dtype=F32)
    x64, w64 = x[tail].double(), w.double()
    bounded(y[tail], x64 @ w64.t(), H * U32 * (x64.abs() @ w64.abs().t()), F32, "linear")
    off = torch.tensor([0, 5, T], dtype=torch.int32, device="cuda")
    idx = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")
    y = moe.moe_fp4_grouped_forward(x, torch.stack([w, -w]), off, rows=idx, out_dtype=F32)
    h64 = x[T - 5:].double().flip(0)
    bounded(y[:5], h64 @ w64.t(), H * U32 * (h64.abs() @ w64.abs().t()), F32, "gathered, first expert")
    n, mean, rstd = moe.moe_fp4_norm(x, save_stats=True)
    m = x64.mean(1, keepdim=True)
    sd = torch.sqrt((x64 - m).square().mean(1, keepdim=True) + 1e-6)
    assert ((n[tail].double() - (x64 - m) / sd).abs() <= 2 * half_step(BF) * ((x64 - m) / sd).abs() + 1e-4).all()
    dx, _, _ = moe.moe_fp4_norm_backward(x, x, None, mean, rstd)
    hat = (x64 - m) / sd
    want = (x64 - x64.mean(1, keepdim=True) - hat * (x64 * hat).mean(1, keepdim=True)) / sd
    # what is left after the projections is rounding of the terms, of order 1
    assert (dx[tail].double() - want).abs().max().item() <= 1e-4
