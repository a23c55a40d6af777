"""The router's losses, the gradients' clipping and the 4-bit product as a program uses them:
a training step of a router with the operators around it, a served layer, replays from HIP
graphs, several streams and host threads."""
import threading

import pytest
import torch

from block_common import gen, randn

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_routed_expert_router_amd as m
    return m


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,H", [(96, 24, 3, 128), (300, 64, 6, 256)])
def test_a_routers_training_step(moe, T, E, k, H, score):
    """norm -> router logits -> route -> losses; their gradient with the gates' through the router's
    product and the norm, then the gradients' norm and clipping: against autograd of the same
    in 64 bits with this run's choices.  u and dlogits are rounded to bf16 on the way (2^-8
    relative each); norms of the differences stay within 2^-5."""
    g = gen(T + E)
    x, gamma, beta = randn(g, T, H), 1 + 0.1 * randn(g, H), 0.1 * randn(g, H)
    w = randn(g, E, H, dtype=BF, scale=2 * H ** -0.5)
    v = randn(g, T, E)  # what an expert's output is worth to the loss
    seqs = torch.tensor([0, T // 3, T], dtype=torch.int32, device="cuda")
    mask = torch.rand(T, generator=g, device="cuda") < 0.8
    a, b = torch.tensor([0.3, 0.5], device="cuda"), torch.tensor([0.02, 0.01], device="cuda")
    sc = moe.SCORE_SIGMOID if score == "sigmoid" else moe.SCORE_SOFTMAX

    u, mean, rstd = moe.moe_fp4_norm(x, gamma, beta, out_dtype=BF, save_stats=True)
    logits = moe.moe_fp4_router_logits(u, w)
    route = moe.moe_fp4_route(logits, k)
    loss = moe.moe_fp4_router_loss(logits, route.topk_idx, score=sc, seqs=seqs, mask=mask)
    dgates = v.gather(1, route.topk_idx.long())
    dlogits = moe.moe_fp4_router_loss_backward(logits, route.topk_idx, loss, dbalance=a, dz=b, gates=route.gates, dgates=dgates,
                                               score=sc, seqs=seqs, mask=mask)
    du, dw, _ = moe.moe_fp4_linear_backward(dlogits, u, w, need_db=False, dw_dtype=F32)
    dx, dgamma, dbeta = moe.moe_fp4_norm_backward(du, x, gamma, mean, rstd)
    grads = [dw, dgamma, dbeta]
    before = [t.clone() for t in grads]
    norm = moe.moe_fp4_grad_clip(grads, moe.moe_fp4_grad_sumsq(grads), 0.1)

    q = [t.double().requires_grad_(True) for t in (w, gamma, beta, x)]
    with torch.enable_grad():
        xm = q[3] - q[3].mean(1, keepdim=True)
        u64 = xm / torch.sqrt(xm.square().mean(1, keepdim=True) + 1e-6) * q[1] + q[2]
        l = u64 @ q[0].t()
        p = torch.softmax(l, 1) if score == "softmax" else torch.sigmoid(l) / torch.sigmoid(l).sum(1, keepdim=True)
        total = (torch.softmax(l.gather(1, route.topk_idx.long()), 1) * dgates.double())[mask].sum()
        lse = torch.logsumexp(l, 1)
        for s, (lo, hi) in enumerate(((0, T // 3), (T // 3, T))):
            m = mask[lo:hi]
            n = int(m.sum())
            counts = torch.bincount(route.topk_idx[lo:hi][m].flatten().long(), minlength=E).double()
            bal = E / (k * n * n) * (counts * p[lo:hi][m].sum(0)).sum()
            z = lse[lo:hi][m].square().sum() / n
            assert abs(loss.balance[s].item() - bal.item()) <= 2.0 ** -7 * bal.item() and int(loss.tokens[s]) == n
            assert abs(loss.z[s].item() - z.item()) <= 2.0 ** -5 * z.item()
            total = total + a[s].double() * bal + b[s].double() * z
        total.backward()
    for name, got, want in (("w", before[0], q[0].grad), ("gamma", before[1], q[1].grad), ("beta", before[2], q[2].grad),
                            ("x", dx, q[3].grad)):
        rel = ((got.double() - want).norm() / want.norm()).item()
        print(f"  {name}: rel {rel:.2e}", flush=True)
        assert rel <= 2.0 ** -5, (name, rel)
    whole = torch.cat([t.flatten() for t in before]).double().norm().item()
    assert abs(norm.item() - whole) <= 1e-6 * whole and whole > 0.1
    clipped = torch.cat([t.flatten() for t in grads]).double().norm().item()
    assert abs(clipped - 0.1) <= 1e-5


def test_a_served_dense_layer_in_four_bits(moe):
    """norm -> up -> down with the residual added, one token and a batch, in both formats: the
    16-bit operator's results on the decoded weights, but for roundings of h (2^-8)."""
    g = gen(3)
    H, I = 512, 768
    e2m1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6], device="cuda")

    def make(N, K, mx):
        codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        c = torch.stack([codes & 15, codes >> 4], dim=2).reshape(N, K)
        if mx:
            s = torch.randint(117, 120, (N, K // 32), generator=g, device="cuda", dtype=torch.uint8)
            return moe.W4Weights(codes, s), (e2m1[c.long()] * torch.exp2(s.float() - 127).repeat_interleave(32, 1)).to(BF)
        s = torch.full((N, K // 64), 2.0 ** -7, device="cuda", dtype=BF)
        return moe.W4Weights(codes, s, None, 64), ((c.float() - 8) * 2.0 ** -7).to(BF)

    for mx in (True, False):
        up, up16 = make(I, H, mx)
        down, down16 = make(H, I, mx)
        for M in (1, 5, 40):
            x = randn(g, M, H)
            u = moe.moe_fp4_norm(x, kind=moe.NORM_RMS, out_dtype=BF)
            y = moe.moe_fp4_linear_w4(moe.moe_fp4_linear_w4(u, up, act=moe.ACT_SILU), down, residual=x, out_dtype=F32)
            want = moe.moe_fp4_linear(moe.moe_fp4_linear(u, up16, act=moe.ACT_SILU), down16, residual=x, out_dtype=F32)
            assert ((y - want).norm() / (want - x).norm()).item() <= 2.0 ** -8, (mx, M)


def inputs(moe, g, T, E, k, S, K):
    logits = randn(g, T, E, scale=2.0)
    top = torch.topk(logits, k, dim=1)
    cuts = torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda").sort().values
    seqs = torch.cat([torch.zeros(1, device="cuda"), cuts, torch.full((1,), T, device="cuda")]).to(torch.int32)
    grads = [randn(g, n, dtype=dt) for n, dt in ((70001, F32), (5, BF), (40000, HF))]
    x = [randn(g, m, K, dtype=BF) for m in (1, 7, 40)]
    codes = torch.randint(0, 256, (200, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    wide = torch.randint(0, 256, (20481, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.randint(118, 124, (20481, K // 32), generator=g, device="cuda", dtype=torch.uint8)
    int4 = randn(g, 200, (K + 63) // 64, dtype=BF)
    return [logits, top.indices.to(torch.int32), torch.softmax(top.values, 1), randn(g, T, k), seqs,
            torch.rand(T, generator=g, device="cuda") < 0.8, randn(g, S), randn(g, S)] + grads + x + [codes, wide, scales, int4]


def calls(moe, logits, idx, gates, dgates, seqs, mask, a, b, g0, g1, g2, x0, x1, x2, codes, wide, scales, int4):
    """Every operator, in each of its kernels; all results."""
    outs = []
    for sc in (moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID):
        r = moe.moe_fp4_router_loss(logits, idx, score=sc, seqs=seqs, mask=mask)
        outs += list(vars(r).values())
        outs.append(moe.moe_fp4_router_loss_backward(logits, idx, r, dbalance=a, dz=b, gates=gates, dgates=dgates, score=sc, seqs=seqs,
                                                     mask=mask))
    r = moe.moe_fp4_router_loss(logits[:60], idx[:60])
    outs += list(vars(r).values())
    ss = moe.moe_fp4_grad_sumsq([g0, g1, g2])
    clipped = [torch.empty_like(t) for t in (g0, g1, g2)]
    outs += [ss, moe.moe_fp4_grad_clip([g0, g1, g2], ss, 1.0, out=clipped)] + clipped
    ws = [moe.W4Weights(codes, scales[:200]), moe.W4Weights(codes, int4, None, 64), moe.W4Weights(wide, scales)]
    outs += [moe.moe_fp4_linear_w4(x, w, act=moe.ACT_SILU, out_dtype=F32) for w in ws for x in (x0, x1, x2)]
    return outs


SIZES = [(700, 48, 4, 3, 1024), (5000, 384, 6, 9, 1184)]


@pytest.mark.parametrize("size", SIZES)
def test_graph_replays_equal_eager(moe, size):
    """Captured once, replayed with new inputs in the captured buffers and eager work between the
    replays: the same bits as eager calls."""
    bufs = inputs(moe, gen(1), *size)
    calls(moe, *bufs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = calls(moe, *bufs)
    for turn in range(4):
        new = inputs(moe, gen(10 + turn), *size)
        for p, q in zip(bufs, new):
            p.copy_(q)
        graph.replay()
        want = calls(moe, *new)
        torch.cuda.synchronize()
        for i, (p, q) in enumerate(zip(outs, want)):
            assert torch.equal(p, q), (turn, i)


@pytest.mark.parametrize("size", SIZES)
def test_streams_and_threads(moe, size):
    """Four streams at once, then four host threads with a stream each, every one with its own
    data: the results of calls made alone."""
    sets = [inputs(moe, gen(100 + i), *size) for i in range(4)]
    want = [calls(moe, *s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [None] * 4
    for _ in range(3):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                got[i] = calls(moe, *sets[i])
    torch.cuda.synchronize()
    for p, q in zip(got, want):
        assert all(torch.equal(s, t) for s, t in zip(p, q))
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
    for p, q in zip(got, want):
        assert all(torch.equal(s, t) for s, t in zip(p, q))


def test_many_tensors_in_a_graph(moe):
    """More tensors than one launch's arguments hold, in place, replayed."""
    g = gen(7)
    grads = [randn(g, 100 + i, dtype=(F32, BF)[i % 2]) for i in range(300)]
    keep = [t.clone() for t in grads]
    graph = torch.cuda.CUDAGraph()
    moe.moe_fp4_grad_clip(grads, moe.moe_fp4_grad_sumsq(grads), 1.0)
    want = [t.clone() for t in grads]
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        norm = moe.moe_fp4_grad_clip(grads, moe.moe_fp4_grad_sumsq(grads), 1.0)
    whole = torch.stack([t.double().square().sum() for t in keep]).sum().sqrt().item()
    for _ in range(3):
        for t, k in zip(grads, keep):
            t.copy_(k)
        graph.replay()
        torch.cuda.synchronize()
        assert abs(norm.item() - whole) <= 1e-6 * whole
        assert all(torch.equal(a, b) for a, b in zip(grads, want))
