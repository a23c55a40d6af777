"""The router's losses and their gradients against 64-bit references: every type,
both scores, expert counts from one to the most, ragged and empty sequences,
masks, masked experts, dropped and repeated choices, strides, and the gradients against
differences."""
import pytest
import torch

from block_common import U32, bounded, gen, padded, randn

pytestmark = pytest.mark.gpu

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
H32 = U32 / 2  # half a step of fp32
TINY = 2.0 ** -120  # what exponentials below the normal numbers may leave


@pytest.fixture(scope="module")
def moe():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mxfp4_routed_expert_router_amd as m
    return m


def scores64(l, sigmoid):
    """p, 1 - sigmoid (or 1), lse, softmax, and relative bounds of p, lse's absolute one.

    An exponential of l - m: the difference and the product with log2 e are rounded and
    log2 e is itself, 3 half steps of the exponent; the instruction adds a step.  For the
    softmax m is the row's largest; with sigmoids it may be 0, and |l - m| is below |l| +
    (largest - l) either way.  A row's sum has at most 24 + 6 additions; reciprocal and
    product 2 steps."""
    E = l.shape[1]
    m = l.amax(1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    e = torch.exp(l - m)
    s = e.sum(1, keepdim=True)
    inv = torch.where(s > 0, 1 / s, torch.zeros_like(s))
    soft = e * inv
    adds = 30
    far = torch.where(torch.isinf(l), torch.zeros_like(l), m - l)
    if sigmoid:
        far = far + torch.where(torch.isinf(l), torch.zeros_like(l), l.abs())
    r_e = 3 * H32 * far + U32
    r_s = (r_e * soft).sum(1, keepdim=True) + adds * U32
    r_soft = r_e + r_s + 2 * U32
    lse = torch.where(s > 0, m + torch.log(s), torch.zeros_like(s))
    e_lse = r_s + U32 * (m.abs() + 2 * torch.log(s.clamp(min=1)).abs() + lse.abs() + 1)
    if not sigmoid:
        return soft, torch.ones_like(l), lse, soft, r_soft, r_soft, torch.zeros_like(l), e_lse
    # log sigmoid keeps its digits where the sigmoids are all tiny
    ls = torch.nn.functional.logsigmoid(l)
    u = torch.exp(ls - torch.where(torch.isinf(ls.amax(1, keepdim=True)), torch.zeros_like(m), ls.amax(1, keepdim=True)))
    su = u.sum(1, keepdim=True)
    p = torch.where(su > 0, u / su, torch.zeros_like(u))
    # 1 / (1 + e e^m), off by what e and e^m are (|m| <= |l| where m < 0), the product, the sum and
    # the reciprocal by a step each; its product with e once more
    r_down = 3 * H32 * far + 5 * U32
    r_u = r_e + r_down + U32
    r_p = r_u + (r_u * p).sum(1, keepdim=True) + (adds + 2) * U32
    return p, torch.sigmoid(-l), lse, soft, r_soft, r_p, r_down, e_lse


def cuts_of(seqs, T):
    return [(0, T)] if seqs is None else list(zip(seqs.tolist(), seqs.tolist()[1:]))


def forward64(logits, idx, sigmoid, seqs, mask):
    l = logits.double()
    T, E = l.shape
    k = idx.shape[1]
    live = torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask.bool()
    p, _, lse, _, _, r_p, _, e_lse = scores64(torch.where(live[:, None], l, torch.zeros_like(l)), sigmoid)
    out = {n: [] for n in ("counts", "tokens", "probs", "balance", "z", "e_probs", "e_balance", "e_z")}
    for lo, hi in cuts_of(seqs, T):
        m = live[lo:hi]
        n = int(m.sum())
        ids = idx[lo:hi][m].reshape(-1).long()
        cnt = torch.bincount(ids[(ids >= 0) & (ids < E)], minlength=E).double()
        pr = p[lo:hi][m].sum(0)
        e_pr = (p[lo:hi][m] * r_p[lo:hi][m]).sum(0) + n * (U32 * pr + TINY)
        zz = lse[lo:hi][m].square().sum()
        e_zz = (2 * lse[lo:hi][m].abs() * e_lse[lo:hi][m] + e_lse[lo:hi][m] ** 2).sum() + (n + 2) * U32 * zz
        q, d = max(n, 1), E / (k * max(n, 1) ** 2)
        for name, v in zip(out, (cnt.int(), torch.tensor(n, dtype=torch.int32, device="cuda"), pr, d * (cnt * pr).sum(), zz / q,
                                 e_pr, d * (cnt * e_pr).sum() + U32 * d * (cnt * pr).sum(), e_zz / q)):
            out[name].append(v)
    return {n: torch.stack(v) for n, v in out.items()}


def check_forward(moe, logits, idx, sigmoid, seqs, mask):
    r = moe.moe_fp4_router_loss(logits, idx, score=int(sigmoid), seqs=seqs, mask=mask)
    w = forward64(logits, idx, sigmoid, seqs, mask)
    assert torch.equal(r.counts, w["counts"]) and torch.equal(r.tokens, w["tokens"])
    bounded(r.probs, w["probs"], w["e_probs"], F32, "probs")
    bounded(r.balance, w["balance"], w["e_balance"], F32, "balance")
    bounded(r.z, w["z"], w["e_z"], F32, "z")
    return r


def backward64(logits, idx, loss, dbalance, dz, gates, dgates, sigmoid, seqs, mask):
    """dlogits and its bound before the rounding; rows of no sequence are NaN."""
    l = logits.double()
    T, E = l.shape
    k = idx.shape[1]
    live = torch.ones(T, dtype=torch.bool, device="cuda") if mask is None else mask.bool()
    p, down, lse, soft, r_soft, r_p, r_down, e_lse = scores64(torch.where(live[:, None], l, torch.zeros_like(l)), sigmoid)
    d, e = torch.full_like(l, float("nan")), torch.zeros_like(l)
    adds = 30
    for s, (lo, hi) in enumerate(cuts_of(seqs, T)):
        if lo >= hi:
            continue
        n = max(1, int(loss.tokens[s]))
        c = (dbalance[s].double() * E / (k * n * n) * loss.counts[s].double()) if dbalance is not None else torch.zeros_like(l[0])
        q = p[lo:hi]
        a = q @ c
        e_a = ((r_p[lo:hi] + (adds + 4) * U32) * q) @ c.abs()
        t = q * (c - a[:, None]) * down[lo:hi]
        e_t = t.abs() * (r_p[lo:hi] + r_down[lo:hi] + 4 * U32) + q * down[lo:hi] * (e_a[:, None] + 4 * U32 * (c.abs() + a.abs()[:, None]))
        zc = 2 * dz[s].double() / n if dz is not None else torch.zeros((), dtype=torch.float64, device="cuda")
        zt = zc * lse[lo:hi] * soft[lo:hi]
        e_z = zt.abs() * (r_soft[lo:hi] + 4 * U32) + zc.abs() * e_lse[lo:hi] * soft[lo:hi]
        d[lo:hi] = t + zt
        e[lo:hi] = e_t + e_z + U32 * (t.abs() + zt.abs()) + TINY
    none = torch.isnan(d).all(1)
    if gates is not None:
        g, dg = gates.double(), dgates.double()
        inner, mag = (g * dg).sum(1, keepdim=True), (g * dg).abs().sum(1, keepdim=True)
        v = g * (dg - inner)
        e_v = g.abs() * ((k + 6) * U32 * (dg.abs() + mag))
        for j in range(k):
            ok = ((idx[:, j] >= 0) & (idx[:, j] < E)).nonzero()[:, 0]
            at = idx[ok, j].long()
            d[ok, at] += v[ok, j]
            e[ok, at] += e_v[ok, j] + U32 * d[ok, at].abs().nan_to_num() + U32 * v[ok, j].abs()
    d[~live & ~none] = 0
    e[~live] = 0
    return d, e, none


def batch(g, T, E, k, S, dt, masked, holes=False):
    logits = (randn(g, T, E, scale=3.0) + randn(g, E)).to(dt)
    if holes:  # experts that are out for some tokens; every token keeps those that it chose
        out = torch.rand(T, E, generator=g, device="cuda") < 0.3
        out.scatter_(1, torch.topk(logits.float(), k, dim=1).indices, False)
        logits[out] = float("-inf")
    top = torch.topk(logits.float(), k, dim=1)
    idx, gates = top.indices.to(torch.int32), torch.softmax(top.values, 1)
    seqs = None
    if S:
        c = torch.randint(0, T + 1, (S - 1,), generator=g, device="cuda").sort().values
        seqs = torch.cat([torch.zeros(1, device="cuda"), c, torch.full((1,), T, device="cuda")]).to(torch.int32)
    mask = (torch.rand(T, generator=g, device="cuda") < 0.7) if masked else None
    if masked:  # nothing of a masked token is read
        logits[~mask] = float("nan")
        idx[~mask] = 0
        gates[~mask] = float("nan")
    return logits, idx, gates, seqs, mask


SHAPES = [(1, 1, 1, 0), (1, 384, 6, 0), (5, 7, 2, 3), (64, 384, 6, 1), (33, 129, 16, 40), (300, 256, 4, 2), (257, 1024, 8, 5),
          (1000, 17, 3, 9), (5000, 384, 6, 8), (4099, 600, 2, 1), (700, 513, 5, 700), (9000, 64, 1, 3)]


@pytest.mark.parametrize("dt", [F32, BF, HF], ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,S", SHAPES)
def test_forward_and_backward(moe, T, E, k, S, score, dt):
    sigmoid = score == "sigmoid"
    for masked in (False, True):
        g = gen(T + E + masked)
        logits, idx, gates, seqs, mask = batch(g, T, E, k, S, dt, masked, holes=E > 20)
        r = check_forward(moe, logits, idx, sigmoid, seqs, mask)
        n = max(S, 1)
        dbal, dz, dg = randn(g, n), randn(g, n), randn(g, T, k)
        for out, db_, dz_, dg_ in ((dt, dbal, dz, dg), (F32, dbal, None, None), (F32, None, dz, None), (F32, None, None, dg),
                                   (BF if dt == F32 else dt, None, dz, dg)):
            got = moe.moe_fp4_router_loss_backward(logits, idx, r, dbalance=db_, dz=dz_, gates=gates if dg_ is not None else None,
                                                   dgates=dg_, score=int(sigmoid), seqs=seqs, mask=mask, out_dtype=out)
            want, e, none = backward64(logits, idx, r, db_, dz_, gates if dg_ is not None else None, dg_, sigmoid, seqs, mask)
            assert got.dtype == out and not bool(none.any())
            bounded(got, want, e, out, f"dlogits {out}")
            if masked:
                assert bool((got[~mask] == 0).all())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,S", [(40, 33, 3, 4), (17, 384, 6, 0)])
def test_gradients_against_differences(moe, T, E, k, S, score):
    """f(l) = sum_s a_s balance_s + b_s z_s + sum c gates, in 64 bits with the choices held:
    central differences along random directions."""
    sigmoid = score == "sigmoid"
    g = gen(T * E)
    logits, idx, gates, seqs, _ = batch(g, T, E, k, S, F32, False)
    r = moe.moe_fp4_router_loss(logits, idx, score=int(sigmoid), seqs=seqs)
    n = max(S, 1)
    a, b, c = randn(g, n), randn(g, n), randn(g, T, k)
    got = moe.moe_fp4_router_loss_backward(logits, idx, r, dbalance=a, dz=b, gates=gates, dgates=c, score=int(sigmoid),
                                           seqs=seqs).double()

    def f(l):
        p = torch.sigmoid(l) / torch.sigmoid(l).sum(1, keepdim=True) if sigmoid else torch.softmax(l, 1)
        lse = torch.logsumexp(l, 1)
        v = (torch.softmax(l.gather(1, idx.long()), 1) * c.double()).sum()
        for s, (lo, hi) in enumerate(cuts_of(seqs, T)):
            m = hi - lo
            if m > 0:
                v = v + a[s].double() * E / (k * m * m) * (r.counts[s].double() * p[lo:hi].sum(0)).sum()
                v = v + b[s].double() * lse[lo:hi].square().sum() / m
        return v

    h = 2.0 ** -14
    for _ in range(3):
        v = randn(g, T, E).double()
        diff = ((f(logits.double() + h * v) - f(logits.double() - h * v)) / (2 * h)).item()
        along = (got * v).sum().item()
        scale = (got.abs() * v.abs()).sum().item() + c.double().abs().sum().item() + b.double().abs().sum().item()
        # h^2 / 6 of third derivatives (of the terms' order times v^3, v below 5), the gates' fp32
        assert abs(diff - along) <= (32 * h * h + (E + 32) * U32) * scale, (diff, along)


@pytest.mark.parametrize("pad,offset", [(8, 8), (1, 0), (3, 1)])
@pytest.mark.parametrize("dt", [F32, BF])
def test_strides_alignment_and_rows_of_no_sequence(moe, dt, pad, offset):
    g = gen(pad)
    T, E, k = 50, 131, 4
    logits, idx, gates, _, _ = batch(g, T, E, k, 0, dt, False)
    seqs = torch.tensor([3, 3, 20, 41], dtype=torch.int32, device="cuda")
    view, _ = padded(logits, pad, offset)
    r = check_forward(moe, view, idx, False, seqs, None)
    out, buf = padded(torch.full((T, E), 7.0, dtype=dt, device="cuda"), pad, offset, fill=7.0)
    one, dg = torch.ones(3, device="cuda"), randn(g, T, k)
    moe.moe_fp4_router_loss_backward(view, idx, r, dbalance=one, dz=one, gates=gates, dgates=dg, seqs=seqs, dlogits=out)
    want, e, none = backward64(logits, idx, r, one, one, gates, dg, False, seqs, None)
    assert none.nonzero()[:, 0].tolist() == [0, 1, 2] + list(range(41, 50))
    bounded(out[~none], want[~none], e[~none], dt, "dlogits")
    left = buf.clone()
    left.as_strided(out.shape, out.stride(), offset)[~none] = 7.0
    assert bool((left == 7.0).all())


def test_accumulate_and_in_place(moe):
    g = gen(5)
    T, E, k = 70, 96, 3
    logits, idx, gates, seqs, mask = batch(g, T, E, k, 4, F32, True)
    logits = logits.nan_to_num()
    r = moe.moe_fp4_router_loss(logits, idx, seqs=seqs, mask=mask)
    a, dg = randn(g, 4), randn(g, T, k)
    kw = dict(dbalance=a, dz=a, gates=gates, dgates=dg, seqs=seqs, mask=mask)
    alone = moe.moe_fp4_router_loss_backward(logits, idx, r, **kw)
    for dt in (F32, BF):
        base = randn(g, T, E, dtype=dt)
        acc = base.clone()
        moe.moe_fp4_router_loss_backward(logits, idx, r, dlogits=acc, accumulate=True, **kw)
        if dt == F32:
            assert torch.equal(acc, base + alone)
        assert torch.equal(acc[~mask], base[~mask])
        bounded(acc, base.double() + alone.double(), U32 * (base.double() + alone.double()).abs(), dt, "+=")
    own = logits.clone()
    moe.moe_fp4_router_loss_backward(own, idx, r, dlogits=own, **kw)
    assert torch.equal(own, alone)


def test_dropped_and_repeated_choices(moe):
    g = gen(6)
    T, E, k = 30, 12, 4
    logits, idx, gates, _, _ = batch(g, T, E, k, 0, F32, False)
    idx[::2, 1] = idx[::2, 0]
    idx[1::3, 2] = -1
    idx[2::5, 3] = E
    idx[3::7, 0] = 2**31 - 1
    r = check_forward(moe, logits, idx, False, None, None)
    dg = randn(g, T, k)
    got = moe.moe_fp4_router_loss_backward(logits, idx, r, dbalance=torch.ones(1, device="cuda"), gates=gates, dgates=dg)
    want, e, _ = backward64(logits, idx, r, torch.ones(1, device="cuda"), None, gates, dg, False, None, None)
    bounded(got, want, e, F32, "dlogits")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_far_logits(moe, score):
    """Logits of 1e4 either way, a row of the lowest fp32 values, one of -inf alone, one with a
    single expert left."""
    sigmoid = score == "sigmoid"
    g = gen(7)
    T, E, k = 8, 70, 2
    logits = randn(g, T, E)
    logits[0] += 1e4
    logits[1] -= 1e4
    logits[2] = torch.finfo(F32).min
    logits[3] = float("-inf")
    logits[4] = float("-inf")
    logits[4, 5] = -300.0
    logits[5, :40] = -200.0 - torch.arange(40, device="cuda")
    logits[6] = -200.0 - torch.arange(70, device="cuda")
    idx = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    for rows in ([0], [1], [3], [4], [5], [6], [7], [0, 1, 3, 4, 5, 6, 7]):
        check_forward(moe, logits[rows], idx[rows], sigmoid, None, None)
    r = moe.moe_fp4_router_loss(logits[2:3], idx[2:3], score=int(sigmoid))
    # its square passes fp32
    assert torch.allclose(r.probs, torch.full_like(r.probs, 1 / E), rtol=1e-5) and r.z.item() == float("inf")
    one = torch.ones(1, device="cuda")
    r = moe.moe_fp4_router_loss(logits, idx, score=int(sigmoid))
    rows = [0, 1, 3, 4, 5, 6, 7]
    got = moe.moe_fp4_router_loss_backward(logits, idx, r, dbalance=one, dz=one, score=int(sigmoid))
    want, e, _ = backward64(logits[rows], idx[rows], r, one, one, None, None, sigmoid, None, None)
    bounded(got[rows], want, e, F32, "dlogits")
    assert bool((got[3] == 0).all())


def test_nan_and_inf_stay_in_their_sequence(moe):
    g = gen(8)
    logits = randn(g, 40, 20)
    logits[3, 7], logits[25, 0] = float("nan"), float("inf")
    idx = torch.zeros(40, 2, dtype=torch.int32, device="cuda")
    seqs = torch.tensor([0, 10, 20, 30, 40], dtype=torch.int32, device="cuda")
    r = moe.moe_fp4_router_loss(logits, idx, seqs=seqs)
    for t in (r.balance, r.z):
        assert torch.isnan(t).tolist() == [True, False, True, False]
    one = torch.ones(4, device="cuda")
    d = moe.moe_fp4_router_loss_backward(logits, idx, r, dbalance=one, dz=one, seqs=seqs)
    assert (~torch.isfinite(d).all(1)).nonzero()[:, 0].tolist() == [3, 25]


def test_no_tokens_and_empty_sequences(moe):
    for T, seqs in ((0, None), (0, [0, 0, 0]), (6, [0, 0, 6, 6]), (6, [6, 6])):
        s = None if seqs is None else torch.tensor(seqs, dtype=torch.int32, device="cuda")
        logits = torch.randn(T, 9, device="cuda")
        idx = torch.zeros(T, 2, dtype=torch.int32, device="cuda")
        r = check_forward(moe, logits, idx, False, s, None)
        one = torch.ones(r.balance.numel(), device="cuda")
        d = moe.moe_fp4_router_loss_backward(logits, idx, r, dbalance=one, dz=one, seqs=s)
        assert d.shape == (T, 9)
    # all tokens masked
    mask = torch.zeros(6, dtype=torch.bool, device="cuda")
    r = moe.moe_fp4_router_loss(logits, idx, mask=mask)
    assert r.tokens.item() == 0 and r.balance.item() == 0 and r.z.item() == 0 and not bool(r.probs.any())
    one = torch.ones(1, device="cuda")
    assert not bool(moe.moe_fp4_router_loss_backward(logits, idx, r, dbalance=one, dz=one, mask=mask).any())


def test_offsets_out_of_range_stay_inside(moe):
    """Offsets past the tokens or not ascending: no defined value, no access outside."""
    logits = torch.randn(50, 40, device="cuda")
    idx = torch.zeros(50, 2, dtype=torch.int32, device="cuda")
    for seqs in ([-5, 20, 1000], [40, 10, 30], [50, 0, 50]):
        s = torch.tensor(seqs, dtype=torch.int32, device="cuda")
        r = moe.moe_fp4_router_loss(logits, idx, seqs=s)
        one = torch.ones(2, device="cuda")
        moe.moe_fp4_router_loss_backward(logits, idx, r, dbalance=one, dz=one, seqs=s)
    s = torch.tensor([-5, 20, 1000], dtype=torch.int32, device="cuda")
    assert moe.moe_fp4_router_loss(logits, idx, seqs=s).tokens.tolist() == [20, 30]


def test_ranks_that_balance_together(moe):
    """Two halves of a batch with summed counts and tokens give the whole batch's gradient."""
    g = gen(9)
    logits, idx, _, _, _ = batch(g, 64, 24, 3, 0, F32, False)
    one = torch.ones(1, device="cuda")
    whole = moe.moe_fp4_router_loss(logits, idx)
    want = moe.moe_fp4_router_loss_backward(logits, idx, whole, dbalance=one, dz=one)
    halves = [moe.moe_fp4_router_loss(logits[r], idx[r]) for r in (slice(0, 20), slice(20, 64))]
    total = moe.RouterLoss(halves[0].counts + halves[1].counts, halves[0].tokens + halves[1].tokens,
                           halves[0].probs + halves[1].probs, None, None)
    got = torch.cat([moe.moe_fp4_router_loss_backward(logits[r], idx[r], total, dbalance=one, dz=one)
                     for r in (slice(0, 20), slice(20, 64))])
    assert torch.equal(got, want)


def test_route_gives_the_choices(moe):
    """A route's own choices and gates: its counts, and the gates' gradient against autograd."""
    g = gen(10)
    T, E, k = 90, 48, 6
    logits = randn(g, T, E)
    route = moe.moe_fp4_route(logits, k)
    r = moe.moe_fp4_router_loss(logits, route.topk_idx)
    assert torch.equal(r.counts[0], route.counts)
    dg = randn(g, T, k)
    got = moe.moe_fp4_router_loss_backward(logits, route.topk_idx, gates=route.gates, dgates=dg)
    want, e, _ = backward64(logits, route.topk_idx, r, None, None, route.gates, dg, False, None, None)
    bounded(got, want, e, F32, "dlogits")


def test_same_bits_twice_and_any_workspace(moe):
    g = gen(11)
    logits, idx, _, seqs, mask = batch(g, 6000, 384, 6, 5, BF, True)
    n = moe.moe_fp4_router_loss_workspace_size(6000, 384, 5)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    one = moe.moe_fp4_router_loss(logits, idx, seqs=seqs, mask=mask)
    two = moe.moe_fp4_router_loss(logits, idx, seqs=seqs, mask=mask, workspace=ws)
    for a, b in zip(vars(one).values(), vars(two).values()):
        assert torch.equal(a, b)
    with pytest.raises(moe.MoeFp4Error):
        moe.moe_fp4_router_loss(logits, idx, seqs=seqs, workspace=ws[:n - 4])


def test_rows_past_32_bits(moe):
    """2^20 tokens of 1024 experts at a row stride of 4200: element offsets past 2^32."""
    T, E = 1 << 20, 1024
    free, _ = torch.cuda.mem_get_info()
    if free < 30 << 30:
        pytest.skip("needs 30 GB")
    g = gen(12)
    buf = torch.empty(T, 4200, dtype=BF, device="cuda").normal_(generator=g)
    logits = buf[:, :E]
    idx = torch.arange(T, device="cuda", dtype=torch.int32)[:, None] % E
    seqs = torch.tensor([0, T - 100, T], dtype=torch.int32, device="cuda")
    r = moe.moe_fp4_router_loss(logits, idx, seqs=seqs)
    tail = logits[T - 100:]
    w = forward64(tail, idx[T - 100:], False, None, None)
    assert r.tokens.tolist() == [T - 100, 100] and torch.equal(r.counts[1], w["counts"][0])
    bounded(r.probs[1], w["probs"][0], w["e_probs"][0], F32, "probs")
    one = torch.ones(2, device="cuda")
    moe.moe_fp4_router_loss_backward(logits, idx, r, dbalance=one, dz=one, seqs=seqs, dlogits=logits)
    assert r.counts.sum().item() == T


def test_binding_refusals(moe):
    logits = torch.zeros(4, 8, device="cuda")
    idx = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    r = moe.moe_fp4_router_loss(logits, idx)
    one = torch.ones(1, device="cuda")
    with pytest.raises(TypeError):
        moe.moe_fp4_router_loss(logits.double(), idx)
    with pytest.raises(TypeError):
        moe.moe_fp4_router_loss(logits, idx.long())
    with pytest.raises(TypeError):
        moe.moe_fp4_router_loss(logits, None)
    with pytest.raises(ValueError):
        moe.moe_fp4_router_loss(logits, idx[:3])
    with pytest.raises(ValueError):
        moe.moe_fp4_router_loss(logits, idx, mask=torch.ones(5, dtype=torch.bool, device="cuda"))
    with pytest.raises(TypeError):
        moe.moe_fp4_router_loss(logits, idx, seqs=torch.tensor([0, 4], device="cuda"))
    with pytest.raises(moe.MoeFp4Error):
        moe.moe_fp4_router_loss(logits, idx, seqs=torch.zeros(1, dtype=torch.int32, device="cuda"))
    with pytest.raises(moe.MoeFp4Error):
        moe.moe_fp4_router_loss(logits, idx, score=2)
    with pytest.raises(moe.MoeFp4Error):
        moe.moe_fp4_router_loss(logits, torch.zeros(4, 9, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_fp4_router_loss_backward(logits, idx, r)
    with pytest.raises(ValueError):
        moe.moe_fp4_router_loss_backward(logits, idx, r, gates=torch.zeros(4, 2, device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_fp4_router_loss_backward(logits, idx, dz=one)
    with pytest.raises(ValueError):
        moe.moe_fp4_router_loss_backward(logits, idx, r, dz=one, accumulate=True)
    with pytest.raises(ValueError):
        moe.moe_fp4_router_loss_backward(logits, idx, r, dz=torch.ones(2, device="cuda"))
    with pytest.raises(TypeError):
        moe.moe_fp4_router_loss_backward(logits.to(BF), idx, r, dz=one, out_dtype=HF)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E", [(50001, 100), (30001, 384), (17001, 600)])
def test_tokens_behind_a_late_first_sequence(moe, T, E, score):
    """Sequences that start behind tokens of none, several tokens a group of lanes: every token from the
    first offset on has its gradient, the ones before keep what they held."""
    sigmoid = score == "sigmoid"
    g = gen(T)
    k = 3
    logits, idx, gates, _, _ = batch(g, T, E, k, 0, F32, False)
    a, b, dg = randn(g, 3), randn(g, 3), randn(g, T, k)
    for start in (1, 6, T // 2 + 1):
        seqs = torch.tensor([start, start + 4000, start + 4000, T - 2], dtype=torch.int32, device="cuda")
        r = moe.moe_fp4_router_loss(logits, idx, score=int(sigmoid), seqs=seqs)
        got = torch.full((T, E), 7.0, device="cuda")
        moe.moe_fp4_router_loss_backward(logits, idx, r, dbalance=a, dz=b, gates=gates, dgates=dg, score=int(sigmoid), seqs=seqs,
                                         dlogits=got)
        want, e, none = backward64(logits, idx, r, a, b, gates, dg, sigmoid, seqs, None)
        assert none.nonzero()[:, 0].tolist() == list(range(start)) + [T - 2, T - 1]
        assert bool((got[none] == 7.0).all())
        bounded(got[~none], want[~none], e[~none], F32, f"dlogits from {start} on")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradients_past_32_bits(moe, score):
    """2^20 tokens of 1024 experts at a row stride of 4200, the gradient over the logits: rows at both
    ends and between, and nothing beside the rows."""
    sigmoid = score == "sigmoid"
    T, E = 1 << 20, 1024
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GB")
    g = gen(15)
    buf = torch.empty(T, 4200, dtype=BF, device="cuda").normal_(generator=g)
    logits = buf[:, :E]
    idx = (torch.rand(T, 1, generator=g, device="cuda").square() * (E - 1)).to(torch.int32)
    start, cut = 37, T - 100
    seqs = torch.tensor([start, cut, T - 9], dtype=torch.int32, device="cuda")
    r = moe.moe_fp4_router_loss(logits, idx, score=int(sigmoid), seqs=seqs)
    assert r.tokens.tolist() == [cut - start, T - 9 - cut]
    rows = torch.cat([torch.arange(a, a + 300, device="cuda") for a in (0, T // 2 - 7, T - 300)])
    before, beside = logits[rows], buf[:, E:].clone()
    a, b = torch.tensor([1e6, 1.0], device="cuda"), torch.tensor([1e6, 1.0], device="cuda")
    moe.moe_fp4_router_loss_backward(logits, idx, r, dbalance=a, dz=b, score=int(sigmoid), seqs=seqs, dlogits=logits)
    assert torch.equal(buf[:, E:], beside)
    got = logits[rows]
    none = (rows < start) | (rows >= T - 9)
    assert torch.equal(got[none], before[none])
    for s, (lo, hi) in enumerate(((start, cut), (cut, T - 9))):
        of = (rows >= lo) & (rows < hi)
        one = moe.RouterLoss(r.counts[s:s + 1], r.tokens[s:s + 1], None, None, None)
        want, e, _ = backward64(before[of], idx[rows][of], one, a[s:s + 1], b[s:s + 1], None, None, sigmoid, None, None)
        bounded(got[of], want, e, BF, f"dlogits of sequence {s}")


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("size", [1e5, 1.1e6, 3e7, 1e9, 2e9, 1e10, 3e10, 1e20, 9e29, 2e30, 1e38])
def test_logits_of_any_magnitude(moe, size, score, dt):
    """Rows whose largest logits all lie at +-size: alone, or above others that are further down by
    `size`, whose exponentials are exactly 0.  The largest ones' exponentials are equal, off
    by a step; a sum of them by 30 additions, reciprocal and products by 6 more steps.  lse is off
    by that and its own roundings: of m log2 e and of the sum with m."""
    sigmoid = score == "sigmoid"
    T, E, k = 4, 70, 2
    logits = torch.empty(T, E, device="cuda")
    for t, c in enumerate((size, -size)):
        logits[2 * t], logits[2 * t + 1] = c, c - size
        logits[2 * t + 1, 5:12] = c
    logits = logits.to(dt)
    idx = torch.tensor([[5, 6]] * T, dtype=torch.int32, device="cuda")
    one = torch.ones(1, device="cuda")
    for t in range(T):
        row, ids = logits[t:t + 1], idx[t:t + 1]
        l = row.double()
        soft, lse = torch.softmax(l, 1), torch.logsumexp(l, 1).item()
        u = torch.nn.functional.logsigmoid(l)
        p, down = (torch.softmax(u, 1), torch.sigmoid(-l)) if sigmoid else (soft, torch.ones_like(l))
        r = moe.moe_fp4_router_loss(row, ids, score=int(sigmoid))
        bounded(r.probs, p, 36 * U32 * p, F32, f"probs {t}")
        counts = torch.zeros(1, E, dtype=torch.float64, device="cuda")
        counts[0, 5:7] = 1
        balance = E / k * (counts * p).sum(1)
        bounded(r.balance, balance, 37 * U32 * balance, F32, f"balance {t}")
        e_lse = U32 * (3 * abs(lse) + 44)
        if lse * lse < 3.3e38:
            assert abs(r.z.item() - lse * lse) <= 2 * abs(lse) * e_lse + e_lse ** 2 + U32 * lse * lse
        else:
            assert r.z.item() == float("inf")
        c = E / k * counts
        along = (p * c).sum(1, keepdim=True)
        d1 = p * (c - along) * down
        e1 = 80 * U32 * p * (c + along) * down
        d2 = 2 * lse * soft
        e2 = (44 * U32 * abs(lse) + e_lse) * 2 * soft
        for db, dz, want, e in ((one, None, d1, e1), (None, one, d2, e2), (one, one, d1 + d2, e1 + e2)):
            got = moe.moe_fp4_router_loss_backward(row, ids, r, dbalance=db, dz=dz, score=int(sigmoid), out_dtype=F32)
            bounded(got, want, e + TINY, F32, f"dlogits {t}")


def test_sigmoid_of_an_infinite_logit(moe):
    """Its probability and the balance loss's gradient are finite: that of its own logit is 0."""
    g = gen(13)
    T, E, k = 6, 40, 2
    logits = randn(g, T, E)
    logits[0, 4] = logits[1, 0] = logits[1, 1] = logits[3, 39] = float("inf")
    logits[3, 2], logits[3, 3] = 100.0, float("-inf")
    idx = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    r = moe.moe_fp4_router_loss(logits, idx, score=moe.SCORE_SIGMOID)
    s = torch.sigmoid(logits.double())
    p = s / s.sum(1, keepdim=True)
    # |l| below 8 or the sigmoid is 1 in fp32 (100: off by 2^-144): the exponent 24 half steps, 40 steps else
    rel = 64 * U32
    bounded(r.probs, p.sum(0)[None], (rel + T * U32) * p.sum(0)[None], F32, "probs")
    one = torch.ones(1, device="cuda")
    got = moe.moe_fp4_router_loss_backward(logits, idx, r, dbalance=one, score=moe.SCORE_SIGMOID)
    c = E / (k * T * T) * r.counts.double()
    along = p @ c.t()
    down = torch.sigmoid(-logits.double())
    bounded(got, p * (c - along) * down, 2 * rel * p * (c + along) * down + TINY, F32, "dlogits")
    assert not bool(got[torch.isinf(logits)].any())
    d = moe.moe_fp4_router_loss_backward(logits, idx, r, dbalance=one, dz=one, score=moe.SCORE_SIGMOID)
    assert (~torch.isfinite(d).all(1)).nonzero()[:, 0].tolist() == [0, 1, 3]


@pytest.mark.parametrize("E", [33, 384])
def test_gradients_of_saturated_sigmoids(moe, E):
    """1 - sigmoid of logits up to 90: e^-l keeps its digits down to the smallest normal numbers."""
    g = gen(14)
    T, k = 40, 4
    logits = (torch.arange(T, device="cuda")[:, None] * 2.25 + randn(g, T, E)).clamp(max=80.0)
    logits[::4, ::3] -= 30.0
    idx = torch.topk(logits, k, dim=1).indices.to(torch.int32)
    r = check_forward(moe, logits, idx, True, None, None)
    dbal = torch.full((1,), 1000.0, device="cuda")
    got = moe.moe_fp4_router_loss_backward(logits, idx, r, dbalance=dbal, score=moe.SCORE_SIGMOID)
    want, e, _ = backward64(logits, idx, r, dbal, None, None, None, True, None, None)
    bounded(got, want, e, F32, "dlogits")


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,starts", [(1000, 384, [7, 7, 300, 301, 301, 990]), (6000, 40, [2500, 2500, 5990, 5999]),
                                        (300, 700, [299, 300, 300]), (90, 20, [4 * i for i in range(11, 22)]), (4096, 130, [4096, 4096])])
def test_forward_of_late_sequences(moe, T, E, starts, score):
    """Tokens in front of the first sequence and behind the last one, which are in none."""
    g = gen(T + E)
    logits, idx, _, _, mask = batch(g, T, E, 2, 0, F32, True)
    seqs = torch.tensor(starts, dtype=torch.int32, device="cuda")
    r = check_forward(moe, logits, idx, score == "sigmoid", seqs, mask)
    assert int(r.tokens.sum()) == int(mask[starts[0]:starts[-1]].sum())


@pytest.mark.parametrize("dt", [F32, BF], ids=["f32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,S", [(60001, 40, 16, 1500), (40001, 384, 6, 700), (20001, 700, 16, 30)])
def test_several_sequences_of_a_group_of_lanes(moe, T, E, k, S, score, dt):
    """Batches that give a group of lanes several tokens, of several sequences, some of them empty or
    masked: into new results, added to what is there, over the logits."""
    sigmoid = score == "sigmoid"
    g = gen(T + S)
    logits, idx, gates, seqs, mask = batch(g, T, E, k, S, dt, True)
    logits = logits.nan_to_num()
    r = check_forward(moe, logits, idx, sigmoid, seqs, mask)
    a, b, dg = randn(g, S), randn(g, S), randn(g, T, k)
    kw = dict(dbalance=a, dz=b, gates=gates, dgates=dg, score=int(sigmoid), seqs=seqs, mask=mask)
    got = moe.moe_fp4_router_loss_backward(logits, idx, r, **kw)
    want, e, none = backward64(logits, idx, r, a, b, gates, dg, sigmoid, seqs, mask)
    assert not bool(none.any())
    bounded(got, want, e, dt, "dlogits")
    base = randn(g, T, E)
    acc = moe.moe_fp4_router_loss_backward(logits, idx, r, dlogits=base.clone(), accumulate=True, **kw)
    bounded(acc, base.double() + want, e + U32 * (base.double() + want).abs(), F32, "+=")
    assert torch.equal(acc[~mask], base[~mask])
    moe.moe_fp4_router_loss_backward(logits, idx, r, dlogits=logits, **kw)
    assert torch.equal(logits, got)
