"""The operators that a routed layer's training step and its serving need beside its
products, as they are used: the router's losses with the gradient of its logits,
the gradients' global norm with clipping, and the dense product with 4-bit
weights and group scales.

A case names one pass.  `prepare` makes what a program holds before it, `run`
makes the calls: in plain torch operations in 32 bits, or, where `own` is true,
through this repository's package.  `exact` gives the same outputs from the
definitions in 64 bits.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
NORM_EPS = 1e-6


# ---------------------------------------------------------------- the cases
def listed():
    H, I, E, k = 5120, 2304, 384, 6  # the layer's sizes
    return [
        # one micro-batch of a few tokens through the router's losses: latency alone
        {"name": "router_loss_few_tokens", "op": "router", "dir": "fwd", "type": "f32", "out": "f32", "score": "softmax",
         "T": 64, "E": E, "k": k, "S": 1, "pad": 0.0},
        # a training batch of eight ragged sequences, an eighth of it padding; balance by sequence
        {"name": "router_loss_batch", "op": "router", "dir": "fwd", "type": "f32", "out": "f32", "score": "softmax",
         "T": 16384, "E": E, "k": k, "S": 8, "pad": 0.125},
        # its gradient: both losses and the gates', into fp32 logits' gradients
        {"name": "router_backward_batch", "op": "router", "dir": "bwd", "type": "f32", "out": "f32", "score": "softmax",
         "T": 16384, "E": E, "k": k, "S": 8, "pad": 0.125},
        # the longest batch, sigmoid scores, 16-bit logits
        {"name": "router_backward_long", "op": "router", "dir": "bwd", "type": "bf16", "out": "bf16", "score": "sigmoid",
         "T": 65536, "E": E, "k": k, "S": 64, "pad": 0.0},
        # the gradients of a block's norms, biases and router: a few small tensors
        {"name": "clip_small", "op": "clip", "types": "f32", "out": "same", "count": 7, "lo": 384, "hi": 36864,
         "step": 1, "max_norm": 1.0},
        # a model's dense gradients in 16 bits: many tensors, odd sizes among them
        {"name": "clip_many", "op": "clip", "types": "bf16", "out": "same", "count": 150, "lo": 1024, "hi": 4000000,
         "step": 1, "max_norm": 1.0},
        # one GPU's 48 experts: their fp32 main gradients, and 16-bit ones beside
        {"name": "clip_experts", "op": "clip", "types": "f32,bf16", "out": "same", "count": 2, "lo": 48 * I * H,
         "hi": 48 * I * H, "step": 8, "max_norm": 1.0},
        # one token through one GPU's share of a projection, in the checkpoint's 4-bit format
        {"name": "w4_share_of_8_one_token", "op": "w4", "type": "bf16", "out": "bf16", "code": "mx", "group": 32,
         "M": 1, "N": I // 8, "K": H, "zeros": False, "act": "none", "bias": False, "residual": False},
        # one token through a dense layer's up product
        {"name": "w4_one_token", "op": "w4", "type": "bf16", "out": "bf16", "code": "mx", "group": 32,
         "M": 1, "N": 4 * I, "K": H, "zeros": False, "act": "silu", "bias": False, "residual": False},
        # a decode batch through its down product, added to the 32-bit residual stream
        {"name": "w4_batch", "op": "w4", "type": "bf16", "out": "f32", "code": "int4", "group": 128,
         "M": 16, "N": H, "K": 4 * I, "zeros": False, "act": "none", "bias": True, "residual": True},
        # odd sizes, zero points, the other type
        {"name": "w4_odd", "op": "w4", "type": "f16", "out": "f16", "code": "int4", "group": 64,
         "M": 5, "N": 1001, "K": I, "zeros": True, "act": "gelu", "bias": True, "residual": False},
        # a larger decode batch on the widest weight
        {"name": "w4_wide", "op": "w4", "type": "bf16", "out": "bf16", "code": "mx", "group": 32,
         "M": 64, "N": 65536, "K": H, "zeros": False, "act": "none", "bias": False, "residual": False},
    ]


def _size(rng, lo, hi, step):
    """A size between lo and hi, even over its logarithm: a multiple of `step`, or any."""
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))
    if rng.random() < 0.7:
        v = (v + step // 2) // step * step
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["router", "router", "clip", "w4", "w4", "w4"])
    ty = rng.choice(["bf16", "bf16", "f16"])
    if op == "router":
        lt = rng.choice(["f32", "f32", ty])
        E = _size(rng, 2, 1024, 8)
        T = _size(rng, 1, 65536, 8)
        while T * E > 65536 * 384:
            T = max(1, T // 2)
        return {"op": op, "dir": rng.choice(["fwd", "bwd"]), "type": lt, "out": "bf16" if lt == "bf16" and rng.random() < 0.5 else "f32",
                "score": rng.choice(["softmax", "sigmoid"]), "T": T, "E": E, "k": rng.randint(1, min(E, 8)),
                "S": min(T, _size(rng, 1, 64, 1)), "pad": rng.choice([0.0, 0.125, 0.5])}
    if op == "clip":
        count = _size(rng, 1, 200, 1)
        hi = _size(rng, 1000, 48 * 2304 * 5120 // max(8, count), 8)
        return {"op": op, "types": rng.choice(["f32", "bf16", "f16", "f32,bf16"]), "out": rng.choice(["same", "same", "bf16"]),
                "count": count, "lo": max(1, hi // rng.choice([1, 10, 1000])), "hi": hi, "step": rng.choice([1, 8]),
                "max_norm": rng.choice([1.0, 1.0, 1e9])}
    code = rng.choice(["mx", "int4"])
    M, N, K = _size(rng, 1, 64, 1), _size(rng, 32, 65536, 32), 32 * _size(rng, 1, 288, 4)
    while N * K > 65536 * 5120:
        N = max(32, N // 2)
    return {"op": op, "type": ty, "out": rng.choice([ty, "f32"]), "code": code,
            "group": 32 if code == "mx" else rng.choice([32, 64, 128]), "M": M, "N": N, "K": K,
            "zeros": code == "int4" and rng.random() < 0.5, "act": rng.choice(["none", "gelu", "silu"]),
            "bias": rng.random() < 0.5, "residual": rng.random() < 0.5}


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 2 + 1)
    return g


def _randn(g, *shape, dtype, scale=1.0):
    t = torch.randn(*shape, generator=g, device="cuda", dtype=dtype)
    return t if scale == 1.0 else t.mul_(scale)


def _cuts(g, T, S):
    """Ragged sequences end to end: S + 1 offsets from 0 to T, none of them empty."""
    inner = torch.randperm(T - 1, generator=g, device="cuda")[:S - 1].sort().values + 1
    ends = torch.tensor([0, T], device="cuda")
    return torch.cat([ends[:1], inner, ends[1:]]).to(torch.int32)


def _sizes(case):
    """The tensors' sizes: even over their logarithm, small ones among large ones."""
    lo, hi, step, count = case["lo"], case["hi"], case["step"], case["count"]
    n = [int(lo * (hi / lo) ** ((i + 0.5) / count)) for i in range(count)]
    n = [max(1, min(hi, (v + step - 1) // step * step)) for v in n]
    return n[0::3] + n[1::3] + n[2::3]


def _flat(tensors, kinds, dtypes):
    """A buffer of zeros for the tensors of each of `kinds`, and their places in it."""
    at, size = [], {}
    for t, kind in zip(tensors, kinds):
        at.append(size.get(kind, 0))
        size[kind] = at[-1] + (t.numel() + 7) // 8 * 8
    kind_dtype = dict(zip(kinds, dtypes))
    flat = {kind: torch.zeros(n, dtype=kind_dtype[kind], device="cuda") for kind, n in size.items()}
    return list(flat.values()), [flat[kind][a:a + t.numel()] for t, kind, a in zip(tensors, kinds, at)]


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case)
    if case["op"] == "router":
        T, E, k, S = (case[n] for n in ("T", "E", "k", "S"))
        s["dt"], s["odt"] = DT[case["type"]], DT[case["out"]]
        # logits with popular experts; a sequence's last tokens are padding
        bias = torch.randn(E, generator=g, device="cuda")
        s["logits"] = (1.5 * torch.randn(T, E, generator=g, device="cuda") + bias).to(s["dt"])
        top = torch.topk(s["logits"].float(), k, dim=1)
        s["idx"] = top.indices.to(torch.int32)
        s["gates"] = torch.softmax(top.values, 1)
        s["seqs"] = _cuts(g, T, S)
        s["cuts"] = s["seqs"].tolist()  # the program packed the batch
        lens = (s["seqs"][1:] - s["seqs"][:-1]).long()
        s["seg"] = torch.repeat_interleave(torch.arange(S, device="cuda"), lens)
        place = torch.arange(T, device="cuda") - s["seqs"][:-1].long()[s["seg"]]
        s["mask"] = place < (lens.double() * (1 - case["pad"])).ceil()[s["seg"]] if case["pad"] else None
        if case["dir"] == "bwd":
            # what the forward pass left, and the gradients of the losses (their weights) and gates
            s.update(_router_plain(s))
            s["dbalance"] = 0.01 * (0.5 + torch.rand(S, generator=g, device="cuda"))
            s["dz"] = 0.001 * (0.5 + torch.rand(S, generator=g, device="cuda"))
            s["dgates"] = 0.01 * torch.randn(T, k, generator=g, device="cuda")
    elif case["op"] == "clip":
        types = [DT[t] for t in case["types"].split(",")]
        # gradients: each tensor at its own scale
        s["grads"] = [_randn(g, n, dtype=types[i % len(types)], scale=10.0 ** -(i % 4)) for i, n in enumerate(_sizes(case))]
        # where the clipped ones go: flat buffers of each type, every tensor on a 16-byte boundary
        odt = [t.dtype if case["out"] == "same" or t.dtype != torch.float32 else DT[case["out"]] for t in s["grads"]]
        s["flat"], s["outs"] = _flat(s["grads"], odt, odt)
    else:
        M, N, K, group = (case[n] for n in ("M", "N", "K", "group"))
        s["dt"], s["odt"] = DT[case["type"]], DT[case["out"]]
        s["x"] = _randn(g, M, K, dtype=s["dt"])
        s["codes"] = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        G = (K + group - 1) // group
        down = 2 - int(math.log2(K) / 2)  # scales about 1 / sqrt(K)
        s["zeros"] = None
        if case["code"] == "mx":
            s["scales"] = torch.randint(125 + down - 4, 125 + down, (N, G), generator=g, device="cuda", dtype=torch.uint8)
        else:
            s["scales"] = ((0.5 + torch.rand(N, G, generator=g, device="cuda")) * 2.0 ** (down - 4)).to(s["dt"])
            if case["zeros"]:
                s["zeros"] = torch.randint(4, 12, (N, G), generator=g, device="cuda", dtype=torch.uint8)
        s["b"] = _randn(g, N, dtype=s["dt"]) if case["bias"] else None
        s["r"] = _randn(g, M, N, dtype=s["odt"]) if case["residual"] else None
        if own:
            import mxfp4_routed_expert_router_amd as moe
            s["w"] = moe.W4Weights(s["codes"], s["scales"], s["zeros"], group)
    return s


# ---------------------------------------------------------------- the plain forms
def _scores(l, score):
    """The probabilities of rows of logits, and the sigmoids where they are made of those."""
    if score == "softmax":
        e = torch.exp(l - l.amax(1, keepdim=True))
        return e / e.sum(1, keepdim=True), None
    sg = 1 / (1 + torch.exp(-l))
    return sg / sg.sum(1, keepdim=True), sg


def _lse(l):
    m = l.amax(1)
    return m + torch.log(torch.exp(l - m[:, None]).sum(1))


def _router_plain(s):
    l = s["logits"].float()
    S, E, k = s["S"], s["E"], s["k"]
    live = s["mask"] if s["mask"] is not None else torch.ones_like(s["seg"], dtype=torch.bool)
    p, _ = _scores(l, s["score"])
    p = torch.where(live[:, None], p, 0.0)
    counts = torch.zeros(S * E, dtype=torch.int32, device=l.device)
    at = (s["seg"][:, None] * E + s["idx"].long())[live].reshape(-1)
    counts.index_add_(0, at, torch.ones_like(at, dtype=torch.int32))
    counts = counts.view(S, E)
    tokens = torch.zeros(S, dtype=torch.int32, device=l.device)
    tokens.index_add_(0, s["seg"], live.to(torch.int32))
    # long sums of many small terms, and squares: in 64 bits
    zz = torch.where(live, _lse(l).double().square(), 0.0)
    at = list(zip(s["cuts"], s["cuts"][1:]))
    probs = torch.stack([p[lo:hi].sum(0, dtype=torch.float64) for lo, hi in at])
    zsum = torch.stack([zz[lo:hi].sum() for lo, hi in at])
    n = torch.clamp(tokens, min=1).double()
    balance = (counts.double() * probs).sum(1) * (E / k) / (n * n)
    return {"counts": counts, "tokens": tokens, "probs": probs.float(), "balance": balance.float(), "z": (zsum / n).float()}


def _router_backward_plain(s):
    l = s["logits"].float()
    E, k, seg = s["E"], s["k"], s["seg"]
    n = torch.clamp(s["tokens"], min=1).float()
    c = (s["counts"].float() * (s["dbalance"] * (E / k) / (n * n))[:, None])[seg]
    p, sg = _scores(l, s["score"])
    d = p * (c - (p * c).sum(1, keepdim=True))
    if sg is not None:
        d = d * (1 - sg)
    lse = _lse(l)
    d = d + (2 * (s["dz"] / n)[seg] * lse)[:, None] * torch.exp(l - lse[:, None])
    gg = s["gates"] * (s["dgates"] - (s["gates"] * s["dgates"]).sum(1, keepdim=True))
    d.scatter_add_(1, s["idx"].long(), gg)
    if s["mask"] is not None:
        d = torch.where(s["mask"][:, None], d, 0.0)
    return {"dlogits": d.to(s["odt"])}


def _clip_plain(s):
    total = torch.zeros((), dtype=torch.float64, device="cuda")
    for t in s["grads"]:  # long sums: the parts of a tensor in 32 bits, their sum in 64
        head = t.numel() // 1024 * 1024
        total = total + t[:head].view(-1, 1024).float().square().sum(1).double().sum() + t[head:].float().square().sum().double()
    norm = torch.sqrt(total)
    factor = torch.clamp(s["max_norm"] / (norm + NORM_EPS), max=1.0).float()
    for t, o in zip(s["grads"], s["outs"]):
        o.copy_(t.float() * factor)
    return {"norm": norm.float().reshape(1), "clipped": s["flat"]}


_E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _w4_plain(s):
    N, K, group = s["N"], s["K"], s["group"]
    c = torch.stack([s["codes"] & 15, s["codes"] >> 4], dim=2).view(N, K)
    if s["code"] == "mx":
        w = torch.tensor(_E2M1, device="cuda")[c.int()]
        scale = torch.exp2(s["scales"].float() - 127)
    else:
        w = c.float() - (s["zeros"].float().repeat_interleave(group, 1)[:, :K] if s["zeros"] is not None else 8.0)
        scale = s["scales"].float()
    w = w * scale.repeat_interleave(group, 1)[:, :K]
    z = s["x"].float() @ w.t()
    if s["b"] is not None:
        z = z + s["b"].float()
    if s["act"] == "gelu":
        z = 0.5 * z * (1 + torch.erf(z * (1 / math.sqrt(2))))
    elif s["act"] == "silu":
        z = z / (1 + torch.exp(-z))
    if s["r"] is not None:
        z = z + s["r"].float()
    return {"y": z.to(s["odt"])}


# ---------------------------------------------------------------- one pass
def run(s):
    if own:
        import mxfp4_routed_expert_router_amd as moe
        if s["op"] == "router":
            score = moe.SCORE_SOFTMAX if s["score"] == "softmax" else moe.SCORE_SIGMOID
            if s["dir"] == "fwd":
                r = moe.moe_fp4_router_loss(s["logits"], s["idx"], score=score, seqs=s["seqs"], mask=s["mask"])
                return {"counts": r.counts, "tokens": r.tokens, "probs": r.probs, "balance": r.balance, "z": r.z}
            loss = moe.RouterLoss(s["counts"], s["tokens"], s["probs"], s["balance"], s["z"])
            return {"dlogits": moe.moe_fp4_router_loss_backward(
                s["logits"], s["idx"], loss, dbalance=s["dbalance"], dz=s["dz"], gates=s["gates"], dgates=s["dgates"],
                score=score, seqs=s["seqs"], mask=s["mask"], out_dtype=s["odt"])}
        if s["op"] == "clip":
            sumsq = moe.moe_fp4_grad_sumsq(s["grads"])
            norm = moe.moe_fp4_grad_clip(s["grads"], sumsq, s["max_norm"], eps=NORM_EPS, out=s["outs"])
            return {"norm": norm, "clipped": s["flat"]}
        act = {"none": moe.ACT_NONE, "gelu": moe.ACT_GELU, "silu": moe.ACT_SILU}[s["act"]]
        return {"y": moe.moe_fp4_linear_w4(s["x"], s["w"], bias=s["b"], act=act, residual=s["r"], out_dtype=s["odt"])}
    if s["op"] == "router":
        return _router_plain(s) if s["dir"] == "fwd" else _router_backward_plain(s)
    return _clip_plain(s) if s["op"] == "clip" else _w4_plain(s)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "router":
        T, E, k, S = (case[n] for n in ("T", "E", "k", "S"))
        small = T * k * 4 + (T if case["pad"] else 0) + S * 4
        if case["dir"] == "fwd":
            return {"bytes": T * E * BYTES[case["type"]] + small + S * E * 8 + S * 12, "flops": 8 * T * E}
        return {"bytes": T * E * (BYTES[case["type"]] + BYTES[case["out"]]) + small + T * k * 8 + S * E * 4 + S * 12,
                "flops": 16 * T * E}
    if case["op"] == "clip":
        types, n = case["types"].split(","), _sizes(case)
        bytes_ = 0
        for i, v in enumerate(n):
            t = types[i % len(types)]
            bytes_ += v * (BYTES[t] + BYTES[t if case["out"] == "same" or t != "f32" else case["out"]])
        return {"bytes": bytes_, "flops": 3 * sum(n)}
    M, N, K = case["M"], case["N"], case["K"]
    G = (K + case["group"] - 1) // case["group"]
    b = N * K // 2 + N * G * ((1 if case["code"] == "mx" else 2) + case["zeros"]) + M * K * 2
    return {"bytes": b + M * N * BYTES[case["out"]] * (1 + case["residual"]) + N * 2 * case["bias"], "flops": 2 * M * N * K}


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f = torch.float64
    if s["op"] == "router":
        l = s["logits"].to(f)
        cut, E, k = s["cuts"], case["E"], case["k"]
        lse = torch.logsumexp(l, 1)
        soft = torch.exp(l - lse[:, None])
        sig = torch.sigmoid(l)
        p = soft if case["score"] == "softmax" else sig / sig.sum(1, keepdim=True)
        live = s["mask"] if s["mask"] is not None else torch.ones(case["T"], dtype=torch.bool, device="cuda")
        if case["dir"] == "fwd":
            o = {"counts": [], "tokens": [], "probs": [], "balance": [], "z": []}
            for lo, hi in zip(cut, cut[1:]):
                m = live[lo:hi]
                n = int(m.sum())
                cnt = torch.bincount(s["idx"][lo:hi][m].reshape(-1).long(), minlength=E)
                o["counts"].append(cnt.to(torch.int32))
                o["tokens"].append(torch.tensor(n, dtype=torch.int32, device="cuda"))
                o["probs"].append(p[lo:hi][m].sum(0))
                share = cnt.to(f) / max(1, n * k)
                o["balance"].append(E * (share * o["probs"][-1] / max(1, n)).sum())
                o["z"].append((lse[lo:hi][m] ** 2).sum() / max(1, n))
            return {n: torch.stack(v) for n, v in o.items()}
        d = torch.zeros_like(l)
        for i, (lo, hi) in enumerate(zip(cut, cut[1:])):
            n = max(1, int(s["tokens"][i]))
            # the gradient of a row's probabilities, then through the scores
            up = s["dbalance"][i].to(f) * E * s["counts"][i].to(f) / (k * n) / n
            q = p[lo:hi]
            centred = up[None, :] - (q @ up)[:, None]
            d[lo:hi] = q * centred * (1 if case["score"] == "softmax" else torch.sigmoid(-l[lo:hi]))
            d[lo:hi] += soft[lo:hi] * (s["dz"][i].to(f) * 2 * lse[lo:hi] / n)[:, None]
        g, dg = s["gates"].to(f), s["dgates"].to(f)
        inner = (g * dg).sum(1)
        rows = torch.arange(case["T"], device="cuda")
        for j in range(k):
            d[rows, s["idx"][:, j].long()] += g[:, j] * (dg[:, j] - inner)
        d[~live] = 0
        return {"dlogits": d}
    if s["op"] == "clip":
        total = 0.0
        for t in s["grads"]:
            for part in t.split(1 << 26):
                v = part.to(f)
                total += float(torch.dot(v, v))
        norm = math.sqrt(total)
        factor = min(1.0, case["max_norm"] / (norm + NORM_EPS))
        flat, places = _flat(s["grads"], [o.dtype for o in s["outs"]], [f] * len(s["outs"]))
        for t, o in zip(s["grads"], places):
            o.copy_(t).mul_(factor)
        return {"norm": torch.tensor([norm], dtype=f, device="cuda"), "clipped": flat}
    M, N, K, group = (case[n] for n in ("M", "N", "K", "group"))
    y = torch.empty(M, N, dtype=f, device="cuda")
    x = s["x"].to(f)
    for lo in range(0, N, 8192):
        r = slice(lo, min(N, lo + 8192))
        by = s["codes"][r].long()
        q = torch.empty(by.shape[0], K, dtype=torch.long, device="cuda")
        q[:, 0::2], q[:, 1::2] = by % 16, by // 16
        of = torch.arange(K, device="cuda") // group
        if case["code"] == "mx":
            # sign, two bits of exponent (bias 1), one of mantissa; no exponent: halves
            mag, sign = q % 8, 1.0 - 2.0 * (q // 8).to(f)
            ex, ma = mag // 2, (mag % 2).to(f)
            v = torch.where(ex == 0, ma / 2, (1 + ma / 2) * torch.pow(2.0, (ex - 1).to(f))) * sign
            scale = torch.pow(2.0, s["scales"][r].to(f) - 127)
        else:
            v = (q - (s["zeros"][r].long()[:, of] if s["zeros"] is not None else 8)).to(f)
            scale = s["scales"][r].to(f)
        y[:, r] = x @ (v * scale[:, of]).t()
    if s["b"] is not None:
        y += s["b"].to(f)
    if case["act"] == "gelu":
        y = y * torch.special.ndtr(y)
    elif case["act"] == "silu":
        y = y * torch.sigmoid(y)
    if s["r"] is not None:
        y = y + s["r"].to(f)
    return {"y": y}
