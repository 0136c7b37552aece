"""Cases of the router's balance loss, the router's backward pass and the expert products on
4-bit weights: their inputs, plain forms, exact values and the work of one pass.

`own` chooses what `run` does: the plain form in elementary torch operations (32 bits), or the
library's calls (`capacity_routing_expert_amd.binding`).  `exact` evaluates the definitions in
64 bits.
"""
import math

import torch

own = False

DEV = "cuda:0"
# magnitudes of the 4-bit code's low three bits (2 exponent bits, 1 mantissa bit); bit 3 is the sign
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------- the cases
def listed():
    bal = lambda name, T, E, k, masked: dict(name=name, op="balance", T=T, E=E, k=k, masked=masked)
    rb = lambda name, T, d, E, k, dtype, masked, add: dict(
        name=name, op="route_backward", T=T, d=d, E=E, k=k, dtype=dtype, masked=masked, add=add)
    ffn = lambda name, T, d, f, E, k, group, gated: dict(
        name=name, op="ffn", T=T, d=d, f=f, E=E, k=k, group=group, gated=gated)
    return [
        # the decode layer's router watched for balance: one small batch, bound by latency
        bal("balance_decode_T64_E8", 64, 8, 2, False),
        # a training step's router over the fine layer's 64 experts
        bal("balance_fine_T16384_E64", 16384, 64, 6, False),
        # many small experts, a padded batch with an odd number of tokens
        bal("balance_padded_T32771_E256", 32771, 256, 8, True),
        # router tuning on a handful of tokens, fp32 with odd sizes
        rb("route_bwd_f32_T37_d136_E5", 37, 136, 5, 2, "f32", False, False),
        # the mid layer's router, bf16
        rb("route_bwd_mid_T4096_d2048_E8", 4096, 2048, 8, 2, "bf16", False, False),
        # the fine layer's router, added to the residual's gradient, a padded batch
        rb("route_bwd_fine_T16384_d2048_E64", 16384, 2048, 64, 6, "bf16", True, True),
        # the collapse layer's router: the longest batch and widest rows
        rb("route_bwd_collapse_T32768_d4096_E8", 32768, 4096, 8, 2, "bf16", False, True),
        # one token through the decode layer's experts at 4 bits: two experts' weights stream
        ffn("ffn_single_token_d2048_f8192_E8", 1, 2048, 8192, 8, 2, 32, False),
        # the decode batch: every expert's weights stream for about 16 rows each
        ffn("ffn_decode_T64_d2048_f8192_E8", 64, 2048, 8192, 8, 2, 32, False),
        # gated experts at the flow diagram's width, coarser groups, an odd batch
        ffn("ffn_gated_T37_d2048_f768_E8", 37, 2048, 768, 8, 2, 128, True),
        # many small experts with tens of rows each
        ffn("ffn_fine_T512_d2048_f1408_E64", 512, 2048, 1408, 64, 6, 64, False),
        # the mid layer's batch: bound by the matrix cores
        ffn("ffn_mid_T4096_d2048_f8192_E8", 4096, 2048, 8192, 8, 2, 128, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("balance", "route_backward", "ffn"))
    if op == "balance":
        E = _log(rng, 2, 256)
        return dict(op=op, T=_log(rng, 1, 32768), E=E, k=rng.randint(1, min(E, 8)),
                    masked=rng.random() < 0.5)
    if op == "route_backward":
        E = _log(rng, 2, 128)
        dtype = rng.choice(("bf16", "bf16", "f32"))
        d = 8 * _log(rng, 8, 512)
        T = _log(rng, 1, min(32768, (1 << 25) // d, (1 << 31) // (d * E)))
        return dict(op=op, T=T, d=d, E=E, k=rng.randint(1, min(E, 8)), dtype=dtype,
                    masked=rng.random() < 0.5, add=rng.random() < 0.5)
    E = _log(rng, 1, 64)
    k = rng.randint(1, min(E, 6))
    gated = rng.random() < 0.4
    d = 8 * _log(rng, 32, 256)
    f = 8 * _log(rng, 32, min(1024, (1 << 24) // (8 * d * E) * (4 if E > 1 else 8)))
    T = _log(rng, 1, 4096)
    return dict(op=op, T=T, d=d, f=f, E=E, k=k, group=rng.choice((32, 64, 128)), gated=gated)


# ---------------------------------------------------------------- inputs
def _generator(seed, salt):
    return torch.Generator(device=DEV).manual_seed((seed * 1000003 + salt) & 0x7FFFFFFF)


def _routing(g, T, E, k, spread):
    """Router logits with a mild preference among the experts, and each token's k best."""
    logits = torch.randn(T, E, generator=g, device=DEV)
    logits += spread * torch.randn(E, generator=g, device=DEV)
    ids = torch.topk(logits, k, dim=1).indices.to(torch.int32).contiguous()
    return logits, ids


def _padding(g, T):
    """A batch padded at its end and, here and there, inside: 1 for a real token."""
    mask = torch.rand(T, generator=g, device=DEV) < 0.95
    mask[T - T // 8:] = False
    return mask.to(torch.uint8)


def _quantize(w, group):
    """Codes (uint8, one a weight) and bf16 scales of w [E, rows, cols]: the scale of a group is
    max |w| / 6 rounded to bf16, the code the nearest magnitude, ties to the even code."""
    E, rows, cols = w.shape
    G = -(-cols // group)
    v = torch.nn.functional.pad(w.float(), (0, G * group - cols)).view(E, rows, G, group)
    scales = (v.abs().amax(-1) / 6.0).to(torch.bfloat16)
    s = scales.float().unsqueeze(-1)
    a = torch.where(s > 0, v.abs() / s, torch.zeros_like(v))
    code = torch.zeros(a.shape, dtype=torch.uint8, device=w.device)
    for bound, up in ((0.25, False), (0.75, True), (1.25, False), (1.75, True), (2.5, False),
                      (3.5, True), (5.0, False)):
        code += (a >= bound) if up else (a > bound)
    code += 8 * torch.signbit(v).to(torch.uint8)
    return code.view(E, rows, G * group)[:, :, :cols].contiguous(), scales


def _ffn_weights(case, g):
    """bf16 expert weights and biases (gated experts have none), one expert at a time."""
    E, d, f = case["E"], case["d"], case["f"]
    rows1 = 2 * f if case["gated"] else f
    w1 = torch.empty(E, rows1, d, dtype=torch.bfloat16, device=DEV)
    w2 = torch.empty(E, d, f, dtype=torch.bfloat16, device=DEV)
    for e in range(E):
        w1[e] = torch.randn(rows1, d, generator=g, device=DEV) / math.sqrt(d)
        w2[e] = torch.randn(d, f, generator=g, device=DEV) / math.sqrt(f)
    if case["gated"]:
        return w1, None, w2, None
    b1 = (0.02 * torch.randn(E, f, generator=g, device=DEV)).to(torch.bfloat16)
    b2 = (0.02 * torch.randn(E, d, generator=g, device=DEV)).to(torch.bfloat16)
    return w1, b1, w2, b2


def _inputs(case, seed):
    """The tensors of one case, from the seed alone."""
    op, T, E, k = case["op"], case["T"], case["E"], case["k"]
    g = _generator(seed, {"balance": 1, "route_backward": 2, "ffn": 3}[op])
    if op == "balance":
        logits, ids = _routing(g, T, E, k, 1.0)
        return dict(logits=logits, ids=ids, mask=_padding(g, T) if case["masked"] else None,
                    coef=0.01, grad_scale=1.0)
    if op == "route_backward":
        d, dt = case["d"], torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        x = torch.randn(T, d, generator=g, device=DEV).to(dt)
        w = (torch.randn(E, d, generator=g, device=DEV) / math.sqrt(d)).to(dt)
        logits = torch.empty(T, E, device=DEV)
        for t in range(0, T, 4096):
            logits[t:t + 4096] = (x[t:t + 4096].double() @ w.double().T).float()
        ids = torch.topk(logits, k, dim=1).indices.to(torch.int32).contiguous()
        dgates = 0.02 * torch.randn(T, k, generator=g, device=DEV)
        dgates[torch.rand(T, k, generator=g, device=DEV) < 0.15] = 0.0  # dropped assignments
        dlogits = 0.001 * torch.randn(T, E, generator=g, device=DEV)
        add = (0.05 * torch.randn(T, d, generator=g, device=DEV)).to(dt) if case["add"] else None
        return dict(x=x, w=w, logits=logits, ids=ids, dgates=dgates, dlogits=dlogits, add=add,
                    mask=_padding(g, T) if case["masked"] else None)
    d = case["d"]
    w1, b1, w2, b2 = _ffn_weights(case, g)
    x = torch.randn(T, d, generator=g, device=DEV).to(torch.bfloat16)
    _, ids = _routing(g, T, E, k, 0.25)
    order = torch.sort(ids.flatten().long(), stable=True).indices
    counts = torch.bincount(ids.flatten().long(), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0).to(torch.int32)
    return dict(x=x, w1=w1, b1=b1, w2=w2, b2=b2, row_token=(order // k).to(torch.int32),
                offsets=offsets)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "ffn":
        # the program keeps the weights at 4 bits only
        group = case["group"]
        w1, w2 = s.pop("w1"), s.pop("w2")
        s["bounds"] = s["offsets"].tolist()
        if own:
            from capacity_routing_expert_amd import binding as B
            from capacity_routing_expert_amd import layer as L
            s["shape"] = B.make_shape(T, case["d"], case["f"], E, k, T, B.MOE_BF16)
            s["experts"] = L.quantize_experts(w1, s["b1"], w2, s["b2"], group, case["gated"])
            s["ws"] = L.workspace(s["shape"], DEV)
            s["y"] = torch.empty(T * k, case["d"], dtype=torch.bfloat16, device=DEV)
        else:
            E1, E2 = torch.empty_like(w1, dtype=torch.uint8), torch.empty_like(w2, dtype=torch.uint8)
            S1, S2 = [], []
            for e in range(E):
                E1[e:e + 1], sc = _quantize(w1[e:e + 1], group)
                S1.append(sc)
                E2[e:e + 1], sc = _quantize(w2[e:e + 1], group)
                S2.append(sc)
            s.update(c1=E1, s1=torch.cat(S1), c2=E2, s2=torch.cat(S2))
            s["magnitudes"] = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=DEV)
    elif own:
        from capacity_routing_expert_amd import binding as B
        if case["op"] == "balance":
            s["shape"] = B.make_shape(T, 8, 8, E, k, 0, B.MOE_F32)
            n = B.workspace_bytes_balance(s["shape"])
            s.update(loss=torch.empty(1, device=DEV), counts=torch.empty(E, dtype=torch.int32, device=DEV),
                     probs=torch.empty(E, device=DEV), grad=torch.empty(T, E, device=DEV))
        else:
            dt = B.MOE_BF16 if case["dtype"] == "bf16" else B.MOE_F32
            s["shape"] = B.make_shape(T, case["d"], 8, E, k, 0, dt)
            n = B.workspace_bytes_route_backward(s["shape"])
            s.update(dx=torch.empty_like(s["x"]), dw=torch.empty(E, case["d"], device=DEV),
                     db=torch.empty(E, device=DEV))
        s["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if own:
        return {"balance": _own_balance, "route_backward": _own_route_backward,
                "ffn": _own_ffn}[op](state)
    return {"balance": _plain_balance, "route_backward": _plain_route_backward,
            "ffn": _plain_ffn}[op](state)


def _own_balance(s):
    from capacity_routing_expert_amd import binding as B
    B.moe_balance_loss(s["shape"], s["logits"], s["ids"], s["loss"], expert_counts=s["counts"],
                       expert_probs=s["probs"], dlogits=s["grad"], token_mask=s["mask"],
                       coef=s["coef"], grad_scale=s["grad_scale"], ws=s["ws"])
    return {"loss": s["loss"], "counts": s["counts"], "probs": s["probs"], "dlogits": s["grad"]}


def _own_route_backward(s):
    from capacity_routing_expert_amd import binding as B
    B.moe_route_backward(s["shape"], s["x"], s["w"], s["logits"], s["ids"], s["dgates"],
                         s["dlogits"], dx=s["dx"], dw_router=s["dw"], db_router=s["db"],
                         dx_add=s["add"], token_mask=s["mask"], ws=s["ws"])
    return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}


def _own_ffn(s):
    from capacity_routing_expert_amd import binding as B
    B.moe_expert_ffn_quantized(s["shape"], s["x"], s["row_token"], s["offsets"], s["experts"],
                               s["y"], s["ws"])
    return s["y"]


def _plain_balance(s):
    T, E = s["logits"].shape
    k = s["ids"].shape[1]
    z = s["logits"] - s["logits"].amax(1, keepdim=True)
    p = torch.exp(z)
    p = p / p.sum(1, keepdim=True)
    ids = s["ids"].long()
    hot = torch.zeros(T, E, device=DEV).scatter_add_(1, ids, torch.ones(T, k, device=DEV))
    if s["mask"] is not None:
        valid = s["mask"].float().unsqueeze(1)
        p, hot, n = p * valid, hot * valid, s["mask"].sum().float().clamp(min=1.0)
    else:
        n = torch.full((), float(T), device=DEV)
    counts = hot.sum(0)
    probs = p.sum(0) / n
    loss = s["coef"] * E * (counts / (n * k) * probs).sum()
    # the gradient only sees differences of counts: from the smallest, equal counts give zeros
    scale = s["grad_scale"] * s["coef"] * E / (n * k) / n
    over = counts - counts.amin()
    grad = scale * p * (over - (p * over).sum(1, keepdim=True))
    return {"loss": loss.reshape(1), "counts": counts.to(torch.int32), "probs": probs,
            "dlogits": grad}


def _plain_route_backward(s):
    T, E = s["logits"].shape
    p = torch.exp(s["logits"] - s["logits"].amax(1, keepdim=True))
    p = p / p.sum(1, keepdim=True)
    dp = torch.zeros(T, E, device=DEV).scatter_add_(1, s["ids"].long(), s["dgates"])
    dl = p * (dp - (p * dp).sum(1, keepdim=True)) + s["dlogits"]
    if s["mask"] is not None:
        dl = dl * s["mask"].float().unsqueeze(1)
    x = s["x"].float()
    dx = dl @ s["w"].float()
    if s["add"] is not None:
        dx = dx + s["add"].float()
    return {"dx": dx.to(s["x"].dtype), "dw": dl.T @ x, "db": dl.sum(0)}


def _plain_ffn(s):
    case = s["case"]
    group, f = case["group"], case["f"]
    y = torch.empty(s["row_token"].shape[0], case["d"], dtype=torch.bfloat16, device=DEV)

    def weights(codes, scales):
        w = s["magnitudes"][codes.long()]
        return w * torch.repeat_interleave(scales.float(), group, dim=1)[:, :w.shape[1]]

    for e in range(case["E"]):
        lo, hi = s["bounds"][e], s["bounds"][e + 1]
        if lo == hi:
            continue
        xe = s["x"][s["row_token"][lo:hi].long()].float()
        h = xe @ weights(s["c1"][e], s["s1"][e]).T
        if case["gated"]:
            h = h[:, :f] / (1.0 + torch.exp(-h[:, :f])) * h[:, f:]
        else:
            h = h + s["b1"][e].float()
            h = h / (1.0 + torch.exp(-h))
        out = h @ weights(s["c2"][e], s["s2"][e]).T
        if not case["gated"]:
            out = out + s["b2"][e].float()
        y[lo:hi] = out.to(torch.bfloat16)
    return y


# ---------------------------------------------------------------- the definitions in 64 bits
def exact(case, seed):
    s = _inputs(case, seed)
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "balance":
        keep = torch.ones(T, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"] > 0
        n = int(keep.sum())
        counts = torch.bincount(s["ids"][keep].flatten().long(), minlength=E)
        p = torch.softmax(s["logits"].double(), dim=1)
        f = counts.double() / max(n * k, 1)
        probs = p[keep].sum(0) / max(n, 1)
        grad = torch.zeros(T, E, dtype=torch.float64, device=DEV)
        pk, above = p[keep], f - f.min()  # sum_j p_j = 1: a common part of f drops out
        grad[keep] = s["grad_scale"] * s["coef"] * E / max(n, 1) * (
            pk * above - pk * (pk @ above).unsqueeze(1))
        return {"loss": (s["coef"] * E * torch.dot(f, probs)).reshape(1), "counts": counts.to(torch.int32),
                "probs": probs, "dlogits": grad}
    if case["op"] == "route_backward":
        p = torch.softmax(s["logits"].double(), dim=1)
        up = torch.zeros_like(p)
        for c in range(k):
            up.scatter_add_(1, s["ids"][:, c:c + 1].long(), s["dgates"][:, c:c + 1].double())
        dl = p * up - p * (p * up).sum(1, keepdim=True) + s["dlogits"].double()
        if s["mask"] is not None:
            dl[s["mask"] == 0] = 0.0
        dw = torch.zeros(E, case["d"], dtype=torch.float64, device=DEV)
        dx = torch.empty(T, case["d"], dtype=torch.float64, device=DEV)
        for t in range(0, T, 8192):
            part = dl[t:t + 8192]
            dw += part.T.contiguous() @ s["x"][t:t + 8192].double()
            dx[t:t + 8192] = part @ s["w"].double()
            if s["add"] is not None:
                dx[t:t + 8192] += s["add"][t:t + 8192].double()
        return {"dx": dx, "dw": dw, "db": dl.sum(0)}
    group, f = case["group"], case["f"]
    table = torch.tensor(MAGNITUDES, dtype=torch.float64, device=DEV)
    bounds = s["offsets"].tolist()
    y = torch.empty(T * k, case["d"], dtype=torch.float64, device=DEV)

    def values(w):
        codes, scales = _quantize(w.unsqueeze(0), group)
        c = codes[0].long()
        v = table[c & 7] * (1.0 - 2.0 * (c >> 3).double())
        at = torch.arange(v.shape[1], device=DEV) // group
        return v * scales[0].double()[:, at]

    for e in range(E):
        lo, hi = bounds[e], bounds[e + 1]
        if lo == hi:
            continue
        h = torch.mm(s["x"][s["row_token"][lo:hi].long()].double(), values(s["w1"][e]).t().contiguous())
        if case["gated"]:
            h = h[:, :f] * torch.sigmoid(h[:, :f]) * h[:, f:]
        else:
            h = h + s["b1"][e].double()
            h = h * torch.sigmoid(h)
        o = torch.mm(h, values(s["w2"][e]).t().contiguous())
        y[lo:hi] = o if case["gated"] else o + s["b2"][e].double()
    return y


# ---------------------------------------------------------------- the work of one pass
def work(case):
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "balance":
        return {"bytes": 8 * T * E + 4 * T * k + (T if case["masked"] else 0) + 8 * E + 4,
                "flops": 10 * T * E}
    if case["op"] == "route_backward":
        d, eb = case["d"], 2 if case["dtype"] == "bf16" else 4
        streams = 3 if case["add"] else 2  # x, dx and what dx is added to
        return {"bytes": streams * T * d * eb + E * d * (eb + 4) + 8 * T * E + 8 * T * k +
                (T if case["masked"] else 0) + 4 * E,
                "flops": 4 * T * E * d + 10 * T * E}
    d, f, n = case["d"], case["f"], 3 if case["gated"] else 2
    active = E * (1.0 - (1.0 - k / E) ** T)  # experts that some token picks, at even odds
    weight = 0.5 + 2.0 / case["group"]
    bias = 0 if case["gated"] else 2 * (d + f)
    return {"bytes": int(active * (n * d * f * weight + bias) + 2 * T * d + 4 * T * k + 2 * T * k * d),
            "flops": 2 * n * T * k * d * f}
