"""What is measured of the operators around the grouped GEMMs: the update of
the experts' weights (orthogonalize), the loss over the vocabulary with its
gradients (vocab_cross_entropy) and the whole mixture-of-experts layer for a
few tokens, its router included (moe_layer).

A case is a dict of plain values.  Its sizes are those of the library's
workloads (E, N, K of the 16B and 671B expert shapes: hidden 2048 with expert
width 1408, hidden 7168 with expert width 2048; up to 256 experts) or generic
ones (vocabularies of 32,000 and 128,000, a few odd sizes).
"""
import math

import torch

own = False

DEV = "cuda"
COEFFS = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7
IGNORE = -100


def listed():
    return [
        # the update of one small layer's experts: four matrices, latency counts
        {"name": "ortho_small", "op": "ortho", "E": 4, "N": 128, "K": 256, "dtype": "bf16", "empty": 0},
        # odd sizes, taller than wide, a float32 momentum, and an expert that
        # saw no token (its gradient is zero)
        {"name": "ortho_odd_f32", "op": "ortho", "E": 3, "N": 777, "K": 515, "dtype": "f32", "empty": 1},
        # the 16B shape's gate projections of 8 experts
        {"name": "ortho_16b", "op": "ortho", "E": 8, "N": 1408, "K": 2048, "dtype": "bf16", "empty": 0},
        # the 671B shape's gate/up projections, 4 experts on a rank
        {"name": "ortho_671b", "op": "ortho", "E": 4, "N": 4096, "K": 7168, "dtype": "bf16", "empty": 0},
        # the score of one token: loss alone, the weights are read once
        {"name": "loss_token", "op": "loss", "T": 1, "H": 2048, "V": 32000, "grads": False, "ignored": 0.0},
        # a ragged batch with prompt tokens left out, odd in every size
        {"name": "loss_odd", "op": "loss", "T": 301, "H": 1001, "V": 32003, "grads": True, "ignored": 0.3},
        # a training micro-batch at the 16B hidden size
        {"name": "loss_16b", "op": "loss", "T": 4096, "H": 2048, "V": 128000, "grads": True, "ignored": 0.05},
        # and at the 671B hidden size
        {"name": "loss_671b", "op": "loss", "T": 2048, "H": 7168, "V": 128000, "grads": True, "ignored": 0.0},
        # one token through 2 of 8 experts of the 16B shape: latency counts
        {"name": "moe_token_16b", "op": "moe", "T": 1, "E": 8, "k": 2, "H": 2048, "I": 1408, "off": 0},
        # a few tokens, odd sizes, two slots of the batch empty
        {"name": "moe_odd", "op": "moe", "T": 13, "E": 10, "k": 3, "H": 1120, "I": 416, "off": 2},
        # one token through 8 of 32 experts of the 671B shape
        {"name": "moe_token_671b", "op": "moe", "T": 1, "E": 32, "k": 8, "H": 7168, "I": 2048, "off": 0},
        # a serving batch over 256 experts of the 16B shape: nearly all are read
        {"name": "moe_batch_256e", "op": "moe", "T": 64, "E": 256, "k": 8, "H": 2048, "I": 1408, "off": 0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw(rng):
    op = rng.choice(("ortho", "loss", "moe"))
    if op == "ortho":
        E = _log_int(rng, 1, 16)
        return {"op": op, "E": E, "N": _log_int(rng, 64, 7168), "K": _log_int(rng, 64, 7168),
                "dtype": rng.choice(("bf16", "f32")), "empty": rng.choice((0, 0, 1)) if E > 1 else 0}
    if op == "loss":
        return {"op": op, "T": _log_int(rng, 1, 4096), "H": _log_int(rng, 100, 7168) if rng.random() < 0.5
                else 64 * _log_int(rng, 2, 112), "V": _log_int(rng, 1000, 128000), "grads": rng.random() < 0.7,
                "ignored": rng.choice((0.0, 0.05, 0.5))}
    E = _log_int(rng, 4, 256)
    T = _log_int(rng, 1, 64)
    return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(8, E)), "H": 32 * _log_int(rng, 8, 224),
            "I": 32 * _log_int(rng, 4, 64), "off": rng.choice((0, 0, 1)) if T > 1 else 0}


def draw(rng):
    most = {}
    for c in listed():
        w = work(c)
        most[c["op"]] = tuple(map(max, zip(most.get(c["op"], (0.0, 0.0)), (w["bytes"], w["flops"]))))
    while True:
        c = _draw(rng)
        w = work(c)
        stored = 3 * c["E"] * c["I"] * c["H"] if c["op"] == "moe" else 0
        if w["bytes"] <= most[c["op"]][0] and w["flops"] <= most[c["op"]][1] and stored <= 3 * 256 * 1408 * 2048:
            return c


def work(case):
    """What a pass cannot do without.  ortho: the products of each step, of the
    two symmetric ones half.  loss: the logits, and the two gradients' products.
    moe: the weights of the experts that uniform routing is expected to reach."""
    c = case
    if c["op"] == "ortho":
        n, m = min(c["N"], c["K"]), max(c["N"], c["K"])
        size = 4 if c["dtype"] == "f32" else 2
        return {"bytes": c["E"] * n * m * (size + 2), "flops": c["E"] * STEPS * (3 * n * n * m + n * n * n)}
    if c["op"] == "loss":
        T, H, V = c["T"], c["H"], c["V"]
        once = 2 * (T * H + V * H) + 8 * T
        return {"bytes": 2 * once if c["grads"] else once, "flops": 2 * T * H * V * (3 if c["grads"] else 1)}
    T, E, k, H, I = c["T"] - c["off"], c["E"], c["k"], c["H"], c["I"]
    reached = E * (1.0 - (1.0 - k / E) ** T)
    return {"bytes": int(reached * 3 * H * I * 33 / 32) + 2 * E * H + 4 * c["T"] * H,
            "flops": 6 * T * k * H * I + 2 * T * E * H}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _mx_weights(g, E, R, C):
    """MXFP8 weights [E, R, C] of variance about 1 / C: E4M3 codes that
    fill their range, E8M0 scales around the matching power of two."""
    codes = torch.empty((E, R, C), dtype=torch.uint8, device=DEV)
    scales = torch.empty((E, R, C // 32), dtype=torch.uint8, device=DEV)
    mid = 127 + round(math.log2(1.0 / (120.0 * math.sqrt(C))))
    for e in range(E):
        v = torch.randn((R, C), generator=g, device=DEV).mul_(120.0).clamp_(-448.0, 448.0)
        codes[e] = v.to(torch.float8_e4m3fn).view(torch.uint8)
        scales[e] = torch.randint(mid - 1, mid + 2, (R, C // 32), generator=g, device=DEV, dtype=torch.uint8)
    return codes, scales


def _clear_tokens(g, T, k, router):
    """Tokens whose choice of experts is defined in 32 bits: one whose first
    k + 1 logits hold two nearer than 1e-4 is drawn again."""
    H = router.shape[1]
    r64 = router.double()
    x = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    for _ in range(40):
        top = (x.double() @ r64.t()).sort(dim=1, descending=True).values[:, :k + 1]
        near = ((top[:, :-1] - top[:, 1:]) < 1e-4).any(dim=1)
        fresh = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
        x = torch.where(near[:, None], fresh, x)
    return x


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] == "ortho":
        E, N, K = c["E"], c["N"], c["K"]
        # a gradient: noise of the batch over a few strong directions
        G = torch.randn((E, N, K), generator=g, device=DEV)
        u = torch.randn((E, N, 8), generator=g, device=DEV)
        v = torch.randn((E, 8, K), generator=g, device=DEV)
        G = (G + (u @ v) * 0.35) * 1e-3
        if c["empty"]:
            G[E // 2] = 0.0
        return {"case": c, "G": G if c["dtype"] == "f32" else G.to(torch.bfloat16)}
    if c["op"] == "loss":
        T, H, V = c["T"], c["H"], c["V"]
        x = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
        w = torch.empty((V, H), dtype=torch.bfloat16, device=DEV)
        w.normal_(0.0, 1.5 / math.sqrt(H), generator=g)
        # targets lean to the low indexes, as frequent words do
        y = (torch.rand((T,), generator=g, device=DEV) ** 3 * V).to(torch.int64).clamp_(0, V - 1)
        left_out = torch.rand((T,), generator=g, device=DEV) < c["ignored"]
        left_out[0] = False  # a batch trains on one token at least
        y[left_out] = IGNORE
        return {"case": c, "x": x, "w": w, "y": y}
    T, E, k, H, I = c["T"], c["E"], c["k"], c["H"], c["I"]
    router = (torch.randn((E, H), generator=g, device=DEV) / math.sqrt(H)).to(torch.bfloat16)
    x = _clear_tokens(g, T, k, router)
    wgu, sgu = _mx_weights(g, E, 2 * I, H)
    wd, sd = _mx_weights(g, E, H, I)
    active = None
    if c["off"]:
        active = torch.ones((T,), dtype=torch.bool, device=DEV)
        active[T // 2:T // 2 + c["off"]] = False
    return {"case": c, "x": x, "router": router, "wgu": wgu, "sgu": sgu, "wd": wd, "sd": sd, "active": active}


def _values(codes, scales):
    """The numbers that MXFP8 codes and scales stand for."""
    shape = codes.shape
    v = codes.view(torch.float8_e4m3fn).float().view(*shape[:-1], shape[-1] // 32, 32)
    return (v * torch.exp2(scales.float() - 127.0)[..., None]).view(shape)


def _plain_ortho(G):
    a, b, c = COEFFS
    G = G.float()
    tall = G.shape[1] > G.shape[2]
    X = G.transpose(1, 2) if tall else G
    X = X / (X.square().sum(dim=(1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        A = X @ X.transpose(1, 2)
        X = a * X + (b * A + c * (A @ A)) @ X
    return (X.transpose(1, 2) if tall else X).to(torch.bfloat16).contiguous()


def _plain_loss(x, w, y, grads):
    x, w = x.float(), w.float()
    logits = x @ w.t()
    top = logits.max(dim=1, keepdim=True).values
    p = torch.exp(logits - top)
    total = p.sum(dim=1, keepdim=True)
    used = y != IGNORE
    index = torch.where(used, y, torch.zeros_like(y))[:, None]
    loss = (torch.log(total) + top - logits.gather(1, index))[:, 0]
    loss = torch.where(used, loss, torch.zeros_like(loss))
    if not grads:
        return {"loss": loss}
    scale = 1.0 / used.sum().clamp(min=1).float()
    p = p / total
    p = p.scatter_add(1, index, torch.full_like(index, -1.0, dtype=torch.float32))
    p = torch.where(used[:, None], p, torch.zeros_like(p)) * scale
    return {"loss": loss.sum() * scale, "dx": (p @ w).to(torch.bfloat16), "dw": (p.t() @ x).to(torch.bfloat16)}


def _plain_moe(s):
    c = s["case"]
    T, E, k, I = c["T"], c["E"], c["k"], c["I"]
    x = s["x"].float()
    logits = x @ s["router"].float().t()
    p = torch.exp(logits - logits.max(dim=1, keepdim=True).values)
    p = p / p.sum(dim=1, keepdim=True)
    p, ids = p.sort(dim=1, descending=True, stable=True)
    weights, ids = p[:, :k], ids[:, :k]
    weights = weights / weights.sum(dim=1, keepdim=True)
    if s["active"] is not None:
        weights = torch.where(s["active"][:, None], weights, torch.zeros_like(weights))
    gate = torch.zeros((T, T * k if T * k < E else E), device=x.device)
    if T * k < E:  # few tokens: the weights of each token's experts
        take = ids.reshape(-1)
        gate = gate.scatter(1, torch.arange(T * k, device=x.device).view(T, k), weights)
        wgu, sgu, wd, sd = (s[n][take] for n in ("wgu", "sgu", "wd", "sd"))
    else:          # else every expert on all tokens
        gate = gate.scatter(1, ids, weights)
        wgu, sgu, wd, sd = s["wgu"], s["sgu"], s["wd"], s["sd"]
    gu = x @ _values(wgu, sgu).transpose(1, 2)
    g, u = gu[..., :I], gu[..., I:]
    h = g / (1.0 + torch.exp(-g)) * u * gate.t()[:, :, None]
    out = (h @ _values(wd, sd).transpose(1, 2)).sum(dim=0)
    if s["active"] is not None:
        ids = torch.where(s["active"][:, None], ids, torch.full_like(ids, -1))
    return {"out": out.to(torch.bfloat16), "ids": ids.to(torch.int32), "weights": weights}


def run(state):
    s, c = state, state["case"]
    if own:
        import mxfp8_ragged_grouped_amd as mxw

        if c["op"] == "ortho":
            return mxw.orthogonalize(s["G"], steps=STEPS, coeffs=COEFFS, eps=EPS)
        if c["op"] == "loss":
            if not c["grads"]:
                return {"loss": mxw.vocab_cross_entropy(s["x"], s["w"], s["y"], ignore_index=IGNORE,
                                                        reduction="none", grads=False)}
            loss, dx, dw = mxw.vocab_cross_entropy(s["x"], s["w"], s["y"], ignore_index=IGNORE, reduction="mean")
            return {"loss": loss, "dx": dx, "dw": dw}
        out, ids, weights = mxw.moe_layer(s["x"], s["router"], s["wgu"], s["sgu"], s["wd"], s["sd"], c["k"],
                                          normalize=True, active=s["active"])
        return {"out": out, "ids": ids, "weights": weights}
    if c["op"] == "ortho":
        return _plain_ortho(s["G"])
    if c["op"] == "loss":
        return _plain_loss(s["x"], s["w"], s["y"], c["grads"])
    return _plain_moe(s)


def _decoded(codes, scales):
    """MXFP8 in 64 bits from the formats' definitions: E4M3 is (-1)^s (1 + m/8)
    2^(e-7), m/8 2^-6 where e is 0; E8M0 is 2^(b-127)."""
    b = torch.arange(256, dtype=torch.int64, device=DEV)
    e, m = (b >> 3) & 15, (b & 7).double()
    table = torch.where(e > 0, torch.ldexp(1.0 + m / 8, e - 7), torch.ldexp(m / 8, torch.full_like(e, -6)))
    table = torch.where(b > 127, -table, table)
    return table[codes.long()] * torch.ldexp(torch.ones_like(table), b - 127)[scales.long()].repeat_interleave(32, -1)


def exact(case, seed):
    """The definitions in 64 bits, one matrix, one block of tokens or one
    expert at a time."""
    c, s = case, prepare(case, seed)
    if c["op"] == "ortho":
        out = torch.empty((c["E"], c["N"], c["K"]), dtype=torch.float64, device=DEV)
        for e in range(c["E"]):
            X = s["G"][e].double()
            wide = X.shape[0] <= X.shape[1]
            X = X / (torch.linalg.vector_norm(X) + EPS)
            for _ in range(STEPS):
                # p(X) = a X + b S X + c S S X with the Gram matrix of the short side
                S = X @ X.mT if wide else X.mT @ X
                Y = S @ X if wide else X @ S
                Z = S @ Y if wide else Y @ S
                X = COEFFS[0] * X + COEFFS[1] * Y + COEFFS[2] * Z
            out[e] = X
        return out
    if c["op"] == "loss":
        x, w, y = s["x"].double(), s["w"].double(), s["y"]
        losses, dx, dw = [], [], torch.zeros_like(w)
        count = max(int((y != IGNORE).sum()), 1)
        for i in range(0, c["T"], 512):
            xb, yb = x[i:i + 512], y[i:i + 512]
            lp = torch.log_softmax(xb @ w.mT, dim=1)
            keep = (yb != IGNORE).double()
            pick = torch.where(yb == IGNORE, torch.zeros_like(yb), yb)
            losses.append(-lp[torch.arange(len(yb), device=DEV), pick] * keep)
            if c["grads"]:
                d = lp.exp_()
                d[torch.arange(len(yb), device=DEV), pick] -= 1.0
                d *= keep[:, None] / count
                dx.append(d @ w)
                dw += d.mT @ xb
        loss = torch.cat(losses)
        if not c["grads"]:
            return {"loss": loss}
        return {"loss": loss.sum() / count, "dx": torch.cat(dx), "dw": dw}
    x = s["x"].double()
    prob = torch.softmax(x @ s["router"].double().mT, dim=1)
    ids = torch.argsort(prob, dim=1, descending=True, stable=True)[:, :c["k"]]
    weights = prob.gather(1, ids)
    weights = weights / weights.sum(dim=1, keepdim=True)
    if s["active"] is not None:
        weights = weights * s["active"][:, None]
    out = torch.zeros_like(x)
    for e in torch.unique(ids).tolist():
        share = (weights * (ids == e)).sum(dim=1, keepdim=True)
        gu = x @ _decoded(s["wgu"][e], s["sgu"][e]).mT
        h = torch.nn.functional.silu(gu[:, :c["I"]]) * gu[:, c["I"]:]
        out += share * (h @ _decoded(s["wd"][e], s["sd"][e]).mT)
    return {"out": out, "ids": None, "weights": weights}
