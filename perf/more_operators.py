"""What is measured of the operators that a mixture-of-experts layer needs
between the grouped products: tokens sorted by expert and copied to their rows
(sort_tokens, dispatch_tokens), joined again with their weights (combine_tokens)
and the gradient of that (combine_tokens_grad), the row-wise MXFP8 operands
(quantize_rows), the gradients' norm and clipping (clip_grad_norm, grad_norm),
and dense products of a few tokens with 4-bit weights (linear_4bit).

A case is a dict of plain values.  Its sizes are those of the library's
workloads (experts, hidden and expert width of the 16B and 671B shapes, up to
256 experts) or generic ones (vocabularies of 32,000 and 128,000, odd sizes).
"""
import math

import torch

own = False

DEV = "cuda"
ALIGN = 32
MAX_NORM = 1.0
EPS = 1e-6


def listed():
    return [
        # one token to the experts it chose: latency counts
        {"name": "there_token", "op": "there", "T": 1, "k": 2, "E": 8, "H": 2048, "form": "rows", "type": "bf16",
         "ids": "i64", "empty": 0.0},
        # a ragged batch, odd in every size, a quarter of the slots empty
        {"name": "there_odd", "op": "there", "T": 301, "k": 3, "E": 10, "H": 1001, "form": "rows", "type": "bf16",
         "ids": "i32", "empty": 0.25},
        # the 16B training shape: the bf16 rows for the weight gradient and the
        # MXFP8 rows for the forward product in one pass
        {"name": "there_16b", "op": "there", "T": 98304, "k": 2, "E": 8, "H": 2048, "form": "both", "type": "bf16",
         "ids": "i64", "empty": 0.0},
        # a small batch's way back, with a residual
        {"name": "back_odd", "op": "back", "T": 301, "k": 3, "E": 10, "H": 1120, "type": "bf16", "empty": 0.25,
         "residual": True},
        # 256 experts of the 16B shape, 1,024 tokens each
        {"name": "back_256e", "op": "back", "T": 32768, "k": 8, "E": 256, "H": 2048, "type": "bf16", "empty": 0.0,
         "residual": False},
        # the gradient of the way back at the 671B shape
        {"name": "back_grad_671b", "op": "back_grad", "T": 16384, "k": 8, "E": 32, "H": 7168, "type": "bf16",
         "empty": 0.0},
        # odd activations, float32
        {"name": "rows_odd", "op": "rows", "R": 777, "C": 1120, "type": "f32"},
        # the gate/up weights of 16 experts of the 671B shape
        {"name": "rows_671b", "op": "rows", "R": 65536, "C": 7168, "type": "bf16"},
        # the gradients of a small model: 20 tensors of all sizes
        {"name": "clip_small", "op": "clip", "tensors": 20, "total": 2000000, "clip": True},
        # the gradients of a rank at the 671B shape: four experts and the vocabulary
        {"name": "clip_671b", "op": "clip", "tensors": 12, "total": 1090000000, "clip": True},
        # the words' logits of one token
        {"name": "linear_token", "op": "linear", "T": 1, "K": 2048, "N": 32000, "format": "mxfp4", "group": 32,
         "zeros": False, "f32": True},
        # a serving batch at the 671B hidden size, integer weights
        {"name": "linear_batch", "op": "linear", "T": 64, "K": 7168, "N": 128000, "format": "int4", "group": 128,
         "zeros": True, "f32": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw(rng):
    op = rng.choice(("there", "there", "back", "back_grad", "rows", "clip", "linear", "linear"))
    kind = rng.choice(("bf16", "bf16", "f32"))
    if op in ("there", "back", "back_grad"):
        E = _log_int(rng, 1, 256)
        c = {"op": op, "T": _log_int(rng, 1, 98304), "k": rng.randint(1, min(8, E)), "E": E, "type": kind,
             "H": _log_int(rng, 50, 7168) if rng.random() < 0.4 else 32 * _log_int(rng, 2, 224),
             "empty": rng.choice((0.0, 0.0, 0.25))}
        if op == "there":
            c["form"] = rng.choice(("rows", "mxfp8", "both")) if c["H"] % 32 == 0 else "rows"
            c["ids"] = rng.choice(("i32", "i64"))
        if op == "back":
            c["residual"] = rng.random() < 0.5
        return c
    if op == "rows":
        return {"op": op, "R": _log_int(rng, 1, 65536), "C": 32 * _log_int(rng, 2, 448), "type": kind}
    if op == "clip":
        n = _log_int(rng, 1, 48)
        return {"op": op, "tensors": n, "total": _log_int(rng, 1000 * n, 1000000000), "clip": rng.random() < 0.7}
    form = rng.choice(("mxfp4", "int4"))
    group = 32 if form == "mxfp4" else rng.choice((32, 64, 128))
    return {"op": op, "T": _log_int(rng, 1, 64), "K": 128 * _log_int(rng, 2, 56) if rng.random() < 0.5
            else group * _log_int(rng, 256 // group, 7168 // group), "N": _log_int(rng, 100, 128000), "format": form,
            "group": group, "zeros": form == "int4" and rng.random() < 0.5, "f32": rng.random() < 0.3}


def draw(rng):
    most = {}
    for c in listed():
        most[c["op"]] = max(most.get(c["op"], 0.0), work(c)["bytes"])
    while True:
        c = _draw(rng)
        if work(c)["bytes"] <= most[c["op"]]:
            return c


def _size(case):
    return 4 if case["type"] == "f32" else 2


def work(case):
    """What a pass cannot do without: every input read once, every output written
    once (of the rows those that tokens go to, with half a block of padding for
    each expert where padding is written)."""
    c = case
    if c["op"] in ("there", "back", "back_grad"):
        T, k, E, H, b = c["T"], c["k"], c["E"], c["H"], _size(c)
        n = int(T * k * (1 - c["empty"]))
        padded = n + min(E, n) * ALIGN // 2
        if c["op"] == "there":
            each = {"rows": b, "mxfp8": 33 / 32, "both": b + 33 / 32}[c["form"]]
            return {"bytes": int((4 if c["ids"] == "i32" else 8) * T * k + 4 * T * k + 8 * E + b * T * H
                                 + each * padded * H), "flops": 0}
        if c["op"] == "back":
            return {"bytes": 8 * T * k + b * H * (n + T * (2 if c["residual"] else 1)), "flops": 2 * n * H}
        return {"bytes": 12 * T * k + b * H * (T + n + padded), "flops": 3 * n * H}
    if c["op"] == "rows":
        return {"bytes": int(c["R"] * c["C"] * (_size(c) + 33 / 32)), "flops": 0}
    if c["op"] == "clip":
        b = sum(n * s for n, s in zip(_sizes(c), _item_sizes(c)))
        return {"bytes": 2 * b if c["clip"] else b, "flops": (3 if c["clip"] else 2) * c["total"]}
    T, K, N, G = c["T"], c["K"], c["N"], c["group"]
    scale = 1 if c["format"] == "mxfp4" else 3 if c["zeros"] else 2
    return {"bytes": N * K // 2 + scale * N * (K // G) + 2 * T * K + (4 if c["f32"] else 2) * T * N,
            "flops": 2 * T * N * K}


def _sizes(c):
    """The tensors' element counts: a few hold most, as in a model."""
    n, total = c["tensors"], c["total"]
    share = [1.0 / (1 + i) ** 1.5 for i in range(n)]
    return [max(1, int(total * s / sum(share))) for s in share]


def _item_sizes(c):
    """Every third gradient is float32."""
    return [4 if i % 3 == 2 else 2 for i in range(c["tensors"])]


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _type(case):
    return torch.float32 if case["type"] == "f32" else torch.bfloat16


def _ids(c, g):
    """A skewed router's choices [T, k], int64, -1 in the empty slots."""
    T, k, E = c["T"], c["k"], c["E"]
    lean = torch.randn((E,), generator=g, device=DEV) * 0.4
    ids = (torch.randn((T, E), generator=g, device=DEV) + lean).topk(k, dim=1).indices
    if c["empty"]:
        off = torch.rand((T, k), generator=g, device=DEV) < c["empty"]
        ids = torch.where(off, torch.full_like(ids, -1), ids)
    return ids


def _rows_most(c):
    """Rows that any choice fits in, each expert's run a multiple of ALIGN."""
    n = c["T"] * c["k"]
    return (n + min(n, c["E"]) * (ALIGN - 1)) // ALIGN * ALIGN


def _plain_sort(ids, E):
    """(cumulative ends, counts, the row of every choice) of a stable sort."""
    flat = ids.reshape(-1).to(torch.int64)
    key = torch.where((flat < 0) | (flat >= E), torch.full_like(flat, E), flat)
    counts = torch.zeros((E + 1,), dtype=torch.int64, device=flat.device).scatter_add(0, key, torch.ones_like(key))
    padded = (counts[:E] + ALIGN - 1) // ALIGN * ALIGN
    ends = padded.cumsum(0)
    order = torch.argsort(key, stable=True)
    first = torch.cat([ends - padded - (counts.cumsum(0) - counts)[:E], torch.zeros_like(ends[:1])])
    sorted_key = key[order]
    place = torch.arange(len(flat), device=flat.device) + first[sorted_key]
    rows = torch.empty_like(flat).scatter(0, order, torch.where(sorted_key < E, place, torch.full_like(place, -1)))
    return ends.to(torch.int32), counts[:E].to(torch.int32), rows.to(torch.int32).view(ids.shape)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] in ("there", "back", "back_grad"):
        T, k, E, H, R = c["T"], c["k"], c["E"], c["H"], _rows_most(c)
        ids = _ids(c, g)
        if c["op"] == "there":
            s["ids"] = ids.to(torch.int32) if c["ids"] == "i32" else ids
            s["x"] = torch.randn((T, H), generator=g, device=DEV).to(_type(c))
            # the buffers that a training loop keeps; rows past the last run stay as they are
            if c["form"] != "mxfp8":
                s["xs"] = torch.zeros((R, H), dtype=_type(c), device=DEV)
            if c["form"] != "rows":
                s["q"] = torch.zeros((R, H), dtype=torch.uint8, device=DEV)
                s["s"] = torch.zeros((R, H // 32), dtype=torch.uint8, device=DEV)
            return s
        offs, counts, rows = _plain_sort(ids, E)
        s["plan"] = (offs, counts, rows, R)
        # what fwd left: nothing past the last run
        s["y"] = torch.randn((R, H), generator=g, device=DEV).to(_type(c))
        s["y"][int(offs[-1]):] = float("nan")
        w = torch.rand((T, k), generator=g, device=DEV) + 0.1
        s["w"] = w / w.sum(dim=1, keepdim=True)
        if c["op"] == "back":
            s["residual"] = torch.randn((T, H), generator=g, device=DEV).to(_type(c)) if c["residual"] else None
        else:
            s["dout"] = (torch.randn((T, H), generator=g, device=DEV) * 1e-3).to(_type(c))
            s["dy"] = torch.zeros((R, H), dtype=_type(c), device=DEV)
        return s
    if c["op"] == "rows":
        # activations of uneven size along the rows, a few outliers
        x = torch.randn((c["R"], c["C"]), generator=g, device=DEV)
        x = x * torch.exp2(torch.randint(-6, 3, (c["R"], 1), generator=g, device=DEV).float())
        hot = torch.rand((1, c["C"]), generator=g, device=DEV) < 0.01
        s["x"] = torch.where(hot, x * 30.0, x).to(_type(c))
        return s
    if c["op"] == "clip":
        s["grads"], s["out"] = [], []
        for n, b in zip(_sizes(c), _item_sizes(c)):
            t = torch.empty((n,), dtype=torch.float32 if b == 4 else torch.bfloat16, device=DEV)
            t.normal_(0.0, 0.02, generator=g)
            s["grads"].append(t)
            s["out"].append(torch.empty_like(t))
        return s
    T, K, N, G = c["T"], c["K"], c["N"], c["group"]
    s["x"] = torch.randn((T, K), generator=g, device=DEV).to(torch.bfloat16)
    s["codes"] = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    if c["format"] == "mxfp4":
        mid = 127 + round(math.log2(1.0 / (3.0 * math.sqrt(K))))
        s["scales"] = torch.randint(mid - 1, mid + 2, (N, K // 32), generator=g, device=DEV, dtype=torch.uint8)
    else:
        s["scales"] = ((torch.rand((N, K // G), generator=g, device=DEV) + 0.5) / (4.0 * math.sqrt(K))).to(torch.bfloat16)
    s["zeros"] = torch.randint(5, 11, (N, K // G), generator=g, device=DEV, dtype=torch.uint8) if c["zeros"] else None
    return s


def _power(e):
    """2^e in float32 for whole e from -126 to 127, exactly (exp2 and ldexp may
    be a last bit off on a GPU, which breaks ties)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _plain_mxfp8(x):
    """E4M3 codes and E8M0 scales of float32 x [R, C], 32-element blocks along C."""
    R, C = x.shape
    blocks = x.view(R, C // 32, 32)
    top = blocks.abs().amax(dim=2)
    e = torch.where(top > 0, torch.frexp(top).exponent - 1 - 8, torch.zeros_like(top, dtype=torch.int32))
    e = e.clamp(-127, 126)
    v = (blocks * _power(-e[:, :, None])).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    v = v.view(R, C)
    return torch.where(v.float() == 0, torch.zeros_like(v.float()), v.float()).to(torch.float8_e4m3fn), \
        (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _plain_there(s):
    c = s["case"]
    T, k, H, R = c["T"], c["k"], c["H"], _rows_most(c)
    offs, counts, rows = _plain_sort(s["ids"], c["E"])
    to = rows.reshape(-1).to(torch.int64)
    to = torch.where(to < 0, torch.full_like(to, R), to)
    token = torch.full((R + 1,), -1, dtype=torch.int64, device=to.device)
    token = token.scatter(0, to, torch.arange(T * k, device=to.device) // k)[:R]
    x = s["x"]
    xs = torch.where((token >= 0)[:, None], x[token.clamp(min=0)], torch.zeros((), dtype=x.dtype, device=x.device))
    out = {"offs": offs, "counts": counts, "rows": rows}
    if c["form"] != "mxfp8":
        out["xs"] = xs
    if c["form"] != "rows":
        out["q"], scales = _plain_mxfp8(xs.float())
        # the scale of a padding row's zeros, and nothing behind the last run
        inside = (torch.arange(R, device=to.device) < offs[-1])[:, None]
        out["s"] = torch.where(inside, scales.view(torch.uint8), torch.zeros_like(scales.view(torch.uint8))) \
            .view(torch.float8_e8m0fnu)
    return out


def _gathered(y, rows):
    """float32 y at every choice's row [T, k, H], zeros in the empty slots."""
    at = y.float()[rows.clamp(min=0).to(torch.int64)]
    return torch.where((rows >= 0)[:, :, None], at, torch.zeros_like(at))


def _values4(codes, scales, zeros, group):
    """The numbers that 4-bit weights [N, K/2] stand for: element 2 j in the low
    half of byte j."""
    N = codes.shape[0]
    n = torch.stack([codes & 15, codes >> 4], dim=2).view(N, -1, group)
    if scales.dtype == torch.uint8:
        m, e = (n & 1).float(), ((n >> 1) & 3).float()
        v = torch.where(e > 0, (1.0 + m * 0.5) * _power(e - 1), m * 0.5)
        v = torch.where(n > 7, -v, v)
        scale = _power(scales.to(torch.int32) - 127)
    else:
        v = n.float() - (8.0 if zeros is None else zeros.float()[:, :, None])
        scale = scales.float()
    return (v * scale[:, :, None]).view(N, -1)


def run(state):
    s, c = state, state["case"]
    if own:
        import mxfp8_ragged_grouped_amd as mxw

        if c["op"] == "there":
            plan = mxw.sort_tokens(s["ids"], c["E"], align=ALIGN)
            mxw.dispatch_tokens(s["x"], plan, rows=c["form"] != "mxfp8", mxfp8=c["form"] != "rows", out=s.get("xs"),
                                q=s.get("q"), s=s.get("s"))
            out = {"offs": plan.offs, "counts": plan.counts, "rows": plan.rows}
            if c["form"] != "mxfp8":
                out["xs"] = s["xs"]
            if c["form"] != "rows":
                out["q"], out["s"] = s["q"].view(torch.float8_e4m3fn), s["s"].view(torch.float8_e8m0fnu)
            return out
        if c["op"] == "back":
            return mxw.combine_tokens(s["y"], mxw.TokenPlan(*s["plan"]), weights=s["w"], residual=s["residual"])
        if c["op"] == "back_grad":
            dy, dw = mxw.combine_tokens_grad(s["dout"], s["y"], mxw.TokenPlan(*s["plan"]), s["w"], dy=s["dy"])
            return {"dy": dy, "dw": dw}
        if c["op"] == "rows":
            q, scales = mxw.quantize_rows(s["x"])
            return {"q": q.view(torch.float8_e4m3fn), "s": scales.view(torch.float8_e8m0fnu)}
        if c["op"] == "clip":
            if not c["clip"]:
                return {"norm": mxw.grad_norm(s["grads"])}
            return {"norm": mxw.clip_grad_norm(s["grads"], MAX_NORM, eps=EPS, out=s["out"]), "grads": s["out"]}
        return mxw.linear_4bit(s["x"], s["codes"], s["scales"], zeros=s["zeros"],
                               dtype=torch.float32 if c["f32"] else torch.bfloat16)
    if c["op"] == "there":
        return _plain_there(s)
    if c["op"] == "back":
        out = (_gathered(s["y"], s["plan"][2]) * s["w"][:, :, None]).sum(dim=1)
        if s["residual"] is not None:
            out = out + s["residual"].float()
        return out.to(_type(c))
    if c["op"] == "back_grad":
        offs, counts, rows, R = s["plan"]
        dout = s["dout"].float()
        dw = (_gathered(s["y"], rows) * dout[:, None, :]).sum(dim=2)
        each = (dout[:, None, :] * s["w"][:, :, None]).view(-1, c["H"])
        to = rows.reshape(-1).to(torch.int64)
        to = torch.where(to < 0, torch.full_like(to, R), to)
        dy = torch.zeros((R + 1, c["H"]), device=to.device).scatter(0, to[:, None].expand(-1, c["H"]), each)[:R]
        return {"dy": dy.to(_type(c)), "dw": dw}
    if c["op"] == "rows":
        q, scales = _plain_mxfp8(s["x"].float())
        return {"q": q, "s": scales}
    if c["op"] == "clip":
        squares = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]])
        norm = squares.sum().sqrt()
        if not c["clip"]:
            return {"norm": norm.float()}
        factor = (MAX_NORM / (norm + EPS)).clamp(max=1.0).float()
        return {"norm": norm.float(), "grads": [(g.float() * factor).to(g.dtype) for g in s["grads"]]}
    out = s["x"].float() @ _values4(s["codes"], s["scales"], s["zeros"], c["group"]).t()
    return out if c["f32"] else out.to(torch.bfloat16)


def _two_to(e):
    """2^e in 64 bits by its bits, exactly."""
    return ((e.to(torch.int64) + 1023) * 2 ** 52).view(torch.float64)


def _exact_mxfp8(x):
    """E4M3 by its definition: 4 significant bits from 2^-6 up, steps of 2^-9
    below, ties to even, at most 448; the scale 2^(floor(log2 top) - 8)."""
    R, C = x.shape
    blocks = x.view(R, C // 32, 32)
    top = blocks.abs().amax(dim=2, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top).exponent - 9, torch.zeros_like(top, dtype=torch.int32)).clamp(-127, 127)
    y = blocks * _two_to(-e)
    step = _two_to(torch.frexp(y).exponent.clamp(min=-5) - 4)
    return (torch.round(y / step) * step).clamp(-448.0, 448.0).view(R, C), _two_to(e)[:, :, 0]


def exact(case, seed):
    """The definitions in 64 bits."""
    c, s = case, prepare(case, seed)
    if c["op"] == "there":
        x, k, R = s["x"], c["k"], _rows_most(c)
        # where every choice goes, expert by expert
        flat = s["ids"].reshape(-1)
        token = torch.full((R,), -1, dtype=torch.int64, device=DEV)
        end = 0
        for e in range(c["E"]):
            mine = torch.nonzero(flat == e)[:, 0]
            token[end:end + len(mine)] = mine // k
            end += -(-len(mine) // ALIGN) * ALIGN
        xs = x.double()[token.clamp(min=0)]
        xs[token < 0] = 0.0
        out = {"offs": None, "counts": None, "rows": None}
        if c["form"] != "mxfp8":
            out["xs"] = xs
        if c["form"] != "rows":
            out["q"], out["s"] = _exact_mxfp8(xs)
            out["s"][end:] = 2.0 ** -127
        return out
    if c["op"] in ("back", "back_grad"):
        offs, counts, rows, R = s["plan"]
        total = torch.zeros((c["T"], c["H"]), dtype=torch.float64, device=DEV)
        if c["op"] == "back":
            for j in range(c["k"]):
                used = rows[:, j] >= 0
                total[used] += s["w"][used, j].double()[:, None] * s["y"][rows[used, j].long()].double()
            return total if s["residual"] is None else total + s["residual"].double()
        dy = torch.zeros((R, c["H"]), dtype=torch.float64, device=DEV)
        dw = torch.zeros(rows.shape, dtype=torch.float64, device=DEV)
        for j in range(c["k"]):
            used = rows[:, j] >= 0
            at, d = rows[used, j].long(), s["dout"][used].double()
            dy[at] = s["w"][used, j].double()[:, None] * d
            dw[used, j] = (d * s["y"][at].double()).sum(dim=1)
        return {"dy": dy, "dw": dw}
    if c["op"] == "rows":
        q, scales = _exact_mxfp8(s["x"].double())
        return {"q": q, "s": scales}
    if c["op"] == "clip":
        norm = math.sqrt(sum(float(g.double().square().sum()) for g in s["grads"]))
        at = torch.tensor(norm, dtype=torch.float64)
        if not c["clip"]:
            return {"norm": at}
        return {"norm": at, "grads": [g.double() * min(1.0, MAX_NORM / (norm + EPS)) for g in s["grads"]]}
    out = torch.empty((c["T"], c["N"]), dtype=torch.float64, device=DEV)
    E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=DEV)
    x = s["x"].double()
    for n0 in range(0, c["N"], 8192):
        codes = s["codes"][n0:n0 + 8192].long()
        n = torch.empty((codes.shape[0], c["K"]), dtype=torch.int64, device=DEV)
        n[:, 0::2], n[:, 1::2] = codes % 16, codes // 16
        scales = s["scales"][n0:n0 + 8192]
        if c["format"] == "mxfp4":
            v = E2M1[n % 8] * (1 - 2 * (n // 8))
            scales = _two_to(scales.long() - 127)
        else:
            z = 8 if s["zeros"] is None else s["zeros"][n0:n0 + 8192].long().repeat_interleave(c["group"], 1)
            v = (n - z).double()
        out[:, n0:n0 + 8192] = x @ (v * scales.double().repeat_interleave(c["group"], 1)).mT
    return out
