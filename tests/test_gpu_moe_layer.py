"""mxw.moe_layer against the definition in 64 bits (needs an MI355X).

Tolerances.  A sum of H exact FP32-accumulated products is off by about
sqrt(H) 2^-24 of the sum of magnitudes; twice that is allowed.  Call that d for
the logits, the gate and the up values.  Weights: 2 d + 2^-20, relative.  Out,
element by element: weight * h is rounded to bf16 (2^-8 of each term at most) and
so is the result; the gate's and up's d pass through silu (slope <= 1.1):

    2^-8 |ref| + sum_j w_j sum_i |Wd| (1.05 2^-8 |h| + 1.1 |u| d_g + |silu g| d_u)

plus the weights' relative error times sum_j w_j sum_i |Wd| |h|.  ids are exact:
tokens whose first k + 1 logits come nearer than 4 d are drawn again.
"""
import math

import pytest
import torch

import mxfp8_ragged_grouped_amd as mxw

pytestmark = pytest.mark.gpu

DEV = "cuda"


def say(msg):
    print("[gpu-case] " + msg, flush=True)


def decode(codes, scales):
    b = torch.arange(256, dtype=torch.int64, device=DEV)
    e, m = (b >> 3) & 15, (b & 7).double()
    t = torch.where(e > 0, torch.ldexp(1 + m / 8, e - 7), torch.ldexp(m / 8, torch.full_like(e, -6)))
    t = torch.where(b > 127, -t, t)
    t[127] = t[255] = float("nan")
    s = torch.ldexp(torch.ones(256, dtype=torch.float64, device=DEV), b - 127)
    s[255] = float("nan")
    return t[codes.long()] * s[scales.long()].repeat_interleave(32, -1)


def mx(g, E, R, C):
    codes = (torch.randn((E, R, C), generator=g, device=DEV) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    mid = 127 + round(math.log2(1 / (100 * math.sqrt(C))))
    scales = torch.randint(mid - 2, mid + 3, (E, R, C // 32), generator=g, device=DEV, dtype=torch.uint8)
    return codes.view(torch.uint8), scales


def make(T, E, k, H, I, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    router = (torch.randn((E, H), generator=g, device=DEV) / math.sqrt(H)).to(torch.bfloat16)
    x = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    for _ in range(30):
        d = sum_error(x, router)
        top = (x.double() @ router.double().mT).sort(dim=1, descending=True).values[:, :k + 1]
        near = ((top[:, :-1] - top[:, 1:]) < 4 * d.max()).any(1) if top.shape[1] > 1 else torch.zeros(T, dtype=torch.bool)
        x = torch.where(near.to(DEV)[:, None], torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16), x)
    wgu, sgu = mx(g, E, 2 * I, H)
    wd, sd = mx(g, E, H, I)
    return dict(x=x, router=router, wgu=wgu, sgu=sgu, wd=wd, sd=sd)


def sum_error(x, w):
    return 2 * math.sqrt(x.shape[1]) * 2.0 ** -24 * (x.double().abs() @ w.double().abs().mT)


def route(x, router, k, normalize=True, scale=1.0, active=None):
    p = torch.softmax(x.double() @ router.double().mT, 1)
    ids = torch.argsort(p, dim=1, descending=True, stable=True)[:, :k]
    w = p.gather(1, ids)
    if normalize:
        w = w / w.sum(1, keepdim=True)
    w = w * scale
    if active is not None:
        w = torch.where(active[:, None], w, torch.zeros_like(w))
        ids = torch.where(active[:, None], ids, torch.full_like(ids, -1))
    return ids, w


def experts(a, ids, w, wrel=0.0):
    """out in 64 bits and its tolerance."""
    x = a["x"].double()
    out, tol = torch.zeros_like(x), torch.zeros_like(x)
    I = a["wd"].shape[2]
    for e in sorted(set(ids.flatten().tolist())):
        if not 0 <= e < a["wd"].shape[0]:
            continue
        share = torch.where(ids == e, w, torch.zeros_like(w)).sum(1, keepdim=True)
        rows = (ids == e).any(1)
        Wgu, Wd = decode(a["wgu"][e], a["sgu"][e]), decode(a["wd"][e], a["sd"][e])
        xe = x[rows]
        gu, d = xe @ Wgu.mT, sum_error(xe, Wgu)
        g, u, dg, du = gu[:, :I], gu[:, I:], d[:, :I], d[:, I:]
        silu = g / (1 + torch.exp(-g))
        h = silu * u
        out[rows] += share[rows] * (h @ Wd.mT)
        terms = (1.05 * 2.0 ** -8 + wrel) * h.abs() + 1.1 * u.abs() * dg + silu.abs() * du
        tol[rows] += share[rows].abs() * (terms @ Wd.abs().mT)
    return out, tol + 2.0 ** -8 * out.abs()


def check(got, a, k, normalize=True, scale=1.0, active=None):
    out, ids, weights = got
    rids, rw = route(a["x"], a["router"], k, normalize, scale, active)
    assert torch.equal(ids.long(), rids)
    wrel = 2 * float(sum_error(a["x"], a["router"]).max()) + 2.0 ** -20
    assert ((weights.double() - rw).abs() <= wrel * rw.abs()).all()
    ref, tol = experts(a, rids, rw, wrel)
    bad = (out.double() - ref).abs() > tol
    assert not bad.any(), "%d of %d outside, worst %.2f of its tolerance" % (
        int(bad.sum()), bad.numel(), float(((out.double() - ref).abs() / tol.clamp(min=1e-30)).max()))


SIZES = [(1, 1, 1, 32, 32), (1, 8, 2, 2048, 1408), (2, 3, 2, 64, 96), (16, 16, 4, 256, 128), (17, 5, 5, 160, 32),
         (13, 10, 3, 1120, 416), (33, 17, 1, 96, 2048), (40, 4, 4, 288, 352), (64, 256, 8, 64, 64), (64, 2, 1, 1024, 512),
         (64, 16, 16, 128, 160), (3, 65, 6, 4128, 32), (1, 32, 8, 7168, 2048), (64, 130, 8, 512, 352)]


@pytest.mark.parametrize("T,E,k,H,I", SIZES)
def test_against_64_bits(T, E, k, H, I):
    say("moe_layer T=%d E=%d k=%d H=%d I=%d" % (T, E, k, H, I))
    a = make(T, E, k, H, I, 3000 + T + E + H + I)
    out = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    got = mxw.moe_layer(**a, top_k=k, out=out)
    assert got[0] is out
    check(got, a, k)


@pytest.mark.parametrize("T,E,k,H,I", [(4, 130, 8, 512, 352), (5, 130, 8, 512, 352), (12, 64, 4, 1024, 96),
                                       (40, 8, 2, 2048, 704), (17, 8, 2, 2048, 256), (1, 16, 8, 4096, 1568)])
def test_either_side_of_the_rules(T, E, k, H, I):
    """The choices in the gate kernel or by a launch, the down product whole or by
    items, one group of rows a wave or two."""
    say("moe_layer rules T=%d E=%d k=%d H=%d I=%d" % (T, E, k, H, I))
    a = make(T, E, k, H, I, 4000 + T + E + H + I)
    check(mxw.moe_layer(**a, top_k=k), a, k)


@pytest.mark.parametrize("normalize,scale", [(True, 2.5), (False, 1.0), (False, 0.3)])
def test_weights(normalize, scale):
    a = make(9, 24, 5, 192, 64, 1)
    check(mxw.moe_layer(**a, top_k=5, normalize=normalize, scale=scale), a, 5, normalize, scale)


@pytest.mark.parametrize("T,E,k,H,I", [(2, 4, 2, 160, 96), (16, 16, 16, 96, 1056), (20, 6, 3, 288, 32)])
def test_infinities_in_x(T, E, k, H, I):
    """x[t][0] infinite, every weight positive (row lengths that end inside a
    step of 128 columns): the outputs are inf, not the NaN of inf times a zero
    that fills a step up; the choices are the experts whose logit is inf."""
    say("moe_layer infinities T=%d E=%d k=%d H=%d I=%d" % (T, E, k, H, I))
    a = make(T, E, k, H, I, 21)
    a["wgu"], a["wd"] = (a["wgu"] & 0x70) | 0x08, (a["wd"] & 0x70) | 0x08
    a["x"] = a["x"].abs()
    a["x"][:, 0] = float("inf")
    ids = torch.arange(T * k, device=DEV, dtype=torch.int32).reshape(T, k) % E
    weights = torch.full((T, k), 0.5, device=DEV)
    b = dict(a)
    b.pop("router")
    out = mxw.moe_layer(router=None, routing=(ids, weights), top_k=k, **b)[0]
    assert (out == float("inf")).all()
    router = a["router"].abs() + 0.01
    router[: E - k, 0] *= -1
    got = mxw.moe_layer(**dict(a, router=router), top_k=k)
    assert torch.equal(got[1].long(), torch.arange(E - k, E, device=DEV).expand(T, k)) and got[2].isnan().all()


def test_tokens_that_are_not_there():
    """Their x is not used (NaN), their rows are zero, no expert is read for
    them; a batch of none at all."""
    a = make(20, 12, 3, 160, 96, 2)
    active = torch.ones(20, dtype=torch.bool, device=DEV)
    active[[0, 7, 19]] = False
    clean = dict(a)
    a["x"] = torch.where(active[:, None], a["x"], torch.full_like(a["x"], float("nan")))
    clean["x"] = torch.where(active[:, None], a["x"], torch.zeros_like(a["x"]))
    got = mxw.moe_layer(**a, top_k=3, active=active)
    check(got, clean, 3, active=active)
    assert (got[0][~active] == 0).all()
    out, ids, w = mxw.moe_layer(**a, top_k=3, active=torch.zeros_like(active))
    assert (out == 0).all() and (ids == -1).all() and (w == 0).all()


def test_ties_go_to_the_lower_expert():
    a = make(6, 40, 4, 128, 64, 3)
    a["router"][1::2] = a["router"][0::2]
    _, ids, w = mxw.moe_layer(**a, top_k=4)
    top = (a["x"].double() @ a["router"].double().mT).sort(dim=1, descending=True, stable=True).indices[:, :4]
    assert torch.equal(ids.long(), top)
    a["router"][:] = 0
    _, ids, w = mxw.moe_layer(**a, top_k=4)
    assert (ids == torch.arange(4, device=DEV)).all() and (w == 0.25).all()


def test_routing_of_ones_own():
    """Empty slots, ids outside the experts, one expert twice, weights as given
    (negative too), an expert with all 64 tokens."""
    a = make(64, 9, 1, 128, 160, 4)
    a.pop("router")
    g = torch.Generator(device=DEV).manual_seed(5)
    ids = torch.randint(-2, 11, (64, 3), generator=g, device=DEV, dtype=torch.int32)
    ids[:, 0] = 4
    ids[5] = torch.tensor([2, 2, 2], dtype=torch.int32)
    ids[6] = -1
    w = torch.randn((64, 3), generator=g, device=DEV)
    out, _, _ = mxw.moe_layer(a["x"], None, a["wgu"], a["sgu"], a["wd"], a["sd"], 3, routing=(ids, w))
    ref, tol = experts(a, ids.long(), w.double())
    # weights of one expert given twice may cancel: their sum is FP32
    assert ((out.double() - ref).abs() <= tol + 1e-6).all() and (out[6] == 0).all()


def test_only_chosen_experts_matter():
    """NaN codes and 0xFF scales in experts nobody chose change no bit; a chosen
    expert's reach its tokens alone."""
    a = make(5, 32, 2, 96, 64, 6)
    want, ids, _ = mxw.moe_layer(**a, top_k=2)
    b = {k: v.clone() for k, v in a.items()}
    idle = [e for e in range(32) if e not in set(ids.flatten().tolist())]
    for e in idle:
        b["wgu"][e] = 0x7F
        b["sd"][e] = 0xFF
    assert torch.equal(mxw.moe_layer(**b, top_k=2)[0], want)
    e = int(ids[2, 0])
    b["sgu"][e, 3, 1] = 0xFF
    out = mxw.moe_layer(**b, top_k=2)[0]
    hit = (ids == e).any(1)
    assert out[hit].isnan().all() and torch.equal(out[~hit], want[~hit])


def test_broken_tokens_stay_alone():
    a = make(18, 6, 2, 64, 64, 7)
    want = mxw.moe_layer(**a, top_k=2)
    b = dict(a, x=a["x"].clone())
    b["x"][4, 9] = float("nan")
    b["x"][17, 63] = float("inf")
    out, ids, w = mxw.moe_layer(**b, top_k=2)
    good = torch.ones(18, dtype=torch.bool, device=DEV)
    good[[4, 17]] = False
    assert torch.equal(out[good], want[0][good]) and torch.equal(ids[good], want[1][good])
    assert out[~good].isnan().all() and w[~good].isnan().all()
    assert ((ids >= 0) & (ids < 6)).all() and (ids[:, 0] != ids[:, 1]).all()


def test_every_code_and_wide_scales():
    """All E4M3 codes but NaN, scales from 2^-100 to 2^100 in matching pairs."""
    a = make(4, 2, 1, 256, 256, 8)
    codes = torch.arange(256, device=DEV, dtype=torch.int64)
    codes = torch.where((codes & 127) == 127, torch.zeros_like(codes), codes).to(torch.uint8)
    a["wgu"][:] = codes
    a["wd"][:] = codes.flip(0)
    a["sgu"][:, :256] = 127 - 10
    a["sgu"][:, 256:] = 27
    a["sd"][:] = 127 + 90
    check(mxw.moe_layer(**a, top_k=1), a, 1)


def test_strides_and_types():
    a = make(7, 10, 3, 96, 64, 9)
    want = mxw.moe_layer(**a, top_k=3)
    buf = torch.full((7, 120), float("nan"), dtype=torch.bfloat16, device=DEV)
    b = dict(a, x=buf[:, 8:104], wgu=a["wgu"].view(torch.float8_e4m3fn), wd=a["wd"].view(torch.float8_e4m3fn))
    b["x"].copy_(a["x"])
    got = mxw.moe_layer(**b, top_k=3)
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    bad = torch.zeros((7, 97), dtype=torch.bfloat16, device=DEV)[:, :96]
    with pytest.raises(mxw.MxwError):
        mxw.moe_layer(**dict(a, x=bad), top_k=3)     # rows not a multiple of 8 elements apart


def test_weights_past_32_bit_offsets():
    """More than 4 GiB of gate/up codes: the first and the last expert."""
    E, H, I = 160, 7168, 2048
    a = make(3, 2, 1, H, I, 10)
    wgu = torch.zeros((E, 2 * I, H), dtype=torch.uint8, device=DEV)
    sgu = torch.full((E, 2 * I, H // 32), 127, dtype=torch.uint8, device=DEV)
    wd = torch.zeros((E, H, I), dtype=torch.uint8, device=DEV)
    sd = torch.full((E, H, I // 32), 127, dtype=torch.uint8, device=DEV)
    for to, e in ((0, 0), (E - 1, 1)):
        wgu[to], sgu[to], wd[to], sd[to] = a["wgu"][e], a["sgu"][e], a["wd"][e], a["sd"][e]
    ids = torch.tensor([[0, E - 1], [E - 1, -1], [0, -1]], dtype=torch.int32, device=DEV)
    small = torch.tensor([[0, 1], [1, -1], [0, -1]], dtype=torch.int32, device=DEV)
    w = torch.tensor([[0.25, 0.75], [1.0, 0.0], [1.0, 0.0]], device=DEV)
    out, _, _ = mxw.moe_layer(a["x"], None, wgu, sgu, wd, sd, 2, routing=(ids, w))
    ref, tol = experts(a, small.long(), w.double())
    assert ((out.double() - ref).abs() <= tol).all()


def test_repeats_streams_and_graphs():
    a = make(24, 20, 4, 320, 192, 11)
    want = mxw.moe_layer(**a, top_k=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = mxw.moe_layer(**a, top_k=4, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(other, want))
    need = mxw.moe_workspace_size(24, 20, 4, 320, 192)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.empty_like(a["x"])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = mxw.moe_layer(**a, top_k=4, out=out, workspace=ws)
    for i in range(3):
        a["x"].copy_(a["x"].roll(1, 0))
        graph.replay()
        torch.cuda.synchronize()
        now = mxw.moe_layer(**a, top_k=4)
        assert all(torch.equal(p, q) for p, q in zip(got, now)), "replay %d" % i
    with pytest.raises(ValueError):
        mxw.moe_layer(**a, top_k=4, workspace=ws[:need - 1])


@pytest.mark.parametrize("T,E,k,H,I", [(2, 16, 2, 2048, 1408), (4, 32, 2, 1024, 704), (3, 20, 3, 4128, 576),
                                       (16, 24, 2, 512, 192), (20, 12, 2, 256, 320), (64, 9, 2, 96, 448),
                                       (8, 64, 4, 512, 704), (40, 40, 3, 288, 832)])
def test_neighbours_do_not_move_a_bit(T, E, k, H, I):
    """A token's result is bit for bit the same whatever the other tokens of the
    batch hold and choose, and whether they are there, in both forms of the down
    product.  The second half of every expert's hidden values repeats the first
    with the opposite down weights, so out is nothing but its sums' rounding
    errors, which another order or grouping of the terms changes nearly everywhere."""
    say("moe_layer neighbours T=%d E=%d k=%d H=%d I=%d" % (T, E, k, H, I))
    a = make(T, E, k, H, I, 5000 + T + E + H + I)
    h = I // 2
    for n in ("wgu", "sgu"):
        a[n][:, h:I], a[n][:, I + h:] = a[n][:, :h].clone(), a[n][:, I:I + h].clone()
    a["wd"][..., h:], a["sd"][..., h // 32:] = a["wd"][..., :h] ^ 0x80, a["sd"][..., :h // 32].clone()
    want = mxw.moe_layer(**a, top_k=k)
    for t in sorted({0, T // 2, T - 1}):
        alone = torch.zeros(T, dtype=torch.bool, device=DEV)
        alone[t] = True
        few = alone.clone()
        few[(t + 1) % T] = True
        others = dict(a, x=torch.where(alone[:, None], a["x"], a["x"].flip(1)))
        for b, active in ((a, alone), (a, few), (others, None), (others, few)):
            got = mxw.moe_layer(**b, top_k=k, active=active)
            assert all(torch.equal(p[t], q[t]) for p, q in zip(got, want)), "token %d" % t


@pytest.mark.parametrize("T,E,k,H,I", [(64, 16, 16, 64, 256), (64, 14, 14, 64, 288), (16, 7, 7, 4096, 1728),
                                       (16, 256, 16, 4096, 32)])
def test_down_at_the_room_for_its_sums(T, E, k, H, I):
    """Partial sums of every step and choice that just fit in LDS, that do not
    (by items then), and the most experts."""
    say("moe_layer down sums T=%d E=%d k=%d H=%d I=%d" % (T, E, k, H, I))
    a = make(T, E, k, H, I, 6000 + T + E + H + I)
    check(mxw.moe_layer(**a, top_k=k), a, k)


def test_minus_infinite_router_logit():
    """An expert whose logit is -inf is never chosen and changes nothing else;
    where it has to be chosen its weight is 0."""
    a = make(9, 8, 3, 96, 64, 31)
    a["x"] = a["x"].abs() + 0.1
    fewer = {n: torch.cat([t[:2], t[3:]]) if n != "x" else t for n, t in a.items()}
    want = mxw.moe_layer(**fewer, top_k=3)
    a["router"][2] = -float("inf")
    got = mxw.moe_layer(**a, top_k=3)
    assert torch.equal(got[1], torch.where(want[1] >= 2, want[1] + 1, want[1])) and torch.isfinite(got[2]).all()
    # the weights' sums run over the lanes in another order
    assert (got[2] - want[2]).abs().max() <= 2.0 ** -20
    assert (got[0].double() - want[0].double()).norm() <= 2.0 ** -8 * want[0].double().norm()
    out, ids, w = mxw.moe_layer(**a, top_k=8)
    assert (ids[:, 7] == 2).all() and (w[:, 7] == 0).all() and torch.isfinite(w).all() and torch.isfinite(out).all()
