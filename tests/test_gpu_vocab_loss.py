"""mxw.vocab_cross_entropy against the definition in 64 bits (needs an MI355X).

Tolerances.  Loss: the logits are FP32 sums of H exact products (error about
sqrt(H) 2^-24 of the sum of magnitudes A, taken twice for the largest of many),
the exponentials and the logarithm are good to a few 2^-24:
2 sqrt(H) 2^-24 A + 2^-21 max(1, |lse|).  Gradients, element by element: g is
rounded to bf16 (half an ulp: 2^-8 of each term at most) and so is the result:
2^-8 |ref| + 1.05 2^-8 sum |g| |w| (likewise sum |g| |x| for dw); the FP32
errors of g fit in the 0.05.
"""
import math

import pytest
import torch

import mxfp8_ragged_grouped_amd as mxw

pytestmark = pytest.mark.gpu

DEV = "cuda"
IGNORE = -100


def say(msg):
    print("[gpu-case] " + msg, flush=True)


def make(T, H, V, seed, ignored=0.2, scale=1.5, int32=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((T, H), generator=g, device=DEV).to(torch.bfloat16)
    w = (torch.randn((V, H), generator=g, device=DEV) * (scale / math.sqrt(H))).to(torch.bfloat16)
    y = torch.randint(0, V, (T,), generator=g, device=DEV)
    y[torch.rand((T,), generator=g, device=DEV) < ignored] = IGNORE
    y[-1] = V - 1
    return x, w, y.to(torch.int32) if int32 else y


def reference(x, w, y, reduction="mean", grad_scale=1.0, ignore=IGNORE):
    x, w = x.double(), w.double()
    logits = x @ w.mT
    lse = torch.logsumexp(logits, dim=1)
    used = y != ignore
    idx = torch.where(used, y, torch.zeros_like(y)).long()
    rows = torch.where(used, lse - logits.gather(1, idx[:, None])[:, 0], torch.zeros_like(lse))
    n = max(int(used.sum()), 1)
    g = torch.exp(logits - lse[:, None])
    g[torch.arange(len(y), device=DEV), idx] -= 1.0
    g = g * used[:, None] * (grad_scale / n if reduction == "mean" else grad_scale)
    loss = rows if reduction == "none" else rows.sum() / (n if reduction == "mean" else 1)
    A = (x.abs() @ w.abs().mT).max().item()
    tol = 2 * math.sqrt(x.shape[1]) * 2.0 ** -24 * A + 2.0 ** -21 * max(1.0, lse.abs().max().item())
    if reduction == "sum":
        tol *= n
    return dict(loss=loss, dx=g @ w, dw=g.mT @ x, tol=tol, dx_terms=g.abs() @ w.abs(), dw_terms=g.abs().mT @ x.abs())


def check(got, ref, what=""):
    loss, dx, dw = got
    assert (loss.double() - ref["loss"]).abs().max().item() <= ref["tol"], what
    for name, t in (("dx", dx), ("dw", dw)):
        r = ref[name]
        bad = (t.double() - r).abs() > 2.0 ** -8 * r.abs() + 1.05 * 2.0 ** -8 * ref[name + "_terms"] + 1e-37
        assert not bad.any() and torch.isfinite(t).all(), "%s %s: %d of %d outside" % (what, name, int(bad.sum()),
                                                                                       bad.numel())


SIZES = [(1, 1, 1), (1, 1, 7), (1, 64, 1), (2, 3, 257), (5, 192, 1000), (31, 128, 255), (32, 64, 256), (33, 65, 300),
         (129, 256, 513), (127, 1001, 999), (256, 128, 4096), (300, 320, 2049), (513, 72, 3001), (1, 2048, 32000),
         (64, 128, 70001)]


@pytest.mark.parametrize("T,H,V", SIZES)
def test_against_64_bits(T, H, V):
    say("vocab loss T=%d H=%d V=%d" % (T, H, V))
    x, w, y = make(T, H, V, 2000 + T + H + V, int32=bool(T & 1))
    dx = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    dw = torch.full((V, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    got = mxw.vocab_cross_entropy(x, w, y, dx=dx, dw=dw)
    assert got[1] is dx and got[2] is dw
    ref = reference(x, w, y)
    check(got, ref, "T=%d H=%d V=%d" % (T, H, V))
    alone = mxw.vocab_cross_entropy(x, w, y, grads=False)
    assert torch.equal(alone, got[0])


def test_several_pieces():
    """A vocabulary walked in several pieces (g of all of it would take over
    256 MiB), aligned and padded operands, ragged last piece."""
    for T, H in ((4100, 64), (4100, 66)):
        V = 70003
        say("vocab loss in pieces T=%d H=%d V=%d" % (T, H, V))
        x, w, y = make(T, H, V, 77 + H)
        check(mxw.vocab_cross_entropy(x, w, y), reference(x, w, y), "H=%d" % H)


@pytest.mark.parametrize("T,H,V", [(4100, 1024, 33001), (4100, 64, 3001), (40, 1100, 20003), (33, 4992, 3001)])
def test_logits_kept_or_made_twice(T, H, V):
    """With room for the logits and without: the same bits, against 64 bits; in
    several pieces, padded operands, narrow and wide tiles."""
    say("vocab loss kept logits T=%d H=%d V=%d" % (T, H, V))
    x, w, y = make(T, H, V, 90 + H)
    small = mxw.vocab_loss_workspace_size(x.data_ptr(), H, w.data_ptr(), H, T, H, V, 11)
    assert small <= mxw.vocab_loss_workspace_size(x.data_ptr(), H, w.data_ptr(), H, T, H, V) - 4 * T * V
    got = mxw.vocab_cross_entropy(x, w, y)
    check(got, reference(x, w, y), "T=%d H=%d V=%d" % (T, H, V))
    again = mxw.vocab_cross_entropy(x, w, y, keep_logits=False)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    ws = torch.empty(small, dtype=torch.uint8, device=DEV)
    again = mxw.vocab_cross_entropy(x, w, y, keep_logits=False, workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_reductions_and_scale(reduction):
    x, w, y = make(70, 96, 700, 3)
    got = mxw.vocab_cross_entropy(x, w, y, reduction=reduction, grad_scale=0.37)
    assert got[0].shape == ((70,) if reduction == "none" else ())
    check(got, reference(x, w, y, reduction, 0.37), reduction)


def test_ignored_tokens():
    """Ignored tokens give zero rows; a batch without a counting token gives
    loss 0 and zero gradients; another ignore_index; an ignored row of NaN
    leaves the others alone in loss and dx."""
    x, w, y = make(40, 64, 300, 4, ignored=0.5)
    loss, dx, dw = mxw.vocab_cross_entropy(x, w, y, reduction="none")
    assert (loss[y == IGNORE] == 0).all() and (dx[y == IGNORE] == 0).all()
    none = torch.full_like(y, IGNORE)
    loss, dx, dw = mxw.vocab_cross_entropy(x, w, none)
    assert loss.item() == 0.0 and (dx == 0).all() and (dw == 0).all()
    y7 = torch.where(y == IGNORE, torch.full_like(y, 7), y)
    check(mxw.vocab_cross_entropy(x, w, y7, ignore_index=7), reference(x, w, y7, ignore=7), "ignore 7")


@pytest.mark.parametrize("T,H,V", [(40, 64, 300), (40, 65, 300), (300, 320, 2049), (3, 128, 513)])
def test_what_ignored_tokens_hold_is_not_used(T, H, V):
    """NaN and infinities in the x of tokens that do not count, or whose target
    is no word: the same bits as zeros there."""
    say("ignored tokens of NaN T=%d H=%d V=%d" % (T, H, V))
    x, w, y = make(T, H, V, 15, ignored=0.4)
    y[0], y[1] = IGNORE, V + 5
    out = (y < 0) | (y >= V)
    zeros = torch.where(out[:, None], torch.zeros_like(x), x)
    junk = torch.where(out[:, None], torch.full_like(x, float("nan")), x)
    junk[0] = float("inf")
    a = mxw.vocab_cross_entropy(zeros, w, y, reduction="none")
    b = mxw.vocab_cross_entropy(junk, w, y, reduction="none")
    assert a[0][1].isnan() and b[0][1].isnan() and (b[0][y == IGNORE] == 0).all()
    assert torch.equal(a[0][~out], b[0][~out]) and torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    assert torch.isfinite(b[1]).all() and torch.isfinite(b[2]).all()
    alone = mxw.vocab_cross_entropy(junk, w, y, reduction="none", grads=False)
    assert torch.equal(alone[~out], b[0][~out])


def test_targets_outside_the_vocabulary():
    x, w, y = make(20, 64, 300, 5, ignored=0.0)
    want = mxw.vocab_cross_entropy(x, w, y, reduction="none")
    bad = y.clone()
    bad[3], bad[11], bad[12] = 300, -1, 2 ** 40
    loss, dx, dw = mxw.vocab_cross_entropy(x, w, bad, reduction="none")
    out = torch.zeros(20, dtype=torch.bool, device=DEV)
    out[[3, 11, 12]] = True
    assert loss[out].isnan().all() and torch.equal(loss[~out], want[0][~out])
    assert (dx[out] == 0).all() and torch.equal(dx[~out], want[1][~out]) and torch.isfinite(dw).all()
    assert mxw.vocab_cross_entropy(x, w, bad, grads=False).isnan()


def test_large_logits_infinities_and_nan():
    """Logits of several hundred (a one-hot softmax), a weight row of -inf (its
    word is never said), NaN in one token."""
    x, w, y = make(40, 64, 300, 6, ignored=0.1, scale=200.0)
    check(mxw.vocab_cross_entropy(x, w, y), reference(x, w, y), "large logits")
    x, w, y = make(40, 64, 300, 7, ignored=0.0)
    x, xn = x.abs(), None
    y[y == 9] = 10
    want = mxw.vocab_cross_entropy(x, torch.cat([w[:9], w[10:]]), torch.where(y > 9, y - 1, y), reduction="none",
                                   grads=False)
    gone = w.clone()
    gone[9] = -float("inf")
    loss = mxw.vocab_cross_entropy(x, gone, y, reduction="none", grads=False)
    assert (loss - want).abs().max() < 1e-5
    broken = x.clone()
    broken[5, 3] = float("nan")
    rows = mxw.vocab_cross_entropy(broken, w, y, reduction="none", grads=False)
    assert rows[5].isnan() and torch.isfinite(rows[torch.arange(40, device=DEV) != 5]).all()


def test_gradients_against_differences():
    """The slope of the loss along a direction of x, and of w, from losses on
    either side (64-bit reference of the loss on perturbed bf16 inputs' exact
    values), against the gradients: both come from 2^-8-exact numbers, the
    difference quotient adds its third-order term."""
    x, w, y = make(24, 64, 200, 8)
    _, dx, dw = mxw.vocab_cross_entropy(x, w, y, reduction="sum")
    g = torch.Generator(device=DEV).manual_seed(1)
    for which, t, grad in (("x", x, dx), ("w", w, dw)):
        d = torch.randn(t.shape, generator=g, device=DEV).double()
        h = 1e-4

        def loss(sign):
            xs = x.double() + (sign * h * d if which == "x" else 0)
            ws = w.double() + (sign * h * d if which == "w" else 0)
            logits = xs @ ws.mT
            used = y != IGNORE
            rows = torch.logsumexp(logits, 1) - logits.gather(1, y.clamp(min=0)[:, None])[:, 0]
            return (rows * used).sum()

        slope = (loss(1) - loss(-1)) / (2 * h)
        assert abs((grad.double() * d).sum() - slope) <= 2.0 ** -8 * (grad.double() * d).abs().sum()


def test_strides_and_alignment():
    """Rows apart, odd first elements, an odd stride: in place and padded reads
    give the same bits."""
    x, w, y = make(50, 128, 700, 9)
    want = mxw.vocab_cross_entropy(x, w, y)
    for pad, first in ((8, 0), (64, 8), (1, 0), (8, 1), (3, 5)):
        xb = torch.full((51 * (128 + pad) + 16,), float("nan"), dtype=torch.bfloat16, device=DEV)
        wb = torch.full((701 * (128 + pad) + 16,), float("nan"), dtype=torch.bfloat16, device=DEV)
        xs = xb.as_strided((50, 128), (128 + pad, 1), first)
        ws = wb.as_strided((700, 128), (128 + pad, 1), first)
        xs.copy_(x)
        ws.copy_(w)
        got = mxw.vocab_cross_entropy(xs, ws, y)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), (pad, first)
    dw = torch.empty(700 * 128 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(700, 128)
    dx = torch.empty(50 * 128 + 1, dtype=torch.bfloat16, device=DEV)[1:].view(50, 128)
    got = mxw.vocab_cross_entropy(x, w, y, dx=dx, dw=dw)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_weights_past_32_bit_offsets():
    """A vocabulary of more than 4 GiB: the last words' logits and gradients."""
    T, H, V = 3, 7168, 320001
    x, _, _ = make(T, H, 8, 13)
    w = torch.zeros((V, H), dtype=torch.bfloat16, device=DEV)
    last = make(T, H, 500, 14)[1]
    w[-500:] = last
    y = torch.tensor([V - 1, V - 500, 3], device=DEV)
    loss, dx, dw = mxw.vocab_cross_entropy(x, w, y, reduction="none")
    # the words of zero weight share logit 0: one word of weight V - 500
    logits = x.double() @ last.double().mT
    both = torch.cat([logits, torch.full((T, 1), math.log(V - 500), dtype=torch.float64, device=DEV)], 1)
    lse = torch.logsumexp(both, 1)
    ref = lse - torch.stack([logits[0, 499], logits[1, 0], torch.zeros((), dtype=torch.float64, device=DEV)])
    A = (x.double().abs() @ last.double().abs().mT).max().item()
    assert (loss.double() - ref).abs().max() <= 2 * math.sqrt(H) * 2.0 ** -24 * A + 2.0 ** -21 * lse.max()
    g = torch.exp(logits - lse[:, None])
    g[0, 499] -= 1
    g[1, 0] -= 1
    for t, r, terms in ((dw[-500:], g.mT @ x.double(), g.abs().mT @ x.double().abs()),
                        (dx, g @ last.double(), g.abs() @ last.double().abs())):
        assert ((t.double() - r).abs() <= 2.0 ** -8 * r.abs() + 1.05 * 2.0 ** -8 * terms + 1e-37).all()


def test_far_apart_rows():
    """Row strides beyond what a tile's 32-bit offsets reach (3 Mi elements)."""
    x, w, y = make(30, 64, 40, 15)
    want = mxw.vocab_cross_entropy(x, w, y)
    far = torch.empty((40, 3 << 20), dtype=torch.bfloat16, device=DEV)
    far[:, :64] = w
    got = mxw.vocab_cross_entropy(x, far[:, :64], y)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("which", [1, 2])
def test_one_gradient_alone(which):
    """The C entry with dx or dw left out."""
    x, w, y = make(70, 128, 900, 16)
    want = mxw.vocab_cross_entropy(x, w, y)
    loss = torch.empty((), device=DEV)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    need = mxw.vocab_loss_workspace_size(x.data_ptr(), 128, w.data_ptr(), 128, 70, 128, 900, which)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    rc = mxw.mxw_vocab_loss(x.data_ptr(), 128, w.data_ptr(), 128, y.data_ptr(), 8, IGNORE, 70, 128, 900, 1, 1.0,
                            loss.data_ptr(), dx.data_ptr() if which == 1 else 0, dw.data_ptr() if which == 2 else 0,
                            ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and torch.equal(loss, want[0])
    assert torch.equal(dx, want[1]) if which == 1 else torch.equal(dw, want[2])


def test_repeats_streams_and_graphs():
    x, w, y = make(300, 192, 3000, 10)
    want = mxw.vocab_cross_entropy(x, w, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = mxw.vocab_cross_entropy(x, w, y, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(other, want))
    need = mxw.vocab_loss_workspace_size(x.data_ptr(), 192, w.data_ptr(), 192, 300, 192, 3000)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        loss, _, _ = mxw.vocab_cross_entropy(x, w, y, dx=dx, dw=dw, workspace=ws)
    for i in range(3):
        x.copy_(x.roll(1, 0))
        graph.replay()
        torch.cuda.synchronize()
        now = mxw.vocab_cross_entropy(x, w, y)
        assert all(torch.equal(a, b) for a, b in zip((loss, dx, dw), now)), "replay %d" % i
    with pytest.raises(ValueError):
        mxw.vocab_cross_entropy(x, w, y, workspace=ws[:need - 1])


def test_room_for_less_than_the_logits():
    """With memory for the smaller workspace but not for the logits, the call
    makes them twice instead of failing: the same bits."""
    T, H, V = 2000, 1024, 30000
    x, w, y = make(T, H, V, 21)
    want = mxw.vocab_cross_entropy(x, w, y)
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    small = mxw.vocab_loss_workspace_size(x.data_ptr(), H, w.data_ptr(), H, T, H, V, 11)
    assert mxw.vocab_loss_workspace_size(x.data_ptr(), H, w.data_ptr(), H, T, H, V) >= small + 4 * T * V
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    room = torch.cuda.memory_reserved() + small + (64 << 20)  # the logits take 240 MB
    torch.cuda.set_per_process_memory_fraction(room / torch.cuda.get_device_properties(0).total_memory)
    try:
        got = mxw.vocab_cross_entropy(x, w, y, dx=dx, dw=dw)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_minus_infinite_logits():
    """A word of weights -inf (x positive) is never said: the losses and the dw of
    the other words are those without it, its own dw is 0, and dx is the NaN of
    g = 0 times its weights.  As a target it makes the loss inf."""
    x, w, y = make(40, 64, 300, 22, ignored=0.0)
    x = x.abs() + 0.01
    y[y == 9] = 10
    without = torch.cat([w[:9], w[10:]])
    gone = w.clone()
    gone[9] = -float("inf")
    loss, dx, dw = mxw.vocab_cross_entropy(x, gone, y, reduction="none")
    ref = reference(x, without, torch.where(y > 9, y - 1, y), reduction="none")
    assert ((loss.double() - ref["loss"]).abs() <= ref["tol"]).all() and dx.isnan().all() and (dw[9] == 0).all()
    rest = torch.cat([dw[:9], dw[10:]]).double()
    assert ((rest - ref["dw"]).abs() <= 2.0 ** -8 * ref["dw"].abs() + 1.05 * 2.0 ** -8 * ref["dw_terms"] + 1e-37).all()
    y[3] = 9
    loss = mxw.vocab_cross_entropy(x, gone, y, reduction="none", grads=False)
    assert loss[3] == float("inf") and torch.isfinite(loss[torch.arange(40, device=DEV) != 3]).all()
