"""clip_grad_norm and grad_norm against 64 bits (needs an MI355X).

Tolerances: the norm's sum is in 64 bits (its roundings, at most 2^-53 of each partial sum,
are far below) and rounded once to float32: 2^-24, and the largest magnitude is exact.  A
scaled gradient takes the factor's rounding, 2^-24, the product's, 2^-24, and for bf16 the
result's, 2^-8; results below the normal range may be off by the smallest subnormal besides.
"""
import math

import pytest
import torch

import mxfp8_ragged_grouped_amd as mxw

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
INF = float("inf")


def say(msg):
    print("[gpu-case] " + msg, flush=True)


def tensors(sizes, seed, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [(torch.randn((n,), generator=g, device=DEV) * scale).to(F32 if i % 3 == 2 else BF16) for i, n in enumerate(sizes)]


def norm_of(grads, norm_type=2):
    if norm_type == INF:
        return max([float(g.double().abs().max()) for g in grads if g.numel()], default=0.0)
    return math.sqrt(sum(float(g.double().square().sum()) for g in grads))


def close(got, g, factor):
    ref = g.double() * factor
    rel = 2.0 ** -23 + (2.0 ** -8 if g.dtype == BF16 else 0.0)
    least = 2.0 ** -133 if g.dtype == BF16 else 2.0 ** -149
    bad = ~((got.double() - ref).abs() <= rel * (1 + 2.0 ** -10) * ref.abs() + least)
    assert got.dtype == g.dtype and got.shape == g.shape and not bad.any(), int(bad.sum())


SIZES = [[1], [7], [8], [9], [2047, 1, 0, 5], [8191], [8192], [8193], [1 << 20, 3, 70000, 0, 8192 * 3 + 5],
         [100 + 37 * i for i in range(97)], [1 + i % 50 for i in range(300)], [3 * 10 ** 7, 11], [0, 0, 0]]


@pytest.mark.parametrize("norm_type", [2, INF])
@pytest.mark.parametrize("case", range(len(SIZES)))
def test_against_64_bits(case, norm_type):
    sizes = SIZES[case]
    say("clip %d tensors, %d elements, norm %s" % (len(sizes), sum(sizes), norm_type))
    grads = tensors(sizes, case)
    n = norm_of(grads, norm_type)
    assert abs(mxw.grad_norm(grads, norm_type).item() - n) <= 2.0 ** -24 * n
    for max_norm in (0.25 * n + 1e-3, 4 * n + 1):
        factor = min(1.0, max_norm / (n + 1e-6))
        out = [torch.full_like(g, float("nan")) for g in grads]
        got = mxw.clip_grad_norm(grads, max_norm, norm_type, out=out)
        assert abs(got.item() - n) <= 2.0 ** -24 * n and got.dtype == F32 and got.shape == ()
        inside = [g.clone() for g in grads]
        again = mxw.clip_grad_norm(inside, max_norm, norm_type)
        assert again.item() == got.item()
        for g, o, i in zip(grads, out, inside):
            close(o, g, factor)
            assert torch.equal(i, o)
            if factor == 1.0:
                assert torch.equal(i.view(torch.uint8), g.view(torch.uint8))


@pytest.mark.parametrize("scale", [1e-42, 1e-30, 1e-19, 1e15, 1e30, 3e37])
def test_squares_out_of_float32s_range(scale):
    grads = [g for g in tensors([3, 100, 5000], 1)]
    grads = [(g.double() * scale).to(g.dtype) for g in grads]
    n = norm_of(grads)
    got = mxw.grad_norm(grads).item()
    if n >= 2.0 ** 128:  # 3e37 sqrt(5103) = 2.1e39 is past float32's 3.4e38: its rounding is infinity
        assert got == INF
    else:
        assert abs(got - n) <= 2.0 ** -24 * n + 2.0 ** -149
    out = [torch.empty_like(g) for g in grads]
    mxw.clip_grad_norm(grads, n / 3, eps=0.0, out=out)
    for g, o in zip(grads, out):
        close(o, g, 1 / 3)


def test_a_norm_past_float32():
    """The norm shows as infinity, but the factor is the finite one's."""
    g = torch.full((100,), 3e38, device=DEV)
    out = torch.empty_like(g)
    assert mxw.clip_grad_norm([g], 1.0, out=[out]).item() == INF
    close(out, g, 1 / (norm_of([g]) + 1e-6))


def test_nan_and_infinity():
    for bad in (float("nan"), INF, -INF):
        for norm_type in (2, INF):
            for at in (0, 8191, 20000):
                grads = tensors([300, 8200, 20001], 3)
                g = grads[at % 3]
                g[min(at, g.numel() - 1)] = bad
                out = [torch.zeros_like(t) for t in grads]
                norm = mxw.clip_grad_norm(grads, 1.0, norm_type, out=out).item()
                assert math.isnan(norm) if math.isnan(bad) else norm == INF
                for t, o in zip(grads, out):
                    if math.isnan(bad):
                        assert o.isnan().all()
                    else:
                        assert (o[t.isfinite()] == 0).all() and o[~t.isfinite()].isnan().all()
    assert mxw.clip_grad_norm(tensors([50], 4), INF, out=[torch.empty(50, dtype=BF16, device=DEV)]).isfinite()


def test_edges_of_max_norm():
    grads = tensors([1000, 50], 5)
    out = [torch.empty_like(g) for g in grads]
    mxw.clip_grad_norm(grads, 0.0, out=out)
    assert all((o == 0).all() for o in out)
    zero = [torch.zeros(10, device=DEV)]
    assert mxw.clip_grad_norm(zero, 1.0, eps=0.0).item() == 0 and (zero[0] == 0).all()
    mxw.clip_grad_norm(grads, INF, out=out)
    assert all(torch.equal(g, o) for g, o in zip(grads, out))


@pytest.mark.parametrize("norm_type", [2, INF])
@pytest.mark.parametrize("max_norm", [2.0 ** -126 * (1 - 2.0 ** -30), 2.0 ** -126 * (1 - 2.0 ** -20), 2.0 ** -126,
                                      2.0 ** -126 * (1 + 2.0 ** -30), 2.0 ** -127, 1.7 * 2.0 ** -133, 2.0 ** -149])
def test_factors_below_float32s_normal_range(max_norm, norm_type):
    """In place as into other tensors.  The norm is 1 exactly, so the factor is max_norm,
    and 2^-126 (1 - 2^-30) is 2^-126 and a rest that rounds to 1."""
    say("clip in place by a factor of %g, norm %s" % (max_norm, norm_type))
    first = torch.zeros(9000, device=DEV)
    first[[0, 700, 8191, 8999]] = torch.tensor([0.5, -0.5, 0.5, -0.5], device=DEV) if norm_type == 2 else \
        torch.tensor([0.5, -1.0, 0.25, 0.75], device=DEV)
    grads = [first, torch.zeros(300, dtype=BF16, device=DEV)]
    if norm_type == INF:
        grads[1][7:9] = torch.tensor([-1.0, 0.375])
    assert norm_of(grads, norm_type) == 1.0
    out = [torch.full_like(g, float("nan")) for g in grads]
    assert mxw.clip_grad_norm(grads, max_norm, norm_type, eps=0.0, out=out).item() == 1.0
    inside = [g.clone() for g in grads]
    assert mxw.clip_grad_norm(inside, max_norm, norm_type, eps=0.0).item() == 1.0
    for g, o, i in zip(grads, out, inside):
        close(o, g, max_norm)
        close(i, g, max_norm)
        assert torch.equal(i, o)


@pytest.mark.parametrize("norm_type", [2, INF])
def test_zeros_with_nothing_to_divide_by(norm_type):
    """norm, eps and max_norm all 0: zeros stay zeros, of their sign, in place and elsewhere."""
    for max_norm in (0.0, 1.0):
        grads = [torch.zeros(9000, device=DEV), -torch.zeros(11, dtype=BF16, device=DEV)]
        out = [torch.full_like(g, float("nan")) for g in grads]
        assert mxw.clip_grad_norm(grads, max_norm, norm_type, eps=0.0, out=out).item() == 0
        assert all(torch.equal(o.view(torch.uint8), g.view(torch.uint8)) for o, g in zip(out, grads))
        assert mxw.clip_grad_norm(grads, max_norm, norm_type, eps=0.0).item() == 0
        assert all(torch.equal(o.view(torch.uint8), g.view(torch.uint8)) for o, g in zip(out, grads))


def test_shapes_alignment_and_none():
    g = torch.Generator(device=DEV).manual_seed(6)
    room = torch.randn((3, 40, 50), generator=g, device=DEV)
    turned = room.to(BF16).permute(2, 0, 1)          # fills its memory in another order
    odd = torch.randn((1001,), generator=g, device=DEV).to(BF16)[1:]   # 2-byte aligned
    odd32 = torch.randn((777,), generator=g, device=DEV)[3:]
    whole = [turned, None, odd, odd32, torch.tensor(2.0, device=DEV)]
    grads = [t for t in whole if t is not None]
    n, kept = norm_of(grads), [t.clone() for t in grads]
    assert abs(mxw.clip_grad_norm(whole, 1.0).item() - n) <= 2.0 ** -24 * n
    for t, k in zip(grads, kept):
        close(t, k, 1 / (n + 1e-6))
    one = torch.randn((100,), generator=g, device=DEV)
    n = norm_of([one])
    assert abs(mxw.grad_norm(one).item() - n) <= 2.0 ** -24 * n
    kept = one.clone()
    mxw.clip_grad_norm(one, 0.5)
    close(one, kept, 0.5 / (n + 1e-6))
    with pytest.raises(ValueError):
        mxw.grad_norm([room[:, :, :49]])


def test_shared_memory_is_refused():
    room = torch.zeros(4000, device=DEV)
    a, b, c = room[:1000], room[999:2000], room[2000:3000]
    mxw.grad_norm([a, b, a])  # reading twice is fine
    for grads, out in (([a, a], None), ([a, b], None), ([a, c], [c, torch.empty_like(c)]), ([a], [room[1:1001]]),
                       ([a, c], [b[:1000], b[:1000]])):
        with pytest.raises(mxw.MxwError, match="overlaps"):
            mxw.clip_grad_norm(grads, 1.0, out=out)
    mxw.clip_grad_norm([a, c], 1.0, out=[room[1000:2000], room[3000:]])


def test_repeats_streams_and_graphs():
    grads = tensors([50000, 300, 12345] + [64] * 100, 7)
    out = [torch.empty_like(g) for g in grads]
    want = mxw.clip_grad_norm(grads, 1.0, out=out).item()
    kept = [o.clone() for o in out]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mxw.clip_grad_norm(grads, 1.0, out=out, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert got.item() == want and all(torch.equal(o, k) for o, k in zip(out, kept))
    ws = torch.full((mxw.clip_workspace_size(len(grads)),), 0xFF, dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        norm = mxw.clip_grad_norm(grads, 1.0, out=out, workspace=ws)
    eager = [torch.empty_like(g) for g in grads]
    for i in range(3):
        for g in grads:
            g.mul_(-1.25)
        graph.replay()
        torch.cuda.synchronize()
        assert mxw.clip_grad_norm(grads, 1.0, out=eager).item() == norm.item()
        assert all(torch.equal(o, e) for o, e in zip(out, eager))


@pytest.mark.parametrize("norm_type", [2, INF])
def test_more_than_the_caches_hold(norm_type):
    """Over 256 MB in all, where loads and stores go past the caches: float32 and bf16, ends
    inside 8 elements, more tensors than a launch takes, to others and in place."""
    sizes = [30000003, 70000005, 20000001, 5, 8193] + [1000 + 7 * i for i in range(100)]
    say("clip %d tensors, %d elements, norm %s" % (len(sizes), sum(sizes), norm_type))
    grads = tensors(sizes, 8)
    assert sum(g.numel() * g.element_size() for g in grads) > 1 << 28
    n = norm_of(grads, norm_type)
    assert abs(mxw.grad_norm(grads, norm_type).item() - n) <= 2.0 ** -24 * n
    for max_norm in (0.25 * n, 4 * n):
        out = [torch.full_like(g, float("nan")) for g in grads]
        got = mxw.clip_grad_norm(grads, max_norm, norm_type, out=out)
        assert abs(got.item() - n) <= 2.0 ** -24 * n
        for g, o in zip(grads, out):
            close(o, g, min(1.0, max_norm / (n + 1e-6)))
        kept = [g.clone() for g in grads]
        assert mxw.clip_grad_norm(grads, max_norm, norm_type).item() == got.item()
        assert all(torch.equal(g, o) for g, o in zip(grads, out))
        grads = kept


def test_offsets_past_32_bits():
    """A tensor of over 2^31 elements whose last ones count."""
    n = (1 << 31) + 12345
    say("clip %d elements" % n)
    g = torch.zeros(n, dtype=BF16, device=DEV)
    g[-5:] = 3.0
    g[0] = 4.0
    want = math.sqrt(5 * 9 + 16)
    assert abs(mxw.clip_grad_norm([g], 1.0).item() - want) <= 2.0 ** -24 * want
    close(g[-5:], torch.full((5,), 3.0, dtype=BF16, device=DEV), 1 / (want + 1e-6))
    close(g[:1], torch.full((1,), 4.0, dtype=BF16, device=DEV), 1 / (want + 1e-6))
