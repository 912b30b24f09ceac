"""linear_4bit against the formats' definitions in 64 bits (needs an MI355X).

Tolerance.  MXFP4: the weights enter exactly, each product of two bf16 numbers is exact in
float32, and a sum of K terms rounds at most K times by half a step of 2^-24 (a whole one,
2^-23, if the matrix unit cuts instead) of a partial sum that the sum of magnitudes S
bounds: K 2^-23 S.  Integers: code and zero enter apart, so S is that of x code s and of x zero s,
and there are four more roundings for each group.  The result's rounding to bf16 adds 2^-8 of it.
"""
import pytest
import torch

import mxfp8_ragged_grouped_amd as mxw

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0] + [-0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                    dtype=torch.float64, device=DEV if torch.cuda.is_available() else "cpu")


def say(msg):
    print("[gpu-case] " + msg, flush=True)


def make(T, K, N, group, seed, zeros=False):
    """x, codes, scales, zeros; group None: MXFP4."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((T, K), generator=g, device=DEV).to(BF16)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8)
    if group is None:
        return x, codes, torch.randint(118, 130, (N, K // 32), generator=g, device=DEV, dtype=torch.uint8), None
    scales = (torch.randn((N, K // group), generator=g, device=DEV) * 0.1).to(BF16)
    return x, codes, scales, torch.randint(0, 16, scales.shape, generator=g, device=DEV, dtype=torch.uint8) if zeros else None


def reference(x, codes, scales, zeros):
    """(result, sum of magnitudes) in 64 bits."""
    N, K = codes.shape[0], 2 * codes.shape[1]
    n = torch.empty((N, K), dtype=torch.int64, device=DEV)
    n[:, 0::2], n[:, 1::2] = codes.long() % 16, codes.long() // 16
    group = K // scales.shape[1]
    if scales.dtype == torch.uint8:
        v = E2M1[n] * torch.exp2(scales.double() - 127).repeat_interleave(32, 1)
        size = v.abs()
    else:
        s = scales.double().repeat_interleave(group, 1)
        z = 8 if zeros is None else zeros.long().repeat_interleave(group, 1)
        v, size = (n - z) * s, (n + z) * s.abs()
    return x.double() @ v.mT, x.double().abs() @ size.mT


def check(got, x, codes, scales, zeros, what):
    ref, size = reference(x, codes, scales, zeros)
    K = x.shape[1]
    terms = K + (0 if scales.dtype == torch.uint8 else 4 * scales.shape[1])
    eps = 2.0 ** -8 if got.dtype == BF16 else 0.0
    bad = ~((got.double() - ref).abs() <= eps * (1 + 2.0 ** -10) * ref.abs() + 2 * terms * 2.0 ** -24 * size + 2.0 ** -133)
    assert not bad.any(), "%s: %d of %d outside, first %s" % (what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist())
    # the bound above is the worst case; the errors are like random ones, and of their 2-norm a
    # sixteenth of it is never passed by a right kernel with sums of a hundred terms and more
    off = (got.double() - ref).norm()
    assert off <= (eps + 2.0 ** -20) * ref.norm() + 2.0 ** -24 * size.norm() * terms ** 0.5


def poisoned(T, N, dtype):
    return torch.full((T, N), float("nan"), dtype=dtype, device=DEV)


FORMS = [(None, False), (32, False), (32, True), (64, True), (128, False), (128, True)]


@pytest.mark.parametrize("group,zeros", FORMS)
@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 31, 33, 48, 49, 64])
def test_tokens(T, group, zeros):
    for K, N in ((128, 16), (640, 100), (1152, 1025)):
        say("linear_4bit T=%d K=%d N=%d group=%s zeros=%s" % (T, K, N, group, zeros))
        args = make(T, K, N, group, T + K, zeros)
        for dtype in (BF16, F32):
            got = mxw.linear_4bit(*args, dtype=dtype, out=poisoned(T, N, dtype))
            check(got, *args, "T=%d K=%d N=%d" % (T, K, N))


@pytest.mark.parametrize("group,zeros", FORMS)
@pytest.mark.parametrize("N", [1, 2, 15, 17, 63, 64, 65, 4999])
def test_rows_of_weights(N, group, zeros):
    for T, K in ((1, 256), (5, 2048), (40, 384)):
        say("linear_4bit T=%d K=%d N=%d group=%s" % (T, K, N, group))
        args = make(T, K, N, group, N, zeros)
        check(mxw.linear_4bit(*args, dtype=F32, out=poisoned(T, N, F32)), *args, "N=%d" % N)


@pytest.mark.parametrize("K", [32, 64, 96, 160, 192, 224, 480, 544, 1120, 4128, 7168, 65536])
def test_lengths(K):
    for group, zeros in FORMS:
        if group and K % group:
            continue
        for T, N in ((1, 40), (20, 33)):
            say("linear_4bit T=%d K=%d N=%d group=%s" % (T, K, N, group))
            args = make(T, K, N, group, K, zeros)
            check(mxw.linear_4bit(*args, dtype=F32), *args, "K=%d" % K)


@pytest.mark.parametrize("group", [None, 32, 128])
def test_many_rows(group):
    """Enough rows that waves take whole rows, up to a vocabulary's."""
    for T, K, N in ((1, 2048, 32003), (64, 512, 70001), (17, 256, 128000)):
        say("linear_4bit T=%d K=%d N=%d group=%s" % (T, K, N, group))
        args = make(T, K, N, group, N, group is not None)
        check(mxw.linear_4bit(*args), *args, "N=%d" % N)


@pytest.mark.parametrize("group,zeros", FORMS)
@pytest.mark.parametrize("T,K,N", [(1, 7200, 34001), (9, 7200, 36017), (16, 4192, 33000), (23, 4192, 40001), (32, 2144, 66000),
                                   (37, 1120, 40001), (64, 2080, 33041),      # two tiles of rows a wave
                                   (16, 7200, 20001), (20, 7200, 20001), (48, 2080, 20001), (64, 3104, 17000),
                                   (12, 12320, 700), (20, 7200, 3001), (32, 4192, 16384), (33, 2080, 3001),
                                   (64, 7200, 100), (64, 65536, 40)])
def test_every_form(T, K, N, group, zeros):
    """Tokens that fit in LDS and that come in pieces, one and two row tiles a wave, parts of K,
    several rounds of workgroups, and ends inside a step, with rows and tokens to spare."""
    K = K // (group or 32) * (group or 32)
    say("linear_4bit T=%d K=%d N=%d group=%s zeros=%s" % (T, K, N, group, zeros))
    args = make(T, K, N, group, T + N, zeros)
    check(mxw.linear_4bit(*args, dtype=F32, out=poisoned(T, N, F32)), *args, "T=%d K=%d N=%d" % (T, K, N))


def test_each_code_and_place():
    """One token with a single 1: every code of every place comes out as its value."""
    K = 288
    codes = torch.arange(16, dtype=torch.uint8, device=DEV)
    both = (codes[:, None] | (codes.flip(0)[:, None] << 4)).expand(16, K // 2).contiguous()
    x = torch.eye(64, K, dtype=BF16, device=DEV)
    for first in (0, 64, 224):
        xt = torch.roll(x, first, 1)
        v = torch.where(torch.arange(64, device=DEV)[:, None] % 2 == 0, E2M1[codes.long()], E2M1[codes.flip(0).long()])
        got = mxw.linear_4bit(xt, both, torch.full((16, K // 32), 128, dtype=torch.uint8, device=DEV), dtype=F32)
        assert torch.equal(got.double(), 2 * v)
        s = torch.full((16, K // 32), 0.25, dtype=BF16, device=DEV)
        z = torch.arange(16, dtype=torch.uint8, device=DEV)[:, None].expand(16, K // 32).contiguous()
        n = torch.where(torch.arange(64, device=DEV)[:, None] % 2 == 0, codes, codes.flip(0)).double()
        assert torch.equal(mxw.linear_4bit(xt, both, s, dtype=F32).double(), (n - 8) / 4)
        assert torch.equal(mxw.linear_4bit(xt, both, s, zeros=z, dtype=F32).double(), (n - codes.double()) / 4)


def test_scales_at_the_ends():
    """MXFP4 scales 0 and 254 (numbers below bf16's normal range may be 0, beyond it
    infinity), and the NaN scale, which stays in its row."""
    x, codes, scales, _ = make(3, 256, 48, None, 1)
    scales[5, 2] = 255
    scales[7] = 254
    scales[9] = 0
    got = mxw.linear_4bit(x, codes, scales, dtype=F32)
    keep = torch.ones(48, dtype=torch.bool, device=DEV)
    keep[[5, 7, 9]] = False
    assert got[:, 5].isnan().all() and (got[:, 9].abs() <= 2.0 ** -110).all()
    check(got[:, keep], x, codes[keep], scales[keep], None, "other rows")
    x, codes, scales, _ = make(3, 256, 48, 64, 2)
    scales[5, 2], scales[7, 0] = float("nan"), float("inf")
    got = mxw.linear_4bit(x, codes, scales, dtype=F32)
    keep[9] = True
    assert got[:, 5].isnan().all() and not got[:, 7].isfinite().any()
    check(got[:, keep], x, codes[keep], scales[keep], None, "other rows")


@pytest.mark.parametrize("scale", [255, 254, 253, 251, 2, 1, 0])
def test_a_single_weight_under_scales_at_the_ends(scale):
    """MXFP4: one code a row and one 1 a token (2^60 under the lowest scales, so that the
    result is far from float32's ends), the rest zeros, so that an output is a single
    weight: exact in bf16's range and below its normal numbers (2^-128 is among its
    subnormals), past the range infinity (0 stays 0), and under the NaN scale NaN."""
    x0 = 1.0 if scale > 127 else 2.0 ** 60
    for K, T, N in ((32, 1, 16), (288, 3, 16), (288, 20, 16 * 2100)):   # the last: two row tiles a wave
        for place in (0, 13, K - 1):
            codes = torch.zeros((N, K // 2), dtype=torch.uint8, device=DEV)
            code = torch.arange(N, dtype=torch.uint8, device=DEV) % 16
            codes[:, place // 2] = code << 4 * (place % 2)
            scales = torch.full((N, K // 32), 127, dtype=torch.uint8, device=DEV)
            scales[:, place // 32] = scale
            x = torch.zeros((T, K), dtype=BF16, device=DEV)
            x[T - 1, place] = x0
            got = mxw.linear_4bit(x, codes, scales, dtype=F32, out=poisoned(T, N, F32))[T - 1].double()
            if scale == 255:
                assert got.isnan().all()
                continue
            v = E2M1[code.long()] * 2.0 ** (scale - 127)
            say("scale %d K=%d place %d" % (scale, K, place))
            assert torch.equal(got, torch.where(v.abs() < 2.0 ** 128, v * x0, torch.sign(v) * float("inf")))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("scale,tokens", [(126, -100), (124, -60), (-126, 100), (-133, 60)])
def test_integers_under_scales_at_the_ends(scale, tokens, group):
    """Scales that times a zero leave float32's range, or that are bf16's smallest, with
    tokens that bring the result back: the definition's value."""
    for T, K, N, zeros in ((1, 256, 40, True), (5, 640, 100, False), (40, 1152, 33, True), (20, 256, 34000, True)):
        say("linear_4bit scale 2^%d T=%d K=%d N=%d group=%d" % (scale, T, K, N, group))
        x, codes, scales, z = make(T, K, N, group, K + group, zeros)
        size = torch.rand(scales.shape, generator=torch.Generator(device=DEV).manual_seed(3), device=DEV) + 1.0
        scales = (torch.copysign(size, scales.float()) * 2.0 ** scale).to(BF16)
        x = (x.float() * 2.0 ** tokens).to(BF16)
        check(mxw.linear_4bit(x, codes, scales, zeros=z, dtype=F32), x, codes, scales, z, "scale 2^%d" % scale)


@pytest.mark.parametrize("group", [None, 32, 128])
def test_tokens_stay_apart(group):
    """No token's bits depend on the others' values, NaN and infinity among them."""
    for T in (2, 16, 37, 64):
        args = make(T, 512, 200, group, T)
        want = mxw.linear_4bit(*args, dtype=F32)
        x = args[0].clone()
        x[T // 2, 100], x[T // 2 + 1 if T > 2 else T // 2, 3] = float("nan"), float("inf")
        got = mxw.linear_4bit(x, *args[1:], dtype=F32)
        assert got[T // 2].isnan().all()
        others = torch.ones(T, dtype=torch.bool)
        others[T // 2], others[min(T // 2 + 1, T - 1) if T > 2 else T // 2] = False, False
        assert torch.equal(got[others], want[others])


def test_strides_streams_and_graphs():
    x, codes, scales, zeros = make(9, 1152, 333, 64, 3, True)
    want = mxw.linear_4bit(x, codes, scales, zeros)
    wide = torch.full((9, 1200), float("nan"), dtype=BF16, device=DEV)
    wide[:, 16:16 + 1152] = x
    assert torch.equal(mxw.linear_4bit(wide[:, 16:16 + 1152], codes, scales, zeros), want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mxw.linear_4bit(x, codes, scales, zeros, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    assert mxw.linear_4bit(x[:0], codes, scales, zeros).shape == (0, 333)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = mxw.linear_4bit(x, codes, scales, zeros)
    for _ in range(3):
        x.copy_(x.roll(1, 0) * 1.5)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mxw.linear_4bit(x, codes, scales, zeros))


def test_weights_that_quantize_rows_made():
    g = torch.Generator(device=DEV).manual_seed(5)
    w, x = torch.randn((300, 640), generator=g, device=DEV), torch.randn((4, 640), generator=g, device=DEV).to(BF16)
    q, s = mxw.quantize_rows(w, "mxfp4")
    got = mxw.linear_4bit(x, q, s, dtype=F32)
    check(got, x, q, s, None, "quantised")
    want = x.double() @ w.double().mT
    assert (got.double() - want).norm() < 0.2 * want.norm()


def test_scales_past_32_bits():
    """A scale plane of over 1.6 GB, K ending inside a step: nothing past K comes in."""
    K, N = 65312, 820000
    say("linear_4bit K=%d N=%d" % (K, N))
    codes = torch.zeros((N, K // 2), dtype=torch.uint8, device=DEV)
    scales = torch.full((N, K // 32), 255, dtype=torch.uint8, device=DEV)  # NaN, where nothing is looked at
    rows = [0, 1, 15, 16, 300000, N - 17, N - 1]
    x, some, ss, _ = make(1, K, len(rows), None, 7)
    codes[rows], scales[rows] = some, ss
    got = mxw.linear_4bit(x, codes, scales, dtype=F32)
    check(got[:, rows].contiguous(), x, some, ss, None, "rows")
    del codes, scales
    torch.cuda.empty_cache()


def test_weights_past_32_bits():
    """Codes of over 2^31 bytes."""
    K, N = 65536, 70000
    say("linear_4bit K=%d N=%d" % (K, N))
    codes = torch.zeros((N, K // 2), dtype=torch.uint8, device=DEV)
    scales = torch.full((N, K // 32), 127, dtype=torch.uint8, device=DEV)
    x, last, ls, _ = make(2, K, 40, None, 6)
    codes[-40:], scales[-40:] = last, ls
    got = mxw.linear_4bit(x, codes, scales, dtype=F32)
    assert (got[:, :-40] == 0).all()
    check(got[:, -40:].contiguous(), x, last, ls, None, "last rows")
