"""mxw.orthogonalize against the same products in 64 bits (needs an MI355X).

Tolerance, by the 2-norm of a whole matrix.  Every step rounds X, S and P to f16
(relative 2^-12 at most, independent and zero-mean over the entries), and an
error already in X is multiplied by at most |s f'(s) / f(s)| <= 1.64 per step
for the singular values the inputs here keep (f = 3.4445 s - 4.775 s^3 +
2.0315 s^5, s from 0.5 up) and by at most 3.45 / 3.4445 ~ 1 below, where f is
linear.  Added in squares over five steps: sqrt(1 + 1.64^2 + ... + 1.64^8) = 9.1
times sqrt(3) 2^-12 / sqrt(3); three times that, plus the result's own rounding
to bf16 (2^-8 at most, less than 2^-9 in the 2-norm): 2^-9 + 3 * 9.1 * 2^-12 = 0.0086.
"""
import pytest
import torch

import mxfp8_ragged_grouped_amd as mxw

pytestmark = pytest.mark.gpu

DEV = "cuda"
TOL = 2.0 ** -9 + 3 * 9.1 * 2.0 ** -12
COEFFS = (3.4445, -4.7750, 2.0315)


def say(msg):
    print("[gpu-case] " + msg, flush=True)


def reference(G, coeffs, eps=1e-7):
    X = G.double()
    X = X / (X.square().sum(dim=(-2, -1), keepdim=True).sqrt() + eps)
    for a, b, c in coeffs:
        S = X @ X.mT
        X = a * X + (b * S + c * S @ S) @ X
    return X


def spread(E, N, K, seed, low=0.2):
    """Matrices whose singular values lie in [low, 1], with random vectors."""
    g = torch.Generator().manual_seed(seed)
    n = min(N, K)
    out = []
    for _ in range(E):
        u = torch.linalg.qr(torch.randn(N, n, generator=g, dtype=torch.float64)).Q
        v = torch.linalg.qr(torch.randn(K, n, generator=g, dtype=torch.float64)).Q
        s = low + (1 - low) * torch.rand(n, generator=g, dtype=torch.float64)
        out.append((u * s) @ v.T)
    return torch.stack(out).to(DEV)


def poisoned(shape):
    t = torch.empty(shape, dtype=torch.bfloat16, device=DEV)
    t.view(torch.int16).fill_(0x7FC0)
    return t


def close(got, ref, what):
    for e in range(ref.shape[0]):
        err = (got[e].double() - ref[e]).norm() / ref[e].norm()
        assert err <= TOL, "%s, matrix %d: off by %.2e of its norm" % (what, e, float(err))


SIZES = [(1, 1, 1), (2, 1, 65), (2, 65, 1), (1, 70, 3), (3, 3, 70), (2, 63, 64), (2, 64, 63), (4, 128, 256),
         (2, 129, 257), (2, 257, 129), (1, 256, 256), (3, 300, 520), (1, 777, 515), (9, 100, 100), (1, 1000, 2050),
         (1, 2050, 1000)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("E,N,K", SIZES)
def test_against_64_bits(E, N, K, dtype):
    say("orthogonalize E=%d N=%d K=%d %s" % (E, N, K, dtype))
    G = (3e-4 * spread(E, N, K, 1000 + N + K)).to(dtype)
    out = poisoned(G.shape)
    got = mxw.orthogonalize(G, out=out)
    assert got is out
    close(got, reference(G, [COEFFS] * 5), "N=%d K=%d" % (N, K))


def test_large_tiles():
    """Sizes that run the 256 x 256 tiles, wide and tall, edges included."""
    for E, N, K in ((8, 1400, 2000), (8, 2000, 1400)):
        say("orthogonalize E=%d N=%d K=%d" % (E, N, K))
        g = torch.Generator(device=DEV).manual_seed(N)
        G = torch.randn((E, N, K), generator=g, device=DEV).to(torch.bfloat16)
        close(mxw.orthogonalize(G), reference(G, [COEFFS] * 5), "N=%d K=%d" % (N, K))


@pytest.mark.parametrize("E,N,K", [(2, 150, 3000), (1, 3000, 150), (1, 64, 8200), (3, 33, 2300), (4, 2100, 130)])
def test_long_and_narrow(E, N, K):
    """A short side over a long one: the long sum is split over workgroups."""
    say("orthogonalize E=%d N=%d K=%d" % (E, N, K))
    G = (2e-2 * spread(E, N, K, 2000 + N + K)).to(torch.bfloat16)
    close(mxw.orthogonalize(G, out=poisoned(G.shape)), reference(G, [COEFFS] * 5), "N=%d K=%d" % (N, K))


@pytest.mark.parametrize("E,N,K", [(5, 1500, 1100), (4, 1100, 4100), (9, 900, 600), (8, 2300, 2400)])
def test_whole_rounds_and_quarters(E, N, K):
    """Sizes that take other tile edges, and 256-tiles with the rest in quarters:
    the same bits as each matrix alone."""
    say("orthogonalize E=%d N=%d K=%d" % (E, N, K))
    g = torch.Generator(device=DEV).manual_seed(N + K)
    G = torch.randn((E, N, K), generator=g, device=DEV).to(torch.bfloat16)
    out = mxw.orthogonalize(G, out=poisoned(G.shape))
    close(out, reference(G, [COEFFS] * 5), "N=%d K=%d" % (N, K))
    assert torch.equal(out[E // 2], mxw.orthogonalize(G[E // 2]))


@pytest.mark.parametrize("E,N,K,split", [(6, 2300, 2400, False), (6, 2400, 2300, False), (17, 900, 3900, True),
                                         (12, 1000, 1300, False)])
def test_whole_rounds_and_smaller_tiles(E, N, K, split):
    """256-tiles with the rest cut into 64- or 128-tiles, in either form of the
    products: the same bits as each matrix alone (split: one alone has few tiles
    of S, and its sums over the long axis are joined from two parts)."""
    say("orthogonalize cut tiles E=%d N=%d K=%d" % (E, N, K))
    g = torch.Generator(device=DEV).manual_seed(N + K)
    G = torch.randn((E, N, K), generator=g, device=DEV).to(torch.bfloat16)
    out = mxw.orthogonalize(G, out=poisoned(G.shape))
    close(out, reference(G, [COEFFS] * 5), "N=%d K=%d" % (N, K))
    for e in (0, E - 1):
        assert split or torch.equal(out[e], mxw.orthogonalize(G[e]))


def test_singular_values_come_near_one():
    G = spread(2, 200, 333, 5).to(torch.bfloat16)
    s = torch.linalg.svdvals(mxw.orthogonalize(G).double())
    assert float(s.min()) > 0.6 and float(s.max()) < 1.3


@pytest.mark.parametrize("coeffs,steps", [((2.0, -1.5, 0.5), 8), ([(3.4445, -4.775, 2.0315)] * 2 + [(2.0, -1.5, 0.5)], 3),
                                          ((1.5, -0.5, 0.0), 1)])
def test_other_coefficients(coeffs, steps):
    G = spread(2, 96, 160, 6).float()
    each = list(coeffs) if hasattr(coeffs[0], "__len__") else [coeffs] * steps
    close(mxw.orthogonalize(G, steps=steps, coeffs=coeffs), reference(G, each), "coeffs %s" % (coeffs,))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_strides_and_alignment(dtype):
    """Padded rows, gaps between experts, an odd first element, 2-D inputs and
    one matrix repeated: the same bits as contiguous inputs."""
    G = spread(3, 90, 136, 7).to(dtype)
    want = mxw.orthogonalize(G)
    flat = torch.full((4 * 100 * 200 + 64,), float("nan"), dtype=dtype, device=DEV)
    for first in (0, 1, 3, 8):
        for rows, experts in ((144, 14400), (137, 12463), (200, 20000)):
            view = flat.as_strided((3, 90, 136), (experts, rows, 1), first)
            view.copy_(G)
            assert torch.equal(mxw.orthogonalize(view), want), (first, rows, experts)
            view.fill_(float("nan"))
    assert torch.equal(mxw.orthogonalize(G[1]), want[1])
    again = mxw.orthogonalize(G[1:2].expand(4, -1, -1))
    assert all(torch.equal(again[i], want[1]) for i in range(4))
    odd = torch.empty(3 * 90 * 136 + 1, dtype=torch.bfloat16, device=DEV)
    out = odd[1:].view(3, 90, 136)  # 2-byte aligned
    assert torch.equal(mxw.orthogonalize(G, out=out), want)


def test_rows_past_32_bit_offsets():
    G = spread(1, 2200, 64, 12).to(torch.bfloat16)[0]
    far = torch.empty(2200 << 20, dtype=torch.bfloat16, device=DEV).view(2200, 1 << 20)[:, 5:69]
    far.copy_(G)
    assert torch.equal(mxw.orthogonalize(far), mxw.orthogonalize(G))


def test_empty_and_broken_experts_stay_alone():
    """A zero gradient gives zeros; NaN and infinity stay in their expert."""
    G = spread(5, 130, 200, 8).to(torch.bfloat16)
    want = mxw.orthogonalize(G)
    bad = G.clone()
    bad[1] = 0
    bad[2, 5, 7] = float("nan")
    bad[3, 129, 199] = float("inf")
    out = poisoned(G.shape)
    mxw.orthogonalize(bad, out=out)
    assert torch.equal(out[0], want[0]) and torch.equal(out[4], want[4])
    assert (out[1] == 0).all()
    assert out[2].isnan().any() and out[3].isnan().any()


def test_scale_does_not_matter():
    """Powers of two on G change no bit (eps = 0): squares of large and small
    gradients stay in range."""
    G = spread(2, 64, 80, 9).float()
    want = mxw.orthogonalize(G, eps=0.0)
    for p in (-90, -30, 30, 100):
        assert torch.equal(mxw.orthogonalize(G * 2.0 ** p, eps=0.0), want), p


def test_repeats_streams_and_graphs():
    G = spread(3, 200, 260, 10).to(torch.bfloat16)
    want = mxw.orthogonalize(G)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = mxw.orthogonalize(G, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(other, want)
    ws = torch.empty(mxw.orthogonalize_workspace_size(3, 200, 260), dtype=torch.uint8, device=DEV)
    ws.fill_(0xFF)
    out = poisoned(G.shape)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        mxw.orthogonalize(G, out=out, workspace=ws)
    for i in range(3):
        G.copy_(G.roll(1, 0))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, mxw.orthogonalize(G)), "replay %d" % i


def test_workspace_is_checked():
    G = spread(1, 64, 64, 11).to(torch.bfloat16)
    need = mxw.orthogonalize_workspace_size(1, 64, 64)
    with pytest.raises(ValueError):
        mxw.orthogonalize(G, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
    big = torch.empty(need + 256, dtype=torch.uint8, device=DEV)
    with pytest.raises(mxw.MxwError):
        mxw.orthogonalize(G, workspace=big[1:])


@pytest.mark.parametrize("eps", [0.0, 1e-45, 1e-38])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,K", [(40, 70), (70, 40), (130, 200), (200, 130)])
def test_zero_tiny_and_huge_experts_with_a_small_eps(N, K, dtype, eps):
    """An expert without a gradient gives zeros for every eps; norms from below
    2^-118, where their reciprocal leaves float32's range, up to above 2^127."""
    say("orthogonalize small eps N=%d K=%d %s eps=%g" % (N, K, dtype, eps))
    G = spread(5, N, K, 40 + N).float()
    G[1] = 0
    G[2] *= 2.0 ** -122
    G[3] *= 2.0 ** -124
    G[4] /= G[4].abs().max()
    G[4] *= 2.0 ** 127
    G = G.to(dtype)
    assert torch.isfinite(G).all()
    out = mxw.orthogonalize(G, eps=eps, out=poisoned(G.shape))
    assert (out[1] == 0).all()
    live = [0, 2, 3, 4]
    close(out[live], reference(G[live], [COEFFS] * 5, eps), "eps=%g" % eps)


@pytest.mark.parametrize("E,N,K", [(4, 128, 256), (3, 100, 400), (2, 257, 129), (3, 300, 520), (1, 777, 515), (2, 150, 3000),
                                   (4, 2100, 130), (8, 1400, 2000), (8, 2000, 1400), (5, 1500, 1100), (12, 1000, 1300),
                                   (6, 2300, 2400), (6, 2400, 2300)])
def test_every_element(E, N, K):
    """Every entry, so that one wrong chunk of a tile shows.  Of the tolerance at
    the top the f16 part, 3 * 9.1 * 2^-12 of the 2-norm, is a rounding noise that
    the random directions of these inputs spread evenly: that times the matrix's
    rms is an entry's standard deviation at most, and six of them are passed by
    none of 10^8 entries; the result's rounding to bf16 adds 2^-8 of the entry.
    An entry from a wrong place is off by about 1.4 rms, 35 times the noise's share."""
    say("orthogonalize every element E=%d N=%d K=%d" % (E, N, K))
    g = torch.Generator(device=DEV).manual_seed(5 * N + K)
    G = torch.randn((E, N, K), generator=g, device=DEV).to(torch.bfloat16)
    out = mxw.orthogonalize(G, out=poisoned(G.shape))
    ref = reference(G, [COEFFS] * 5)
    for e in range(E):
        rms = ref[e].square().mean().sqrt()
        bad = ~((out[e].double() - ref[e]).abs() <= 2.0 ** -8 * ref[e].abs() + 6 * 3 * 9.1 * 2.0 ** -12 * rms)
        assert not bad.any(), "matrix %d: %d of %d outside, first %s" % (e, int(bad.sum()), bad.numel(),
                                                                         bad.nonzero()[0].tolist())
