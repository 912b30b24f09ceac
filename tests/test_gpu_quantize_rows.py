"""quantize_rows against the oracle's quantiser and the formats' definitions, byte for
byte (needs an MI355X)."""
import numpy as np
import pytest
import torch

import mxfp8_ragged_grouped_amd as mxw
import oracle
from test_oracle_quant_pins import tricky_block

pytestmark = pytest.mark.gpu

DEV = "cuda"
E4M3 = [0.0] + [m * 2.0 ** -9 for m in range(1, 8)] + [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
E4M3 = np.array(E4M3[:127])  # 448 is the largest, 0x7F is NaN
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def say(msg):
    print("[gpu-case] " + msg, flush=True)


def nearest(v, table):
    """Index of the number of `table` nearest to |v|, ties to the even index, saturated."""
    a = np.minimum(np.abs(v), table[-1])
    hi = np.searchsorted(table, a)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - table[lo], table[hi] - a
    return np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def reference(x, format):
    """(codes one to a byte, scales) from the definition, in 64 bits."""
    table, b, top = (E4M3, 8, 0x80) if format == "mxfp8" else (E2M1, 2, 8)
    R, C = x.shape
    v = x.astype(np.float64).reshape(R, C // 32, 32)
    amax = np.abs(v).max(axis=2)
    fine = np.isfinite(amax)
    e = np.where(fine & (amax > 0), np.frexp(np.where(fine, amax, 1.0))[1] - 1, b)
    s = np.clip(e - b + 127, 0, 254)
    y = np.where(fine[..., None], np.nan_to_num(v), 0.0) * 2.0 ** (127.0 - s)[..., None]
    q = nearest(y, table)
    q = np.where((q > 0) & (y < 0), q + top, q)
    q = np.where(fine[..., None], q, 0x7F if format == "mxfp8" else 0)
    return q.reshape(R, C).astype(np.uint8), np.where(fine, s, 255).astype(np.uint8)


def unpack(q):
    q = q.cpu().numpy()
    return np.stack([q & 15, q >> 4], axis=-1).reshape(q.shape[:-1] + (-1,))


def check(x, format):
    C = x.shape[-1]
    q = torch.full(x.shape[:-1] + (C if format == "mxfp8" else C // 2,), 0xAA, dtype=torch.uint8, device=DEV)
    s = torch.full(x.shape[:-1] + (C // 32,), 0xAA, dtype=torch.uint8, device=DEV)
    got = mxw.quantize_rows(x, format, q=q, s=s)
    assert got[0].data_ptr() == q.data_ptr() and got[1].data_ptr() == s.data_ptr()
    rq, rs = reference(x.float().cpu().numpy().reshape(-1, C), format)
    np.testing.assert_array_equal(s.cpu().numpy().reshape(-1, C // 32), rs)
    np.testing.assert_array_equal((q.cpu().numpy() if format == "mxfp8" else unpack(q)).reshape(-1, C), rq)


def tricky(R, C, seed, dtype):
    rng = np.random.default_rng(seed)
    x = np.concatenate([tricky_block(rng, int(rng.integers(-60, 60))) for _ in range(R * C // 32)]).reshape(R, C)
    return torch.from_numpy(x).to(dtype).to(DEV)


@pytest.mark.parametrize("format", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("R,C", [(1, 32), (3, 64), (33, 96), (7, 1120), (100, 2048), (1, 65536), (513, 224)])
def test_against_the_definition(R, C, dtype, format):
    say("quantize_rows R=%d C=%d %s %s" % (R, C, dtype, format))
    check(tricky(R, C, R + C, dtype), format)
    g = torch.Generator(device=DEV).manual_seed(R)
    x = torch.randn((R, C), generator=g, device=DEV)
    check((x * torch.exp2(torch.randint(-100, 100, (R, C // 32, 1), generator=g, device=DEV).float())
           .expand(-1, -1, 32).reshape(R, C)).to(dtype), format)


@pytest.mark.parametrize("format", ["mxfp8", "mxfp4"])
def test_every_bf16_value(format):
    """Every finite bf16 number under scales from far above it to its own."""
    bits = torch.arange(1 << 16, dtype=torch.int32, device=DEV).to(torch.int16).view(torch.bfloat16)
    bits = bits[bits.isfinite()].float()
    n = (len(bits) + 30) // 31 * 31
    x = torch.zeros(n, device=DEV)
    x[:len(bits)] = bits
    x = x.view(-1, 31)
    for up in (0, 1, 3, 8, 12):
        top = x.abs().amax(1, keepdim=True) * 2.0 ** up
        top = torch.where(top.isfinite(), top, x.abs().amax(1, keepdim=True))
        check(torch.cat([x, top], 1).to(torch.bfloat16).contiguous(), format)


def test_same_bytes_as_the_token_axis_quantiser():
    g = torch.Generator(device=DEV).manual_seed(1)
    x = torch.randn((256, 320), generator=g, device=DEV).to(torch.bfloat16)
    q, s = mxw.quantize_rows(x)
    qt, st = mxw.quantize_tokens(x.t().contiguous())
    assert torch.equal(q, qt) and torch.equal(s, st)
    rq, rs = oracle.quantize_tokens(x.t().contiguous().view(torch.int16).cpu().numpy().view(np.uint16))
    np.testing.assert_array_equal(q.cpu().numpy(), rq)
    np.testing.assert_array_equal(s.cpu().numpy(), rs)


@pytest.mark.parametrize("format", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_zeros_extremes_and_broken_blocks(format, dtype):
    big = torch.finfo(dtype).max
    tiny = 2.0 ** -133 if dtype == torch.bfloat16 else 2.0 ** -149
    x = torch.zeros((12, 64), dtype=dtype, device=DEV)
    x[1, :32], x[1, 32:] = -0.0, big
    x[2, 3], x[2, 40] = -big, tiny
    x[3, 0], x[3, 33] = float("nan"), 1.0
    x[4, 31], x[4, 32] = float("inf"), -2.0
    x[5, 5], x[5, 6], x[5, 63] = float("-inf"), float("nan"), -float("nan")
    x[6] = 2.0 ** -126
    x[7, ::2] = 2.0 ** -127
    x[8, 1::2] = -2.0 ** -130
    x[9, 0], x[9, 1] = 1.0, 2.0 ** -133
    x[10, 0], x[10, 1], x[10, 32:] = big, 1.0, torch.tensor(-1.0)
    check(x, format)
    q, s = mxw.quantize_rows(x, format)
    assert s[3, 0] == 255 and s[3, 1] != 255 and s[4, 0] == 255 and (s[5] == 255).all()


def test_shapes_and_strides():
    g = torch.Generator(device=DEV).manual_seed(2)
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.randn((3, 5, 7, 96), generator=g, device=DEV).to(dtype)
        for format in ("mxfp8", "mxfp4"):
            q, s = mxw.quantize_rows(x, format)
            flat = mxw.quantize_rows(x.view(-1, 96), format)
            assert q.shape[:3] == s.shape[:3] == (3, 5, 7) and torch.equal(q.view(105, -1), flat[0])
            # rows apart, starting on any element
            wide = torch.randn((105 * 131 + 5,), generator=g, device=DEV).to(dtype)
            for start, ld in ((0, 96), (1, 97), (3, 131), (2, 128)):
                v = torch.as_strided(wide, (105, 96), (ld, 1), start)
                got, want = mxw.quantize_rows(v, format), mxw.quantize_rows(v.contiguous(), format)
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (start, ld)
        one = mxw.quantize_rows(x[0, 0, 0])
        assert one[0].shape == (96,) and one[1].shape == (3,)
    empty = mxw.quantize_rows(x[:0])
    assert empty[0].shape == (0, 5, 7, 96) and empty[1].shape == (0, 5, 7, 3)
    with pytest.raises(ValueError):
        mxw.quantize_rows(x.transpose(0, 1))
    with pytest.raises(ValueError):
        mxw.quantize_rows(x[..., :33])


def test_offsets_past_32_bits():
    R, C = 70000, 32768
    say("quantize_rows R=%d C=%d" % (R, C))
    x = torch.zeros((R, C), dtype=torch.bfloat16, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(3)
    x[-3:] = torch.randn((3, C), generator=g, device=DEV).to(torch.bfloat16)
    for format in ("mxfp8", "mxfp4"):
        q, s = mxw.quantize_rows(x, format)
        want = mxw.quantize_rows(x[-3:].clone(), format)
        assert torch.equal(q[-3:], want[0]) and torch.equal(s[-3:], want[1])
        assert (q[:-3] == 0).all() and (s[:-3] == 127).all()


@pytest.mark.parametrize("format", ["mxfp8", "mxfp4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_more_than_the_caches_hold(dtype, format):
    """Over 256 MB in all, where loads and stores go past the caches: the bytes of the same
    rows a part at a time, from rows together and from rows that start on any element."""
    C, ld = 2080, 2083
    R = (1 << 28) // (C * (5 if dtype == torch.float32 else 3)) + 777
    say("quantize_rows R=%d C=%d %s %s" % (R, C, dtype, format))
    g = torch.Generator(device=DEV).manual_seed(6)
    wide = (torch.randn((R * ld + 1,), generator=g, device=DEV) * 3.0).to(dtype)
    apart = torch.as_strided(wide, (R, C), (ld, 1), 1)
    together = apart.contiguous()
    parts = [mxw.quantize_rows(t, format) for t in together.split(R // 4 + 1)]
    want = [torch.cat([p[i] for p in parts]) for i in range(2)]
    for x in (together, apart):
        q, s = mxw.quantize_rows(x, format, q=torch.full_like(want[0], 0xAA), s=torch.full_like(want[1], 0xAA))
        assert torch.equal(q, want[0]) and torch.equal(s, want[1])


def test_streams_and_graphs():
    g = torch.Generator(device=DEV).manual_seed(4)
    x = torch.randn((300, 160), generator=g, device=DEV)
    want = mxw.quantize_rows(x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = mxw.quantize_rows(x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        q, s = mxw.quantize_rows(x)
    for _ in range(3):
        x.copy_(x.roll(1, 0) * 1.3)
        graph.replay()
        torch.cuda.synchronize()
        want = mxw.quantize_rows(x)
        assert torch.equal(q, want[0]) and torch.equal(s, want[1])
