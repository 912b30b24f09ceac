"""sort_tokens, dispatch_tokens, combine_tokens and combine_tokens_grad against plain
forms in whole numbers and 64 bits (needs an MI355X).

Sorting and copying are compared bit for bit.  Tolerances of sums, from the formulas'
roundings (half a step each): out of combine_tokens takes k products joined by fused
multiply-adds and one addition in FP32, each off by at most 2^-24 of a partial sum that
the sum of all magnitudes S bounds, so (k + 1) 2^-24 S, and one rounding to the output's
type, half of whose step is eps / 2 of the value; dy takes one product, 2^-24, and the
type's rounding; a dot product of H terms (H + 12) 2^-24 S.  Subnormal results do not
occur in the inputs here.
"""
import pytest
import torch

import mxfp8_ragged_grouped_amd as mxw

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def say(msg):
    print("[gpu-case] " + msg, flush=True)


def plain_sort(ids, E, align):
    """The definition, one choice after the other."""
    flat = ids.cpu().reshape(-1).tolist()
    counts = [0] * E
    for e in flat:
        if 0 <= e < E:
            counts[e] += 1
    offs, end = [], 0
    for c in counts:
        end += -(-c // align) * align
        offs.append(end)
    place = [0] + offs[:-1]
    rows = []
    for e in flat:
        if 0 <= e < E:
            rows.append(place[e])
            place[e] += 1
        else:
            rows.append(-1)
    return offs, counts, rows


def make_ids(T, k, E, seed, empty=0.0, dtype=torch.int64, skew=True):
    g = torch.Generator().manual_seed(seed)
    u = torch.rand((T, k), generator=g)
    ids = ((u ** 2 if skew else u) * E).long().clamp_(max=E - 1)  # an expert may come twice
    off = torch.rand((T, k), generator=g) < empty
    ids[off] = torch.where(torch.rand((T, k), generator=g)[off] < 0.5, -1, E + 3)
    return ids.to(dtype).to(DEV)


def values(shape, seed, dtype=BF16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV).to(dtype)


def poison(shape, dtype):
    t = torch.empty(shape, dtype=dtype, device=DEV)
    return t.fill_(0xA5 if dtype == torch.uint8 else float("nan"))


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ---- sort ---------------------------------------------------------------------

@pytest.mark.parametrize("T,k,E,align,empty", [
    (0, 2, 8, 32, 0), (1, 1, 1, 32, 0), (1, 2, 8, 32, 0), (1, 64, 256, 1, 0), (5, 3, 10, 7, 0.3), (64, 8, 256, 32, 0),
    (301, 3, 10, 32, 0.25), (300, 4, 3, 1024, 0.1), (1000, 1, 255, 16, 0), (4095, 4, 129, 32, 0), (4096, 4, 129, 32, 0),
    (1024, 1, 8, 32, 0), (1025, 1, 8, 32, 0.1), (2049, 1, 256, 32, 0), (4097, 1, 2, 32, 0.5), (16385, 1, 2, 32, 0.5),
    (5000, 9, 256, 32, 0.05), (40, 2, 8, 32, 1.0), (70000, 2, 37, 32, 0)])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(T, k, E, align, empty, dtype):
    say("sort T=%d k=%d E=%d align=%d empty=%g %s" % (T, k, E, align, empty, dtype))
    ids = make_ids(T, k, E, T + k, empty, dtype)
    plan = mxw.sort_tokens(ids, E, align=align)
    offs, counts, rows = plain_sort(ids, E, align)
    assert plan.offs.tolist() == offs and plan.counts.tolist() == counts
    assert plan.rows.reshape(-1).tolist() == rows
    assert plan.size == mxw.token_rows(T, k, E, align) >= (offs[-1] if offs else 0) and plan.size % align == 0


def test_sort_one_expert_takes_all():
    for E, e in ((1, 0), (256, 255), (256, 0), (64, 63)):
        ids = torch.full((9000, 2), e, dtype=torch.int32, device=DEV)
        plan = mxw.sort_tokens(ids, E)
        assert torch.equal(plan.rows.view(-1), torch.arange(18000, dtype=torch.int32, device=DEV))
        assert plan.offs[e].item() == 18016 and plan.offs[-1].item() == 18016


def test_sort_ids_beyond_32_bits_and_strided():
    ids = make_ids(200, 4, 16, 5)
    ids[3, 1] = (1 << 32) + 2      # 2 in its low half
    ids[7, 0] = -(1 << 40)
    wide = torch.full((200, 9), 77, dtype=torch.int64, device=DEV)
    wide[:, 2:6] = ids
    for t in (ids, wide[:, 2:6]):
        plan = mxw.sort_tokens(t, 16)
        offs, counts, rows = plain_sort(ids, 16, 32)
        assert plan.rows.reshape(-1).tolist() == rows and plan.offs.tolist() == offs and plan.counts.tolist() == counts
        assert plan.rows[3, 1].item() == -1


@pytest.mark.parametrize("T", [75000, 100000, 1 << 20])
def test_sort_many(T):
    """525,000, 700,000 and 7,340,032 choices against a stable sort."""
    ids = make_ids(T, 7, 200, 9, 0.01, torch.int32)
    plan = mxw.sort_tokens(ids, 200)
    flat = ids.view(-1).long()
    flat = torch.where((flat < 0) | (flat >= 200), 200, flat)
    order = torch.argsort(flat, stable=True)
    counts = torch.bincount(flat, minlength=201)
    ends = ((counts[:200] + 31) // 32 * 32).cumsum(0)
    first = torch.cat([torch.zeros(1, dtype=torch.int64, device=DEV), ends[:-1]]) - (counts.cumsum(0) - counts)[:200]
    rows = torch.full_like(flat, -1)
    n = int(counts[:200].sum())
    rows[order[:n]] = torch.arange(n, device=DEV) + first[flat[order[:n]]]
    assert torch.equal(plan.rows.view(-1).long(), rows) and torch.equal(plan.offs.long(), ends)


# ---- dispatch -----------------------------------------------------------------

def plain_dispatch(x, plan, xs):
    """xs with the rows that the definition writes."""
    offs, counts = plan.offs.tolist(), plan.counts.tolist()
    start = 0
    for end, n in zip(offs, counts):
        xs[start + n:end] = 0
        start = end
    used = plan.rows >= 0
    token = torch.arange(x.shape[0], device=DEV)[:, None].expand_as(plan.rows)
    xs[plan.rows[used].long()] = x[token[used]]
    return xs


HS = [1, 7, 8, 9, 33, 64, 505, 511, 512, 513, 520, 1001, 1024, 1030, 1536, 1540, 2047, 2048, 2052, 4100, 8200]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", HS)
def test_dispatch_copies(H, dtype):
    say("dispatch H=%d %s" % (H, dtype))
    T, k, E = 37, 3, 5
    plan = mxw.sort_tokens(make_ids(T, k, E, H, 0.2), E)
    x = values((T, H), H, dtype)
    x[0, 0], x[1, H - 1], x[2, H // 2] = float("nan"), float("inf"), -0.0
    got = mxw.dispatch_tokens(x, plan, out=poison((plan.size, H), dtype))
    assert same_bits(got, plain_dispatch(x, plan, poison((plan.size, H), dtype)))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", [32, 96, 512, 544, 2048, 2080, 7168])
@pytest.mark.parametrize("rows", [True, False])
def test_dispatch_mxfp8_is_quantize_rows(H, dtype, rows):
    say("dispatch mxfp8 H=%d %s rows=%s" % (H, dtype, rows))
    T, k, E = 29, 2, 4
    plan = mxw.sort_tokens(make_ids(T, k, E, H + 1, 0.1), E)
    x = values((T, H), H + 2, dtype) * 3.0
    x[3, 5], x[4, 31], x[5, :32] = float("nan"), float("-inf"), 0.0
    u8 = torch.uint8
    q, s = poison((plan.size, H), u8), poison((plan.size, H // 32), u8)
    got = mxw.dispatch_tokens(x, plan, rows=rows, mxfp8=True, q=q, s=s)
    xs = plain_dispatch(x, plan, torch.full((plan.size, H), 5.0, dtype=dtype, device=DEV))
    wq, ws = mxw.quantize_rows(xs)
    end = plan.offs[-1].item()
    assert got[-2].data_ptr() == q.data_ptr() and got[-1].data_ptr() == s.data_ptr()
    assert torch.equal(q[:end], wq[:end]) and torch.equal(s[:end], ws[:end])
    assert (q[end:] == 0xA5).all() and (s[end:] == 0xA5).all()
    if rows:
        assert same_bits(got[0][:end], xs[:end])


def test_dispatch_strides_and_alignment():
    """Rows of any stride, and tensors that start on any element."""
    T, k, E, H = 40, 2, 6, 260
    plan = mxw.sort_tokens(make_ids(T, k, E, 3), E)
    for dtype in (BF16, F32):
        big = values((T * 300 + 9,), 4, dtype)
        for start, ld in ((0, 260), (1, 261), (3, 297), (0, 300)):
            x = torch.as_strided(big, (T, H), (ld, 1), start)
            room = poison((plan.size * H + 3,), dtype)
            out = room[1:1 + plan.size * H].view(plan.size, H)
            mxw.dispatch_tokens(x, plan, out=out)
            assert same_bits(out, plain_dispatch(x, plan, poison((plan.size, H), dtype)))
            assert room[0].isnan() and room[-2:].isnan().all()


def test_dispatch_fewer_rows_than_the_plan():
    """Rows that the outputs do not have are skipped, and nothing outside is written."""
    T, k, E, H = 64, 2, 6, 96
    plan = mxw.sort_tokens(make_ids(T, k, E, 6), E)
    x = values((T, H), 6)
    full = mxw.dispatch_tokens(x, plan, out=torch.zeros((plan.size, H), dtype=BF16, device=DEV))
    for R in (1, 33, 100):
        room = poison((plan.size, H), BF16)
        got = mxw.dispatch_tokens(x, plan, out=room[:R])
        assert same_bits(got, full[:R]) and room[R:].isnan().all()
    assert mxw.dispatch_tokens(x, plan, out=room[:0]).shape == (0, H)


def test_malformed_plans_stay_inside():
    T, k, E, H, R = 32, 2, 4, 64, 96
    x, y = values((T, H), 7), values((R, H), 8)
    rows = torch.randint(-(1 << 31), (1 << 31) - 1, (T, k), dtype=torch.int32, device=DEV)
    offs = torch.tensor([50, -7, 1 << 30, 20], dtype=torch.int32, device=DEV)
    counts = torch.tensor([-5, 1 << 30, 3, -(1 << 31)], dtype=torch.int32, device=DEV)
    plan = mxw.TokenPlan(offs, counts, rows, R)
    room = poison((3 * R, H), BF16)
    q, s = poison((3 * R, H), torch.uint8), poison((3 * R, H // 32), torch.uint8)
    mxw.dispatch_tokens(x, plan, mxfp8=True, out=room[R:2 * R], q=q[R:2 * R], s=s[R:2 * R])
    w = torch.rand((T, k), device=DEV)
    mxw.combine_tokens_grad(x, y, plan, w, dy=room[R:2 * R])
    out = mxw.combine_tokens(y, plan, w)
    torch.cuda.synchronize()
    for t in (room, q, s):
        edge = torch.cat([t[:R], t[2 * R:]])
        assert (edge == 0xA5).all() if t.dtype == torch.uint8 else edge.isnan().all()
    assert (out[((rows < 0) | (rows >= R)).all(1)] == 0).all()


# ---- combine ------------------------------------------------------------------

def plain_combine(y, plan, w, residual=None):
    """(result, sum of magnitudes) in 64 bits."""
    at = y.double()[plan.rows.clamp(min=0).long()]
    at = torch.where((plan.rows >= 0)[..., None], at, 0.0)
    terms = at if w is None else at * torch.where(plan.rows >= 0, w, 0.0).double()[..., None]
    out, size = terms.sum(1), terms.abs().sum(1)
    if residual is not None:
        out, size = out + residual.double(), size + residual.double().abs()
    return out, size


def check(got, ref, size, roundings, what):
    eps = torch.finfo(got.dtype).eps / 2 if got.dtype != F32 else 0.0
    bad = ~((got.double() - ref).abs() <= eps * (1 + 2.0 ** -10) * ref.abs() + (1 + eps) * roundings * 2.0 ** -24 * size)
    assert not bad.any(), "%s: %d of %d outside, first %s" % (what, int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", HS)
def test_combine(H, dtype):
    for T, k, E, empty, weighted, with_residual in ((37, 3, 5, 0.2, True, False), (9, 8, 16, 0.0, True, True),
                                                    (5, 17, 3, 0.1, False, True), (1, 1, 1, 0.0, False, False)):
        say("combine H=%d T=%d k=%d %s" % (H, T, k, dtype))
        plan = mxw.sort_tokens(make_ids(T, k, E, H + T, empty), E)
        y = values((plan.size, H), H, dtype)
        y[plan.offs[-1].item():] = float("nan")
        w = None
        if weighted:
            w = torch.rand((T, k), device=DEV) - 0.3
            w[plan.rows < 0] = float("nan")
        r = values((T, H), H + 1, dtype) if with_residual else None
        got = mxw.combine_tokens(y, plan, w, residual=r, out=poison((T, H), dtype))
        ref, size = plain_combine(y, plan, w, r)
        check(got, ref, size, k + 1, "H=%d T=%d k=%d" % (H, T, k))


def test_combine_tokens_without_choices():
    T, k, E, H = 6, 2, 3, 70
    ids = make_ids(T, k, E, 1)
    ids[2], ids[4] = -1, 99
    plan = mxw.sort_tokens(ids, E)
    y, r = values((plan.size, H), 2), values((T, H), 3)
    out = mxw.combine_tokens(y, plan, torch.ones((T, k), device=DEV))
    assert (out[2] == 0).all() and (out[4] == 0).all()
    out = mxw.combine_tokens(y, plan, residual=r)
    assert same_bits(out[2], r[2]) and same_bits(out[4], r[4])
    none = mxw.sort_tokens(torch.full((T, k), -1, dtype=torch.int32, device=DEV), E)
    assert none.offs.tolist() == [0, 0, 0]
    assert (mxw.combine_tokens(torch.full_like(y, float("nan")), none) == 0).all()
    assert (mxw.combine_tokens(y[:0], none) == 0).all()


def test_combine_residual_in_place_and_strides():
    T, k, E, H = 50, 4, 8, 1001
    plan = mxw.sort_tokens(make_ids(T, k, E, 11), E)
    w = torch.rand((T, k), device=DEV)
    for dtype in (BF16, F32):
        wide = values((plan.size, H + 5), 12, dtype)
        y = wide[:, 3:3 + H]
        res = values((T, H + 2), 13, dtype)[:, 1:1 + H]
        want = mxw.combine_tokens(y.contiguous(), plan, w, residual=res.contiguous())
        assert same_bits(mxw.combine_tokens(y, plan, w, residual=res), want)
        acc = res.contiguous()
        assert mxw.combine_tokens(y, plan, w, residual=acc, out=acc) is acc and same_bits(acc, want)


def test_broken_rows_stay_with_their_tokens():
    T, k, E, H = 30, 2, 4, 600
    plan = mxw.sort_tokens(make_ids(T, k, E, 14), E)
    w = torch.rand((T, k), device=DEV) + 0.1
    y = values((plan.size, H), 15)
    want = mxw.combine_tokens(y, plan, w)
    y[plan.rows[7, 1].item(), 100] = float("inf")
    y[plan.rows[9, 0].item(), 599] = float("nan")
    got = mxw.combine_tokens(y, plan, w)
    assert got[7, 100].isinf() and got[9, 599].isnan()
    got[7, 100], got[9, 599] = want[7, 100], want[9, 599]
    assert same_bits(got, want)


# ---- the gradient -------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", HS)
def test_grad(H, dtype):
    for T, k, E, empty in ((37, 3, 5, 0.2), (9, 8, 16, 0.0), (5, 17, 3, 0.1), (1, 1, 1, 0.0)):
        say("combine grad H=%d T=%d k=%d %s" % (H, T, k, dtype))
        plan = mxw.sort_tokens(make_ids(T, k, E, H + T, empty), E)
        y, dout = values((plan.size, H), H, dtype), values((T, H), H + 1, dtype)
        end = plan.offs[-1].item()
        y[end:] = float("nan")
        w = torch.rand((T, k), device=DEV) - 0.3
        w[plan.rows < 0] = float("nan")
        dy, dw = mxw.combine_tokens_grad(dout, y, plan, w, dy=poison((plan.size, H), dtype))
        used = plan.rows >= 0
        token = torch.arange(T, device=DEV)[:, None].expand_as(plan.rows)
        ref = torch.zeros((plan.size, H), dtype=torch.float64, device=DEV)
        ref[plan.rows[used].long()] = w[used].double()[:, None] * dout.double()[token[used]]
        check(dy[:end], ref[:end], ref[:end].abs(), 1, "dy H=%d T=%d" % (H, T))
        assert dy[end:].isnan().all()
        at = torch.where(used[..., None], y.double()[plan.rows.clamp(min=0).long()], 0.0) * dout.double()[:, None]
        check(dw, at.sum(2), at.abs().sum(2), H + 12, "dw H=%d T=%d" % (H, T))
        assert (dw[~used] == 0).all()


@pytest.mark.parametrize("H", [32, 512, 544, 2048, 7168])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_grad_mxfp8_is_quantize_rows(H, dtype):
    T, k, E = 21, 3, 4
    say("combine grad mxfp8 H=%d %s" % (H, dtype))
    plan = mxw.sort_tokens(make_ids(T, k, E, H, 0.1), E)
    y, dout, w = values((plan.size, H), H, dtype), values((T, H), 1, dtype), torch.rand((T, k), device=DEV)
    dy, dw = mxw.combine_tokens_grad(dout, y, plan, w)
    end = plan.offs[-1].item()
    wq, ws = mxw.quantize_rows(dy[:end])
    both = mxw.combine_tokens_grad(dout, y, plan, w, mxfp8=True)
    codes = mxw.combine_tokens_grad(dout, y, plan, w, rows=False, mxfp8=True)
    assert len(both) == 4 and len(codes) == 3
    assert same_bits(both[0][:end], dy[:end]) and same_bits(both[3], dw) and same_bits(codes[2], dw)
    for q, s in (both[1:3], codes[:2]):
        assert torch.equal(q[:end], wq) and torch.equal(s[:end], ws)


def test_grad_in_y_itself():
    T, k, E, H = 60, 9, 12, 1001
    plan = mxw.sort_tokens(make_ids(T, k, E, 20, 0.1), E)
    for dtype in (BF16, F32):
        y, dout, w = values((plan.size, H), 21, dtype), values((T, H), 22, dtype), torch.rand((T, k), device=DEV)
        end = plan.offs[-1].item()
        dy, dw = mxw.combine_tokens_grad(dout, y, plan, w)
        got, again = mxw.combine_tokens_grad(dout, y, plan, w, dy=y)
        assert got is y and same_bits(y[:end], dy[:end]) and same_bits(again, dw)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", [3, 7, 8, 9, 15, 115, 501, 1001, 2047, 3949])
def test_in_place_at_row_ends(H, dtype):
    """Rows that end inside a lane's 8 columns: the same bits in place (out over the
    residual, dy over y) as into other tensors, again and again."""
    T, k, E = 700, 9, 16
    say("in place %s H=%d" % (dtype, H))
    ids = make_ids(T, k, E, 70, 0.2)
    plan = mxw.sort_tokens(ids, E)
    x, w = values((T, H), 71, dtype), torch.rand((T, k), device=DEV)
    y = values((plan.size, H), 72, dtype)
    out = mxw.combine_tokens(y, plan, w, residual=x)
    dy, dw = mxw.combine_tokens_grad(x, y, plan, w)
    end = plan.offs[-1].item()
    for _ in range(4):
        there = x.clone()
        assert same_bits(mxw.combine_tokens(y, plan, w, residual=there, out=there), out)
        there = y.clone()
        got, gw = mxw.combine_tokens_grad(x, there, plan, w, dy=there)
        assert got is there and same_bits(got[:end], dy[:end]) and same_bits(gw, dw)
        assert same_bits(got[end:], y[end:])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", [9, 15, 115, 2047])
def test_infinities_before_a_row_end(H, dtype):
    """An infinity in a column that lanes share counts once, as an infinity, and a NaN in
    y's meets no other."""
    T, k, E = 40, 2, 4
    ids = make_ids(T, k, E, 73)
    plan = mxw.sort_tokens(ids, E)
    for col in {max(H - 8, 0), H // 8 * 8 - 1, H - 1}:
        dout = torch.ones((T, H), dtype=dtype, device=DEV)
        y = torch.ones((plan.size, H), dtype=dtype, device=DEV)
        dout[3, col] = float("inf")
        y[plan.rows[7, 1].item(), col] = float("nan")
        w = torch.ones((T, k), device=DEV)
        dy, dw = mxw.combine_tokens_grad(dout, y, plan, w)
        want = torch.full((T, k), float(H), device=DEV)
        want[3] = float("inf")
        want[7, 1] = float("nan")
        assert torch.equal(dw.nan_to_num(nan=-1.0), want.nan_to_num(nan=-1.0))
        out = mxw.combine_tokens(y, plan, w)
        bad = out.isnan()
        assert bad[7, col] and bad.sum() == 1


def test_gradients_against_differences():
    """f(y, w) = <out, d> in float32: its central differences along random directions.
    f is linear in y and in w, so that a difference over 2 h is exact but for roundings:
    f's are at most (k + 1) 2^-24 of its terms' magnitudes (the sum over out is in 64
    bits), twice over 2 h with h = 1, and those of the gradients below them."""
    T, k, E, H = 23, 3, 4, 777
    plan = mxw.sort_tokens(make_ids(T, k, E, 30, 0.1), E)
    end = plan.offs[-1].item()
    y, v = values((plan.size, H), 31, F32), values((plan.size, H), 32, F32)
    w, u = torch.rand((T, k), device=DEV), torch.randn((T, k), device=DEV)
    d = values((T, H), 33, F32)
    dy, dw = mxw.combine_tokens_grad(d, y, plan, w)

    def f(y, w):
        return (mxw.combine_tokens(y, plan, w).double() * d.double()).sum().item()

    def size(y, w):
        return (plain_combine(y, plan, w)[1] * d.double().abs()).sum().item()

    got = (dy[:end].double() * v[:end].double()).sum().item()
    assert abs((f(y + v, w) - f(y - v, w)) / 2 - got) <= (k + 4) * 2.0 ** -23 * (size(y.abs() + v.abs(), w) + 1)
    used = plan.rows >= 0
    got = (dw[used].double() * u[used].double()).sum().item()
    assert abs((f(y, w + u) - f(y, w - u)) / 2 - got) <= (H + 20) * 2.0 ** -23 * size(y, w.abs() + u.abs())
    # dispatch's gradient is combine without weights: <dispatch(x), g> = <x, combine(g)>
    x, g = values((T, H), 34, F32), values((plan.size, H), 35, F32)
    left = (mxw.dispatch_tokens(x, plan)[:end].double() * g[:end].double()).sum()
    right = (x.double() * mxw.combine_tokens(g, plan).double()).sum()
    size = (plain_combine(g.abs(), plan, None)[1] * x.double().abs()).sum()
    assert (left - right).abs() <= (k + 1) * 2.0 ** -24 * size


def test_no_tokens():
    plan = mxw.sort_tokens(torch.empty((0, 2), dtype=torch.int64, device=DEV), 4)
    assert plan.size == 0 and plan.rows.shape == (0, 2) and plan.offs.tolist() == [0, 0, 0, 0]
    x = torch.empty((0, 64), dtype=BF16, device=DEV)
    assert mxw.dispatch_tokens(x, plan).shape == (0, 64)
    room = poison((32, 64), BF16)
    assert mxw.dispatch_tokens(x, plan, out=room).isnan().all()
    assert mxw.combine_tokens(room, plan).shape == (0, 64)
    dy, dw = mxw.combine_tokens_grad(x, room, plan, torch.empty((0, 2), device=DEV))
    assert dy.shape == (32, 64) and dw.shape == (0, 2)


# ---- use ----------------------------------------------------------------------

def test_repeats_streams_and_graphs():
    """Two streams at once, and a captured run of all four replayed on new ids and values
    with eager work between: the same bits as eagerly."""
    T, k, E, H = 9000, 2, 8, 544  # two pieces of the sort
    ids, x, dout = make_ids(T, k, E, 40), values((T, H), 41), values((T, H), 42)
    w = torch.rand((T, k), device=DEV)

    def all_of(ids, x, dout, w, **more):
        plan = mxw.sort_tokens(ids, E, **more)
        more.pop("workspace", None)
        xs, q, s = mxw.dispatch_tokens(x, plan, mxfp8=True, **more)
        out = mxw.combine_tokens(xs, plan, w, residual=x, **more)
        dy, dw = mxw.combine_tokens_grad(dout, xs, plan, w, **more)
        return plan, xs, q, s, out, dy, dw

    def same(a, b):
        end = b[0].offs[-1].item()
        assert all(torch.equal(p, r) for p, r in zip(a[0][:3], b[0][:3]))
        for p, r in zip(a[1:], b[1:]):
            n = end if p.shape[0] == b[0].size else p.shape[0]
            assert same_bits(p[:n], r[:n])

    want = all_of(ids, x, dout, w)
    sides = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = []
    for s in sides:
        s.wait_stream(torch.cuda.current_stream())
        got.append(all_of(ids, x, dout, w, stream=s))
    for s, g in zip(sides, got):
        torch.cuda.current_stream().wait_stream(s)
        same(g, want)
    ws = torch.full((mxw.sort_workspace_size(T, k, E),), 0xEE, dtype=torch.uint8, device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kept = all_of(ids, x, dout, w, workspace=ws)
    for i in range(4):
        ids.copy_(ids.roll(17, 0))
        x.mul_(-1.5)
        w.copy_(w.roll(1, 0))
        graph.replay()
        torch.cuda.synchronize()
        same(kept, all_of(ids, x, dout, w))


def past_the_caches(H, dtype, k=4, E=8):
    """(plan, parts of it with a quarter of the tokens) of a call that moves over 256 MB,
    where loads and stores go past the caches; a part's call moves less."""
    T = (1 << 28) // (H * dtype.itemsize * (k + 1)) + 1001
    say("over 256 MB: T=%d k=%d H=%d %s" % (T, k, H, dtype))
    plan = mxw.sort_tokens(make_ids(T, k, E, H, 0.05), E)
    cuts = [(a, min(a + T // 4 + 1, T)) for a in range(0, T, T // 4 + 1)]
    return plan, [(slice(a, b), plan._replace(rows=plan.rows[a:b].contiguous())) for a, b in cuts]


LONG = [501, 512, 901, 1024, 1501, 1701, 2048]   # one, two and four waves a token, whole rows and shared ends


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", LONG)
def test_dispatch_past_the_caches(H, dtype):
    plan, parts = past_the_caches(H, dtype)
    x = values((plan.rows.shape[0], H), 70, dtype)
    got, want = poison((plan.size, H), dtype), poison((plan.size, H), dtype)
    mxw.dispatch_tokens(x, plan, out=got)
    for at, part in parts:
        mxw.dispatch_tokens(x[at], part, out=want)
    assert same_bits(got, want) and not got[:plan.offs[-1].item()].isnan().any()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", [480, 992, 1504])
@pytest.mark.parametrize("rows", [True, False])
def test_dispatch_mxfp8_past_the_caches(H, dtype, rows):
    plan, parts = past_the_caches(H, dtype, k=8 if dtype == BF16 else 4)
    T, k = plan.rows.shape
    if not rows:   # codes alone are fewer bytes: the tokens count more than once
        T = (1 << 28) // (H * (dtype.itemsize + k)) + 1001
        plan = mxw.sort_tokens(make_ids(T, k, 8, H, 0.05), 8)
        parts = [(slice(a, a + T // 4 + 1), plan._replace(rows=plan.rows[a:a + T // 4 + 1].contiguous()))
                 for a in range(0, T, T // 4 + 1)]
    x = values((T, H), 71, dtype)
    both = []
    for _ in range(2):
        both.append((poison((plan.size, H), dtype) if rows else None, poison((plan.size, H), torch.uint8),
                     poison((plan.size, H // 32), torch.uint8)))
    mxw.dispatch_tokens(x, plan, rows=rows, mxfp8=True, out=both[0][0], q=both[0][1], s=both[0][2])
    for at, part in parts:
        mxw.dispatch_tokens(x[at], part, rows=rows, mxfp8=True, out=both[1][0], q=both[1][1], s=both[1][2])
    for got, want in zip(*both):
        assert got is want is None or same_bits(got, want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", LONG)
def test_combine_past_the_caches(H, dtype):
    """With weights and a residual, into another tensor and into the residual itself."""
    plan, parts = past_the_caches(H, dtype)
    T, k = plan.rows.shape
    y, r = values((plan.size, H), 72, dtype), values((T, H), 73, dtype)
    w = torch.rand((T, k), device=DEV)
    want = torch.cat([mxw.combine_tokens(y, part, w[at].contiguous(), residual=r[at]) for at, part in parts])
    got = mxw.combine_tokens(y, plan, w, residual=r, out=poison((T, H), dtype))
    assert same_bits(got, want) and not got.isnan().any()
    mxw.combine_tokens(y, plan, w, residual=r, out=r)
    assert same_bits(r, want)
    want = torch.cat([mxw.combine_tokens(y, part) for at, part in parts])
    assert same_bits(mxw.combine_tokens(y, plan, out=poison((T, H), dtype)), want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("H", LONG)
def test_grad_past_the_caches(H, dtype):
    """Into other tensors, with MXFP8 rows where the row has whole blocks, and over y itself."""
    plan, parts = past_the_caches(H, dtype)
    T, k = plan.rows.shape
    y, dout = values((plan.size, H), 74, dtype), values((T, H), 75, dtype)
    w = torch.rand((T, k), device=DEV)
    mx = H % 32 == 0

    def outputs():
        both = dict(dy=poison((plan.size, H), dtype))
        if mx:
            both.update(q=poison((plan.size, H), torch.uint8), s=poison((plan.size, H // 32), torch.uint8))
        return both

    got, want = outputs(), outputs()
    dw = mxw.combine_tokens_grad(dout, y, plan, w, mxfp8=mx, **got)[-1]
    dws = [mxw.combine_tokens_grad(dout[at], y, part, w[at].contiguous(), mxfp8=mx, **want)[-1] for at, part in parts]
    assert all(same_bits(got[n], want[n]) for n in got) and same_bits(dw, torch.cat(dws))
    assert not dw.isnan().any() and not got["dy"][:plan.offs[-1].item()].isnan().any()
    dw = mxw.combine_tokens_grad(dout, y, plan, w, dy=y)[-1]
    end = plan.offs[-1].item()
    assert same_bits(dw, torch.cat(dws)) and same_bits(y[:end], want["dy"][:end])


def test_offsets_past_32_bits():
    """Rows whose offsets pass 2^31 elements and 2^32 bytes."""
    T, k, E, H = 40000, 8, 4, 7168
    say("tokens R=%d H=%d" % (T * k, H))
    ids = make_ids(T, k, E, 50, dtype=torch.int32)
    plan = mxw.sort_tokens(ids, E)
    assert plan.size * H > 1 << 31
    x = values((T, H), 51)
    xs, q, s = mxw.dispatch_tokens(x, plan, mxfp8=True)
    end = plan.offs[-1].item()
    for t in (0, 1, T // 2, T - 2, T - 1):
        want = mxw.quantize_rows(x[t:t + 1])
        for r in plan.rows[t].tolist():
            assert same_bits(xs[r], x[t]) and torch.equal(q[r], want[0][0]) and torch.equal(s[r], want[1][0])
    del q, s
    last = plan.rows == plan.offs[-2] + plan.counts[-1] - 1
    assert last.any() and not xs[end - 32:end].isnan().any()
    w = torch.full((T, k), 0.125, device=DEV)
    assert same_bits(mxw.combine_tokens(xs, plan, w), x)  # eight equal rows, an eighth each
    dy, dw = mxw.combine_tokens_grad(x, xs, plan, w, dy=xs)
    for t in (0, T // 2, T - 1):
        for r in plan.rows[t].tolist():
            assert same_bits(dy[r], x[t] * 0.125)
    norm = x.double().square().sum(1)
    assert ((dw.double() - norm[:, None]).abs() <= (H + 12) * 2.0 ** -24 * norm[:, None]).all()


def test_a_layer_of_grouped_products():
    """sort, dispatch to MXFP8, two grouped products, combine, and back: the layer of a
    mixture of experts against its definition on the same operands in 64 bits, and the
    weight gradient from the rows.  Operands are the decoded codes, so what is left is
    the products' rounding to bf16 (2^-8) and those below it."""
    T, k, E, H, N = 700, 2, 5, 256, 96
    ids = make_ids(T, k, E, 60, 0.05)
    x, w = values((T, H), 61), torch.rand((T, k), device=DEV)
    weight = values((E, N, H), 62) * 0.1
    plan = mxw.sort_tokens(ids, E)
    xs, q, s = mxw.dispatch_tokens(x, plan, mxfp8=True)
    wq, wsc = mxw.quantize_rows(weight)
    y = mxw.fwd(q, s, wq, wsc, plan.offs)
    out = mxw.combine_tokens(y, plan, w)

    def decode(q, s):
        v = q.view(torch.float8_e4m3fn).double().view(*s.shape, 32)
        return (v * torch.exp2(s.double() - 127)[..., None]).view(q.shape)

    X, W = decode(*mxw.quantize_rows(x)), decode(wq, wsc)
    ref, size = torch.zeros((T, N), dtype=torch.float64, device=DEV), torch.zeros((T, N), dtype=torch.float64, device=DEV)
    for e in range(E):
        share = (w.double() * (ids == e)).sum(1, keepdim=True)
        each = X @ W[e].mT
        ref += share * each
        size += share * (each.abs() + X.abs() @ W[e].abs().mT * H * 2.0 ** -16)
    bad = (out.double() - ref).abs() > 2.0 ** -8 * 2.02 * size
    assert not bad.any(), int(bad.sum())
    dout = values((T, N), 63)
    dy, dw = mxw.combine_tokens_grad(dout, y, plan, w)
    for t in dy, xs:
        t[plan.offs[-1].item():] = 0
    grad = mxw.wgrad(*mxw.quantize_tokens(dy, plan.offs), *mxw.quantize_tokens(xs, plan.offs), plan.offs)
    for e in range(E):
        share = (w.double() * (ids == e)).sum(1, keepdim=True)
        want = (dout.double() * share).mT @ x.double()
        assert (grad[e].double() * want).sum() / (grad[e].double().norm() * want.norm()) > 0.998
