"""The host checks of the tokens' operators, quantize_rows, clip_grad_norm and linear_4bit:
bad arguments come back as status codes or exceptions before any device access (CPU only)."""
import pytest
import torch

import mxfp8_ragged_grouped_amd as mxw

P = 0x10000  # a fake, never-dereferenced device address
BIG = 1 << 50
BF16 = torch.bfloat16


def call(f, base, over):
    return f(**dict(base, **over))


SORT = dict(ids=P, id_bytes=8, ld=2, T=4, k=2, E=8, align=32, offs=P, counts=P, rows=P, workspace=P, workspace_bytes=BIG)


@pytest.mark.parametrize("over,code", [
    (dict(ids=0), -1), (dict(offs=0), -1), (dict(counts=0), -1), (dict(rows=0), -1),
    (dict(id_bytes=2), -2), (dict(ld=1), -2), (dict(T=-1), -2), (dict(k=0), -2), (dict(k=65, ld=65), -2), (dict(E=0), -2),
    (dict(E=257), -2), (dict(align=0), -2), (dict(align=1025), -2), (dict(T=1 << 23, k=2), -2),
    (dict(T=(1 << 23) - 8, k=1, E=256, align=1024), -2),   # its rows are over the most
    (dict(ids=P + 4), -3), (dict(offs=P + 2), -3), (dict(counts=P + 1), -3), (dict(rows=P + 2), -3),
    (dict(T=9000, workspace=0), -6), (dict(T=9000, workspace=P + 16), -6), (dict(T=9000, workspace_bytes=63), -6),
])
def test_sort_host_checks(over, code):
    assert call(mxw.mxw_sort_tokens, SORT, over) == code


def test_sizes():
    assert mxw.token_rows(0, 2, 8) == 0 and mxw.token_rows(1, 2, 8) == 64 and mxw.token_rows(1, 2, 1) == 32
    assert mxw.token_rows(100, 2, 8) == (200 + 8 * 31) // 32 * 32 and mxw.token_rows(5, 3, 10, 1) == 15
    assert mxw.sort_workspace_size(2048, 2, 8) == 0 and mxw.sort_workspace_size(2049, 2, 8) == 3 * 8 * 4
    assert mxw.clip_workspace_size(0) > 0 and mxw.clip_workspace_size(96) < mxw.clip_workspace_size(97)
    for f, args in ((mxw.token_rows, (1 << 23, 2, 8)), (mxw.token_rows, (4, 2, 0)), (mxw.token_rows, (4, 2, 8, 0)),
                    (mxw.sort_workspace_size, (4, 65, 8)), (mxw.clip_workspace_size, (-1,)),
                    (mxw.clip_workspace_size, (65537,))):
        with pytest.raises(mxw.MxwError):
            f(*args)


DISPATCH = dict(x=P, dtype=0, ldx=64, offs=P, counts=P, rows=P, T=4, k=2, E=8, H=64, R=64, xs=P, q=P, s=P)


@pytest.mark.parametrize("over,code", [
    (dict(x=0), -1), (dict(offs=0), -1), (dict(counts=0), -1), (dict(rows=0), -1), (dict(xs=0, q=0, s=0), -1),
    (dict(q=0), -1), (dict(s=0), -1),
    (dict(dtype=2), -2), (dict(ldx=63), -2), (dict(T=-1), -2), (dict(k=0), -2), (dict(E=0), -2), (dict(H=0), -2),
    (dict(H=48), -2), (dict(H=65568, ldx=65568), -2), (dict(R=-1), -2), (dict(R=(1 << 23) + 1), -2),
    (dict(x=P + 1), -3), (dict(dtype=1, x=P + 2), -3), (dict(xs=P + 1), -3), (dict(q=P + 4), -3), (dict(rows=P + 2), -3),
    (dict(offs=P + 2), -3), (dict(counts=P + 1), -3),
])
def test_dispatch_host_checks(over, code):
    assert call(mxw.mxw_dispatch_tokens, DISPATCH, over) == code


COMBINE = dict(y=P, dtype=0, ldy=64, rows=P, weights=P, residual=P, ldr=64, T=4, k=2, H=64, R=64, out=P)


@pytest.mark.parametrize("over,code", [
    (dict(y=0), -1), (dict(rows=0), -1), (dict(out=0), -1),
    (dict(dtype=-1), -2), (dict(ldy=63), -2), (dict(ldr=63), -2), (dict(T=-1), -2), (dict(k=65), -2), (dict(H=0), -2),
    (dict(H=65537, ldy=1 << 20, ldr=1 << 20), -2), (dict(R=-1), -2),
    (dict(y=P + 1), -3), (dict(residual=P + 1), -3), (dict(out=P + 1), -3), (dict(weights=P + 2), -3), (dict(rows=P + 1), -3),
    (dict(dtype=1, out=P + 2), -3),
])
def test_combine_host_checks(over, code):
    assert call(mxw.mxw_combine_tokens, COMBINE, over) == code


GRAD = dict(dout=P, dtype=0, ldo=64, y=P, ldy=64, offs=P, counts=P, rows=P, weights=P, T=4, k=2, E=8, H=64, R=64, dy=P, q=P,
            s=P, dweights=P)


@pytest.mark.parametrize("over,code", [
    (dict(dout=0), -1), (dict(y=0), -1), (dict(offs=0), -1), (dict(counts=0), -1), (dict(rows=0), -1), (dict(weights=0), -1),
    (dict(dy=0, q=0, s=0, dweights=0), -1), (dict(q=0), -1), (dict(s=0), -1),
    (dict(dtype=2), -2), (dict(ldo=63), -2), (dict(ldy=63), -2), (dict(E=257), -2), (dict(H=40), -2), (dict(R=-1), -2),
    (dict(dout=P + 1), -3), (dict(y=P + 1), -3), (dict(dy=P + 1), -3), (dict(q=P + 2), -3), (dict(dweights=P + 2), -3),
])
def test_grad_host_checks(over, code):
    assert call(mxw.mxw_combine_tokens_grad, GRAD, over) == code


ROWS = dict(x=P, dtype=0, ldx=64, R=10, C=64, format=0, q=P, s=P)


@pytest.mark.parametrize("over,code", [
    (dict(x=0), -1), (dict(q=0), -1), (dict(s=0), -1),
    (dict(dtype=2), -2), (dict(ldx=63), -2), (dict(R=-1), -2), (dict(R=(1 << 31) + 1), -2), (dict(C=0), -2), (dict(C=40), -2),
    (dict(C=65568, ldx=65568), -2), (dict(format=2), -2), (dict(R=1 << 31, C=65536, ldx=65536), -2),
    (dict(x=P + 1), -3), (dict(dtype=1, x=P + 2), -3), (dict(q=P + 4), -3),
])
def test_quantize_rows_host_checks(over, code):
    assert call(mxw.mxw_quantize_rows, ROWS, over) == code


CLIP = dict(grads=[P, 2 * P], outs=[P, 2 * P], sizes=[100, 200], types=[0, 1], norm_type=2, max_norm=1.0, eps=1e-6, norm=P,
            workspace=P, workspace_bytes=BIG)


@pytest.mark.parametrize("over,code", [
    (dict(grads=[0, P]), -1), (dict(outs=[P, 0]), -1), (dict(norm=0), -1),
    (dict(types=[0, 2]), -2), (dict(sizes=[100, -1]), -2), (dict(sizes=[100, (1 << 40) + 1]), -2), (dict(norm_type=1), -2),
    (dict(max_norm=-1.0), -2), (dict(max_norm=float("nan")), -2), (dict(eps=-1e-9), -2), (dict(eps=float("nan")), -2),
    (dict(grads=[P + 1, 2 * P], outs=None), -3), (dict(grads=[P, 2 * P + 2], outs=None), -3), (dict(norm=P + 2), -3),
    (dict(workspace=0), -6), (dict(workspace=P + 128), -6), (dict(workspace_bytes=16), -6),
    (dict(grads=[P, P], outs=[P, P]), -8), (dict(grads=[P, P + 196], outs=[P, P + 196]), -8),
    (dict(outs=[P + 2, 2 * P]), -8), (dict(outs=[2 * P, 3 * P]), -8), (dict(outs=[3 * P, 3 * P]), -8),
])
def test_clip_host_checks(over, code):
    assert call(mxw.mxw_clip_grads, CLIP, over) == code


LINEAR = dict(x=P, ldx=256, codes=P, scales=P, zeros=0, format=1, group=32, T=4, K=256, N=100, out=P, out_type=0)
INT = dict(format=2, group=64, zeros=P)


@pytest.mark.parametrize("over,code", [
    (dict(x=0), -1), (dict(codes=0), -1), (dict(scales=0), -1), (dict(out=0), -1),
    (dict(format=0), -2), (dict(format=3), -2), (dict(group=64), -2), (dict(zeros=P), -2), (dict(T=-1), -2), (dict(T=65), -2),
    (dict(K=0), -2), (dict(K=48), -2), (dict(K=65568, ldx=65568), -2), (dict(N=0), -2), (dict(N=(1 << 20) + 1), -2),
    (dict(ldx=248), -2), (dict(ldx=260), -2), (dict(ldx=(1 << 23) + 8), -2), (dict(out_type=2), -2), (dict(INT, group=16), -2), (dict(INT, group=48), -2),
    (dict(INT, group=128, K=192, ldx=192), -2),
    (dict(x=P + 8), -3), (dict(codes=P + 4), -3), (dict(out=P + 1), -3), (dict(out_type=1, out=P + 2), -3),
    (dict(INT, scales=P + 1), -3),
])
def test_linear_host_checks(over, code):
    assert call(mxw.mxw_linear_4bit, LINEAR, over) == code


def apart(base, **sizes):
    """The call's arguments, every address its own MiB."""
    names = [n for n, v in base.items() if v == P]
    return dict(base, **{n: (i + 1) << 20 for i, n in enumerate(names)}, **sizes)


@pytest.mark.parametrize("f,base,pairs", [
    (mxw.mxw_sort_tokens, apart(SORT, T=9000), [("offs", "ids"), ("rows", "ids"), ("counts", "offs"), ("workspace", "rows")]),
    (mxw.mxw_dispatch_tokens, apart(DISPATCH), [("xs", "x"), ("q", "x"), ("s", "q"), ("xs", "s"), ("xs", "offs"), ("q", "rows"),
                                                ("s", "counts")]),
    (mxw.mxw_combine_tokens, apart(COMBINE), [("out", "y"), ("out", "rows"), ("out", "weights")]),
    (mxw.mxw_combine_tokens_grad, apart(GRAD), [("dy", "dout"), ("q", "dout"), ("dy", "q"), ("s", "y"), ("q", "y"),
                                                ("dweights", "weights"), ("dweights", "y"), ("dy", "rows"), ("dy", "dweights")]),
    (mxw.mxw_quantize_rows, apart(ROWS), [("q", "x"), ("s", "x"), ("s", "q")]),
    (mxw.mxw_linear_4bit, apart(LINEAR), [("out", "x"), ("out", "codes"), ("out", "scales")]),
])
def test_overlaps_are_refused(f, base, pairs):
    """An output at an input's address or another output's, or that begins in its last
    bytes (a workspace lies on 256)."""
    for out, other in pairs:
        by = 256 if out == "workspace" else 16
        assert f(**dict(base, **{out: base[other]})) == -8, (out, other)
        assert f(**dict(base, **{out: base[other] + by})) == -8, (out, other)
        assert f(**dict(base, **{other: base[out] + by})) == -8, (out, other)


def test_overlaps_that_are_meant():
    """The residual in place and dy over y pass this check (and meet the next), other
    strides do not, nor does a residual that begins inside the output."""
    c, g = apart(COMBINE), apart(GRAD)
    past = mxw.mxw_combine_tokens(**dict(c, T=0))   # what a call that passes every check gives here
    assert past != -8
    same = dict(c, residual=c["out"])
    assert call(mxw.mxw_combine_tokens, same, dict(residual=c["out"] + 2)) == -8
    assert call(mxw.mxw_combine_tokens, same, dict(ldr=72)) == -8
    same = dict(g, dy=g["y"])
    assert call(mxw.mxw_combine_tokens_grad, same, dict(dy=g["y"] + 2)) == -8
    assert call(mxw.mxw_combine_tokens_grad, same, dict(ldy=72)) == -8
    if not torch.cuda.is_available():   # with a device these would run
        assert mxw.mxw_combine_tokens(**dict(c, residual=c["out"])) == past
        assert mxw.mxw_combine_tokens_grad(**same) == past
        # an output that ends where the input begins
        assert call(mxw.mxw_quantize_rows, apart(ROWS), dict(q=(1 << 20) - 640, s=9 << 20)) == past
    # the norm inside a gradient that is scaled
    far = dict(CLIP, grads=[P, 2 * P], outs=[P, 2 * P], workspace=16 * P)
    assert call(mxw.mxw_clip_grads, far, dict(norm=P + 196)) == -8


CLIP_APART = dict(CLIP, grads=[1 << 20, 2 << 20], outs=[3 << 20, 4 << 20], norm=5 << 20, workspace=6 << 20)   # bf16 [100], float32 [200]


@pytest.mark.parametrize("outs", [CLIP_APART["outs"], CLIP_APART["grads"], None])
def test_clip_norm_and_workspace_lie_apart(outs):
    """The norm's four bytes and the workspace are written: they may share nothing with a
    gradient, an output or each other, for the norm alone as for clipping."""
    need = mxw.clip_workspace_size(2)
    base = dict(CLIP_APART, outs=outs)
    for at, size in list(zip(base["grads"], (200, 800))) + list(zip(outs or [], (200, 800))):
        for norm in (at, at + 4, at + size - 4):
            assert call(mxw.mxw_clip_grads, base, dict(norm=norm)) == -8, (at, norm)
        for ws in (at, at + size // 256 * 256 - (256 if size % 256 == 0 else 0), at - need + 256 - need % 256):
            assert ws % 256 == 0 and ws < at + size and ws + need > at
            assert call(mxw.mxw_clip_grads, base, dict(workspace=ws)) == -8, (at, ws)
    # a bf16 tensor may begin inside the norm
    for name in ("grads", "outs"):
        if base[name]:
            assert call(mxw.mxw_clip_grads, base, {name: [base["norm"] + 2, base[name][1]]}) == -8, name
    ws = base["workspace"]
    for norm in (ws, ws + 256, ws + need - 4):
        assert call(mxw.mxw_clip_grads, base, dict(norm=norm)) == -8, norm
    if not torch.cuda.is_available():   # with a device these would run
        past = mxw.mxw_combine_tokens(**dict(apart(COMBINE), T=0))   # what a call that passes every check gives here
        for fine in (dict(), dict(norm=ws - 4), dict(norm=ws + need), dict(norm=base["grads"][0] - 4),
                     dict(norm=base["grads"][0] + 200), dict(workspace=base["grads"][1] + 1024),
                     dict(workspace=base["grads"][0] - need - (256 - need % 256) % 256)):
            assert call(mxw.mxw_clip_grads, base, fine) == past != -8, fine


def test_sizes_past_32_bits_are_refused():
    """They would reach the library cut to 32 bits."""
    big = 1 << 32
    for f in (lambda: mxw.token_rows(big + 4, 2, 8), lambda: mxw.sort_workspace_size(4, 2, big + 8),
              lambda: mxw.token_rows(4, 2, 8, big + 32)):
        with pytest.raises(ValueError):
            f()


def test_sizes_past_32_bits_of_either_sign_are_refused():
    """Cut to 32 bits, all of these would be sizes that the library takes."""
    big = 1 << 32
    for f in (lambda: mxw.token_rows(4 - big, 2, 8), lambda: mxw.token_rows(4, 2, 8 - big), lambda: mxw.token_rows(4, 2, 8, 32 - big),
              lambda: mxw.sort_workspace_size(9000 - big, 2, 8), lambda: mxw.clip_workspace_size(big),
              lambda: mxw.clip_workspace_size(big + 5), lambda: mxw.clip_workspace_size(5 - big)):
        with pytest.raises(ValueError):
            f()


def test_python_faces_validate():
    """CPU tensors (there is no host fallback), types, shapes and strides."""
    ids = torch.zeros((4, 2), dtype=torch.int64)
    x, y, w = torch.zeros((4, 64), dtype=BF16), torch.zeros((64, 64), dtype=BF16), torch.zeros((4, 2))
    i32 = torch.int32
    plan = mxw.TokenPlan(torch.zeros(8, dtype=i32), torch.zeros(8, dtype=i32), torch.zeros((4, 2), dtype=i32), 64)
    codes, scales = torch.zeros((100, 32), dtype=torch.uint8), torch.zeros((100, 2), dtype=torch.uint8)
    for error, f in (
            (ValueError, lambda: mxw.sort_tokens(ids, 8)), (TypeError, lambda: mxw.sort_tokens(ids.short(), 8)),
            (ValueError, lambda: mxw.sort_tokens(ids[0], 8)), (ValueError, lambda: mxw.sort_tokens(ids[:, :0], 8)),
            (ValueError, lambda: mxw.dispatch_tokens(x, plan)), (TypeError, lambda: mxw.dispatch_tokens(x.half(), plan)),
            (ValueError, lambda: mxw.combine_tokens(y, plan)), (TypeError, lambda: mxw.combine_tokens(y.half(), plan)),
            (ValueError, lambda: mxw.combine_tokens_grad(x, y, plan, w)),
            (TypeError, lambda: mxw.combine_tokens_grad(x.half(), y, plan, w)),
            (ValueError, lambda: mxw.quantize_rows(x)), (TypeError, lambda: mxw.quantize_rows(x.half())),
            (ValueError, lambda: mxw.quantize_rows(x, "mxfp6")),
            (ValueError, lambda: mxw.clip_grad_norm([x], 1.0)), (ValueError, lambda: mxw.grad_norm([])),
            (TypeError, lambda: mxw.grad_norm([x.half()])), (ValueError, lambda: mxw.grad_norm([x], norm_type=1)),
            (ValueError, lambda: mxw.clip_grad_norm([x], -1.0)), (ValueError, lambda: mxw.clip_grad_norm([x], float("nan"))),
            (ValueError, lambda: mxw.linear_4bit(x, codes, scales)), (TypeError, lambda: mxw.linear_4bit(x.float(), codes, scales)),
            (TypeError, lambda: mxw.linear_4bit(x, codes, scales.half())),
            (TypeError, lambda: mxw.linear_4bit(x, codes, scales, dtype=torch.float16))):
        with pytest.raises(error):
            f()


def test_strerror_names_overlap():
    assert "overlap" in mxw.strerror(-8)
