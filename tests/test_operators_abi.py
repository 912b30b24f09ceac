"""The host checks of orthogonalize, vocab_cross_entropy and moe_layer: bad arguments come
back as status codes or exceptions before any device access (CPU only)."""
import ctypes

import pytest
import torch

import mxfp8_ragged_grouped_amd as mxw

P = 0x10000  # a fake, never-dereferenced device address
C5 = [3.4445, -4.7750, 2.0315] * 5


@pytest.mark.parametrize("args,code", [
    ((0, 0, 0, 256, 1, 128, 256, C5, 1e-7, P, P, 1 << 40), -1),            # NULL G
    ((P, 0, 0, 256, 1, 128, 256, C5, 1e-7, 0, P, 1 << 40), -1),            # NULL out
    ((P, 2, 0, 256, 1, 128, 256, C5, 1e-7, P, P, 1 << 40), -2),            # unknown type
    ((P, 0, 0, 256, 0, 128, 256, C5, 1e-7, P, P, 1 << 40), -2),            # E = 0
    ((P, 0, 0, 256, 257, 128, 256, C5, 1e-7, P, P, 1 << 40), -2),          # too many experts
    ((P, 0, 0, 256, 1, 0, 256, C5, 1e-7, P, P, 1 << 40), -2),              # N = 0
    ((P, 0, 0, 1 << 17, 1, 128, 65537, C5, 1e-7, P, P, 1 << 40), -2),      # K too large
    ((P, 0, 0, 255, 1, 128, 256, C5, 1e-7, P, P, 1 << 40), -2),            # rows overlap
    ((P, 0, -1, 256, 1, 128, 256, C5, 1e-7, P, P, 1 << 40), -2),           # negative stride
    ((P, 0, 0, 256, 1, 128, 256, [], 1e-7, P, P, 1 << 40), -2),            # no steps
    ((P, 0, 0, 256, 1, 128, 256, C5 * 7, 1e-7, P, P, 1 << 40), -2),        # 35 steps
    ((P, 0, 0, 256, 1, 128, 256, C5, -1.0, P, P, 1 << 40), -2),            # eps < 0
    ((P, 0, 0, 256, 1, 128, 256, C5, float("nan"), P, P, 1 << 40), -2),    # eps NaN
    ((P + 1, 0, 0, 256, 1, 128, 256, C5, 1e-7, P, P, 1 << 40), -3),        # bf16 on an odd address
    ((P + 2, 1, 0, 256, 1, 128, 256, C5, 1e-7, P, P, 1 << 40), -3),        # float32 on half a word
    ((P, 0, 0, 256, 1, 128, 256, C5, 1e-7, P + 1, P, 1 << 40), -3),        # out on an odd address
    ((P, 0, 0, 256, 1, 128, 256, C5, 1e-7, P, 0, 1 << 40), -6),            # no workspace
    ((P, 0, 0, 256, 1, 128, 256, C5, 1e-7, P, P, 100), -6),                # short workspace
    ((P, 0, 0, 256, 1, 128, 256, C5, 1e-7, P, P + 16, 1 << 40), -6),       # misaligned workspace
])
def test_orthogonalize_host_checks(args, code):
    assert mxw.mxw_orthogonalize(*args) == code


def test_orthogonalize_workspace_size():
    n = mxw.orthogonalize_workspace_size(8, 1408, 2048)
    assert n >= 2 * 8 * (2 * 1408 * 2048 + 2 * 1408 * 1408)
    for bad in ((0, 8, 8), (1, 0, 8), (1, 8, 65537), (257, 8, 8), (256, 65536, 65536)):
        with pytest.raises(mxw.MxwError):
            mxw.orthogonalize_workspace_size(*bad)


def test_orthogonalize_python_face_validates():
    G = torch.zeros((2, 64, 32), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        mxw.orthogonalize(G)                              # CPU tensor: no host fallback
    with pytest.raises(TypeError):
        mxw.orthogonalize(G.half())
    with pytest.raises(ValueError):
        mxw.orthogonalize(G[0, 0])
    with pytest.raises(ValueError):
        mxw.orthogonalize(G[:, :0])


BIG = 1 << 50


@pytest.mark.parametrize("args,code", [
    ((0, 64, P, 64, P, 8, -100, 4, 64, 100, 1, 1.0, P, P, P, P, BIG), -1),        # NULL x
    ((P, 64, 0, 64, P, 8, -100, 4, 64, 100, 1, 1.0, P, P, P, P, BIG), -1),        # NULL w
    ((P, 64, P, 64, 0, 8, -100, 4, 64, 100, 1, 1.0, P, P, P, P, BIG), -1),        # NULL targets
    ((P, 64, P, 64, P, 8, -100, 4, 64, 100, 1, 1.0, 0, P, P, P, BIG), -1),        # NULL loss
    ((P, 64, P, 64, P, 8, -100, 0, 64, 100, 1, 1.0, P, P, P, P, BIG), -2),        # no tokens
    ((P, 64, P, 64, P, 8, -100, 131073, 64, 100, 1, 1.0, P, P, P, P, BIG), -2),   # too many tokens
    ((P, 64, P, 64, P, 8, -100, 4, 0, 100, 1, 1.0, P, P, P, P, BIG), -2),         # H = 0
    ((P, 64, P, 64, P, 8, -100, 4, 64, 0, 1, 1.0, P, P, P, P, BIG), -2),          # V = 0
    ((P, 64, P, 64, P, 8, -100, 4, 64, (1 << 20) + 1, 1, 1.0, P, P, P, P, BIG), -2),  # V too large
    ((P, 63, P, 64, P, 8, -100, 4, 64, 100, 1, 1.0, P, P, P, P, BIG), -2),        # rows of x overlap
    ((P, 64, P, 63, P, 8, -100, 4, 64, 100, 1, 1.0, P, P, P, P, BIG), -2),        # rows of w overlap
    ((P, 64, P, 64, P, 2, -100, 4, 64, 100, 1, 1.0, P, P, P, P, BIG), -2),        # 16-bit targets
    ((P, 64, P, 64, P, 8, -100, 4, 64, 100, 3, 1.0, P, P, P, P, BIG), -2),        # unknown reduction
    ((P + 1, 64, P, 64, P, 8, -100, 4, 64, 100, 1, 1.0, P, P, P, P, BIG), -3),    # x on an odd address
    ((P, 64, P, 64, P + 4, 8, -100, 4, 64, 100, 1, 1.0, P, P, P, P, BIG), -3),    # int64 targets on half a word
    ((P, 64, P, 64, P, 8, -100, 4, 64, 100, 1, 1.0, P + 2, P, P, P, BIG), -3),    # loss misaligned
    ((P, 64, P, 64, P, 8, -100, 4, 64, 100, 1, 1.0, P, P, P + 1, P, BIG), -3),    # dw on an odd address
])
def test_vocab_loss_host_checks(args, code):
    assert mxw.mxw_vocab_loss(*args) == code


def test_vocab_loss_workspace_size_host_checks():
    lib = mxw._load()
    assert lib.mxw_vocab_loss_workspace_size(P, 64, P, 64, 0, 64, 100, 3) == -2
    assert lib.mxw_vocab_loss_workspace_size(P, 63, P, 64, 4, 64, 100, 3) == -2
    assert lib.mxw_vocab_loss_workspace_size(P, 64, P, 64, 4, 64, 100, 4) == -2
    if not torch.cuda.is_available():
        assert lib.mxw_vocab_loss_workspace_size(P, 64, P, 64, 4, 64, 100, 3) == -4
        assert mxw.mxw_vocab_loss(P, 64, P, 64, P, 8, -100, 4, 64, 100, 1, 1.0, P, P, P, P, BIG) == -4


def test_vocab_loss_python_face_validates():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    w = torch.zeros((100, 64), dtype=torch.bfloat16)
    y = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(ValueError):
        mxw.vocab_cross_entropy(x, w, y)                       # CPU tensors: no host fallback
    with pytest.raises(TypeError):
        mxw.vocab_cross_entropy(x.float(), w, y)
    with pytest.raises(TypeError):
        mxw.vocab_cross_entropy(x, w, y.to(torch.int16))
    with pytest.raises(ValueError):
        mxw.vocab_cross_entropy(x, w, y, reduction="max")
    with pytest.raises(ValueError):
        mxw.vocab_cross_entropy(x, w[:, :32], y)
    with pytest.raises(ValueError):
        mxw.vocab_cross_entropy(x, w, y[:3])
    with pytest.raises(ValueError):
        mxw.vocab_cross_entropy(x[:0], w, y[:0])


def moe_args(**over):
    a = dict(x=P, ldx=64, router=P, wgu=P, sgu=P, wd=P, sd=P, active=0, T=4, E=8, k=2, H=64, I=32, normalize=1,
             scale=1.0, ids=P, weights=P, out=P, workspace=P, workspace_bytes=BIG)
    a.update(over)
    return tuple(a.values())


@pytest.mark.parametrize("over,code", [
    (dict(x=0), -1), (dict(wgu=0), -1), (dict(sgu=0), -1), (dict(wd=0), -1), (dict(sd=0), -1), (dict(ids=0), -1),
    (dict(weights=0), -1), (dict(out=0), -1),
    (dict(T=0), -2), (dict(T=65), -2), (dict(E=0), -2), (dict(E=257), -2), (dict(k=0), -2), (dict(k=9), -2),
    (dict(E=32, k=17), -2), (dict(H=48), -2), (dict(H=0), -2), (dict(I=16), -2), (dict(I=65568), -2),
    (dict(ldx=63), -2), (dict(ldx=68), -2),
    (dict(x=P + 8), -3), (dict(router=P + 2), -3), (dict(wgu=P + 4), -3), (dict(wd=P + 8), -3), (dict(out=P + 1), -3),
    (dict(ids=P + 2), -3), (dict(weights=P + 1), -3), (dict(sgu=P + 2), -3), (dict(sd=P + 1), -3),
    (dict(workspace=0), -6), (dict(workspace_bytes=64), -6), (dict(workspace=P + 128), -6),
])
def test_moe_host_checks(over, code):
    assert mxw.mxw_moe_layer(*moe_args(**over)) == code


def test_moe_workspace_size():
    assert mxw.moe_workspace_size(64, 256, 8, 2048, 1408) >= 64 * 8 * 1408 * 2
    with pytest.raises(mxw.MxwError):
        mxw.moe_workspace_size(65, 8, 2, 64, 32)


def test_moe_python_face_validates():
    u8 = torch.uint8
    a = dict(x=torch.zeros((4, 64), dtype=torch.bfloat16), router=torch.zeros((8, 64), dtype=torch.bfloat16),
             wgu=torch.zeros((8, 64, 64), dtype=u8), sgu=torch.zeros((8, 64, 2), dtype=u8),
             wd=torch.zeros((8, 64, 32), dtype=u8), sd=torch.zeros((8, 64, 1), dtype=u8), top_k=2)
    ids, w = torch.zeros((4, 2), dtype=torch.int32), torch.zeros((4, 2))
    for error, over in ((ValueError, {}),                                   # CPU tensors: no host fallback
                        (TypeError, dict(x=a["x"].float())), (TypeError, dict(wgu=a["wgu"].to(torch.int8))),
                        (ValueError, dict(sgu=a["sgu"][..., :1])), (ValueError, dict(x=a["x"][:, :32])),
                        (ValueError, dict(router=a["router"][:7])), (ValueError, dict(router=None)),
                        (ValueError, dict(routing=(ids, w))),               # a router and a routing
                        (ValueError, dict(router=None, routing=(ids.long(), w))),
                        (ValueError, dict(router=None, routing=(ids[:, :1], w))),
                        (ValueError, dict(active=torch.zeros(3, dtype=torch.bool)))):
        with pytest.raises(error):
            mxw.moe_layer(**dict(a, **over))
