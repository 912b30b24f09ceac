"""MI355X-native MXFP8 ragged grouped GEMMs.

    out = wgrad(A, sA, B, sB, offs)        # bf16 [E, N, K]
    out = wgrad(..., plain=True)           # the entry point that takes no workspace
    out = wgrad_bf16(A, B, offs)           # bf16 [E, N, K] from bf16 operands
    out = fwd(A, sA, B, sB, offs)          # bf16 [R, N]
    q, s = quantize_tokens(x, offs)        # MXFP8 operand [H, M] from bf16 [M, H]

    update = orthogonalize(out)            # Newton-Schulz on every expert's gradient
    loss, dx, dw = vocab_cross_entropy(x, w, targets)   # over a large vocabulary
    y, ids, weights = moe_layer(x, router, wgu, sgu, wd, sd, top_k)   # a few tokens

    plan = sort_tokens(ids, E)             # tokens grouped by expert: ends, counts, rows
    xs, q, s = dispatch_tokens(x, plan, mxfp8=True)      # to their rows, bf16 and MXFP8
    out = combine_tokens(y, plan, weights)               # and back
    dy, dweights = combine_tokens_grad(dout, y, plan, weights)
    q, s = quantize_rows(x)                # MXFP8 rows, fwd's operands
    norm = clip_grad_norm(grads, 1.0)      # many tensors, in place
    logits = linear_4bit(x, codes, scales) # a few tokens, 4-bit weights

The first group computes, for every expert g (blog "Ragged MXFP8 Weight Gradients: A FlyDSL
Grouped GEMM on MI355X", section 1),

    dW[g] = dY[g]^T X[g]   over expert g's tokens [offs[g-1], offs[g])

from MXFP8 operands A = dY^T [N, M] and B = X^T [K, M] (E4M3 codes, token axis
contiguous) with E8M0 scale planes sA [N, M/32] and sB [K, M/32]; and the
row-ragged GEMM of the same layer (forward and data gradient):

    out[m] = A[m] B[g]^T   for the rows m of expert g, contraction over C

from A [R, C] and B [E, N, C] (contraction innermost, 32-element E8M0 blocks
along it); the same weight gradient on plain bf16 operands A = dY^T [N, M],
B = X^T [K, M] (the XLA blog's "contracting" ragged dot); and the token-axis
quantiser that makes the weight gradient's
operands from bf16 activations / gradients.  The second group is what stands
around those products when such a layer is trained and served: the optimiser's
orthogonalised update of the experts' weights, the loss that the gradients
start from, and the layer for single tokens and small batches (each described
at its function).  The third moves tokens between their own order and the experts'
rows with the gradients of that, makes row-wise operands, clips gradients, and has the
dense products of generation on 4-bit weights.  Everything
runs in the HIP library ``lib/libmxfp8_wgrad.so`` (C ABI in
``include/mxfp8_wgrad.h``); this module only checks tensor metadata and passes
device pointers and the current stream.  There is no fallback: if the library
is missing, or the device is not a gfx950, calls raise.

The weight gradients have two entry points each.  mxfp8_wgrad_grouped (and
bf16_wgrad_grouped) touch no memory but their operands and output: one
workgroup per (expert, output tile).  The _ws variants take a caller-owned
workspace (sized by mxfp8_wgrad_workspace_size) for column mode and the
scale pre-shuffle.  wgrad() and wgrad_bf16() use the _ws variants unless
plain=True, taking the workspace from torch's caching allocator on the
stream the call runs on (or from `workspace`, a uint8 device tensor).
"""
import array
import collections
import ctypes
import functools
import os

import torch

from .build import LIB as _LIB_PATH

__all__ = ["wgrad", "mxfp8_wgrad_grouped", "mxfp8_wgrad_grouped_ws", "mxfp8_wgrad_grouped_noalloc", "workspace_size", "wgrad_bf16",
           "bf16_wgrad_grouped", "bf16_wgrad_grouped_ws", "bf16_workspace_size", "grid_size", "columns",
           "scale_shuffle", "tail_split", "fwd", "mxfp8_grouped_fwd", "fwd_grid_size", "quantize_tokens", "mxfp8_quantize_tokens",
           "orthogonalize", "mxw_orthogonalize", "orthogonalize_workspace_size",
           "vocab_cross_entropy", "mxw_vocab_loss", "vocab_loss_workspace_size",
           "moe_layer", "mxw_moe_layer", "moe_workspace_size",
           "TokenPlan", "sort_tokens", "mxw_sort_tokens", "sort_workspace_size", "token_rows",
           "dispatch_tokens", "mxw_dispatch_tokens", "combine_tokens", "mxw_combine_tokens",
           "combine_tokens_grad", "mxw_combine_tokens_grad", "quantize_rows", "mxw_quantize_rows",
           "clip_grad_norm", "grad_norm", "mxw_clip_grads", "clip_workspace_size", "linear_4bit", "mxw_linear_4bit",
           "strerror", "version", "library_path", "MxwError"]

_lib = None


class MxwError(RuntimeError):
    pass


def library_path():
    return _LIB_PATH


def _load():
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(_LIB_PATH):
        raise MxwError("HIP library not built: %s (run python -m mxfp8_ragged_grouped_amd.build)" % _LIB_PATH)
    lib = ctypes.CDLL(_LIB_PATH)
    P = ctypes.c_void_p
    I = ctypes.c_int
    lib.mxfp8_wgrad_grouped.restype = I
    lib.mxfp8_wgrad_grouped.argtypes = [P, P, P, P, P, I, I, I, I, P, P]
    S = ctypes.c_size_t
    lib.mxfp8_wgrad_grouped_ws.restype = I
    lib.mxfp8_wgrad_grouped_ws.argtypes = [P, P, P, P, P, I, I, I, I, I, P, P, S, P]
    lib.mxfp8_wgrad_grouped_noalloc.restype = I
    lib.mxfp8_wgrad_grouped_noalloc.argtypes = [P, P, P, P, P, I, I, I, I, I, P, P]
    lib.mxfp8_wgrad_workspace_size.restype = ctypes.c_int64
    lib.mxfp8_wgrad_workspace_size.argtypes = [I, I, I, I, I]
    lib.bf16_wgrad_grouped.restype = I
    lib.bf16_wgrad_grouped.argtypes = [P, P, P, I, I, I, I, P, P]
    lib.bf16_wgrad_grouped_ws.restype = I
    lib.bf16_wgrad_grouped_ws.argtypes = [P, P, P, I, I, I, I, P, P, S, P]
    lib.bf16_wgrad_workspace_size.restype = ctypes.c_int64
    lib.bf16_wgrad_workspace_size.argtypes = [I, I, I, I]
    lib.mxw_grid_size.restype = ctypes.c_int64
    lib.mxw_grid_size.argtypes = [I, I, I]
    lib.mxw_strerror.restype = ctypes.c_char_p
    lib.mxw_strerror.argtypes = [I]
    lib.mxw_version.restype = I
    lib.mxw_version.argtypes = []
    lib.mxw_columns.restype = I
    lib.mxw_columns.argtypes = [I, I, I, I]
    lib.mxw_tail_split.restype = I
    lib.mxw_tail_split.argtypes = [I, I, I, I]
    lib.mxw_scale_shuffle.restype = I
    lib.mxw_scale_shuffle.argtypes = [I, I]
    lib.mxfp8_grouped_fwd.restype = I
    lib.mxfp8_grouped_fwd.argtypes = [P, P, P, P, P, I, I, I, I, P, P]
    lib.mxw_fwd_grid_size.restype = ctypes.c_int64
    lib.mxw_fwd_grid_size.argtypes = [I, I, I]
    lib.mxfp8_quantize_tokens.restype = I
    lib.mxfp8_quantize_tokens.argtypes = [P, P, I, I, I, I, P, P, P]
    L = ctypes.c_int64
    F = ctypes.c_float
    lib.mxw_orthogonalize.restype = I
    lib.mxw_orthogonalize.argtypes = [P, I, L, L, I, I, I, ctypes.POINTER(F), I, F, P, P, S, P]
    lib.mxw_orthogonalize_workspace_size.restype = L
    lib.mxw_orthogonalize_workspace_size.argtypes = [I, I, I]
    lib.mxw_vocab_loss.restype = I
    lib.mxw_vocab_loss.argtypes = [P, L, P, L, P, I, L, I, I, I, I, F, P, P, P, P, S, P]
    lib.mxw_vocab_loss_workspace_size.restype = L
    lib.mxw_vocab_loss_workspace_size.argtypes = [P, L, P, L, I, I, I, I]
    lib.mxw_moe_layer.restype = I
    lib.mxw_moe_layer.argtypes = [P, L, P, P, P, P, P, P, I, I, I, I, I, I, F, P, P, P, P, S, P]
    lib.mxw_moe_workspace_size.restype = L
    lib.mxw_moe_workspace_size.argtypes = [I, I, I, I, I]
    lib.mxw_token_rows.restype = L
    lib.mxw_token_rows.argtypes = [I, I, I, I]
    lib.mxw_sort_workspace_size.restype = L
    lib.mxw_sort_workspace_size.argtypes = [I, I, I]
    lib.mxw_sort_tokens.restype = I
    lib.mxw_sort_tokens.argtypes = [P, I, L, I, I, I, I, P, P, P, P, S, P]
    lib.mxw_dispatch_tokens.restype = I
    lib.mxw_dispatch_tokens.argtypes = [P, I, L, P, P, P, I, I, I, I, I, P, P, P, P]
    lib.mxw_combine_tokens.restype = I
    lib.mxw_combine_tokens.argtypes = [P, I, L, P, P, P, L, I, I, I, I, P, P]
    lib.mxw_combine_tokens_grad.restype = I
    lib.mxw_combine_tokens_grad.argtypes = [P, I, L, P, L, P, P, P, P, I, I, I, I, I, P, P, P, P, P]
    lib.mxw_quantize_rows.restype = I
    lib.mxw_quantize_rows.argtypes = [P, I, L, L, I, I, P, P, P]
    lib.mxw_clip_grads.restype = I
    lib.mxw_clip_grads.argtypes = [P, P, P, P, I, I, ctypes.c_double, ctypes.c_double, P, P, S, P]
    lib.mxw_clip_workspace_size.restype = L
    lib.mxw_clip_workspace_size.argtypes = [I]
    lib.mxw_linear_4bit.restype = I
    lib.mxw_linear_4bit.argtypes = [P, L, P, P, P, I, I, I, I, I, P, I, P]
    _lib = lib
    return lib


def strerror(code):
    return _load().mxw_strerror(int(code)).decode()


def version():
    return _load().mxw_version()


def grid_size(E, N, K):
    return int(_load().mxw_grid_size(int(E), int(N), int(K)))


def columns(E, M, N, K):
    """Columns of a column-mode launch for this shape on the current device
    (0: one workgroup per tile).  Raises MxwError on a status code."""
    rc = _load().mxw_columns(int(E), int(M), int(N), int(K))
    if rc < 0:
        raise MxwError("mxw_columns failed: %s" % strerror(rc))
    return rc


def tail_split(E, M, N, K):
    """Output tiles an MXFP8 weight-gradient call without column mode or
    pre-shuffle runs as two half tiles (same bits) on the current device."""
    rc = _load().mxw_tail_split(int(E), int(M), int(N), int(K))
    if rc < 0:
        raise MxwError("mxw_tail_split failed: %s" % strerror(rc))
    return rc


def scale_shuffle(E, M):
    """True if an MXFP8 weight-gradient call of (E, M) runs the scale
    pre-shuffle kernel before the main kernel."""
    rc = _load().mxw_scale_shuffle(int(E), int(M))
    if rc < 0:
        raise MxwError("mxw_scale_shuffle failed: %s" % strerror(rc))
    return bool(rc)


def mxfp8_wgrad_grouped(A, sA, B, sB, offs, E, M, N, K, out, stream=0):
    """Raw C-ABI call on device addresses (ints).  Returns the status code."""
    lib = _load()
    return lib.mxfp8_wgrad_grouped(A, sA, B, sB, offs, int(E), int(M), int(N), int(K), out, stream)


def mxfp8_wgrad_grouped_ws(A, sA, B, sB, offs, E, M, N, K, out, workspace, workspace_bytes, stream=0, ld=0):
    """Raw C-ABI call on device addresses (ints); ld = row stride (0: M).
    Returns the status code."""
    lib = _load()
    return lib.mxfp8_wgrad_grouped_ws(A, sA, B, sB, offs, int(E), int(M), int(ld), int(N), int(K), out, workspace,
                                      int(workspace_bytes), stream)


def mxfp8_wgrad_grouped_noalloc(A, sA, B, sB, offs, E, M, N, K, out, stream=0, ld=0):
    """Raw C-ABI call on device addresses (ints): the workspace entry on the
    library's static scratch (no allocation); ld = row stride (0: M).
    Returns the status code."""
    lib = _load()
    return lib.mxfp8_wgrad_grouped_noalloc(A, sA, B, sB, offs, int(E), int(M), int(ld), int(N), int(K), out, stream)


def workspace_size(E, M, N, K, ld=0):
    """Bytes of workspace mxfp8_wgrad_grouped_ws needs for this shape (row
    stride ld, 0 = M) on the current device (0: none).  Raises MxwError on a
    status code."""
    rc = _load().mxfp8_wgrad_workspace_size(int(E), int(M), int(ld), int(N), int(K))
    if rc < 0:
        raise MxwError("mxfp8_wgrad_workspace_size failed: %s" % strerror(rc))
    return int(rc)


def bf16_workspace_size(E, M, N, K):
    """Bytes of workspace bf16_wgrad_grouped_ws needs (0: none)."""
    rc = _load().bf16_wgrad_workspace_size(int(E), int(M), int(N), int(K))
    if rc < 0:
        raise MxwError("bf16_wgrad_workspace_size failed: %s" % strerror(rc))
    return int(rc)


def _workspace(need, dev, stream, workspace):
    """(pointer, bytes, tensor): the caller's workspace, or a fresh one from
    torch's caching allocator on `stream` (stream-ordered reuse)."""
    if workspace is not None:
        if workspace.device != dev or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on the same GPU")
        nbytes = workspace.numel() * workspace.element_size()
        if nbytes < need:
            raise ValueError("workspace holds %d bytes, the call needs %d" % (nbytes, need))
        return workspace.data_ptr(), nbytes, workspace
    if need == 0:
        return 0, 0, None
    with torch.cuda.stream(stream):
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    return ws.data_ptr(), need, ws


class _On:
    """The device and stream a call runs on (`with` makes the device current;
    switching to what is current already costs several microseconds, so it is
    left out).  handle: the stream as the library takes it; the current one's is
    asked for without making a Stream object, which takes 1.8 us."""

    __slots__ = ("handle", "_stream", "_other_stream", "_dev", "_switch")

    def __init__(self, dev, stream):
        index = dev.index
        current = torch._C._cuda_getCurrentRawStream(index)
        self.handle = current if stream is None else stream.cuda_stream
        self._stream = stream
        self._other_stream = self.handle != current
        self._dev = dev
        self._switch = None if torch._C._cuda_getDevice() == index else torch.cuda.device(dev)

    def __enter__(self):
        if self._switch is not None:
            self._switch.__enter__()
        return self

    def __exit__(self, *exc):
        if self._switch is not None:
            self._switch.__exit__(*exc)

    def new(self, shape, dtype):
        """A fresh tensor that belongs to the stream."""
        if self._other_stream:
            with torch.cuda.stream(self._stream):
                return torch.empty(shape, dtype=dtype, device=self._dev)
        # given its strides torch makes a tensor in 1.2 us instead of 1.6
        n = len(shape)
        if n == 2:
            return torch.empty_strided(shape, (shape[1], 1), dtype=dtype, device=self._dev)
        if n < 2:
            return torch.empty_strided(shape, (1,) * n, dtype=dtype, device=self._dev)
        return torch.empty(shape, dtype=dtype, device=self._dev)

    def workspace(self, need, workspace):
        if workspace is not None:
            return _workspace(need, self._dev, None, workspace)
        ws = self.new((need,), torch.uint8)
        return ws.data_ptr(), need, ws


def _as_u8(t, name):
    if t.dtype == torch.uint8:
        return t
    if t.dtype == getattr(torch, "float8_e4m3fn", None) and name in ("A", "B"):
        return t.view(torch.uint8)
    raise TypeError("%s must be uint8 (or float8_e4m3fn for data), got %s" % (name, t.dtype))


def _row_stride(t, name):
    if t.dim() != 2 or t.stride(1) != 1 or t.stride(0) < t.shape[1]:
        raise ValueError("%s must be a 2-D tensor with unit column stride and rows at least a row apart" % name)
    return t.stride(0)


def wgrad(A, sA, B, sB, offs, out=None, stream=None, workspace=None, plain=False):
    """dW [E, N, K] bf16 from MXFP8 operands (see module docstring).

    A: [N, M] uint8/float8_e4m3fn, sA: [N, M/32] uint8, B: [K, M], sB: [K, M/32],
    offs: [E] int32 cumulative expert ends, all on one CUDA(HIP) device.  A and
    B may be row-strided views ([:, :M] of [rows, ld] buffers, the same ld for
    both, and sA, sB then with row stride ld / 32): the workspace entry reads
    that layout (see mxfp8_wgrad_grouped_ws); the other tensors are
    contiguous.  `out` (optional) is a contiguous bf16 [E, N, K] tensor that is
    fully overwritten.  Runs on `stream` (default: the current stream) and does
    not synchronise.  plain=True calls mxfp8_wgrad_grouped (no workspace);
    otherwise mxfp8_wgrad_grouped_ws with `workspace` (a contiguous device
    tensor of at least workspace_size() bytes) or one taken from torch's
    caching allocator on that stream.
    """
    A = _as_u8(A, "A")
    B = _as_u8(B, "B")
    sA = _as_u8(sA, "sA")
    sB = _as_u8(sB, "sB")
    if A.dim() != 2 or B.dim() != 2 or sA.dim() != 2 or sB.dim() != 2 or offs.dim() != 1:
        raise ValueError("A, sA, B, sB must be 2-D and offs 1-D")
    N, M = A.shape
    K = B.shape[0]
    E = offs.shape[0]
    if B.shape[1] != M or sA.shape != (N, M // 32) or sB.shape != (K, M // 32):
        raise ValueError("shape mismatch: A %s sA %s B %s sB %s" % (tuple(A.shape), tuple(sA.shape),
                                                                     tuple(B.shape), tuple(sB.shape)))
    if offs.dtype != torch.int32:
        raise TypeError("offs must be int32")
    dev = A.device
    for name, t in (("A", A), ("sA", sA), ("B", B), ("sB", sB), ("offs", offs)):
        if t.device != dev or dev.type != "cuda":
            raise ValueError("%s must be on the same GPU as A" % name)
    if not offs.is_contiguous():
        raise ValueError("offs must be contiguous")
    if M == 0:
        ld = 0  # no tokens: nothing is read, the stride is moot
    else:
        ld = _row_stride(A, "A")
        if _row_stride(B, "B") != ld or (ld % 32):
            raise ValueError("A and B must share one row stride, a multiple of 32 (got %d, %d)" % (ld, B.stride(0)))
        for name, t in (("sA", sA), ("sB", sB)):
            if _row_stride(t, name) != ld // 32:
                raise ValueError("%s rows must be ld / 32 = %d bytes apart" % (name, ld // 32))
    if plain and ld not in (0, M):
        raise ValueError("the entry point without a workspace takes contiguous operands (row stride M)")
    if out is None:
        out = torch.empty((E, N, K), dtype=torch.bfloat16, device=dev)
    elif out.dtype != torch.bfloat16 or tuple(out.shape) != (E, N, K) or not out.is_contiguous() or out.device != dev:
        raise ValueError("out must be a contiguous bf16 [E, N, K] tensor on the same device")
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    # with no tokens no operand byte is read (every window is empty and the
    # kernel writes zeros), but torch gives empty tensors NULL addresses
    ptrs = [t.data_ptr() if M else out.data_ptr() for t in (A, sA, B, sB)]
    with torch.cuda.device(dev):
        if plain:
            rc = mxfp8_wgrad_grouped(*ptrs, offs.data_ptr(), E, M, N, K, out.data_ptr(), stream.cuda_stream)
        else:
            wp, wb, ws = _workspace(workspace_size(E, M, N, K, ld), dev, stream, workspace)
            rc = mxfp8_wgrad_grouped_ws(*ptrs, offs.data_ptr(), E, M, N, K, out.data_ptr(), wp, wb,
                                        stream.cuda_stream, ld=ld)
            del ws
    if rc != 0:
        raise MxwError("mxfp8_wgrad_grouped%s failed (%d): %s" % ("" if plain else "_ws", rc, strerror(rc)))
    return out


def bf16_wgrad_grouped(A, B, offs, E, M, N, K, out, stream=0):
    """Raw C-ABI call on device addresses (ints).  Returns the status code."""
    lib = _load()
    return lib.bf16_wgrad_grouped(A, B, offs, int(E), int(M), int(N), int(K), out, stream)


def bf16_wgrad_grouped_ws(A, B, offs, E, M, N, K, out, workspace, workspace_bytes, stream=0):
    """Raw C-ABI call on device addresses (ints).  Returns the status code."""
    lib = _load()
    return lib.bf16_wgrad_grouped_ws(A, B, offs, int(E), int(M), int(N), int(K), out, workspace,
                                     int(workspace_bytes), stream)


def wgrad_bf16(A, B, offs, out=None, stream=None, workspace=None, plain=False):
    """dW [E, N, K] bf16 from bf16 operands: dW[g] = A[:, win_g] B[:, win_g]^T.

    A: [N, M] and B: [K, M] bfloat16 (token axis contiguous), offs: [E] int32
    cumulative expert ends (multiples of 16), all contiguous on one GPU.
    `out` (optional) is a contiguous bf16 [E, N, K] tensor that is fully
    overwritten.  Runs on `stream` (default: the current stream) and does not
    synchronise.  plain / workspace: as for wgrad().
    """
    if A.dtype != torch.bfloat16 or B.dtype != torch.bfloat16:
        raise TypeError("A and B must be bfloat16")
    if A.dim() != 2 or B.dim() != 2 or offs.dim() != 1:
        raise ValueError("A, B must be 2-D and offs 1-D")
    N, M = A.shape
    K = B.shape[0]
    E = offs.shape[0]
    if B.shape[1] != M:
        raise ValueError("shape mismatch: A %s B %s" % (tuple(A.shape), tuple(B.shape)))
    if offs.dtype != torch.int32:
        raise TypeError("offs must be int32")
    dev = A.device
    for name, t in (("A", A), ("B", B), ("offs", offs)):
        if t.device != dev or dev.type != "cuda":
            raise ValueError("%s must be on the same GPU as A" % name)
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
    if out is None:
        out = torch.empty((E, N, K), dtype=torch.bfloat16, device=dev)
    elif out.dtype != torch.bfloat16 or tuple(out.shape) != (E, N, K) or not out.is_contiguous() or out.device != dev:
        raise ValueError("out must be a contiguous bf16 [E, N, K] tensor on the same device")
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    with torch.cuda.device(dev):
        if plain:
            rc = bf16_wgrad_grouped(A.data_ptr(), B.data_ptr(), offs.data_ptr(), E, M, N, K, out.data_ptr(),
                                    stream.cuda_stream)
        else:
            wp, wb, ws = _workspace(bf16_workspace_size(E, M, N, K), dev, stream, workspace)
            rc = bf16_wgrad_grouped_ws(A.data_ptr(), B.data_ptr(), offs.data_ptr(), E, M, N, K, out.data_ptr(),
                                       wp, wb, stream.cuda_stream)
            del ws
    if rc != 0:
        raise MxwError("bf16_wgrad_grouped%s failed (%d): %s" % ("" if plain else "_ws", rc, strerror(rc)))
    return out


def fwd_grid_size(E, R, N):
    return int(_load().mxw_fwd_grid_size(int(E), int(R), int(N)))


def mxfp8_grouped_fwd(A, sA, B, sB, offs, E, R, C, N, out, stream=0):
    """Raw C-ABI call on device addresses (ints).  Returns the status code."""
    lib = _load()
    return lib.mxfp8_grouped_fwd(A, sA, B, sB, offs, int(E), int(R), int(C), int(N), out, stream)


def fwd(A, sA, B, sB, offs, out=None, stream=None):
    """Row-ragged grouped GEMM, bf16 [R, N]: out[m] = A[m] . B[g]^T for the
    rows m of expert g (forward: A = activations, B = weights; data gradient:
    A = output gradient, B = the weights quantized along the other axis).

    A: [R, C] uint8/float8_e4m3fn, sA: [R, C/32] uint8, B: [E, N, C],
    sB: [E, N, C/32], offs: [E] int32 cumulative row ends, all contiguous on
    one GPU.  Rows past offs[E-1] are not written (a new `out` leaves them
    uninitialised).  Runs on `stream` (default: the current stream) and does
    not synchronise.
    """
    A = _as_u8(A, "A")
    B = _as_u8(B, "B")
    sA = _as_u8(sA, "sA")
    sB = _as_u8(sB, "sB")
    if A.dim() != 2 or sA.dim() != 2 or B.dim() != 3 or sB.dim() != 3 or offs.dim() != 1:
        raise ValueError("A, sA must be 2-D, B, sB 3-D and offs 1-D")
    R, C = A.shape
    E, N, C2 = B.shape
    if C2 != C or sA.shape != (R, C // 32) or sB.shape != (E, N, C // 32) or offs.shape[0] != E:
        raise ValueError("shape mismatch: A %s sA %s B %s sB %s offs %s" % (
            tuple(A.shape), tuple(sA.shape), tuple(B.shape), tuple(sB.shape), tuple(offs.shape)))
    if offs.dtype != torch.int32:
        raise TypeError("offs must be int32")
    dev = A.device
    for name, t in (("A", A), ("sA", sA), ("B", B), ("sB", sB), ("offs", offs)):
        if t.device != dev or dev.type != "cuda":
            raise ValueError("%s must be on the same GPU as A" % name)
        if not t.is_contiguous():
            raise ValueError("%s must be contiguous" % name)
    if out is None:
        out = torch.empty((R, N), dtype=torch.bfloat16, device=dev)
    elif out.dtype != torch.bfloat16 or tuple(out.shape) != (R, N) or not out.is_contiguous() or out.device != dev:
        raise ValueError("out must be a contiguous bf16 [R, N] tensor on the same device")
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    with torch.cuda.device(dev):
        rc = mxfp8_grouped_fwd(A.data_ptr(), sA.data_ptr(), B.data_ptr(), sB.data_ptr(), offs.data_ptr(),
                               E, R, C, N, out.data_ptr(), stream.cuda_stream)
    if rc != 0:
        raise MxwError("mxfp8_grouped_fwd failed (%d): %s" % (rc, strerror(rc)))
    return out


def mxfp8_quantize_tokens(x, offs, E, M, H, q, s, stream=0, ld=0):
    """Raw C-ABI call on device addresses (ints; offs may be 0; ld = row stride
    of q, 0 for M).  Returns the status code."""
    return _load().mxfp8_quantize_tokens(x, offs, int(E), int(M), int(ld), int(H), q, s, stream)


def quantize_tokens(x, offs=None, q=None, s=None, stream=None, ld=None):
    """Token-axis MXFP8 quantisation of bf16 x [M, H] -> (codes uint8 [H, M],
    scales uint8 [H, M/32]), the weight gradient's operand layout.  Tokens at
    or past offs[-1] (all tokens are used when offs is None) become code 0.
    With ld (a multiple of 32, >= M) the codes and scales are written into
    [H, ld] and [H, ld/32] buffers and returned as their [:, :M] and
    [:, :M/32] views (the padded rows mxfp8_wgrad_grouped_ws reads best);
    the padding columns are not written.  Runs on `stream` (default: the
    current stream) and does not synchronise."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_contiguous() or x.device.type != "cuda":
        raise ValueError("x must be a contiguous 2-D bf16 tensor on the GPU")
    M, H = x.shape
    dev = x.device
    if offs is not None:
        if offs.dtype != torch.int32 or offs.dim() != 1 or offs.device != dev or not offs.is_contiguous():
            raise ValueError("offs must be a contiguous int32 vector on the same GPU")
    ld = M if ld is None else int(ld)
    if ld < M or ld % 32:
        raise ValueError("ld must be a multiple of 32 and at least M")
    if q is None:
        q = torch.empty((H, ld), dtype=torch.uint8, device=dev)[:, :M]
    if s is None:
        s = torch.empty((H, ld // 32), dtype=torch.uint8, device=dev)[:, :M // 32]
    if tuple(q.shape) != (H, M) or q.dtype != torch.uint8 or q.device != dev or (M and q.stride() != (ld, 1)):
        raise ValueError("q must be a uint8 [H, M] tensor with row stride ld on the same GPU")
    if tuple(s.shape) != (H, M // 32) or s.dtype != torch.uint8 or s.device != dev or (
            M and (s.stride(0) != ld // 32 or s.stride(1) != 1)):
        raise ValueError("s must be a uint8 [H, M/32] tensor with row stride ld / 32 on the same GPU")
    if stream is None:
        stream = torch.cuda.current_stream(dev)
    with torch.cuda.device(dev):
        rc = mxfp8_quantize_tokens(x.data_ptr(), 0 if offs is None else offs.data_ptr(),
                                   1 if offs is None else offs.shape[0], M, H, q.data_ptr(), s.data_ptr(),
                                   stream.cuda_stream, ld=ld)
    if rc != 0:
        raise MxwError("mxfp8_quantize_tokens failed (%d): %s" % (rc, strerror(rc)))
    return q, s


def mxw_orthogonalize(G, dtype, expert_stride, row_stride, E, N, K, coeffs, eps, out, workspace, workspace_bytes,
                      stream=0):
    """Raw C-ABI call on device addresses (ints); coeffs: a flat sequence of
    3 * steps numbers; dtype: 0 bf16, 1 float32.  Returns the status code."""
    host = (ctypes.c_float * max(len(coeffs), 1))(*coeffs)
    return _load().mxw_orthogonalize(G, int(dtype), int(expert_stride), int(row_stride), int(E), int(N), int(K), host,
                                     len(coeffs) // 3, float(eps), out, workspace, int(workspace_bytes), stream)


def orthogonalize_workspace_size(E, N, K):
    """Bytes of workspace orthogonalize needs.  Raises MxwError on a status code."""
    rc = _load().mxw_orthogonalize_workspace_size(int(E), int(N), int(K))
    if rc < 0:
        raise MxwError("mxw_orthogonalize_workspace_size failed: %s" % strerror(rc))
    return int(rc)


def orthogonalize(G, out=None, steps=5, coeffs=(3.4445, -4.7750, 2.0315), eps=1e-7, stream=None, workspace=None):
    """The orthogonalised update of a stack of gradients (or momenta), bf16:
    for every matrix of G, X = G / (|G|_F + eps), then `steps` times
    X <- a X + (b S + c S S) X with S = X X^T (on X^T where it is taller than
    wide), which drives the singular values to about 1.

    G: bf16 or float32 [E, N, K] (as wgrad returns it) or [N, K], any sizes,
    the last axis contiguous, other strides free.  coeffs: (a, b, c), or one
    such triple per step.  `out` (optional) is a contiguous bf16 tensor of G's
    shape, fully overwritten.  A zero matrix gives zeros.  No matrix's result
    depends on another's values; its last bits can depend on how many there are
    (a long side of few matrices is summed in parts).  Runs on `stream`
    (default: the current stream) and does not synchronise; `workspace`: a
    uint8 device tensor of orthogonalize_workspace_size() bytes (default: from
    torch's caching allocator on that stream)."""
    if G.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("G must be bfloat16 or float32, got %s" % G.dtype)
    if G.dim() not in (2, 3) or 0 in G.shape:
        raise ValueError("G must be [E, N, K] or [N, K] with no empty axis, got %s" % (tuple(G.shape),))
    dev = G.device
    if dev.type != "cuda":
        raise ValueError("G must be on the GPU")
    E, N, K = G.shape if G.dim() == 3 else (1,) + tuple(G.shape)
    if K > 1 and G.stride(-1) != 1:
        raise ValueError("G's last axis must be contiguous")
    rs = G.stride(-2) if N > 1 else K
    es = G.stride(0) if G.dim() == 3 and E > 1 else 0
    if rs < K:
        raise ValueError("G's rows must be at least a row apart")
    coeffs = list(coeffs)
    steps = int(steps)
    if len(coeffs) == 3 and not any(hasattr(c, "__len__") for c in coeffs):
        coeffs = [coeffs] * steps
    if steps < 1 or len(coeffs) != steps or any(len(c) != 3 for c in coeffs):
        raise ValueError("coeffs must be one (a, b, c) or one for each of the steps")
    on = _On(dev, stream)
    if out is None:
        out = on.new(G.shape, torch.bfloat16)
    elif out.dtype != torch.bfloat16 or out.shape != G.shape or not out.is_contiguous() or out.device != dev:
        raise ValueError("out must be a contiguous bf16 tensor of G's shape on the same device")
    with on:
        wp, wb, ws = on.workspace(orthogonalize_workspace_size(E, N, K), workspace)
        rc = mxw_orthogonalize(G.data_ptr(), 0 if G.dtype == torch.bfloat16 else 1, es, rs, E, N, K,
                               [float(v) for c in coeffs for v in c], eps, out.data_ptr(), wp, wb, on.handle)
        del ws
    if rc != 0:
        raise MxwError("mxw_orthogonalize failed (%d): %s" % (rc, strerror(rc)))
    return out


def mxw_vocab_loss(x, ldx, w, ldw, targets, target_bytes, ignore_index, T, H, V, reduction, grad_scale, loss, dx, dw,
                   workspace, workspace_bytes, stream=0):
    """Raw C-ABI call on device addresses (ints; dx, dw may be 0); reduction:
    0 none, 1 mean, 2 sum.  Returns the status code."""
    return _load().mxw_vocab_loss(x, int(ldx), w, int(ldw), targets, int(target_bytes), int(ignore_index), int(T),
                                  int(H), int(V), int(reduction), float(grad_scale), loss, dx, dw, workspace,
                                  int(workspace_bytes), stream)


def vocab_loss_workspace_size(x, ldx, w, ldw, T, H, V, grads=3):
    """Bytes of workspace mxw_vocab_loss needs (x, w: device addresses; grads:
    1 for dx, plus 2 for dw, plus 8 for the size without room for the logits).
    Raises MxwError on a status code."""
    rc = _load().mxw_vocab_loss_workspace_size(x, int(ldx), w, int(ldw), int(T), int(H), int(V), int(grads))
    if rc < 0:
        raise MxwError("mxw_vocab_loss_workspace_size failed: %s" % strerror(rc))
    return int(rc)


_REDUCTIONS = {"none": 0, "mean": 1, "sum": 2}


def vocab_cross_entropy(x, w, targets, ignore_index=-100, reduction="mean", grads=True, grad_scale=1.0, dx=None,
                        dw=None, stream=None, workspace=None, keep_logits=True):
    """Softmax cross entropy of hidden states x [T, H] against the vocabulary
    w [V, H] (both bf16, last axis contiguous, rows any stride apart) in bounded
    memory: (loss, dx, dw), or loss alone with grads=False.

    targets: int32 or int64 [T]; tokens whose target is ignore_index have loss
    0 and no gradient, whatever their x holds.  reduction: "mean" over the tokens that count, "sum"
    (loss: a float32 scalar tensor), or "none" (loss: float32 [T]).  dx [T, H]
    and dw [V, H], bf16, are the gradients of grad_scale times the reduced loss
    (of the sum, for "none"); contiguous tensors may be passed for them.  A
    target outside the vocabulary makes the loss NaN.  keep_logits: for the
    gradients the workspace holds the float32 logits if they take at most 4 GiB
    (64 MiB for H < 1024) and there is memory for them; else, or with False,
    they are made twice, which takes up to a quarter more time and gives the
    same bits.  Runs on `stream`
    (default: the current stream) and does not synchronise; `workspace`: a
    uint8 device tensor of vocab_loss_workspace_size() bytes (default: from
    torch's caching allocator on that stream)."""
    if x.dtype != torch.bfloat16 or w.dtype != torch.bfloat16:
        raise TypeError("x and w must be bfloat16")
    if targets.dtype not in (torch.int32, torch.int64):
        raise TypeError("targets must be int32 or int64")
    if reduction not in _REDUCTIONS:
        raise ValueError("reduction must be 'mean', 'sum' or 'none'")
    if x.dim() != 2 or w.dim() != 2 or targets.dim() != 1:
        raise ValueError("x, w must be 2-D and targets 1-D")
    T, H = x.shape
    V = w.shape[0]
    if w.shape[1] != H or targets.shape[0] != T or 0 in (T, H, V):
        raise ValueError("shape mismatch: x %s w %s targets %s" % (tuple(x.shape), tuple(w.shape),
                                                                   tuple(targets.shape)))
    dev = x.device
    for name, t in (("x", x), ("w", w), ("targets", targets)):
        if t.device != dev or dev.type != "cuda":
            raise ValueError("%s must be on the same GPU as x" % name)
    strides = []
    for name, t in (("x", x), ("w", w)):
        if (H > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < H):
            raise ValueError("%s must have a contiguous last axis and rows at least a row apart" % name)
        strides.append(t.stride(0) if t.shape[0] > 1 else H)
    if T > 1 and targets.stride(0) != 1:
        raise ValueError("targets must be contiguous")
    if not grads and (dx is not None or dw is not None):
        raise ValueError("dx and dw are outputs of grads=True")
    on = _On(dev, stream)
    for name, t, shape in (("dx", dx, (T, H)), ("dw", dw, (V, H))):
        if t is not None and (t.dtype != torch.bfloat16 or tuple(t.shape) != shape or not t.is_contiguous()
                              or t.device != dev):
            raise ValueError("%s must be a contiguous bf16 %s tensor on the same device" % (name, list(shape)))
    if grads:
        dx = on.new((T, H), torch.bfloat16) if dx is None else dx
        dw = on.new((V, H), torch.bfloat16) if dw is None else dw
    loss = on.new((T,) if reduction == "none" else (), torch.float32)
    with on:
        def size(which):
            return vocab_loss_workspace_size(x.data_ptr(), strides[0], w.data_ptr(), strides[1], T, H, V, which)

        need = size((3 if keep_logits else 11) if grads else 0)
        try:
            wp, _, ws = on.workspace(need, workspace)
        except torch.OutOfMemoryError:
            if not grads or not keep_logits:
                raise
            need = size(11)
            wp, _, ws = on.workspace(need, None)
        rc = mxw_vocab_loss(x.data_ptr(), strides[0], w.data_ptr(), strides[1], targets.data_ptr(),
                            targets.element_size(), ignore_index, T, H, V, _REDUCTIONS[reduction], grad_scale,
                            loss.data_ptr(), dx.data_ptr() if grads else 0, dw.data_ptr() if grads else 0, wp, need,
                            on.handle)
        del ws
    if rc != 0:
        raise MxwError("mxw_vocab_loss failed (%d): %s" % (rc, strerror(rc)))
    return (loss, dx, dw) if grads else loss


def mxw_moe_layer(x, ldx, router, wgu, sgu, wd, sd, active, T, E, k, H, I, normalize, scale, ids, weights, out, workspace,
                  workspace_bytes, stream=0):
    """Raw C-ABI call on device addresses (ints; router and active may be 0).
    Returns the status code."""
    return _load().mxw_moe_layer(x, ldx, router, wgu, sgu, wd, sd, active, T, E, k, H, I, 1 if normalize else 0, scale,
                                 ids, weights, out, workspace, workspace_bytes, stream)


def moe_workspace_size(T, E, k, H, I):
    """Bytes of workspace moe_layer needs.  Raises MxwError on a status code."""
    rc = _load().mxw_moe_workspace_size(int(T), int(E), int(k), int(H), int(I))
    if rc < 0:
        raise MxwError("mxw_moe_workspace_size failed: %s" % strerror(rc))
    return int(rc)


def moe_layer(x, router, wgu, sgu, wd, sd, top_k, normalize=True, scale=1.0, active=None, routing=None, out=None,
              stream=None, workspace=None):
    """A whole mixture-of-experts layer for a few tokens (up to 64):
    (out [T, H] bf16, ids [T, top_k] int32, weights [T, top_k] float32).

    x: bf16 [T, H] (rows any multiple of 8 elements apart).  router: bf16
    [E, H]; each token goes to the top_k experts of the largest router logits
    (ties: the lower index), weighted by the softmax over all experts, divided
    by the chosen ones' sum if `normalize`, times `scale`.  Or router=None and
    routing=(ids, weights), contiguous int32 and float32 [T, top_k]; ids
    outside [0, E) are empty slots.  wgu, sgu: MXFP8 gate and up weights
    [E, 2 I, H] (codes uint8 or float8_e4m3fn; gate rows first) and
    [E, 2 I, H/32]; wd, sd: down weights [E, H, I] and [E, H, I/32]; an
    expert computes (silu(x Wg^T) * (x Wu^T)) Wd^T.  active: bool [T], False
    for tokens that are not there (out 0; with a router ids -1, weights 0).  Runs on
    `stream` (default: the current stream) and does not synchronise;
    `workspace`: a uint8 device tensor of moe_workspace_size() bytes (default:
    from torch's caching allocator on that stream)."""
    codes = getattr(torch, "float8_e4m3fn", None)
    if wgu.dtype == codes:
        wgu = wgu.view(torch.uint8)
    if wd.dtype == codes:
        wd = wd.view(torch.uint8)
    if x.dtype != torch.bfloat16:
        raise TypeError("x must be bfloat16")
    if not wgu.dtype == sgu.dtype == wd.dtype == sd.dtype == torch.uint8:
        raise TypeError("wgu, sgu, wd, sd must be uint8 (or float8_e4m3fn for codes)")
    dev = x.device
    if dev.type != "cuda":
        raise ValueError("x must be on the GPU")
    for name, t in (("wgu", wgu), ("sgu", sgu), ("wd", wd), ("sd", sd)):
        if t.dim() != 3 or t.device != dev or not t.is_contiguous():
            raise ValueError("%s must be 3-D, contiguous and on the same GPU as x" % name)
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with a contiguous last axis")
    T, H = x.shape
    E, H2, I = wd.shape
    if H2 != H or wgu.shape != (E, 2 * I, H) or sgu.shape != (E, 2 * I, H // 32) or sd.shape != (E, H, I // 32):
        raise ValueError("shape mismatch: x %s wgu %s sgu %s wd %s sd %s" % tuple(
            tuple(t.shape) for t in (x, wgu, sgu, wd, sd)))
    ldx = x.stride(0) if T > 1 else H
    if ldx < H:
        raise ValueError("x's rows must be at least a row apart")
    k = int(top_k)
    if (router is None) == (routing is None):
        raise ValueError("give a router or a routing, and not both")
    on = _On(dev, stream)
    if router is not None:
        if router.dtype != torch.bfloat16 or router.shape != (E, H) or router.device != dev or not router.is_contiguous():
            raise ValueError("router must be a contiguous bf16 [E, H] tensor on the same GPU as x")
        ids = on.new((T, k), torch.int32)
        weights = on.new((T, k), torch.float32)
    else:
        ids, weights = routing
        for name, t, kind in (("ids", ids, torch.int32), ("weights", weights, torch.float32)):
            if t.dtype != kind or t.shape != (T, k) or t.device != dev or not t.is_contiguous():
                raise ValueError("routing: %s must be a contiguous %s [T, top_k] tensor on the same GPU as x" % (name, kind))
    if active is not None and (active.dtype not in (torch.bool, torch.uint8) or active.shape != (T,) or
                               active.device != dev or not active.is_contiguous()):
        raise ValueError("active must be a contiguous bool [T] tensor on the same GPU as x")
    if out is None:
        out = on.new((T, H), torch.bfloat16)
    elif out.dtype != torch.bfloat16 or out.shape != (T, H) or not out.is_contiguous() or out.device != dev:
        raise ValueError("out must be a contiguous bf16 [T, H] tensor on the same device")
    with on:
        wp, wb, ws = on.workspace(moe_workspace_size(T, E, k, H, I), workspace)
        rc = mxw_moe_layer(x.data_ptr(), ldx, 0 if router is None else router.data_ptr(),
                           wgu.data_ptr(), sgu.data_ptr(), wd.data_ptr(), sd.data_ptr(),
                           0 if active is None else active.data_ptr(), T, E, k, H, I, normalize, scale, ids.data_ptr(),
                           weights.data_ptr(), out.data_ptr(), wp, wb, on.handle)
        del ws
    if rc != 0:
        raise MxwError("mxw_moe_layer failed (%d): %s" % (rc, strerror(rc)))
    return out, ids, weights


# ---- tokens to their experts' rows and back -----------------------------------

TokenPlan = collections.namedtuple("TokenPlan", "offs counts rows size")
TokenPlan.__doc__ = """Where sort_tokens puts every token: offs int32 [E], the cumulative ends of the
experts' runs of rows (as the grouped products take them); counts int32 [E], each
expert's choices; rows int32 [T, k], every choice's row, -1 for empty slots; size,
the rows that the runs fit in whatever the ids (a Python number)."""

_TYPES = {torch.bfloat16: 0, torch.float32: 1}


def _fits(*sizes):
    """ctypes would cut sizes past 32 bits without a word."""
    if max(sizes) > 0x7FFFFFFF or min(sizes) < -0x80000000:
        raise ValueError("sizes past 32 bits: %s" % (sizes,))


@functools.lru_cache(maxsize=1024)
def _sort_sizes(T, k, E, align):
    """Rows and workspace of a sort: functions of the sizes alone, and a call of each
    takes 0.5 us."""
    return token_rows(T, k, E, align), sort_workspace_size(T, k, E)


def token_rows(T, k, E, align=32):
    """Rows that T tokens' k choices among E experts fit in, each expert's run a
    multiple of align.  Raises MxwError if that is over 8,388,608."""
    _fits(int(T), int(k), int(E), int(align))
    rc = _load().mxw_token_rows(int(T), int(k), int(E), int(align))
    if rc < 0:
        raise MxwError("mxw_token_rows failed: %s" % strerror(rc))
    return int(rc)


def sort_workspace_size(T, k, E):
    """Bytes of workspace sort_tokens needs (0: none).  Raises MxwError on a
    status code."""
    _fits(int(T), int(k), int(E))
    rc = _load().mxw_sort_workspace_size(int(T), int(k), int(E))
    if rc < 0:
        raise MxwError("mxw_sort_workspace_size failed: %s" % strerror(rc))
    return int(rc)


def mxw_sort_tokens(ids, id_bytes, ld, T, k, E, align, offs, counts, rows, workspace, workspace_bytes, stream=0):
    """Raw C-ABI call on device addresses (ints).  Returns the status code."""
    return _load().mxw_sort_tokens(ids, id_bytes, ld, T, k, E, align, offs, counts, rows, workspace, workspace_bytes,
                                   stream)


def sort_tokens(ids, E, align=32, stream=None, workspace=None):
    """The rows that tokens go to when they are grouped by expert: a TokenPlan.

    ids: int32 or int64 [T, k] (rows any stride apart), each token's experts; an id
    outside [0, E) is an empty slot.  Choices keep their order (token, then choice)
    within an expert, and each expert's run is padded to a multiple of `align` (32: what
    wgrad needs; 16: wgrad_bf16).  Runs on `stream` (default: the current stream) and
    does not synchronise; `workspace`: a uint8 device tensor of sort_workspace_size()
    bytes (default: from torch's caching allocator on that stream)."""
    if ids.dtype not in (torch.int32, torch.int64):
        raise TypeError("ids must be int32 or int64, got %s" % ids.dtype)
    if ids.dim() != 2 or ids.shape[1] == 0:
        raise ValueError("ids must be [T, k], got %s" % (tuple(ids.shape),))
    dev = ids.device
    if dev.type != "cuda":
        raise ValueError("ids must be on the GPU")
    T, k = ids.shape
    if k > 1 and ids.stride(1) != 1 or T > 1 and ids.stride(0) < k:
        raise ValueError("ids must have a contiguous last axis and rows at least a row apart")
    E, align = int(E), int(align)
    _fits(T, k, E, align)
    size, need = _sort_sizes(T, k, E, align)
    on = _On(dev, stream)
    offs, counts, rows = on.new((E,), torch.int32), on.new((E,), torch.int32), on.new((T, k), torch.int32)
    with on:
        wp, wb, ws = on.workspace(need, workspace) if need else (0, 0, None)
        rc = mxw_sort_tokens(ids.data_ptr(), ids.element_size(), ids.stride(0) if T > 1 else k, T, k, E, align,
                             offs.data_ptr(), counts.data_ptr(), rows.data_ptr(), wp, wb, on.handle)
        del ws
    if rc != 0:
        raise MxwError("mxw_sort_tokens failed (%d): %s" % (rc, strerror(rc)))
    return TokenPlan(offs, counts, rows, size)


def _plan(plan, dev):
    """(offs, counts, rows, size, T, k, E) of a plan, checked."""
    offs, counts, rows, size = plan
    i32, index = torch.int32, dev.index
    if (rows.dtype is i32 and offs.dtype is i32 and counts.dtype is i32 and rows.is_contiguous() and offs.is_contiguous()
            and counts.is_contiguous() and rows.get_device() == offs.get_device() == counts.get_device() == index
            and rows.dim() == 2 and offs.dim() == 1 and counts.shape == offs.shape):
        T, k = rows.shape
        return offs, counts, rows, size, T, k, offs.shape[0]
    # what is wrong with it
    if rows.dim() != 2 or offs.dim() != 1 or counts.shape != offs.shape:
        raise ValueError("plan: offs and counts must be [E] and rows [T, k]")
    for name, t in (("offs", offs), ("counts", counts), ("rows", rows)):
        if t.dtype != torch.int32 or t.device != dev or not t.is_contiguous():
            raise ValueError("plan: %s must be a contiguous int32 tensor on the same GPU" % name)
    raise ValueError("plan must be on the same GPU")


def _matrix(t, name, rows, H=None, dtype=None, dev=None):
    """Row stride of a [rows, H] matrix with a contiguous last axis, checked."""
    if t.is_contiguous() and t.dim() == 2 and t.is_cuda and (t.dtype is dtype if dtype is not None else t.dtype in _TYPES):
        shape = t.shape
        if shape[1] and rows in (None, shape[0]) and H in (None, shape[1]) and (dev is None or t.get_device() == dev.index):
            return shape[1]
    if t.dtype not in _TYPES or (dtype is not None and t.dtype != dtype):
        raise TypeError("%s must be %s, got %s" % (name, "bfloat16 or float32" if dtype is None else dtype, t.dtype))
    if t.dim() != 2 or (rows is not None and t.shape[0] != rows) or (H is not None and t.shape[1] != H) or not t.shape[1]:
        raise ValueError("%s must be [%s, %s], got %s" % (name, "rows" if rows is None else rows, "H" if H is None else H,
                                                          tuple(t.shape)))
    if t.device.type != "cuda" or (dev is not None and t.device != dev):
        raise ValueError("%s must be on %s" % (name, "the GPU" if dev is None else dev))
    if (t.shape[1] > 1 and t.stride(1) != 1) or (t.shape[0] > 1 and t.stride(0) < t.shape[1]):
        raise ValueError("%s must have a contiguous last axis and rows at least a row apart" % name)
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _output(t, name, shape, dtype, on):
    """`t` checked, or a new tensor."""
    if t is None:
        return on.new(shape, dtype)
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != on._dev.index:
        raise ValueError("%s must be a contiguous %s %s tensor on the same device" % (name, dtype, list(shape)))
    return t


def _codes_output(q, s, R, H, on):
    if q is not None and q.dtype == getattr(torch, "float8_e4m3fn", None):
        q = q.view(torch.uint8)
    if H % 32:
        raise ValueError("MXFP8 rows need a multiple of 32 columns, got %d" % H)
    return _output(q, "q", (R, H), torch.uint8, on), _output(s, "s", (R, H // 32), torch.uint8, on)


def mxw_dispatch_tokens(x, dtype, ldx, offs, counts, rows, T, k, E, H, R, xs, q, s, stream=0):
    """Raw C-ABI call on device addresses (ints; xs, or q and s, may be 0); dtype:
    0 bf16, 1 float32.  Returns the status code."""
    return _load().mxw_dispatch_tokens(x, dtype, ldx, offs, counts, rows, T, k, E, H, R, xs, q, s, stream)


def dispatch_tokens(x, plan, rows=True, mxfp8=False, out=None, q=None, s=None, stream=None):
    """Tokens x [T, H] (bf16 or float32, rows any stride apart) copied to the rows that
    a TokenPlan gives them: xs [R, H] of x's type, R = plan.size; with mxfp8=True
    (xs, codes uint8 [R, H], scales uint8 [R, H/32]), the codes being what fwd takes;
    with rows=False as well (codes, scales) alone.

    The padding rows of every expert become zeros; rows past the last run are left as
    they were (uninitialised in new tensors; the grouped products do not read them).
    `out`, `q` and `s` (optional) are contiguous tensors of any one number of rows:
    rows that they do not have are skipped.  They may not share memory with an input.
    The gradient with respect to x is combine_tokens(dxs, plan).  Runs on `stream` (default:
    the current stream) and does not synchronise."""
    ldx = _matrix(x, "x", None)
    dev = x.device
    offs, counts, where, R, T, k, E = _plan(plan, dev)
    H = x.shape[1]
    if x.shape[0] != T:
        raise ValueError("x has %d tokens, the plan %d" % (x.shape[0], T))
    if not rows and not mxfp8:
        raise ValueError("nothing to write: rows and mxfp8 are both False")
    if (out is not None and not rows) or ((q is not None or s is not None) and not mxfp8):
        raise ValueError("out is an output of rows=True, q and s are outputs of mxfp8=True")
    for t in (out, q, s):
        if t is not None and t.dim() == 2:
            R = t.shape[0]
    _fits(T, k, E, H, R)
    on = _On(dev, stream)
    if rows:
        out = _output(out, "out", (R, H), x.dtype, on)
    if mxfp8:
        q, s = _codes_output(q, s, R, H, on)
    with on:
        rc = mxw_dispatch_tokens(x.data_ptr(), _TYPES[x.dtype], ldx, offs.data_ptr(), counts.data_ptr(), where.data_ptr(),
                                 T, k, E, H, R, out.data_ptr() if rows else 0, q.data_ptr() if mxfp8 else 0,
                                 s.data_ptr() if mxfp8 else 0, on.handle) if T and R else 0
    if rc != 0:
        raise MxwError("mxw_dispatch_tokens failed (%d): %s" % (rc, strerror(rc)))
    return out if not mxfp8 else (out, q, s) if rows else (q, s)


def mxw_combine_tokens(y, dtype, ldy, rows, weights, residual, ldr, T, k, H, R, out, stream=0):
    """Raw C-ABI call on device addresses (ints; weights and residual may be 0);
    dtype: 0 bf16, 1 float32.  Returns the status code."""
    return _load().mxw_combine_tokens(y, dtype, ldy, rows, weights, residual, ldr, T, k, H, R, out, stream)


def _weights(weights, T, k, dev):
    if (weights.dtype is not torch.float32 or weights.shape != (T, k) or weights.get_device() != dev.index or
            not weights.is_contiguous()):
        raise ValueError("weights must be a contiguous float32 [T, k] tensor on the same GPU")


def combine_tokens(y, plan, weights=None, residual=None, out=None, stream=None):
    """The experts' rows y [R, H] (bf16 or float32, rows any stride apart) joined to
    tokens: out[t] = sum_j weights[t, j] y[plan.rows[t, j]] (+ residual[t]), [T, H] of
    y's type, summed in float32 in the order of j and rounded once.

    weights: float32 [T, k] (None: 1).  residual: [T, H] of y's type, rows any stride
    apart; `out` may be the residual itself.  Empty slots count nothing, whatever their
    weight holds.  Without weights it is the gradient of dispatch_tokens.  Runs on
    `stream` (default: the current stream) and does not synchronise."""
    ldy = _matrix(y, "y", None)
    dev = y.device
    offs, counts, rows, _, T, k, E = _plan(plan, dev)
    R, H = y.shape
    _fits(T, k, H, R)
    ldr = 0 if residual is None else _matrix(residual, "residual", T, H, y.dtype, dev)
    if weights is not None:
        _weights(weights, T, k, dev)
    on = _On(dev, stream)
    out = _output(out, "out", (T, H), y.dtype, on)
    with on:
        rc = mxw_combine_tokens(y.data_ptr(), _TYPES[y.dtype], ldy, rows.data_ptr(),
                                0 if weights is None else weights.data_ptr(),
                                0 if residual is None else residual.data_ptr(), ldr, T, k, H, R, out.data_ptr(),
                                on.handle) if T else 0
    if rc != 0:
        raise MxwError("mxw_combine_tokens failed (%d): %s" % (rc, strerror(rc)))
    return out


def mxw_combine_tokens_grad(dout, dtype, ldo, y, ldy, offs, counts, rows, weights, T, k, E, H, R, dy, q, s, dweights,
                            stream=0):
    """Raw C-ABI call on device addresses (ints; dy, q and s, dweights may be 0);
    dtype: 0 bf16, 1 float32.  Returns the status code."""
    return _load().mxw_combine_tokens_grad(dout, dtype, ldo, y, ldy, offs, counts, rows, weights, T, k, E, H, R, dy, q, s,
                                           dweights, stream)


def combine_tokens_grad(dout, y, plan, weights, rows=True, mxfp8=False, dy=None, q=None, s=None, stream=None):
    """The gradients of combine_tokens(y, plan, weights) from that of its output,
    dout [T, H] (rows any stride apart): (dy [R, H], dweights float32 [T, k]), with
    mxfp8=True (dy, codes, scales, dweights), the codes and scales being those of
    quantize_rows(dy), and with rows=False as well (codes, scales, dweights).

    dy[plan.rows[t, j]] = weights[t, j] dout[t] in dout's type; padding rows become
    zeros, rows past the last run are left as they were.  dweights[t, j] is the dot
    product of dout[t] and y[plan.rows[t, j]] in float32, 0 for empty slots.  The
    residual's gradient is dout.  `dy` may be y itself.  Runs on `stream` (default: the
    current stream) and does not synchronise."""
    ldo = _matrix(dout, "dout", None)
    dev = dout.device
    offs, counts, where, _, T, k, E = _plan(plan, dev)
    H = dout.shape[1]
    if dout.shape[0] != T:
        raise ValueError("dout has %d tokens, the plan %d" % (dout.shape[0], T))
    ldy = _matrix(y, "y", None, H, dout.dtype, dev)
    R = y.shape[0]
    _fits(T, k, E, H, R)
    _weights(weights, T, k, dev)
    if not rows and not mxfp8:
        raise ValueError("nothing to write: rows and mxfp8 are both False")
    if (dy is not None and not rows) or ((q is not None or s is not None) and not mxfp8):
        raise ValueError("dy is an output of rows=True, q and s are outputs of mxfp8=True")
    on = _On(dev, stream)
    dweights = torch.empty_like(weights) if stream is None else on.new((T, k), torch.float32)
    if rows:
        dy = _output(dy, "dy", (R, H), dout.dtype, on)
    if mxfp8:
        q, s = _codes_output(q, s, R, H, on)
    with on:
        rc = mxw_combine_tokens_grad(dout.data_ptr(), _TYPES[dout.dtype], ldo, y.data_ptr(), ldy, offs.data_ptr(),
                                     counts.data_ptr(), where.data_ptr(), weights.data_ptr(), T, k, E, H, R,
                                     dy.data_ptr() if rows and R else 0, q.data_ptr() if mxfp8 and R else 0,
                                     s.data_ptr() if mxfp8 and R else 0, dweights.data_ptr(), on.handle) if T else 0
    if rc != 0:
        raise MxwError("mxw_combine_tokens_grad failed (%d): %s" % (rc, strerror(rc)))
    return ((dy,) if rows else ()) + ((q, s) if mxfp8 else ()) + (dweights,)


# ---- row-wise operands --------------------------------------------------------

_FORMATS = {"mxfp8": 0, "mxfp4": 1}


def mxw_quantize_rows(x, dtype, ldx, R, C, format, q, s, stream=0):
    """Raw C-ABI call on device addresses (ints); dtype: 0 bf16, 1 float32; format:
    0 MXFP8, 1 MXFP4.  Returns the status code."""
    return _load().mxw_quantize_rows(x, dtype, ldx, R, C, format, q, s, stream)


def quantize_rows(x, format="mxfp8", q=None, s=None, stream=None):
    """MX quantisation of bf16 or float32 x [..., C] in blocks of 32 along the last
    axis: (codes, scales uint8 [..., C/32]), as fwd and moe_layer take their operands
    ("mxfp8": codes uint8 [..., C]) and linear_4bit its weights ("mxfp4": codes uint8
    [..., C/2], element 2 i in the low half of byte i).

    Scales and rounding are those of quantize_tokens (MXFP4: the same with the largest
    value 6); a block that holds an infinity or a NaN gets the NaN scale 255.  The last
    axis is contiguous and the rows one stride apart (a transposed weight's operand is
    quantize_tokens of the weight).  Runs on `stream` (default: the current stream) and
    does not synchronise."""
    if x.dtype not in _TYPES:
        raise TypeError("x must be bfloat16 or float32, got %s" % x.dtype)
    if format not in _FORMATS:
        raise ValueError("format must be 'mxfp8' or 'mxfp4'")
    if x.dim() < 1 or not x.is_cuda:
        raise ValueError("x must be a tensor of at least one axis on the GPU")
    shape = x.shape
    C = shape[-1]
    if C == 0 or C % 32:
        raise ValueError("x's last axis must be a multiple of 32, got %d" % C)
    if x.is_contiguous():
        R, ldx = x.numel() // C, C
    else:
        try:
            ldx = _matrix(x.view(-1, C), "x", None)
        except RuntimeError:
            raise ValueError("x's rows must be one stride apart") from None
        R = x.numel() // C
    _fits(C)
    on = _On(x.device, stream)
    if q is not None and q.dtype == getattr(torch, "float8_e4m3fn", None):
        q = q.view(torch.uint8)
    shape = tuple(shape)
    q = _output(q, "q", shape[:-1] + (C if format == "mxfp8" else C // 2,), torch.uint8, on)
    s = _output(s, "s", shape[:-1] + (C // 32,), torch.uint8, on)
    with on:
        rc = mxw_quantize_rows(x.data_ptr(), _TYPES[x.dtype], ldx, R, C, _FORMATS[format], q.data_ptr(), s.data_ptr(),
                               on.handle) if R else 0
    if rc != 0:
        raise MxwError("mxw_quantize_rows failed (%d): %s" % (rc, strerror(rc)))
    return q, s


# ---- gradients together -------------------------------------------------------

def clip_workspace_size(count):
    """Bytes of workspace clip_grad_norm and grad_norm need for so many tensors.
    Raises MxwError on a status code."""
    _fits(int(count))
    rc = _load().mxw_clip_workspace_size(int(count))
    if rc < 0:
        raise MxwError("mxw_clip_workspace_size failed: %s" % strerror(rc))
    return int(rc)


_clip_size = functools.lru_cache(maxsize=1024)(clip_workspace_size)


def mxw_clip_grads(grads, outs, sizes, types, norm_type, max_norm, eps, norm, workspace, workspace_bytes, stream=0):
    """Raw C-ABI call: lists of device addresses (outs None: the norm alone), element
    counts and types (0 bf16, 1 float32); norm_type: 2, or 0 for the largest magnitude.
    Returns the status code."""
    grads, sizes, types = array.array("Q", grads), array.array("q", sizes), array.array("i", types)
    outs = None if outs is None else array.array("Q", outs)
    return _load().mxw_clip_grads(grads.buffer_info()[0], None if outs is None else outs.buffer_info()[0],
                                  sizes.buffer_info()[0], types.buffer_info()[0], len(grads), norm_type, max_norm, eps,
                                  norm, workspace, workspace_bytes, stream)


def _dense(t):
    """Whether a tensor's elements fill its memory from its address on, in any order."""
    if t.is_contiguous():
        return True
    want = 1
    for size, stride in sorted(((n, d) for n, d in zip(t.shape, t.stride()) if n > 1), key=lambda a: a[1]):
        if stride != want:
            return False
        want *= size
    return True


def _grads(grads):
    return [grads] if isinstance(grads, torch.Tensor) else [g for g in grads if g is not None]


def _norm_call(grads, outs, max_norm, norm_type, eps, stream, workspace):
    if norm_type not in (2, float("inf")):
        raise ValueError("norm_type must be 2 or infinity")
    if not grads:
        raise ValueError("no gradients")
    dev = grads[0].device
    index = dev.index
    types = [_TYPES.get(g.dtype, -1) for g in grads]
    if -1 in types:
        raise TypeError("gradients must be bfloat16 or float32, got %s" % grads[types.index(-1)].dtype)
    if dev.type != "cuda" or any([g.get_device() != index for g in grads]):
        raise ValueError("gradients must be on one GPU")
    plain = all([g.is_contiguous() for g in grads])
    if not plain and not all(_dense(g) for g in grads):
        raise ValueError("gradients must fill their memory (contiguous or permuted axes)")
    if outs is not None and outs is not grads:
        outs = [outs] if isinstance(outs, torch.Tensor) else list(outs)
        if len(outs) != len(grads):
            raise ValueError("out must hold a tensor for every gradient")
        if any([o.dtype is not g.dtype or o.get_device() != index or o.shape != g.shape for g, o in zip(grads, outs)]) or not (
                plain and all([o.is_contiguous() for o in outs]) or all(o.stride() == g.stride() for g, o in zip(grads, outs))):
            raise ValueError("out must hold tensors of the gradients' types, shapes, strides and device")
    on = _On(dev, stream)
    norm = on.new((), torch.float32)
    with on:
        wp, wb, ws = on.workspace(_clip_size(len(grads)), workspace)
        rc = mxw_clip_grads([g.data_ptr() for g in grads], None if outs is None else [o.data_ptr() for o in outs],
                            [g.numel() for g in grads], types, 2 if norm_type == 2 else 0,
                            float(max_norm), float(eps), norm.data_ptr(), wp, wb, on.handle)
        del ws
    if rc != 0:
        raise MxwError("mxw_clip_grads failed (%d): %s" % (rc, strerror(rc)))
    return norm


def grad_norm(grads, norm_type=2.0, stream=None, workspace=None):
    """The norm of many gradients together, a float32 scalar tensor: the square root of
    the sum of all squares (in 64 bits), or the largest magnitude (norm_type infinity).

    grads: bf16 and float32 tensors on one GPU, any sizes (None is left out), each
    filling its memory.  Runs on `stream` (default: the current stream) and does not
    synchronise; `workspace`: a uint8 device tensor of clip_workspace_size() bytes
    (default: from torch's caching allocator on that stream)."""
    return _norm_call(_grads(grads), None, 0.0, norm_type, 0.0, stream, workspace)


def clip_grad_norm(grads, max_norm, norm_type=2.0, eps=1e-6, out=None, stream=None, workspace=None):
    """Gradients scaled by min(1, max_norm / (norm + eps)), norm = grad_norm(grads,
    norm_type), in place or into the tensors of `out` (one for every gradient, of its
    type, shape and strides).  Returns the norm before clipping.

    The factor and the product are float32; the product is then rounded to the gradient's
    type.  A NaN makes everything NaN; an infinity makes the norm infinite and the factor 0;
    where norm + eps is 0 the factor is 1.  No two gradients may share memory, nor a gradient
    and the workspace.  Arguments otherwise as grad_norm."""
    if not (max_norm >= 0.0 and eps >= 0.0):
        raise ValueError("max_norm and eps must not be negative")
    grads = _grads(grads)
    return _norm_call(grads, grads if out is None else out, max_norm, norm_type, eps, stream, workspace)


# ---- few tokens, 4-bit weights ------------------------------------------------

def mxw_linear_4bit(x, ldx, codes, scales, zeros, format, group, T, K, N, out, out_type, stream=0):
    """Raw C-ABI call on device addresses (ints; zeros may be 0); format: 1 MXFP4,
    2 integers; out_type: 0 bf16, 1 float32.  Returns the status code."""
    return _load().mxw_linear_4bit(x, ldx, codes, scales, zeros, format, group, T, K, N, out, out_type, stream)


def linear_4bit(x, codes, scales, zeros=None, dtype=torch.bfloat16, out=None, stream=None):
    """x [T, K] (bf16, up to 64 tokens, rows any multiple of 8 elements apart) times
    4-bit weights: out [T, N] = x W^T, bf16 or float32 (`dtype`).

    codes: uint8 [N, K/2], element 2 i of a row in the low half of byte i.  With scales
    uint8 [N, K/32] the weights are MXFP4 (E2M1 and E8M0, as quantize_rows(w, "mxfp4")
    makes them); with scales bf16 [N, K/group], group 32, 64 or 128, they are
    (code - zero) scale, zeros uint8 [N, K/group] or None for 8.  Runs on `stream`
    (default: the current stream) and does not synchronise."""
    if x.dtype != torch.bfloat16:
        raise TypeError("x must be bfloat16")
    if codes.dtype != torch.uint8 or scales.dtype not in (torch.uint8, torch.bfloat16):
        raise TypeError("codes must be uint8, scales uint8 or bfloat16")
    if dtype not in _TYPES:
        raise TypeError("dtype must be bfloat16 or float32")
    dev = x.device
    ldx = _matrix(x, "x", None)
    T, K = x.shape
    if codes.dim() != 2 or scales.dim() != 2 or codes.shape[0] == 0:
        raise ValueError("codes and scales must be 2-D")
    N = codes.shape[0]
    _fits(T, K, N)
    fp4 = scales.dtype == torch.uint8
    groups = scales.shape[1]
    group = K // groups if groups else 0
    if codes.shape[1] * 2 != K or scales.shape[0] != N or group * groups != K or group not in ((32,) if fp4 else (32, 64, 128)):
        raise ValueError("shape mismatch: x %s codes %s scales %s" % (tuple(x.shape), tuple(codes.shape), tuple(scales.shape)))
    if not (codes.is_contiguous() and scales.is_contiguous() and codes.get_device() == scales.get_device() == dev.index):
        raise ValueError("codes and scales must be contiguous and on the same GPU as x")
    if zeros is not None and (fp4 or zeros.dtype != torch.uint8 or zeros.shape != scales.shape or zeros.device != dev or
                              not zeros.is_contiguous()):
        raise ValueError("zeros must be a contiguous uint8 tensor of the scales' shape (with bf16 scales)")
    on = _On(dev, stream)
    out = _output(out, "out", (T, N), dtype, on)
    with on:
        rc = mxw_linear_4bit(x.data_ptr(), ldx, codes.data_ptr(), scales.data_ptr(),
                             0 if zeros is None else zeros.data_ptr(), 1 if fp4 else 2, group, T, K, N, out.data_ptr(),
                             _TYPES[dtype], on.handle) if T else 0
    if rc != 0:
        raise MxwError("mxw_linear_4bit failed (%d): %s" % (rc, strerror(rc)))
    return out
