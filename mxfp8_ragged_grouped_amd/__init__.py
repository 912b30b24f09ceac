"""MI355X-native MXFP8 ragged grouped GEMMs.

    out = wgrad(A, sA, B, sB, offs)        # bf16 [E, N, K]
    out = wgrad(..., plain=True)           # the entry point that takes no workspace
    out = wgrad_bf16(A, B, offs)           # bf16 [E, N, K] from bf16 operands
    out = fwd(A, sA, B, sB, offs)          # bf16 [R, N]
    q, s = quantize_tokens(x, offs)        # MXFP8 operand [H, M] from bf16 [M, H]

    update = orthogonalize(out)            # Newton-Schulz on every expert's gradient
    loss, dx, dw = vocab_cross_entropy(x, w, targets)   # over a large vocabulary
    y, ids, weights = moe_layer(x, router, wgu, sgu, wd, sd, top_k)   # a few tokens

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
at its function).  Everything
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
import ctypes
import os

import torch

from .build import LIB as _LIB_PATH

__all__ = ["wgrad", "mxfp8_wgrad_grouped", "mxfp8_wgrad_grouped_ws", "mxfp8_wgrad_grouped_noalloc", "workspace_size", "wgrad_bf16",
           "bf16_wgrad_grouped", "bf16_wgrad_grouped_ws", "bf16_workspace_size", "grid_size", "columns",
           "scale_shuffle", "tail_split", "fwd", "mxfp8_grouped_fwd", "fwd_grid_size", "quantize_tokens", "mxfp8_quantize_tokens",
           "orthogonalize", "mxw_orthogonalize", "orthogonalize_workspace_size",
           "vocab_cross_entropy", "mxw_vocab_loss", "vocab_loss_workspace_size",
           "moe_layer", "mxw_moe_layer", "moe_workspace_size",
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

    def __init__(self, dev, stream):
        current = torch._C._cuda_getCurrentRawStream(dev.index)
        self.handle = current if stream is None else stream.cuda_stream
        self._stream = stream
        self._other_stream = self.handle != current
        self._dev = dev
        self._switch = None if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)

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
        return torch.empty(shape, dtype=dtype, device=self._dev)

    def workspace(self, need, workspace):
        if workspace is not None:
            return _workspace(need, self._dev, None, workspace)
        ws = self.new(need, torch.uint8)
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
