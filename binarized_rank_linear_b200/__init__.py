"""LittleBit factored linear layer on NVIDIA B200: Python binding of ``liblb.so``.

The layer (sesamedisk.com, "Samsung LittleBit 13B Model", section "What the
method actually computes", Proposition 1) is
``y = h (.) (sign(U) (l (.) (sign(V)^T (g (.) x))))`` per path, with an optional
residual path added on top.  Every step runs in the library's CUDA kernels;
this module only marshals arguments through the C ABI declared in
``include/lb.h``.  PyTorch provides device memory and streams.  There is no
CPU fallback: if ``liblb.so`` is missing or the device is not an sm_100 part,
the calls raise.

A call runs on the current stream, or on the ``stream`` it is given, which then
has to be ordered behind whatever wrote its inputs; memory that the call makes
for itself comes from that stream.

Build the library with ``python -m binarized_rank_linear_b200.build``.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from dataclasses import dataclass

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblb.so")
HEADER_PATH = os.path.join(os.path.dirname(_HERE), "include", "lb.h")

# lb_status
LB_OK = 0
LB_ERR_INVALID_ARGUMENT = 1
LB_ERR_UNSUPPORTED_SHAPE = 2
LB_ERR_MISALIGNED = 3
LB_ERR_CUDA = 4
LB_ERR_DEVICE_TIMEOUT = 5
LB_ERR_NOT_SUPPORTED_DEVICE = 6
LB_ERR_WORKSPACE_TOO_SMALL = 7
LB_ERR_RANGE = 8
# lb_dtype
LB_F32, LB_F16, LB_BF16, LB_I8 = 0, 1, 2, 3
# lb_factor
LB_FACTOR_U, LB_FACTOR_V = 0, 1


class LbPath(ctypes.Structure):
    """``lb_path`` of include/lb.h."""
    _fields_ = [
        ("u_bits", ctypes.c_void_p),
        ("vt_bits", ctypes.c_void_p),
        ("h", ctypes.c_void_p),
        ("g", ctypes.c_void_p),
        ("l", ctypes.c_void_p),
        ("rank", ctypes.c_int64),
        ("u_ld", ctypes.c_int64),
        ("vt_ld", ctypes.c_int64),
    ]


class LbError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {status_string(status)}" if what else status_string(status))


_lock = threading.Lock()
_lib = None


class LbProjection(ctypes.Structure):
    """``lb_projection`` (include/lb.h): one layer of a group that shares x."""
    _fields_ = [("n_out", ctypes.c_int64), ("main", ctypes.POINTER(LbPath)), ("residual", ctypes.POINTER(LbPath)),
                ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64)]


class LbAdapters(ctypes.Structure):
    """``lb_adapters`` (include/lb.h): the adapter pool of one projection."""
    _fields_ = [("a", ctypes.c_void_p), ("b", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("ranks", ctypes.c_void_p),
                ("count", ctypes.c_int64), ("rank", ctypes.c_int64)]


class LbAdapterProjection(ctypes.Structure):
    """``lb_adapter_projection`` (include/lb.h): one projection of an adapters call."""
    _fields_ = [("n_out", ctypes.c_int64), ("adapters", ctypes.POINTER(LbAdapters)), ("base", ctypes.c_void_p),
                ("ldbase", ctypes.c_int64), ("y", ctypes.c_void_p), ("ldy", ctypes.c_int64)]


class LbHeads(ctypes.Structure):
    """``lb_heads`` (include/lb.h): one tensor of heads."""
    _fields_ = [("heads", ctypes.c_int64), ("in_", ctypes.c_void_p), ("ld_in", ctypes.c_int64),
                ("weight", ctypes.c_void_p), ("out", ctypes.c_void_p), ("ld_out", ctypes.c_int64)]


class LbHeadsGrad(ctypes.Structure):
    """``lb_heads_grad`` (include/lb.h): one tensor of heads and its gradients."""
    _fields_ = [("heads", ctypes.c_int64), ("in_", ctypes.c_void_p), ("ld_in", ctypes.c_int64),
                ("weight", ctypes.c_void_p), ("dout", ctypes.c_void_p), ("ld_dout", ctypes.c_int64),
                ("din", ctypes.c_void_p), ("ld_din", ctypes.c_int64), ("dweight", ctypes.c_void_p)]


MAX_SIBLINGS = 4
MAX_ADAPTERS = 1024
MAX_ADAPTER_RANK = 128
MAX_HEADS = 4096  # of a heads call's tensors together
ROTATE_HALVES, ROTATE_PAIRS = 0, 1


def lib() -> ctypes.CDLL:
    """Load ``liblb.so`` (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(
                    f"{LIB_PATH} is missing: build it with `python -m binarized_rank_linear_b200.build`")
            L = ctypes.CDLL(LIB_PATH)
            i64, vp, sz, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int
            L.lb_status_string.restype = ctypes.c_char_p
            L.lb_status_string.argtypes = [i32]
            L.lb_packed_ld_words.restype = i64
            L.lb_packed_ld_words.argtypes = [i64]
            L.lb_packed_bytes.restype = sz
            L.lb_packed_bytes.argtypes = [i32, i64, i64]
            L.lb_rank_for_budget.restype = i32
            L.lb_rank_for_budget.argtypes = [i64, i64, i64, i64, i32, i32, ctypes.POINTER(i64)]
            L.lb_pack_signs.restype = i32
            L.lb_pack_signs.argtypes = [vp, i32, i32, i64, i64, i64, vp, i64, vp]
            L.lb_forward_workspace_bytes.restype = sz
            L.lb_forward_workspace_bytes.argtypes = [i64, i64, i64, i64, i64]
            L.lb_linear_forward.restype = i32
            L.lb_linear_forward.argtypes = [vp, i64, i64, i64, i64, ctypes.POINTER(LbPath),
                                            ctypes.POINTER(LbPath), vp, i64, vp, sz, vp]
            L.lb_latent_forward.restype = i32
            L.lb_latent_forward.argtypes = [vp, i64, i64, i64, ctypes.POINTER(LbPath), ctypes.POINTER(LbPath),
                                            vp, i64, vp]
            L.lb_expand_forward.restype = i32
            L.lb_expand_forward.argtypes = [vp, i64, i64, i64, ctypes.POINTER(LbPath), ctypes.POINTER(LbPath),
                                            vp, i64, vp]
            L.lb_linear_forward_fixed_scratch.restype = i32
            L.lb_linear_forward_fixed_scratch.argtypes = [vp, i64, i64, i64, i64, ctypes.POINTER(LbPath),
                                                          ctypes.POINTER(LbPath), vp, i64, vp]
            L.lb_siblings_workspace_bytes.restype = sz
            L.lb_siblings_workspace_bytes.argtypes = [i64, i64, i32, ctypes.POINTER(LbProjection)]
            L.lb_linear_forward_siblings.restype = i32
            L.lb_linear_forward_siblings.argtypes = [vp, i64, i64, i64, i32, ctypes.POINTER(LbProjection), vp, sz, vp]
            L.lb_linear_forward_host.restype = i32
            L.lb_linear_forward_host.argtypes = [vp, i64, i64, i64, ctypes.POINTER(LbPath), ctypes.POINTER(LbPath),
                                                 vp, vp, vp, vp, sz, vp]
            L.lb_backward_workspace_bytes.restype = sz
            L.lb_backward_workspace_bytes.argtypes = [i64, i64, i64, i64, i64]
            L.lb_linear_backward.restype = i32
            L.lb_linear_backward.argtypes = [vp, vp, i64, i64, i64, i64, i64, ctypes.POINTER(LbPath),
                                             ctypes.POINTER(LbPath), vp, i64, vp, vp, vp, vp, sz, vp]
            L.lb_adapters_workspace_bytes.restype = sz
            L.lb_adapters_workspace_bytes.argtypes = [i64, i64, i32, ctypes.POINTER(LbAdapterProjection)]
            L.lb_adapters_forward.restype = i32
            L.lb_adapters_forward.argtypes = [vp, i64, i64, i64, vp, i32, ctypes.POINTER(LbAdapterProjection), vp, sz, vp]
            L.lb_adapters_backward_workspace_bytes.restype = sz
            L.lb_adapters_backward_workspace_bytes.argtypes = [i64, i64, i64, i64, i64]
            L.lb_adapters_backward.restype = i32
            L.lb_adapters_backward.argtypes = [vp, vp, i64, i64, i64, i64, i64, vp, ctypes.POINTER(LbAdapters), vp, i64,
                                               vp, i64, vp, vp, vp, sz, vp]
            f32 = ctypes.c_float
            L.lb_heads_norm_rotate.restype = i32
            L.lb_heads_norm_rotate.argtypes = [i64, i64, i64, i32, vp, vp, f32, i32, ctypes.POINTER(LbHeads), vp]
            L.lb_heads_backward_workspace_bytes.restype = sz
            L.lb_heads_backward_workspace_bytes.argtypes = [i64]
            L.lb_heads_norm_rotate_backward.restype = i32
            L.lb_heads_norm_rotate_backward.argtypes = [i64, i64, i64, i32, vp, vp, f32, i32,
                                                        ctypes.POINTER(LbHeadsGrad), vp, sz, vp]
            L.lb_device_status.restype = i32
            L.lb_device_status.argtypes = [vp, ctypes.POINTER(i32)]
            L.lb_debug_inject_stall.restype = i32
            L.lb_debug_inject_stall.argtypes = [i32, ctypes.c_uint64]
            L.lb_set_prefill_pairs.restype = i32
            L.lb_set_prefill_pairs.argtypes = [i32]
            _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().lb_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != LB_OK:
        raise LbError(status, what)


# ------------------------------------------------------------------ host-only queries

def packed_ld_words(cols: int) -> int:
    return int(lib().lb_packed_ld_words(cols))


def packed_bytes(kind: int, n_in_or_out: int, rank: int) -> int:
    return int(lib().lb_packed_bytes(kind, n_in_or_out, rank))


def rank_for_budget(n_in: int, n_out: int, eff_num: int, eff_den: int, paths: int = 1,
                    align: int = 32) -> int:
    r = ctypes.c_int64(0)
    _check(lib().lb_rank_for_budget(n_in, n_out, eff_num, eff_den, paths, align, ctypes.byref(r)),
           "lb_rank_for_budget")
    return int(r.value)


def forward_workspace_bytes(tokens: int, n_in: int, n_out: int, rank_main: int,
                            rank_residual: int = 0) -> int:
    return int(lib().lb_forward_workspace_bytes(tokens, n_in, n_out, rank_main, rank_residual))


# ------------------------------------------------------------------ device calls

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _stream_handle(stream) -> ctypes.c_void_p:
    torch = _torch()
    if stream is None:
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        if raw is not None:  # the current stream of the current device, without a Stream object
            return ctypes.c_void_p(raw(torch.cuda.current_device()))
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t) -> int:
    torch = _torch()
    codes = {torch.float32: LB_F32, torch.float16: LB_F16, torch.bfloat16: LB_BF16, torch.int8: LB_I8}
    if t.dtype not in codes:
        raise TypeError(f"unsupported factor dtype {t.dtype}")
    return codes[t.dtype]


def _require(t, name: str, dtype, device: str = "cuda", contiguous: bool = False) -> None:
    """Checks an activation tensor before its pointer crosses the C ABI: the
    library reads the bits as the element type and layout its header states,
    so a tensor of another dtype or with a non-unit inner stride would be read
    as wrong data without an error."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(t.shape)}")
    if t.stride(1) != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must have unit inner stride, got strides {t.stride()}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (rows of exactly {t.shape[1]} elements)")
    if (device == "cuda") != bool(t.is_cuda):
        raise ValueError(f"{name} must be in {'device' if device == 'cuda' else 'host'} memory")


def _require_workspace(ws, device=None) -> None:
    if not ws.is_cuda or not ws.is_contiguous():
        raise ValueError("workspace must be a contiguous device tensor")
    if device is not None and ws.device != device:
        raise ValueError(f"workspace must be on {device}, got {ws.device}")


# Memory that a call makes for itself.  On a stream of the caller's it comes from
# that stream's part of torch's pool: a block of the current stream's may still be
# read by kernels queued there, which the call's stream knows nothing of.

def _new(shape, dtype, device, stream):
    """A dense tensor that a call on `stream` writes and returns.  It may be read
    on the current stream afterwards, so its memory waits for that one too."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream())
    return t


def _new_workspace(like, need: int, stream):
    """Scratch of `need` bytes on the device of the tensor `like`, of two-byte elements."""
    if stream is None:
        return like.new_empty(max(need, 16) + 1 >> 1)
    with _torch().cuda.stream(stream):
        return like.new_empty(max(need, 16) + 1 >> 1)


def pack_signs(src, kind: str, ld_words: int | None = None, stream=None):
    """Pack a device factor (f32 / f16 / bf16 / int8, 2-D, unit column stride)
    with ``lb_pack_signs``.  ``kind`` is ``"U"`` (src = U [n_out, r]) or
    ``"V"`` (src = V [n_in, r], packed as V^T).  Returns an int32 tensor of
    packed words (bit patterns)."""
    if src.dim() != 2 or src.stride(1) != 1 or not src.is_cuda:
        raise ValueError("src must be a 2-D CUDA tensor with unit column stride")
    rows, cols = src.shape
    packed_rows, packed_cols = (rows, cols) if kind == "U" else (cols, rows)
    ld = packed_ld_words(packed_cols) if ld_words is None else int(ld_words)
    dst = _new((packed_rows, ld), _torch().int32, src.device, stream)
    code = LB_FACTOR_U if kind == "U" else LB_FACTOR_V
    _check(lib().lb_pack_signs(src.data_ptr(), _dtype_code(src), code, rows, cols, src.stride(0),
                               dst.data_ptr(), ld, _stream_handle(stream)), "lb_pack_signs")
    return dst


@dataclass(frozen=True)
class PackedPath:
    """One binarized path on the device: packed sign(U) [n_out, u_ld] and
    sign(V)^T [rank, vt_ld] (int32 words) and fp16 scales h [n_out], g [n_in],
    l [rank]."""
    u_bits: object
    vt_bits: object
    h: object
    g: object
    l: object
    rank: int

    @classmethod
    def from_factors(cls, su, sv, h, g, l, stream=None) -> "PackedPath":
        """Pack U [n_out, r] and V [n_in, r] (any supported dtype, on the
        device) and keep the fp16 scales."""
        torch = _torch()
        f16 = lambda t: t.to(device=su.device, dtype=torch.float16).contiguous()
        return cls(pack_signs(su, "U", stream=stream), pack_signs(sv, "V", stream=stream),
                   f16(h), f16(g), f16(l), int(su.shape[1]))

    def as_c(self) -> LbPath:
        """The lb_path struct of this path, built once (the fields are frozen
        and a tensor's storage does not move)."""
        c = self.__dict__.get("_c")
        if c is None:
            torch = _torch()
            for name in ("u_bits", "vt_bits"):
                t = getattr(self, name)
                if t.dtype != torch.int32 or t.dim() != 2 or t.stride(1) != 1 or not t.is_cuda:
                    raise ValueError(f"{name} must be a 2-D int32 device tensor of packed words with unit "
                                     f"inner stride")
            for name in ("h", "g", "l"):
                t = getattr(self, name)
                if t.dtype != torch.float16 or t.dim() != 1 or not t.is_contiguous() or not t.is_cuda:
                    raise ValueError(f"{name} must be a contiguous 1-D float16 device tensor")
            c = LbPath(self.u_bits.data_ptr(), self.vt_bits.data_ptr(), self.h.data_ptr(),
                       self.g.data_ptr(), self.l.data_ptr(), self.rank, self.u_bits.shape[1],
                       self.vt_bits.shape[1])
            object.__setattr__(self, "_c", c)
        return c


def linear_forward(x, main: PackedPath, residual: PackedPath | None = None, y=None,
                   workspace=None, stream=None):
    """``lb_linear_forward``: x bf16 [tokens, n_in] (row stride a multiple of 8)
    -> y bf16 [tokens, n_out].  Allocates y and the workspace with torch when
    not given."""
    torch = _torch()
    _require(x, "x", torch.bfloat16)
    tokens, n_in = x.shape
    n_out = main.h.shape[0]
    if y is None:
        y = _new((tokens, n_out), torch.bfloat16, x.device, stream)
    _require(y, "y", torch.bfloat16)
    if workspace is None:  # a caller's workspace size is checked by the library itself
        need = forward_workspace_bytes(tokens, n_in, n_out, main.rank, residual.rank if residual else 0)
        workspace = _new_workspace(x, need, stream)
    _require_workspace(workspace)
    cm = main.as_c()
    cr = residual.as_c() if residual is not None else None
    _check(lib().lb_linear_forward(
        x.data_ptr(), tokens, n_in, n_out, x.stride(0), ctypes.byref(cm),
        ctypes.byref(cr) if cr is not None else None, y.data_ptr(), y.stride(0),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream_handle(stream)),
        "lb_linear_forward")
    return y


def _projections(layers, ys):
    """ctypes array of lb_projection for [(main, residual or None), ...] and
    their outputs; the LbPath structs are returned too, to keep them alive."""
    keep = []
    arr = (LbProjection * len(layers))()
    for j, ((main, residual), y) in enumerate(zip(layers, ys)):
        cm = main.as_c()
        cr = residual.as_c() if residual is not None else None
        keep += [cm, cr]
        arr[j].n_out = main.h.shape[0]
        arr[j].main = ctypes.pointer(cm)
        arr[j].residual = ctypes.pointer(cr) if cr is not None else None
        arr[j].y = y.data_ptr() if y is not None else None
        arr[j].ldy = y.stride(0) if y is not None else main.h.shape[0]
    return arr, keep


def siblings_workspace_bytes(tokens: int, n_in: int, layers) -> int:
    arr, _keep = _projections(layers, [None] * len(layers))
    return int(lib().lb_siblings_workspace_bytes(tokens, n_in, len(layers), arr))


def linear_forward_siblings(x, layers, ys=None, workspace=None, stream=None, adapters=None, ids=None, rotation=None,
                            positions=None, rotate=None):
    """``lb_linear_forward_siblings``: several layers that read the same x,
    given as [(main, residual or None), ...]; returns their outputs (bf16
    [tokens, n_out_j]), allocated with torch when not given.

    With ``adapters`` (one :class:`AdapterPool` or None per layer) and ``ids``
    each token's adapter is added to the outputs (:func:`adapters_forward`).
    With ``rotation`` (a :class:`HeadRotation`) and ``positions`` (not needed
    for a norm alone) the outputs named by ``rotate``, a dict from the layer's index to its norm weight (or
    None for no norm), then get their heads normed and rotated
    (:func:`heads_norm_rotate`): an attention block's queries and keys."""
    torch = _torch()
    _require(x, "x", torch.bfloat16)
    tokens, n_in = x.shape
    if ys is None:
        ys = [_new((tokens, main.h.shape[0]), torch.bfloat16, x.device, stream) for main, _ in layers]
    for j, y in enumerate(ys):
        _require(y, f"ys[{j}]", torch.bfloat16)
    if adapters is not None and (len(adapters) != len(layers) or ids is None):
        raise ValueError("adapters must name a pool or None for each layer, and ids each token's adapter")
    if rotation is not None and (not rotate or not all(0 <= j < len(layers) for j in rotate)):
        raise ValueError("rotation needs, in rotate, the layers whose outputs are normed and rotated")
    if rotation is not None and positions is None and rotation.rotary_dim:
        raise ValueError("rotation needs positions")
    # what follows the projections is checked before they are launched
    some = [j for j, pool in enumerate(adapters or ()) if pool is not None]
    if some:
        beside = _adapters_call(x, ids, [adapters[j] for j in some], None, [ys[j] for j in some], stream)
        _adapters_checked(lib().lb_adapters_forward, "lb_adapters_forward", tokens, beside[0])
    if rotation is not None:
        which = sorted(rotate)
        turned = [ys[j] for j in which]
        heads = _heads_forward_call(turned, positions, rotation, [rotate[j] for j in which], turned, stream)
        _heads_checked(heads[0])
    arr, _keep = _projections(layers, ys)
    need = int(lib().lb_siblings_workspace_bytes(tokens, n_in, len(layers), arr))
    if workspace is None:
        workspace = _new_workspace(x, need, stream)
    _require_workspace(workspace)
    _check(lib().lb_linear_forward_siblings(
        x.data_ptr(), tokens, n_in, x.stride(0), len(layers), arr, workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_handle(stream)), "lb_linear_forward_siblings")
    if some:
        _adapters_launch(beside, x, None, stream)
    if rotation is not None:
        _check(lib().lb_heads_norm_rotate(*heads[0], _stream_of(stream, heads[1])), "lb_heads_norm_rotate")
    return ys


def linear_forward_host(x_host, main: PackedPath, residual: PackedPath | None, y_host, x_dev, y_dev, workspace,
                        stream=None):
    """``lb_linear_forward_host``: x from pinned host memory (bf16 [tokens,
    n_in], contiguous) through the caller's device buffers x_dev and y_dev to
    y in pinned host memory (bf16 [tokens, n_out]), all on one stream; y_host
    is valid once the stream is synchronised.  For 1-128 tokens on pinned
    buffers x comes in through a gather kernel and y is written to y_host by
    the last kernel (y_dev is then not touched)."""
    torch = _torch()
    _require(x_host, "x_host", torch.bfloat16, device="cpu", contiguous=True)
    _require(y_host, "y_host", torch.bfloat16, device="cpu", contiguous=True)
    _require(x_dev, "x_dev", torch.bfloat16, contiguous=True)
    _require(y_dev, "y_dev", torch.bfloat16, contiguous=True)
    _require_workspace(workspace)
    tokens, n_in = x_host.shape
    n_out = main.h.shape[0]
    if tuple(y_host.shape) != (tokens, n_out) or tuple(x_dev.shape) != (tokens, n_in) \
            or tuple(y_dev.shape) != (tokens, n_out):
        raise ValueError("x_host / x_dev must be [tokens, n_in] and y_host / y_dev [tokens, n_out]")
    cm = main.as_c()
    cr = residual.as_c() if residual is not None else None
    _check(lib().lb_linear_forward_host(
        x_host.data_ptr(), tokens, n_in, n_out, ctypes.byref(cm), ctypes.byref(cr) if cr is not None else None,
        y_host.data_ptr(), x_dev.data_ptr(), y_dev.data_ptr(), workspace.data_ptr(),
        workspace.numel() * workspace.element_size(), _stream_handle(stream)), "lb_linear_forward_host")
    return y_host


def latent_forward(x, main: PackedPath, residual: PackedPath | None = None, z=None, stream=None):
    """``lb_latent_forward``: x bf16 [tokens, n_in] -> z fp16 [tokens, r_main
    + r_residual] (the latent of both paths, main first).  Allocates z with
    torch when not given (the C call allocates nothing)."""
    torch = _torch()
    _require(x, "x", torch.bfloat16)
    tokens, n_in = x.shape
    R = main.rank + (residual.rank if residual is not None else 0)
    if z is None:
        z = _new((tokens, R), torch.float16, x.device, stream)
    _require(z, "z", torch.float16)
    cm = main.as_c()
    cr = residual.as_c() if residual is not None else None
    _check(lib().lb_latent_forward(
        x.data_ptr(), tokens, n_in, x.stride(0), ctypes.byref(cm), ctypes.byref(cr) if cr is not None else None,
        z.data_ptr(), z.stride(0), _stream_handle(stream)), "lb_latent_forward")
    return z


def expand_forward(z, main: PackedPath, residual: PackedPath | None = None, y=None, stream=None):
    """``lb_expand_forward``: z fp16 [tokens, r_main + r_residual] -> y bf16
    [tokens, n_out].  Allocates y with torch when not given."""
    torch = _torch()
    _require(z, "z", torch.float16)
    tokens = z.shape[0]
    n_out = main.h.shape[0]
    if y is None:
        y = _new((tokens, n_out), torch.bfloat16, z.device, stream)
    _require(y, "y", torch.bfloat16)
    cm = main.as_c()
    cr = residual.as_c() if residual is not None else None
    _check(lib().lb_expand_forward(
        z.data_ptr(), tokens, n_out, z.stride(0), ctypes.byref(cm), ctypes.byref(cr) if cr is not None else None,
        y.data_ptr(), y.stride(0), _stream_handle(stream)), "lb_expand_forward")
    return y


def linear_forward_fixed_scratch(x, main: PackedPath, residual: PackedPath | None = None, y=None,
                                 stream=None):
    """``lb_linear_forward_fixed_scratch``: as :func:`linear_forward` for
    1..32 tokens, with the library's fixed device scratch instead of a
    workspace.  Allocates y with torch when not given (the C call itself
    allocates nothing)."""
    torch = _torch()
    _require(x, "x", torch.bfloat16)
    tokens, n_in = x.shape
    n_out = main.h.shape[0]
    if y is None:
        y = _new((tokens, n_out), torch.bfloat16, x.device, stream)
    _require(y, "y", torch.bfloat16)
    cm = main.as_c()
    cr = residual.as_c() if residual is not None else None
    _check(lib().lb_linear_forward_fixed_scratch(
        x.data_ptr(), tokens, n_in, n_out, x.stride(0), ctypes.byref(cm),
        ctypes.byref(cr) if cr is not None else None, y.data_ptr(), y.stride(0), _stream_handle(stream)),
        "lb_linear_forward_fixed_scratch")
    return y


def backward_workspace_bytes(tokens: int, n_in: int, n_out: int, rank_main: int, rank_residual: int = 0) -> int:
    return int(lib().lb_backward_workspace_bytes(tokens, n_in, n_out, rank_main, rank_residual))


def linear_backward(x, dy, main: PackedPath, residual: PackedPath | None = None, dx=None, want_dx: bool = True,
                    workspace=None, stream=None, adapters: "AdapterPool | None" = None, ids=None) -> dict:
    """``lb_linear_backward``: the gradients of a loss with respect to the
    layer's input and scale vectors, given ``dy`` = dL/dy (bf16 [tokens,
    n_out]) and the forward input ``x`` (bf16 [tokens, n_in]).  Returns
    ``{"dx": bf16 [tokens, n_in] or None, "dh": fp32 [paths, n_out], "dg":
    fp32 [paths, n_in], "dl": fp32 [r_main + r_residual]}``; outputs and the
    workspace are allocated with torch when not given.  With ``adapters`` and
    ``ids`` (the layer ran with a pool beside it) dx includes the adapters'
    part, and their gradients "da" and "db" are returned too
    (:func:`adapters_backward`)."""
    torch = _torch()
    _require(x, "x", torch.bfloat16)
    _require(dy, "dy", torch.bfloat16)
    tokens, n_in = x.shape
    n_out = main.h.shape[0]
    if tuple(dy.shape) != (tokens, n_out):
        raise ValueError(f"dy must be [{tokens}, {n_out}], got {tuple(dy.shape)}")
    npaths = 2 if residual is not None else 1
    if adapters is not None and ids is None:
        raise ValueError("adapters need ids, each token's adapter")
    if dx is None and want_dx:
        dx = _new((tokens, n_in), torch.bfloat16, x.device, stream)
    if dx is not None:
        _require(dx, "dx", torch.bfloat16)
    if adapters is not None:  # checked before the layer's own pass is launched
        beside = _adapters_backward_call(x, dy, ids, adapters, None, dx, dx is not None, None, None, stream)
        _adapters_checked(lib().lb_adapters_backward, "lb_adapters_backward", tokens, beside[0])
    dh = _new((npaths, n_out), torch.float32, x.device, stream)
    dg = _new((npaths, n_in), torch.float32, x.device, stream)
    dl = _new((main.rank + (residual.rank if residual is not None else 0),), torch.float32, x.device, stream)
    if workspace is None:
        need = backward_workspace_bytes(tokens, n_in, n_out, main.rank, residual.rank if residual else 0)
        workspace = _new_workspace(x, need, stream)
    _require_workspace(workspace)
    cm = main.as_c()
    cr = residual.as_c() if residual is not None else None
    _check(lib().lb_linear_backward(
        x.data_ptr(), dy.data_ptr(), tokens, n_in, n_out, x.stride(0), dy.stride(0), ctypes.byref(cm),
        ctypes.byref(cr) if cr is not None else None, dx.data_ptr() if dx is not None else None,
        dx.stride(0) if dx is not None else n_in, dh.data_ptr(), dg.data_ptr(), dl.data_ptr(),
        workspace.data_ptr(), workspace.numel() * workspace.element_size(), _stream_handle(stream)),
        "lb_linear_backward")
    out = {"dx": dx, "dh": dh, "dg": dg, "dl": dl}
    if adapters is not None:
        more = _adapters_backward_launch(beside, x, None, stream)
        out["da"], out["db"] = more["da"], more["db"]
    return out


# ------------------------------------------------------------------ adapters

def _require_rows(t, name: str, rows: int, cols: int, dtype, device) -> int:
    """Checks a [rows, cols] tensor of an adapters or heads call and that it
    lives on `device`; returns its row stride in elements."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}], got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    ld, inner = t.stride()
    if inner != 1 and cols > 1:
        raise ValueError(f"{name} must have unit inner stride, got strides {t.stride()}")
    return ld if rows > 1 else cols


def _require_vector(t, name: str, n: int, dtype, device) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{n}] tensor, got shape {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")


def _current(t, name: str):
    """The device of `t`, which must be the current one: the library launches there."""
    device = t.device
    if not t.is_cuda:
        raise ValueError(f"{name} must be in device memory")
    if device.index != _torch().cuda.current_device():
        raise ValueError(f"{name} is on {device}, which is not the current device")
    return device


def _stream_of(stream, device):
    """_stream_handle for a call whose tensors are on `device`, the current one."""
    raw = getattr(_torch()._C, "_cuda_getCurrentRawStream", None)
    if stream is None and raw is not None:
        return raw(device.index)
    return _stream_handle(stream)


# A decode step calls these for microseconds of work on the device, so the calls
# check all of a tensor in one expression and only go through the checks that
# name the fault when it fails, and allocate by the cheapest of torch's calls.

def _new_dense(shape: tuple, strides: tuple, dtype, device, stream):
    """_new, given the strides of a dense tensor too."""
    if stream is None:
        return _torch().empty_strided(shape, strides, dtype=dtype, device=device)
    return _new(shape, dtype, device, stream)


def _rows_ld(t, name: str, rows: int, cols: int, dtype, device) -> int:
    """_require_rows, at once where nothing is wrong."""
    ld, inner = t.stride() if t.ndim == 2 else (0, 0)
    if inner == 1 and t.dtype is dtype and t.shape == (rows, cols) and t.device == device:
        return ld if rows > 1 else cols
    return _require_rows(t, name, rows, cols, dtype, device)


def _vector_ptr(t, name: str, n: int, dtype, device) -> int:
    """_require_vector, at once where nothing is wrong; the vector's address."""
    if t.dtype is not dtype or t.shape != (n,) or t.device != device or not t.is_contiguous():
        _require_vector(t, name, n, dtype, device)
    return t.data_ptr()


@dataclass(frozen=True)
class AdapterPool:
    """The adapters of one projection, on the device: ``a`` bf16 [count, rank,
    n_in], ``b`` bf16 [count, n_out, rank], ``scale`` fp32 [count] or None for
    1, ``ranks`` int32 [count] or None for ``rank`` each (``lb_adapters``)."""
    a: object
    b: object
    scale: object = None
    ranks: object = None

    def as_c(self) -> LbAdapters:
        """The lb_adapters struct of this pool, built once (the fields are
        frozen and a tensor's storage does not move).  ``_c`` is set last: a
        thread that finds it finds the rest too."""
        c = self.__dict__.get("_c")
        if c is None:
            torch = _torch()
            for name in ("a", "b"):
                t = getattr(self, name)
                if t.dtype != torch.bfloat16:
                    raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
                if t.dim() != 3 or not t.is_contiguous() or not t.is_cuda:
                    raise ValueError(f"{name} must be a contiguous 3-D device tensor")
            count, rank, n_in = self.a.shape
            if self.b.shape[0] != count or self.b.shape[2] != rank:
                raise ValueError(f"b must be [{count}, n_out, {rank}], got {tuple(self.b.shape)}")
            if self.b.device != self.a.device:
                raise ValueError("a and b must be on one device")
            if self.scale is not None:
                _require_vector(self.scale, "scale", count, torch.float32, self.a.device)
            if self.ranks is not None:
                _require_vector(self.ranks, "ranks", count, torch.int32, self.a.device)
            c = LbAdapters(self.a.data_ptr(), self.b.data_ptr(),
                           self.scale.data_ptr() if self.scale is not None else None,
                           self.ranks.data_ptr() if self.ranks is not None else None, count, rank)
            object.__setattr__(self, "_p", ctypes.pointer(c))
            object.__setattr__(self, "n_in", n_in)
            object.__setattr__(self, "n_out", self.b.shape[1])
            object.__setattr__(self, "device", self.a.device)
            object.__setattr__(self, "_c", c)
        return c


@functools.lru_cache(maxsize=4096)
def adapters_workspace_bytes(tokens: int, n_in: int, count: int, ranks: tuple) -> int:
    """``lb_adapters_workspace_bytes`` for pools of ``count`` adapters of the given stored ranks."""
    arr = (LbAdapterProjection * max(1, len(ranks)))()
    for j, r in enumerate(ranks):
        arr[j].n_out = 32
        arr[j].adapters = ctypes.pointer(LbAdapters(None, None, None, None, count, r))
    return int(lib().lb_adapters_workspace_bytes(tokens, n_in, len(ranks), arr))


def adapters_forward(x, ids, pools, bases=None, ys=None, workspace=None, stream=None):
    """``lb_adapters_forward``: ``y_j = base_j + s_i B_ij (A_ij x)`` per token,
    i = ids[token], for every pool j of ``pools`` (projections of one x).
    ``ids`` int32 [tokens] on the device, negative for no adapter.  ``bases``
    and ``ys`` are lists of bf16 [tokens, n_out_j]: without ``bases`` the
    ``ys`` are updated in place, without ``ys`` they are allocated.  Returns
    ``ys``."""
    call = _adapters_call(x, ids, pools, bases, ys, stream)
    return _adapters_launch(call, x, workspace, stream)


def _adapters_call(x, ids, pools, bases, ys, stream) -> tuple:
    """What the binding checks of an adapters_forward call, and the arguments of the library's."""
    torch = _torch()
    bf16 = torch.bfloat16
    device = _current(x, "x")
    _require(x, "x", bf16)
    tokens, n_in = x.shape
    ids_ptr = _vector_ptr(ids, "ids", tokens, torch.int32, device)
    n = len(pools)
    if not 1 <= n <= MAX_SIBLINGS:
        raise ValueError(f"1 to {MAX_SIBLINGS} pools, got {n}")
    if bases is None and ys is None:
        raise ValueError("give bases, or ys to update in place")
    if (bases is not None and len(bases) != n) or (ys is not None and len(ys) != n):
        raise ValueError(f"bases and ys must have one tensor for each of the {n} pools")
    arr = (LbAdapterProjection * n)()
    made, ranks = [], []
    for j, pool in enumerate(pools):
        c = pool.as_c()
        if pool.n_in != n_in or pool.device != device:
            raise ValueError(f"pools[{j}] has n_in = {pool.n_in} on {pool.device}, x {n_in} on {device}")
        ranks.append(c.rank)
        n_out, e = pool.n_out, arr[j]
        e.n_out = n_out
        e.adapters = pool._p
        if bases is not None:
            base = bases[j]
            e.ldbase = _rows_ld(base, "bases", tokens, n_out, bf16, device)
            e.base = base.data_ptr()
        if ys is None:
            y = _new_dense((tokens, n_out), (n_out, 1), bf16, device, stream)
            made.append(y)
            e.ldy = n_out
        else:
            y = ys[j]
            e.ldy = _rows_ld(y, "ys", tokens, n_out, bf16, device)
        e.y = y.data_ptr()
    args = (x.data_ptr(), tokens, n_in, x.stride(0) if tokens > 1 else n_in, ids_ptr, n, arr)
    return args, c.count, ranks, device, made if ys is None else ys


def _adapters_launch(call: tuple, x, workspace, stream):
    args, count, ranks, device, ys = call
    if workspace is None:
        workspace = _new_workspace(x, adapters_workspace_bytes(args[1], args[2], count, tuple(ranks)), stream)
    else:
        _require_workspace(workspace, device)
    _check(lib().lb_adapters_forward(*args, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                     _stream_of(stream, device)), "lb_adapters_forward")
    return ys


def _adapters_checked(function, name: str, tokens: int, args: tuple) -> None:
    """Raises what the library refuses of an adapters call that follows another
    launch, before that launch.  A workspace without bytes is the last thing that
    the library finds wrong with a call, before it touches the device."""
    status = function(*args, args[0], 0, None) if tokens else LB_OK
    if status != LB_ERR_WORKSPACE_TOO_SMALL:
        _check(status, name)


@functools.lru_cache(maxsize=4096)
def adapters_backward_workspace_bytes(tokens: int, n_in: int, n_out: int, count: int, rank: int) -> int:
    return int(lib().lb_adapters_backward_workspace_bytes(tokens, n_in, n_out, count, rank))


def adapters_backward(x, dy, ids, pool: AdapterPool, dx_base=None, dx=None, want_dx: bool = True, da=None, db=None,
                      workspace=None, stream=None) -> dict:
    """``lb_adapters_backward``: the gradients of a loss with respect to a
    pool's matrices and to x, given ``dy`` = dL/dy (bf16 [tokens, n_out]) and
    the forward x and ids.  ``dx_base`` is the layer's own dx, to which the
    adapters' part is added; without it ``dx`` is updated in place.  Returns
    ``{"dx": bf16 [tokens, n_in] or None, "da": fp32 [count, rank, n_in],
    "db": fp32 [count, n_out, rank]}``, allocated with torch when not given."""
    call = _adapters_backward_call(x, dy, ids, pool, dx_base, dx, want_dx, da, db, stream)
    return _adapters_backward_launch(call, x, workspace, stream)


def _adapters_backward_call(x, dy, ids, pool, dx_base, dx, want_dx, da, db, stream) -> tuple:
    """_adapters_call for the backward pass."""
    torch = _torch()
    bf16, f32 = torch.bfloat16, torch.float32
    device = _current(x, "x")
    _require(x, "x", bf16)
    c = pool.as_c()
    tokens, n_in = x.shape
    n_out = pool.n_out
    if pool.n_in != n_in or pool.device != device:
        raise ValueError(f"pool has n_in = {pool.n_in} on {pool.device}, x {n_in} on {device}")
    lddy = _rows_ld(dy, "dy", tokens, n_out, bf16, device)
    ids_ptr = _vector_ptr(ids, "ids", tokens, torch.int32, device)
    if want_dx and dx is None:
        if dx_base is None:
            raise ValueError("give dx_base, or dx to update in place, or want_dx=False")
        dx = _new_dense((tokens, n_in), (n_in, 1), bf16, device, stream)
    if not want_dx:
        dx = None
    lddx = _rows_ld(dx, "dx", tokens, n_in, bf16, device) if dx is not None else n_in
    with_base = dx is not None and dx_base is not None
    ldbase = _rows_ld(dx_base, "dx_base", tokens, n_in, bf16, device) if with_base else n_in
    count, rank = c.count, c.rank
    for name, t, shape in (("da", da, (count, rank, n_in)), ("db", db, (count, n_out, rank))):
        if t is not None and (t.dtype != f32 or t.shape != shape or not t.is_contiguous() or t.device != device):
            raise ValueError(f"{name} must be a contiguous {shape} float32 tensor on {device}")
    if da is None:
        da = _new_dense((count, rank, n_in), (rank * n_in, n_in, 1), f32, device, stream)
    if db is None:
        db = _new_dense((count, n_out, rank), (n_out * rank, rank, 1), f32, device, stream)
    args = (x.data_ptr(), dy.data_ptr(), tokens, n_in, n_out, x.stride(0) if tokens > 1 else n_in, lddy, ids_ptr,
            pool._p, dx_base.data_ptr() if with_base else None, ldbase, dx.data_ptr() if dx is not None else None, lddx,
            da.data_ptr(), db.data_ptr())
    return args, (tokens, n_in, n_out, count, rank), device, {"dx": dx, "da": da, "db": db}


def _adapters_backward_launch(call: tuple, x, workspace, stream) -> dict:
    args, sizes, device, out = call
    if workspace is None:
        workspace = _new_workspace(x, adapters_backward_workspace_bytes(*sizes), stream)
    else:
        _require_workspace(workspace, device)
    _check(lib().lb_adapters_backward(*args, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                      _stream_of(stream, device)), "lb_adapters_backward")
    return out


# ------------------------------------------------------------------ heads

@dataclass(frozen=True)
class HeadRotation:
    """What a model's blocks share of the per-head norm and rotation: the head
    size, the rotation's frequencies ``inv_freq`` (fp32 [rotary_dim / 2] on the
    device, or None for a norm alone), which elements form a pair
    (``"halves"``: k and k + rotary_dim / 2, or ``"pairs"``: 2k and 2k + 1) and
    the norm's eps."""
    head_dim: int
    inv_freq: object = None
    rotation: str = "halves"
    eps: float = 1e-6

    def __post_init__(self):
        torch = _torch()
        if self.rotation not in ("halves", "pairs"):
            raise ValueError(f"rotation must be 'halves' or 'pairs', got {self.rotation!r}")
        f = self.inv_freq
        if f is not None and (f.dtype != torch.float32 or f.dim() != 1 or not f.is_contiguous() or not f.is_cuda):
            raise ValueError("inv_freq must be a contiguous 1-D float32 device tensor")
        object.__setattr__(self, "rotary_dim", 2 * f.shape[0] if f is not None else 0)
        object.__setattr__(self, "code", ROTATE_HALVES if self.rotation == "halves" else ROTATE_PAIRS)


def _heads_call(tensors, positions, rotation: HeadRotation, weights, name: str):
    """Checks what both heads calls share; returns (device, tokens, positions' address, frequencies' address)."""
    torch = _torch()
    n = len(tensors)
    if not 1 <= n <= MAX_SIBLINGS:
        raise ValueError(f"1 to {MAX_SIBLINGS} tensors, got {n}")
    if weights is not None and len(weights) != n:
        raise ValueError(f"weights must have one entry for each of the {n} tensors")
    device = _current(tensors[0], name)
    tokens = tensors[0].shape[0]
    if rotation.rotary_dim == 0:
        return device, tokens, None, None
    pos = _vector_ptr(positions, "positions", tokens, torch.int32, device)
    if rotation.inv_freq.device != device:
        raise ValueError(f"inv_freq must be on {device}, got {rotation.inv_freq.device}")
    return device, tokens, pos, rotation.inv_freq.data_ptr()


def _heads_of(t, name: str, head_dim: int) -> tuple:
    """The heads and columns of `t`."""
    shape = t.shape
    if len(shape) != 2 or head_dim < 1 or shape[1] % head_dim:
        raise ValueError(f"{name} must be [tokens, heads * {head_dim}], got {tuple(shape)}")
    return shape[1] // head_dim, shape[1]


def heads_norm_rotate(tensors, positions, rotation: HeadRotation, weights=None, outs=None, stream=None):
    """``lb_heads_norm_rotate``: the RMS norm of each head (where ``weights``
    has a bf16 [head_dim] weight for the tensor) and the rotation by
    ``positions`` (int32 [tokens] on the device; not read where nothing is
    rotated), for up to 4 tensors bf16
    [tokens, heads * head_dim].  ``outs`` may be the tensors themselves; they
    are allocated when not given.  Returns them."""
    args, device, outs = _heads_forward_call(tensors, positions, rotation, weights, outs, stream)
    _check(lib().lb_heads_norm_rotate(*args, _stream_of(stream, device)), "lb_heads_norm_rotate")
    return outs


def _heads_forward_call(tensors, positions, rotation: HeadRotation, weights, outs, stream) -> tuple:
    """What the binding checks of a heads_norm_rotate call, and the arguments of the library's."""
    torch = _torch()
    bf16, d = torch.bfloat16, rotation.head_dim
    device, tokens, pos, freq = _heads_call(tensors, positions, rotation, weights, "tensors")
    if outs is not None and len(outs) != len(tensors):
        raise ValueError(f"outs must have one entry for each of the {len(tensors)} tensors")
    arr = (LbHeads * len(tensors))()
    made = []
    for j, t in enumerate(tensors):
        e = arr[j]
        e.heads, cols = _heads_of(t, "tensors", d)
        e.ld_in = _rows_ld(t, "tensors", tokens, cols, bf16, device)
        e.in_ = t.data_ptr()
        if outs is None:
            o = _new_dense((tokens, cols), (cols, 1), bf16, device, stream)
            made.append(o)
            e.ld_out = cols
        else:
            o = outs[j]
            e.ld_out = _rows_ld(o, "outs", tokens, cols, bf16, device)
        e.out = o.data_ptr()
        if weights is not None and weights[j] is not None:
            e.weight = _vector_ptr(weights[j], "weights", d, bf16, device)
    args = (tokens, d, rotation.rotary_dim, rotation.code, pos, freq, rotation.eps, len(tensors), arr)
    return args, device, made if outs is None else outs


def _heads_checked(args: tuple) -> None:
    """Raises what the library refuses of a heads call that follows another
    launch, before that launch: what it checks of the sizes also where there are
    no tokens, then the limits of its tensors."""
    name = "lb_heads_norm_rotate"
    _check(lib().lb_heads_norm_rotate(0, *args[1:], None), name)
    arr = args[-1]
    if sum(e.heads for e in arr) > MAX_HEADS or any(max(e.ld_in, e.ld_out) > 1 << 30 for e in arr):
        raise LbError(LB_ERR_UNSUPPORTED_SHAPE, name)
    if any(e.heads < 1 or e.ld_in < e.heads * args[1] or e.ld_out < e.heads * args[1] for e in arr):
        raise LbError(LB_ERR_INVALID_ARGUMENT, name)
    if any(v % 16 for e in arr for v in (e.in_ or 0, e.out or 0, e.weight or 0, 2 * e.ld_in, 2 * e.ld_out)):
        raise LbError(LB_ERR_MISALIGNED, name)


@functools.lru_cache(maxsize=256)
def heads_backward_workspace_bytes(head_dim: int) -> int:
    return int(lib().lb_heads_backward_workspace_bytes(head_dim))


def heads_norm_rotate_backward(tensors, douts, positions, rotation: HeadRotation, weights=None, dins=None,
                               want_dweight: bool = True, workspace=None, stream=None) -> list:
    """``lb_heads_norm_rotate_backward``: the gradients of a loss given
    ``douts`` = dL/dout and the forward call's inputs ``tensors``.  Returns a
    dict for each tensor: ``{"din": bf16 [tokens, heads * head_dim]}``, and
    where it has a norm weight (and ``want_dweight``) ``"dweight": fp32
    [head_dim]``.  ``dins`` may be the douts or the tensors; outputs and the
    workspace are allocated with torch when not given."""
    torch = _torch()
    bf16, d = torch.bfloat16, rotation.head_dim
    device, tokens, pos, freq = _heads_call(tensors, positions, rotation, weights, "tensors")
    n = len(tensors)
    if len(douts) != n or (dins is not None and len(dins) != n):
        raise ValueError(f"douts and dins must have one entry for each of the {n} tensors")
    arr = (LbHeadsGrad * n)()
    out = []
    sums = False
    for j, t in enumerate(tensors):
        e = arr[j]
        e.heads, cols = _heads_of(t, "tensors", d)
        e.ld_in = _rows_ld(t, "tensors", tokens, cols, bf16, device)
        e.in_ = t.data_ptr()
        e.ld_dout = _rows_ld(douts[j], "douts", tokens, cols, bf16, device)
        e.dout = douts[j].data_ptr()
        if dins is None:
            din = _new_dense((tokens, cols), (cols, 1), bf16, device, stream)
            e.ld_din = cols
        else:
            din = dins[j]
            e.ld_din = _rows_ld(din, "dins", tokens, cols, bf16, device)
        e.din = din.data_ptr()
        out.append({"din": din})
        if weights is not None and weights[j] is not None:
            e.weight = _vector_ptr(weights[j], "weights", d, bf16, device)
            if want_dweight:
                dw = _new_dense((d,), (1,), torch.float32, device, stream)
                e.dweight = dw.data_ptr()
                out[j]["dweight"] = dw
                sums = True
    if workspace is None:
        workspace = _new_workspace(tensors[0], heads_backward_workspace_bytes(d) if sums else 0, stream)
    else:
        _require_workspace(workspace, device)
    _check(lib().lb_heads_norm_rotate_backward(tokens, d, rotation.rotary_dim, rotation.code, pos, freq, rotation.eps, n,
                                               arr, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                               _stream_of(stream, device)), "lb_heads_norm_rotate_backward")
    return out


def device_status(stream=None) -> int:
    """``lb_device_status``: synchronise the stream, return and clear the
    device status word (an lb_status code)."""
    out = ctypes.c_int(0)
    _check(lib().lb_device_status(_stream_handle(stream), ctypes.byref(out)), "lb_device_status")
    return int(out.value)


def debug_inject_stall(enable: bool, wait_limit_ns: int = 2_000_000_000) -> None:
    """``lb_debug_inject_stall`` (tests only): make the tcgen05 decode kernels
    enqueued afterwards give up their bounded waits after ``wait_limit_ns``
    and skip one stage-barrier arrival, so that they time out and record
    LB_ERR_DEVICE_TIMEOUT; ``enable=False`` restores the defaults."""
    _check(lib().lb_debug_inject_stall(1 if enable else 0, int(wait_limit_ns) if enable else 0),
           "lb_debug_inject_stall")


def set_prefill_pairs(enable: bool) -> None:
    """``lb_set_prefill_pairs``: let prefill contractions run on CTA pairs
    (the default) or keep them on single-CTA tiles."""
    _check(lib().lb_set_prefill_pairs(1 if enable else 0), "lb_set_prefill_pairs")


class LittleBitLinear:
    """A deployed LittleBit layer: one or two packed paths on the device.

    ``layer(x)`` runs ``lb_linear_forward`` on the current stream;
    ``layer(x, adapters=pool, ids=ids)`` adds each token's low-rank adapter
    (:func:`adapters_forward`)."""

    def __init__(self, main: PackedPath, residual: PackedPath | None = None):
        self.main, self.residual = main, residual
        self.n_out = int(main.h.shape[0])
        self.n_in = int(main.g.shape[0])
        self._ws = None

    @classmethod
    def from_factors(cls, paths: list[dict], device="cuda") -> "LittleBitLinear":
        """``paths``: one or two dicts of host or device arrays ``su`` [n_out, r],
        ``sv`` [n_in, r] (+-1, any supported dtype) and fp16 ``h``, ``g``, ``l``."""
        torch = _torch()
        dev = lambda a: torch.as_tensor(a).to(device)
        packed = [PackedPath.from_factors(dev(p["su"]), dev(p["sv"]), dev(p["h"]), dev(p["g"]),
                                          dev(p["l"])) for p in paths]
        return cls(packed[0], packed[1] if len(packed) > 1 else None)

    def workspace(self, tokens: int, device):
        torch = _torch()
        need = forward_workspace_bytes(tokens, self.n_in, self.n_out, self.main.rank,
                                       self.residual.rank if self.residual else 0)
        if self._ws is None or self._ws.numel() < need:
            self._ws = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
        return self._ws

    def __call__(self, x, y=None, stream=None, adapters: AdapterPool | None = None, ids=None):
        if adapters is not None and ids is None:
            raise ValueError("adapters need ids, each token's adapter")
        if adapters is not None:  # checked before the layer is launched
            if y is None:
                y = _new((x.shape[0], self.n_out), _torch().bfloat16, x.device, stream)
            beside = _adapters_call(x, ids, [adapters], None, [y], stream)
            _adapters_checked(lib().lb_adapters_forward, "lb_adapters_forward", x.shape[0], beside[0])
        # the kept workspace belongs to the current stream
        y = linear_forward(x, self.main, self.residual, y=y, stream=stream,
                           workspace=self.workspace(x.shape[0], x.device) if stream is None else None)
        if adapters is not None:
            _adapters_launch(beside, x, None, stream)
        return y
