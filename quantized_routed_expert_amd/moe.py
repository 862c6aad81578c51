"""Python binding of the C ABI in include/moe.h (argument marshalling only).

Every step of the layer runs in the HIP library libmoe_gfx950.so; this module
only turns torch tensors into device pointers and sizes, passes the current
stream as an int64 and raises on a non-zero status.  It never computes any
part of the layer itself and has no fallback: if the library is missing it
raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_gfx950.so")

MOE_OK = 0
MOE_ERR_INVALID_ARG = -1
MOE_ERR_UNSUPPORTED = -2
MOE_ERR_WORKSPACE = -3
MOE_ERR_LAUNCH = -4
MOE_ERR_DEVICE = -5

DTYPE_F32, DTYPE_BF16 = 0, 1
PATH_AUTO, PATH_DECODE, PATH_PREFILL = 0, 1, 2
DECODE_MAX_ROWS = 16
LAYOUT_ROWS, LAYOUT_PREPARED = 0, 1
ACT_NONE, ACT_SILU, ACT_GELU, ACT_GELU_TANH, ACT_RELU = 0, 1, 2, 3, 4

EXPORTS = ["moe_version", "moe_status_string", "moe_expert_bytes", "moe_workspace_bytes",
           "moe_prepare_qweights", "moe_workspace_error", "moe_router_logits", "moe_route", "moe_group", "moe_expert_ffn",
           "moe_layer_forward", "moe_layer_forward_noalloc",
           "moe_linear_workspace_bytes", "moe_linear", "moe_linear_backward",
           "moe_gated_ffn_workspace_bytes", "moe_gated_ffn", "moe_gated_ffn_backward"]
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024

# bits of the workspace error word (moe_workspace_error)
ERR_WAIT_TIMEOUT = 1
ERR_BAD_GROUPING = 2


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} ({status})")
        self.status = status


class QWeights(ctypes.Structure):
    """moe_qweights: device pointer + format and shape of a set of experts."""
    _fields_ = [("data", ctypes.c_void_p), ("bits", ctypes.c_int32), ("n_experts", ctypes.c_int32),
                ("hidden", ctypes.c_int32), ("ffn", ctypes.c_int32), ("layout", ctypes.c_int32),
                ("down_bits", ctypes.c_int32), ("codebook", ctypes.c_int8 * 16)]


class DenseFFN(ctypes.Structure):
    """moe_dense_ffn: device pointers, sizes and activation of a dense gated
    feed-forward block (see dense_ffn, which keeps the tensors alive)."""
    _fields_ = [("gate", ctypes.c_void_p), ("up", ctypes.c_void_p), ("down", ctypes.c_void_p),
                ("hidden", ctypes.c_int32), ("ffn", ctypes.c_int32), ("act", ctypes.c_int32)]


BITS_NL4 = 20  # the non-linear 4-bit format (4-bit layout, codes index a 16-entry int8 table)


def _qw(data_ptr, bits, n_experts, hidden, ffn, layout, down_bits, codebook) -> QWeights:
    q = QWeights(ctypes.c_void_p(data_ptr), bits, n_experts, hidden, ffn, layout, down_bits)
    if codebook is not None:
        cb = [int(v) for v in codebook]
        if len(cb) != 16 or any(v < -128 or v > 127 for v in cb):
            raise ValueError("codebook: 16 values in -128..127")
        q.codebook = (ctypes.c_int8 * 16)(*cb)
    return q


_lib = None


def lib():
    """The loaded library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"HIP library not built: {LIB_PATH} (run quantized_routed_expert_amd.build)")
        L = ctypes.CDLL(LIB_PATH)
        i32, i64, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
        L.moe_version.restype = ctypes.c_int
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_status_string.argtypes = [ctypes.c_int]
        L.moe_expert_bytes.restype = i64
        L.moe_expert_bytes.argtypes = [i32, i32, i32, i32]
        L.moe_workspace_bytes.restype = i64
        L.moe_workspace_bytes.argtypes = [i32] * 7
        L.moe_prepare_qweights.restype = ctypes.c_int
        L.moe_prepare_qweights.argtypes = [ctypes.POINTER(QWeights), vp, i64]
        L.moe_workspace_error.restype = ctypes.c_int
        L.moe_workspace_error.argtypes = [vp, i64, ctypes.POINTER(ctypes.c_uint32), i32, i64]
        L.moe_router_logits.restype = ctypes.c_int
        L.moe_router_logits.argtypes = [vp, i32, i32, i32, vp, i32, vp, i64]
        L.moe_route.restype = ctypes.c_int
        L.moe_route.argtypes = [vp, i32, i32, i32, vp, vp, i64]
        L.moe_group.restype = ctypes.c_int
        L.moe_group.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, i64, i64]
        L.moe_expert_ffn.restype = ctypes.c_int
        L.moe_expert_ffn.argtypes = [vp, i32, i32, ctypes.POINTER(QWeights), vp, vp, vp, vp, i32, vp, i32,
                                     vp, i64, i64]
        L.moe_layer_forward.restype = ctypes.c_int
        L.moe_layer_forward.argtypes = [vp, i32, vp, i32, i32, ctypes.POINTER(QWeights),
                                        ctypes.POINTER(QWeights), vp, vp, vp, vp, i32, vp, i64, i64]
        L.moe_layer_forward_noalloc.restype = ctypes.c_int
        L.moe_layer_forward_noalloc.argtypes = [vp, i32, vp, i32, i32, ctypes.POINTER(QWeights),
                                                ctypes.POINTER(QWeights), vp, vp, vp, vp, i32, i64]
        ffn = ctypes.POINTER(DenseFFN)
        L.moe_linear_workspace_bytes.restype = i64
        L.moe_linear_workspace_bytes.argtypes = [i32] * 3
        L.moe_linear.restype = ctypes.c_int
        L.moe_linear.argtypes = [vp, i32, i32, i32, vp, i32, vp, i32, vp, i32, vp, vp, i32, vp, i64, i64]
        L.moe_linear_backward.restype = ctypes.c_int
        L.moe_linear_backward.argtypes = [vp, i32, i32, i32, vp, vp, vp, i32, vp, vp, vp, i32, i32, vp, i64, i64]
        L.moe_gated_ffn_workspace_bytes.restype = i64
        L.moe_gated_ffn_workspace_bytes.argtypes = [i32] * 3
        L.moe_gated_ffn.restype = ctypes.c_int
        L.moe_gated_ffn.argtypes = [vp, i32, i32, ffn, vp, i32, vp, vp, i32, vp, i64, i64]
        L.moe_gated_ffn_backward.restype = ctypes.c_int
        L.moe_gated_ffn_backward.argtypes = [vp, vp, i32, ffn, vp, vp, vp, vp, vp, i32, i32, vp, i64, i64]
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def _check(rc: int, where: str):
    if rc != MOE_OK:
        raise MoeError(rc, where)


def _ptr(t):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _xcode(x: torch.Tensor) -> int:
    if x.dtype == torch.float32:
        return DTYPE_F32
    if x.dtype == torch.bfloat16:
        return DTYPE_BF16
    raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")


def qweights_at(data_ptr, bits: int, n_experts: int, hidden: int, ffn: int, layout: int,
                down_bits: int = 0, codebook=None) -> QWeights:
    """QWeights for a raw device address (an int or ctypes.c_void_p)."""
    if isinstance(data_ptr, ctypes.c_void_p):
        data_ptr = data_ptr.value
    return _qw(data_ptr, bits, n_experts, hidden, ffn, layout, down_bits, codebook)


def qweights(data: torch.Tensor, bits: int, n_experts: int, hidden: int, ffn: int, layout: int,
             down_bits: int = 0, codebook=None) -> QWeights:
    """Describe a uint8 device tensor holding n_experts expert blobs in the
    given block order (LAYOUT_ROWS or LAYOUT_PREPARED); gate/up in `bits`,
    down in `down_bits` (0: the same); codebook: the 16 int8 values of the
    non-linear format (BITS_NL4)."""
    return _qw(data.data_ptr(), bits, n_experts, hidden, ffn, layout, down_bits, codebook)


def prepare_qweights(data: torch.Tensor, bits: int, n_experts: int, hidden: int, ffn: int, out=None,
                     stream=None, down_bits: int = 0, codebook=None):
    """Blobs in the pages' row-by-row order (uint8 device tensor) -> a new
    tensor in the order the compute calls read; returns (tensor, QWeights)."""
    if out is None:
        out = torch.empty_like(data)
    src = _qw(data.data_ptr(), bits, n_experts, hidden, ffn, LAYOUT_ROWS, down_bits, codebook)
    _check(lib().moe_prepare_qweights(ctypes.byref(src), _ptr(out), _stream(stream)), "moe_prepare_qweights")
    return out, qweights(out, bits, n_experts, hidden, ffn, LAYOUT_PREPARED, down_bits, codebook)


def expert_bytes(bits: int, hidden: int, ffn: int, down_bits: int = 0) -> int:
    return int(lib().moe_expert_bytes(bits, down_bits, hidden, ffn))


def workspace_bytes(T: int, E: int, k: int, hidden: int, ffn: int, shared_ffn: int = 0,
                    path: int = PATH_AUTO) -> int:
    n = int(lib().moe_workspace_bytes(T, E, k, hidden, ffn, shared_ffn, path))
    if n < 0:
        raise MoeError(n, "moe_workspace_bytes")
    return n


def workspace(T, E, k, hidden, ffn, shared_ffn=0, path=PATH_AUTO, device="cuda") -> torch.Tensor:
    """A zero-filled workspace of the required size (uint8 device tensor)."""
    return torch.zeros(max(workspace_bytes(T, E, k, hidden, ffn, shared_ffn, path), 1), dtype=torch.uint8,
                       device=device)


def workspace_error(ws: torch.Tensor, clear: bool = True, stream=None) -> int:
    """The workspace's device error word (0 after correct calls); waits for
    the stream and, with clear, resets the word."""
    v = ctypes.c_uint32(0)
    _check(lib().moe_workspace_error(_ptr(ws), ws.numel(), ctypes.byref(v), 1 if clear else 0, _stream(stream)),
           "moe_workspace_error")
    return int(v.value)


def router_logits(x: torch.Tensor, w_router: torch.Tensor, logits=None, stream=None) -> torch.Tensor:
    """x [T, H] fp32/bf16, w_router [E, H] bf16 (device) -> logits [T, E] fp32."""
    T, H = x.shape
    E = w_router.shape[0]
    if w_router.dtype != torch.bfloat16 or tuple(w_router.shape) != (E, H):
        raise TypeError("w_router must be a bf16 [E, H] tensor")
    if logits is None:
        logits = torch.empty((T, E), dtype=torch.float32, device=x.device)
    _check(lib().moe_router_logits(_ptr(x), _xcode(x), T, H, _ptr(w_router), E, _ptr(logits), _stream(stream)),
           "moe_router_logits")
    return logits


def route(logits: torch.Tensor, k: int, topk_idx=None, topk_w=None, stream=None):
    T, E = logits.shape
    if topk_idx is None:
        topk_idx = torch.empty((T, k), dtype=torch.int32, device=logits.device)
    if topk_w is None:
        topk_w = torch.empty((T, k), dtype=torch.float32, device=logits.device)
    _check(lib().moe_route(_ptr(logits), T, E, k, _ptr(topk_idx), _ptr(topk_w), _stream(stream)), "moe_route")
    return topk_idx, topk_w


def group(topk_idx: torch.Tensor, E: int, ws: torch.Tensor, offsets=None, pairs=None, active=None,
          stream=None):
    T, k = topk_idx.shape
    dev = topk_idx.device
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev) if offsets is None else offsets
    pairs = torch.empty(max(T * k, 1), dtype=torch.int32, device=dev) if pairs is None else pairs
    active = torch.empty(E + 1, dtype=torch.int32, device=dev) if active is None else active
    _check(lib().moe_group(_ptr(topk_idx), T, E, k, _ptr(offsets), _ptr(pairs), _ptr(active), _ptr(ws),
                           ws.numel(), _stream(stream)), "moe_group")
    return offsets, pairs, active


def expert_ffn(x: torch.Tensor, w: QWeights, offsets, pairs, active, k: int, out_pairs: torch.Tensor,
               ws: torch.Tensor, pair_w=None, path: int = PATH_AUTO, stream=None):
    T = x.shape[0]
    _check(lib().moe_expert_ffn(_ptr(x), _xcode(x), T, ctypes.byref(w), _ptr(offsets), _ptr(pairs),
                                _ptr(active), _ptr(pair_w), k, _ptr(out_pairs), path, _ptr(ws), ws.numel(),
                                _stream(stream)), "moe_expert_ffn")
    return out_pairs


def layer_forward(x: torch.Tensor, logits: torch.Tensor, k: int, routed: QWeights, shared: QWeights | None,
                  y: torch.Tensor, ws: torch.Tensor, topk_idx=None, topk_w=None, path: int = PATH_AUTO,
                  stream=None, heat=None):
    """heat: optional int32 [E] device tensor; the call adds its per-expert
    pair counts to it (routing heat)."""
    T = x.shape[0]
    _check(lib().moe_layer_forward(_ptr(x), _xcode(x), _ptr(logits), T, k, ctypes.byref(routed),
                                   ctypes.byref(shared) if shared is not None else None, _ptr(y),
                                   _ptr(topk_idx), _ptr(topk_w), _ptr(heat), path, _ptr(ws), ws.numel(),
                                   _stream(stream)),
           "moe_layer_forward")
    return y


def layer_forward_noalloc(x: torch.Tensor, logits: torch.Tensor, k: int, routed: QWeights,
                          shared: QWeights | None, y: torch.Tensor, topk_idx=None, topk_w=None,
                          path: int = PATH_AUTO, stream=None, heat=None):
    """moe_layer_forward_noalloc: the layer with the library's static device
    scratch instead of a workspace (nothing is allocated)."""
    T = x.shape[0]
    _check(lib().moe_layer_forward_noalloc(_ptr(x), _xcode(x), _ptr(logits), T, k, ctypes.byref(routed),
                                           ctypes.byref(shared) if shared is not None else None, _ptr(y),
                                           _ptr(topk_idx), _ptr(topk_w), _ptr(heat), path, _stream(stream)),
           "moe_layer_forward_noalloc")
    return y


# ---------------------------------------------------------------------------
# Dense operators (bf16 weights): linear and the gated feed-forward block
# ---------------------------------------------------------------------------
_CODES = {torch.float32: DTYPE_F32, torch.bfloat16: DTYPE_BF16}


def _dense(name: str, t, shape: tuple, dtypes: tuple, dev: int):
    """Checks an operand of a dense operator (not None) on device index dev (-1: the host); returns its address."""
    if t.shape == shape and t.dtype in dtypes and t.get_device() == dev and t.is_contiguous():
        return t.data_ptr()
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, other operands are on {f'cuda:{dev}' if dev >= 0 else 'the host'}")
    raise ValueError(f"{name} must be contiguous")


def _need(name: str, t):
    if t is None:
        raise TypeError(f"{name} is required")
    return t


def _code(t) -> int:
    return DTYPE_F32 if t is None else _CODES[t.dtype]


_ANY, _BF16 = (torch.float32, torch.bfloat16), (torch.bfloat16,)


def _dense_device(x: torch.Tensor, ws: torch.Tensor) -> int:
    """The operands' device index: a GPU, the current one (launches go there)."""
    dev = x.get_device()
    if dev < 0:
        raise ValueError("dense operators take device tensors")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"operands on cuda:{dev}, but the current device is cuda:{torch.cuda.current_device()}")
    if ws.get_device() != dev or ws.dtype is not torch.uint8 or not ws.is_contiguous():
        raise ValueError(f"ws must be a contiguous uint8 tensor on cuda:{dev}")
    return dev


def _dense_stream(stream, dev: int) -> int:
    # (the current stream's handle without a Stream object: 0.1 us a call instead of 2.7)
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _dense_new(shape: tuple, dtype: torch.dtype, dev: int, stream) -> torch.Tensor:
    """A new output, allocated for the stream that writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if isinstance(stream, int):  # (0: the null stream)
        stream = torch.cuda.ExternalStream(stream, device=dev) if stream else torch.cuda.default_stream(dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def linear_workspace_bytes(T: int, inner: int, outer: int) -> int:
    n = int(lib().moe_linear_workspace_bytes(T, inner, outer))
    if n < 0:
        raise MoeError(n, "moe_linear_workspace_bytes")
    return n


def linear_workspace(T: int, inner: int, outer: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for linear and linear_backward, up to T rows."""
    return torch.zeros(linear_workspace_bytes(T, inner, outer), dtype=torch.uint8, device=device)


def linear(x: torch.Tensor, w: torch.Tensor, ws: torch.Tensor, bias=None, act: int = ACT_NONE, residual=None, z=None,
           y=None, stream=None) -> torch.Tensor:
    """y = act(x w^T + bias) + residual.  x [T, in] fp32/bf16, w [out, in]
    bf16, bias [out] bf16, residual and y [T, out] fp32/bf16 (y: x's type
    unless given; y may be the residual).  z: bf16 [T, out], receives the
    pre-activation for linear_backward."""
    dev = _dense_device(x, ws)
    T, K = x.shape
    N = w.shape[0]
    if y is None:
        y = _dense_new((T, N), x.dtype, dev, stream)
    out = (T, N)
    px = _dense("x", x, (T, K), _ANY, dev)
    pw = _dense("w", w, (N, K), _BF16, dev)
    pb = None if bias is None else _dense("bias", bias, (N,), _BF16, dev)
    pr = None if residual is None else _dense("residual", residual, out, _ANY, dev)
    pz = None if z is None else _dense("z", z, out, _BF16, dev)
    py = _dense("y", y, out, _ANY, dev)
    rc = lib().moe_linear(px, _CODES[x.dtype], T, K, pw, N, pb, act, pr, _code(residual), pz, py, _CODES[y.dtype],
                          ws.data_ptr(), ws.numel(), _dense_stream(stream, dev))
    if rc:
        raise MoeError(rc, "moe_linear")
    return y


def linear_backward(dy: torch.Tensor, x, w, ws: torch.Tensor, z=None, act: int = ACT_NONE, dx=None, dw=None, dbias=None,
                    accumulate: bool = False, stream=None) -> None:
    """Gradients of linear into the given tensors: dx [T, in] bf16 (needs w),
    dw [out, in] (needs x) and dbias [out] fp32/bf16 of one type; with
    accumulate, dw and dbias are added to.  dy [T, out], x, w bf16; z as
    linear wrote it (needed with an activation)."""
    dev = _dense_device(dy, ws)
    T, N = dy.shape
    K = next((t.shape[-1] for t in (dx, dw, x, w) if t is not None), 8)
    pd = _dense("dy", dy, (T, N), _BF16, dev)
    px = None if dw is None and x is None else _dense("x", _need("x", x), (T, K), _BF16, dev)
    pw = None if dx is None and w is None else _dense("w", _need("w", w), (N, K), _BF16, dev)
    pz = None if act == ACT_NONE and z is None else _dense("z", _need("z", z), (T, N), _BF16, dev)
    pdx = None if dx is None else _dense("dx", dx, (T, K), _BF16, dev)
    pdw = None if dw is None else _dense("dw", dw, (N, K), _ANY, dev)
    pdb = None if dbias is None else _dense("dbias", dbias, (N,), _ANY, dev)
    if dw is not None and dbias is not None and dw.dtype != dbias.dtype:
        raise TypeError("dw and dbias must have one type")
    rc = lib().moe_linear_backward(pd, T, K, N, px, pw, pz, act, pdx, pdw, pdb, _code(dbias if dw is None else dw),
                                   int(accumulate), ws.data_ptr(), ws.numel(), _dense_stream(stream, dev))
    if rc:
        raise MoeError(rc, "moe_linear_backward")


def dense_ffn(gate: torch.Tensor, up: torch.Tensor, down: torch.Tensor, act: int = ACT_SILU) -> DenseFFN:
    """Describe a dense gated feed-forward block: gate, up [ffn, hidden] and
    down [hidden, ffn], bf16 device tensors (kept alive by the result)."""
    F, H = gate.shape
    pg = _dense("gate", gate, (F, H), _BF16, gate.get_device())
    pu = _dense("up", up, (F, H), _BF16, gate.get_device())
    pd = _dense("down", down, (H, F), _BF16, gate.get_device())
    d = DenseFFN(pg, pu, pd, H, F, act)
    d.tensors = (gate, up, down)
    d.device = gate.get_device()
    return d


def _ffn_device(ffn: DenseFFN, dev: int) -> None:
    if getattr(ffn, "device", dev) != dev:  # (a description without tensors: its addresses are the caller's word)
        raise ValueError(f"the block's weights are on device {ffn.device}, the other operands on cuda:{dev}")


def gated_ffn_workspace_bytes(T: int, hidden: int, ffn: int) -> int:
    n = int(lib().moe_gated_ffn_workspace_bytes(T, hidden, ffn))
    if n < 0:
        raise MoeError(n, "moe_gated_ffn_workspace_bytes")
    return n


def gated_ffn_workspace(T: int, hidden: int, ffn: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace for gated_ffn and gated_ffn_backward, up to T rows."""
    return torch.zeros(gated_ffn_workspace_bytes(T, hidden, ffn), dtype=torch.uint8, device=device)


def gated_ffn(x: torch.Tensor, ffn: DenseFFN, ws: torch.Tensor, residual=None, gu=None, y=None, stream=None) -> torch.Tensor:
    """y = (act(x gate^T) * (x up^T)) down^T + residual.  x [T, hidden],
    residual and y [T, hidden] fp32/bf16 (y: x's type unless given; y may be
    the residual).  gu: bf16 [T, 2*ffn], receives gate and up for
    gated_ffn_backward."""
    dev = _dense_device(x, ws)
    _ffn_device(ffn, dev)
    T = x.shape[0]
    H, F = ffn.hidden, ffn.ffn
    if y is None:
        y = _dense_new((T, H), x.dtype, dev, stream)
    out = (T, H)
    px = _dense("x", x, out, _ANY, dev)
    pr = None if residual is None else _dense("residual", residual, out, _ANY, dev)
    pg = None if gu is None else _dense("gu", gu, (T, 2 * F), _BF16, dev)
    py = _dense("y", y, out, _ANY, dev)
    rc = lib().moe_gated_ffn(px, _CODES[x.dtype], T, ffn, pr, _code(residual), pg, py, _CODES[y.dtype], ws.data_ptr(),
                             ws.numel(), _dense_stream(stream, dev))
    if rc:
        raise MoeError(rc, "moe_gated_ffn")
    return y


def gated_ffn_backward(dy: torch.Tensor, x, gu: torch.Tensor, ffn: DenseFFN, ws: torch.Tensor, dx=None, dgate=None,
                       dup=None, ddown=None, accumulate: bool = False, stream=None) -> None:
    """Gradients of gated_ffn into the given tensors: dx [T, hidden] bf16,
    dgate, dup [ffn, hidden] and ddown [hidden, ffn] fp32/bf16 of one type;
    with accumulate, the weight gradients are added to.  dy, x [T, hidden]
    bf16 (x is needed for dgate and dup); gu as gated_ffn wrote it."""
    dev = _dense_device(dy, ws)
    _ffn_device(ffn, dev)
    T = dy.shape[0]
    H, F = ffn.hidden, ffn.ffn
    out = (T, H)
    pd = _dense("dy", dy, out, _BF16, dev)
    px = None if dgate is None and dup is None and x is None else _dense("x", _need("x", x), out, _BF16, dev)
    pg = _dense("gu", _need("gu", gu), (T, 2 * F), _BF16, dev)
    pdx = None if dx is None else _dense("dx", dx, out, _BF16, dev)
    given = [(n, t, s) for n, t, s in (("dgate", dgate, (F, H)), ("dup", dup, (F, H)), ("ddown", ddown, (H, F)))
             if t is not None]
    p = {n: _dense(n, t, s, _ANY, dev) for n, t, s in given}
    if len({t.dtype for _, t, _ in given}) > 1:
        raise TypeError("dgate, dup and ddown must have one type")
    rc = lib().moe_gated_ffn_backward(pd, px, T, ffn, pg, pdx, p.get("dgate"), p.get("dup"), p.get("ddown"),
                                      _code(given[0][1] if given else None), int(accumulate), ws.data_ptr(), ws.numel(),
                                      _dense_stream(stream, dev))
    if rc:
        raise MoeError(rc, "moe_gated_ffn_backward")
