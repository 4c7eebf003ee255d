"""Thin ctypes binding over libgdn (include/gdn.h): argument marshalling only.

Every step of the layer runs in the HIP kernels of libgdn.so.  PyTorch is
used for device memory (tensors are passed by data_ptr) and for the current
HIP stream.  There is no fallback: if the library is missing or fails to
load, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdn.so")

GDN_OK = 0
GDN_ERR_INVALID_ARG = -1
GDN_ERR_UNSUPPORTED = -2
GDN_ERR_BAD_INDEX = -3
GDN_ERR_WORKSPACE = -4
GDN_ERR_HIP = -5
GDN_ERR_RING = -6
GDN_ERR_HOST = -7
GDN_F32 = 0
GDN_BF16 = 1
GDN_VALIDATE = 1
GDN_GROUP_KERNEL = 2
GDN_STATIC_SCRATCH_BYTES = 64 << 20
GDN_BLOCK_NORM_MAX_HIDDEN = 16384
GDN_MX_GROUP = 32
GDN_MX_MAX_IN = 1048576
GDN_BEAM_MAX = 64
GDN_LORA_MAX_RANK = 128

EXPORTED = (
    "gdn_pool_bytes", "gdn_pool_create", "gdn_pool_destroy", "gdn_slot_reset",
    "gdn_decode_step", "gdn_verify_step", "gdn_prefill_workspace_bytes",
    "gdn_prefill_chunked", "gdn_prefill_chunked_static", "gdn_prefill_chunked_ckpt",
    "gdn_slot_copy", "gdn_ring_verify",
    "gdn_ring_commit", "gdn_ring_flush", "gdn_in_proj_workspace_bytes", "gdn_in_proj",
    "gdn_pool_error", "gdn_status_string", "gdn_block_norm", "gdn_gated_norm",
    "gdn_mx_quantize", "gdn_mx_dequantize", "gdn_mx_proj_workspace_bytes", "gdn_mx_proj",
    "gdn_mx_in_proj_workspace_bytes", "gdn_mx_in_proj", "gdn_mx_proj_lora_workspace_bytes",
    "gdn_mx_proj_lora", "gdn_mx_in_proj_lora_workspace_bytes", "gdn_mx_in_proj_lora",
    "gdn_batch_maps", "gdn_beam_select_workspace_bytes", "gdn_beam_select", "gdn_slot_reorder",
)


class GdnError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} ({status})")


class PoolDesc(ctypes.Structure):
    _fields_ = [
        ("n_slots", ctypes.c_int32), ("n_layers", ctypes.c_int32),
        ("h_k", ctypes.c_int32), ("h_v", ctypes.c_int32),
        ("d_k", ctypes.c_int32), ("d_v", ctypes.c_int32),
        ("conv_k", ctypes.c_int32), ("io_dtype", ctypes.c_int32),
        ("q_scale", ctypes.c_float), ("norm_eps", ctypes.c_float),
        ("flags", ctypes.c_uint32), ("ring_len", ctypes.c_int32),
    ]


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libgdn.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libgdn.so not found at {path}; build it with "
                           "`python -m gated_deltanet_state_layer_amd.build`")
    lib = ctypes.CDLL(path)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    F32 = ctypes.c_float
    PSZ = ctypes.POINTER(ctypes.c_size_t)
    sig = {
        "gdn_pool_bytes": [ctypes.POINTER(PoolDesc), PSZ, PSZ],
        "gdn_pool_create": [ctypes.POINTER(PoolDesc), P, P, P, ctypes.POINTER(P)],
        "gdn_pool_destroy": [P],
        "gdn_slot_reset": [P, I32, P, P],
        "gdn_slot_copy": [P, I32, P, P, P],
        "gdn_decode_step": [P, I32, I32, P, P, P, P, P, P, P, P, P],
        "gdn_verify_step": [P, I32, I32, P, I32, P, P, P, P, P, P, P, P, P],
        "gdn_prefill_workspace_bytes": [P, I32, I64, I32, PSZ],
        "gdn_prefill_chunked": [P, I32, I32, P, P, I64, I32, P, P, P, P, P, P, P, P, SZ, P],
        "gdn_prefill_chunked_static": [P, I32, I32, P, P, I64, I32, P, P, P, P, P, P, P, P],
        "gdn_prefill_chunked_ckpt": [P, I32, I32, P, P, I64, I32, P, P, P, P, P, P, P, I32, P, P,
                                     P, SZ, P],
        "gdn_ring_verify": [P, I32, I32, P, I32, P, P, P, P, P, P, P, P],
        "gdn_ring_commit": [P, I32, I32, P, I32, P, P, P, P, P, P, P, P],
        "gdn_ring_flush": [P, I32, I32, P, P],
        "gdn_in_proj_workspace_bytes": [P, I64, I32, PSZ],
        "gdn_in_proj": [P, I64, I32, P, P, P, P, P, P, P, P, SZ, P],
        "gdn_pool_error": [P, P, ctypes.POINTER(I32)],
        "gdn_block_norm": [I64, I32, I32, I32, P, I64, P, F32, P, I64, P, I64, P, F32, F32, P, I64,
                           P],
        "gdn_gated_norm": [P, I64, P, I64, P, I64, P, F32, I32, P, I64, P],
        "gdn_mx_quantize": [I64, I32, I32, P, P, P, P],
        "gdn_mx_dequantize": [I64, I32, P, P, I32, P, P],
        "gdn_mx_proj_workspace_bytes": [I64, I32, I32, PSZ],
        "gdn_mx_proj": [I64, I32, I32, P, I64, P, P, I32, P, I64, P, SZ, P],
        "gdn_mx_in_proj_workspace_bytes": [P, I64, I32, I32, PSZ],
        "gdn_mx_in_proj": [P, I64, I32, P, P, P, P, P, P, P, P, P, P, SZ, P],
        "gdn_mx_proj_lora_workspace_bytes": [I64, I32, I32, I32, PSZ],
        "gdn_mx_proj_lora": [I64, I32, I32, P, I64, P, P, I32, I32, P, P, P, P, I32, P, I64, P, SZ, P],
        "gdn_mx_in_proj_lora_workspace_bytes": [P, I64, I32, I32, I32, PSZ],
        "gdn_mx_in_proj_lora": [P, I64, I32, P, P, P, I32, I32, P, P, P, P, P, P, P, P, P, P, P, SZ, P],
        "gdn_batch_maps": [P, I32, P, I64, P, P, P, P, P, P, I32, P, I32, P, I32, P, P, I32, P],
        "gdn_beam_select_workspace_bytes": [I32, I32, I32, I32, PSZ],
        "gdn_beam_select": [I32, I32, I32, I32, I32, P, I64, P, P, I32, P, P, P, P, P, SZ, P],
        "gdn_slot_reorder": [P, I32, I32, P, P, P, P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = I32
    lib.gdn_status_string.argtypes = [I32]
    lib.gdn_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load_library().gdn_status_string(status).decode()


def _check(status: int, what: str):
    if status != GDN_OK:
        raise GdnError(status, what)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _need(t, name, numel, dtype):
    """Host-side check of a tensor argument before it becomes a raw pointer:
    a contiguous device tensor of `dtype` with at least `numel` elements, so
    that no kernel reads or writes past it.  A call that touches no element
    of it (numel 0) accepts anything, None included."""
    if numel <= 0:
        return
    if t is not None and t.dtype is dtype and t.is_cuda and t.is_contiguous() and t.numel() >= numel:
        return
    if t is None:
        raise ValueError(f"{name}: missing")
    if not t.is_cuda:
        raise ValueError(f"{name}: not a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: not contiguous")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.numel() < numel:
        raise ValueError(f"{name}: {t.numel()} elements, the call needs {numel}")


# The current stream's handle without a Stream object around it: 0.2 us of a
# call's host time in place of 2.9 us, the largest share of a small call's 11.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def _io_torch(io_dtype: int):
    return torch.bfloat16 if io_dtype == GDN_BF16 else torch.float32


def make_desc(n_slots, n_layers, h_k, h_v, d_k, d_v, conv_k, io_dtype=GDN_BF16,
              q_scale=0.0, norm_eps=0.0, flags=0, ring_len=0) -> PoolDesc:
    return PoolDesc(n_slots, n_layers, h_k, h_v, d_k, d_v, conv_k, io_dtype,
                    q_scale, norm_eps, flags, ring_len)


def ring_layout(desc: PoolDesc):
    """Byte offsets of the verify ring inside the aux buffer (the layout
    include/gdn.h documents): (count offset, record offset, floats per
    (slot, layer) record block), or None without a ring."""
    if desc.ring_len == 0:
        return None
    up = lambda x, a: (x + a - 1) // a * a
    io = 2 if desc.io_dtype == GDN_BF16 else 4
    sl = desc.n_slots * desc.n_layers
    c_conv = 2 * desc.h_k * desc.d_k + desc.h_v * desc.d_v
    win = sl * (desc.conv_k - 1) * c_conv * io
    cnt = up(win, 256) + 256 + up(sl * desc.h_k * 4, 256)
    rec = cnt + 2 * up(sl * 4, 256)
    stride = up(desc.ring_len * (desc.h_k * desc.d_k + desc.h_v * desc.d_v + 2 * desc.h_v), 64)
    return cnt, rec, stride


def pool_bytes(desc: PoolDesc):
    lib = load_library()
    sb, ab = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib.gdn_pool_bytes(ctypes.byref(desc), ctypes.byref(sb), ctypes.byref(ab)),
           "gdn_pool_bytes")
    return sb.value, ab.value


_DTYPES = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}


def _dtype(t, name):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name}: dtype {t.dtype}, expected bfloat16 or float32")
    return code


def _rows(t, name, shape, dtype):
    """Host-side check of a device tensor of this shape and dtype whose rows
    (everything behind the first dimension) are contiguous; returns the
    elements between rows."""
    if t is not None and t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t.numel() // shape[0] if shape[0] else 0
    if t is None:
        raise ValueError(f"{name}: missing")
    if not t.is_cuda:
        raise ValueError(f"{name}: not a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if shape[0] and not t[0].is_contiguous():
        raise ValueError(f"{name}: rows are not contiguous")
    return t.stride(0)


# Host time is what a small call costs, so the usual case, dense tensors, is
# checked two tensors at a time, and one by one (with the error's name) only
# where that fails: the norm of one token 7.4 -> 6.9 us.
def _dense(shape, dtype, a, b):
    """Whether a and b are contiguous device tensors of this shape and dtype."""
    return (a is not None and b is not None and a.dtype is dtype and b.dtype is dtype and
            a.shape == shape and b.shape == shape and a.is_cuda and b.is_cuda and
            a.is_contiguous() and b.is_contiguous())


def _hold(numel, dtype, a, b):
    """Whether a and b are contiguous device tensors of this dtype with at
    least numel elements."""
    return (a is not None and b is not None and a.dtype is dtype and b.dtype is dtype and
            a.is_cuda and b.is_cuda and a.is_contiguous() and b.is_contiguous() and
            a.numel() >= numel and b.numel() >= numel)


def block_norm(residual, w, out, y=None, w_post=None, residual_out=None, res_scale=1.0,
               w_offset=0.0, eps=1e-6, stream=None):
    """gdn_block_norm: with a block's output y, residual_out = residual +
    res_scale * y (y normalised with w_post first, if given), and out = the
    norm of that sum times (w_offset + w).  Without y, the norm of residual.
    residual and residual_out share one dtype, y and out another."""
    lib = _lib or load_library()
    shape = residual.shape
    if len(shape) != 2:
        raise ValueError(f"residual: shape {tuple(shape)}, expected [tokens, hidden]")
    n, hidden = shape
    rdt, iodt = _dtype(residual, "residual"), _dtype(out, "out")
    if y is not None and _dense(shape, residual.dtype, residual, residual_out) and \
            _dense(shape, out.dtype, out, y):
        ld_r = ld_x = ld_y = ld_ro = hidden
    else:
        ld_r = _rows(residual, "residual", shape, residual.dtype)
        ld_x = _rows(out, "out", shape, out.dtype)
        ld_y = ld_ro = 0
        if y is not None:
            ld_y = _rows(y, "y", shape, out.dtype)
            ld_ro = _rows(residual_out, "residual_out", shape, residual.dtype)
        elif w_post is not None or residual_out is not None:
            raise ValueError("w_post and residual_out need y")
    _need(w, "w", hidden, torch.float32)
    if w_post is not None:
        _need(w_post, "w_post", hidden, torch.float32)
    _check(lib.gdn_block_norm(n, hidden, iodt, rdt, _ptr(y), ld_y, _ptr(w_post), res_scale,
                              residual.data_ptr(), ld_r, _ptr(residual_out), ld_ro, _ptr(w),
                              w_offset, eps, out.data_ptr(), ld_x, _stream(stream)),
           "gdn_block_norm")
    return out


def mx_quantize(src, codes, scales, stream=None):
    """gdn_mx_quantize: src [rows, cols] (bfloat16 or float32) to 4-bit codes
    [rows, cols/2] and scale bytes [rows, cols/32] (both uint8)."""
    lib = load_library()
    rows, cols = src.shape
    code = _dtype(src, "src")
    _need(src, "src", rows * cols, src.dtype)
    _need(codes, "codes", rows * cols // 2, torch.uint8)
    _need(scales, "scales", rows * cols // GDN_MX_GROUP, torch.uint8)
    _check(lib.gdn_mx_quantize(rows, cols, code, _ptr(src), _ptr(codes), _ptr(scales),
                               _stream(stream)), "gdn_mx_quantize")
    return codes, scales


def mx_dequantize(codes, scales, out, stream=None):
    """gdn_mx_dequantize: the weights [rows, cols] (bfloat16 or float32) that
    codes and scales stand for."""
    lib = load_library()
    rows, cols = out.shape
    code = _dtype(out, "out")
    _need(out, "out", rows * cols, out.dtype)
    _need(codes, "codes", rows * cols // 2, torch.uint8)
    _need(scales, "scales", rows * cols // GDN_MX_GROUP, torch.uint8)
    _check(lib.gdn_mx_dequantize(rows, cols, _ptr(codes), _ptr(scales), code, _ptr(out),
                                 _stream(stream)), "gdn_mx_dequantize")
    return out


def mx_proj_workspace_bytes(n_tok, n_in, n_out):
    lib = load_library()
    n = ctypes.c_size_t()
    _check(lib.gdn_mx_proj_workspace_bytes(n_tok, n_in, n_out, ctypes.byref(n)),
           "gdn_mx_proj_workspace_bytes")
    return n.value


def mx_proj(x, codes, scales, out, workspace=None, stream=None):
    """gdn_mx_proj: out [tokens, n_out] (bfloat16 or float32) = x [tokens,
    n_in] (bfloat16) times the transposed 4-bit weights."""
    lib = load_library()
    if x.dim() != 2 or out.dim() != 2:
        raise ValueError("x and out: expected [tokens, channels]")
    (n_tok, n_in), n_out = x.shape, out.shape[1]
    ld_x = _rows(x, "x", (n_tok, n_in), torch.bfloat16)
    ld_y = _rows(out, "out", (n_tok, n_out), out.dtype)
    code = _dtype(out, "out")
    _need(codes, "codes", n_out * n_in // 2, torch.uint8)
    _need(scales, "scales", n_out * n_in // GDN_MX_GROUP, torch.uint8)
    ws_bytes = 0 if workspace is None else workspace.nbytes
    _check(lib.gdn_mx_proj(n_tok, n_in, n_out, _ptr(x), ld_x, _ptr(codes), _ptr(scales), code,
                           _ptr(out), ld_y, _ptr(workspace), ws_bytes, _stream(stream)),
           "gdn_mx_proj")
    return out


def _current_device():
    """The device the library launches on; -2, which no tensor is on, without a
    GPU."""
    try:
        return _device()
    except (RuntimeError, AssertionError, AttributeError):
        return -2


def _want(dev, t, name, numel, dtype):
    """Host-side check of a contiguous tensor of this dtype on device `dev` (the
    current one, where the library launches) with at least numel elements; numel 0
    accepts anything."""
    if numel > 0 and not (t is not None and t.dtype is dtype and t.get_device() == dev and
                          t.is_contiguous() and t.numel() >= numel):
        _need(t, name, numel, dtype)
        _here(dev, t, name)


def _shaped(dev, t, name, shape, dtype):
    """_want of a matrix of this shape."""
    if t is not None and t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return
    if t is None:
        raise ValueError(f"{name}: missing")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, expected {shape}")
    _want(dev, t, name, shape[0] * shape[1], dtype)


def _here(dev, t, name):
    """A tensor that is not on device `dev` is an error."""
    if t.get_device() != dev and t.numel() > 0:
        raise ValueError(f"{name}: on {t.device}, but the current device is cuda:{dev}")


def _workspace(dev, ws):
    """A workspace's pointer and bytes."""
    if ws is None:
        return None, 0
    if ws.get_device() != dev or not ws.is_contiguous():
        if not ws.is_cuda or not ws.is_contiguous():
            raise ValueError("workspace: not a contiguous device tensor")
        _here(dev, ws, "workspace")
    return ws.data_ptr(), ws.nbytes


def _lora_args(dev, a, b, scale, token_adapter, n_tok, n_in, n_out):
    """Checks the adapters' tensors; their count and rank."""
    if a is None or a.dim() != 3 or a.shape[2] != n_in:
        raise ValueError(f"lora_a: expected [adapters, rank, {n_in}]")
    n, rank, _ = a.shape
    if n:
        if b is None or b.shape != (n, n_out, rank):
            raise ValueError(f"lora_b: expected [{n}, {n_out}, {rank}]")
        _want(dev, a, "lora_a", n * rank * n_in, torch.bfloat16)
        _want(dev, b, "lora_b", n * n_out * rank, torch.bfloat16)
        _want(dev, scale, "lora_scale", n, torch.float32)
        _want(dev, token_adapter, "token_adapter", n_tok, torch.int32)
    return n, rank


def mx_proj_lora_workspace_bytes(n_tok, n_in, n_out, rank):
    lib = load_library()
    n = ctypes.c_size_t()
    _check(lib.gdn_mx_proj_lora_workspace_bytes(n_tok, n_in, n_out, rank, ctypes.byref(n)),
           "gdn_mx_proj_lora_workspace_bytes")
    return n.value


def mx_proj_lora(x, codes, scales, lora_a, lora_b, lora_scale, token_adapter, out, workspace=None,
                 stream=None):
    """gdn_mx_proj_lora: mx_proj, and to each token's row lora_scale[i] (x A_i^T)
    B_i^T of its adapter i = token_adapter[token] (-1: none).  lora_a [adapters,
    rank, n_in] and lora_b [adapters, n_out, rank] are bfloat16."""
    lib = _lib or load_library()
    if x.dim() != 2 or out.dim() != 2:
        raise ValueError("x and out: expected [tokens, channels]")
    (n_tok, n_in), n_out = x.shape, out.shape[1]
    ld_x = _rows(x, "x", (n_tok, n_in), torch.bfloat16)
    ld_y = _rows(out, "out", (n_tok, n_out), out.dtype)
    code, dev = _dtype(out, "out"), _current_device()
    _here(dev, x, "x")
    _here(dev, out, "out")
    _want(dev, codes, "codes", n_out * n_in // 2, torch.uint8)
    _want(dev, scales, "scales", n_out * n_in // GDN_MX_GROUP, torch.uint8)
    n, rank = _lora_args(dev, lora_a, lora_b, lora_scale, token_adapter, n_tok, n_in, n_out)
    ws, ws_bytes = _workspace(dev, workspace)
    _check(lib.gdn_mx_proj_lora(n_tok, n_in, n_out, x.data_ptr(), ld_x, codes.data_ptr(),
                                scales.data_ptr(), n, rank, _ptr(lora_a), _ptr(lora_b),
                                _ptr(lora_scale), _ptr(token_adapter), code, out.data_ptr(), ld_y, ws,
                                ws_bytes, _stream(stream)), "gdn_mx_proj_lora")
    return out


def beam_select_workspace_bytes(n_req, width, vocab, n_out):
    lib = load_library()
    n = ctypes.c_size_t()
    _check(lib.gdn_beam_select_workspace_bytes(n_req, width, vocab, n_out, ctypes.byref(n)),
           "gdn_beam_select_workspace_bytes")
    return n.value


def beam_select(logits, scores, parents, tokens, scores_out, finished=None, finished_out=None, eos=-1,
                workspace=None, stream=None):
    """gdn_beam_select: from logits [requests, width, vocab] (bfloat16 or
    float32; rows may be strided, evenly) and the beams' scores [requests, width],
    the best continuations: parents, tokens (int32) and scores_out (float32)
    [requests, n_out]; finished and finished_out are uint8."""
    lib = _lib or load_library()
    if logits.dim() != 3 or scores_out.dim() != 2:
        raise ValueError("logits: expected [requests, width, vocab], scores_out [requests, n_out]")
    n_req, width, vocab = logits.shape
    n_out, dev = scores_out.shape[1], _current_device()
    code = _dtype(logits, "logits")
    ld = vocab
    if not logits.is_contiguous():
        ld = logits.stride(1) if width > 1 else logits.stride(0)
        if (vocab > 1 and logits.stride(2) != 1) or \
                (n_req > 1 and width > 1 and logits.stride(0) != width * ld):
            raise ValueError("logits: rows are not contiguous and evenly spaced")
    if logits.get_device() != dev:
        _need(logits, "logits", max(1, logits.numel()), logits.dtype)
        _here(dev, logits, "logits")
    wide, kept = (n_req, width), (n_req, n_out)
    _shaped(dev, scores, "scores", wide, torch.float32)
    _shaped(dev, parents, "parents", kept, torch.int32)
    _shaped(dev, tokens, "tokens", kept, torch.int32)
    _shaped(dev, scores_out, "scores_out", kept, torch.float32)
    if finished is not None:
        _shaped(dev, finished, "finished", wide, torch.uint8)
    if finished_out is not None:
        _shaped(dev, finished_out, "finished_out", kept, torch.uint8)
    ws, ws_bytes = _workspace(dev, workspace)
    _check(lib.gdn_beam_select(n_req, width, vocab, n_out, code, logits.data_ptr(), ld,
                               scores.data_ptr(), _ptr(finished), eos, parents.data_ptr(),
                               tokens.data_ptr(), scores_out.data_ptr(), _ptr(finished_out), ws,
                               ws_bytes, _stream(stream)), "gdn_beam_select")
    return parents, tokens, scores_out


class Pool:
    """A slot pool over torch-owned device buffers.

    Attributes `state` ([n_slots, n_layers, h_v, d_v, d_k] fp32) and `window`
    ([n_slots, n_layers, conv_k-1, C_conv] io dtype) are views of the pool's
    device memory in the library's documented layout.
    """

    def __init__(self, desc: PoolDesc, device="cuda", stream=None):
        lib = load_library()
        self.desc = desc
        self.device = torch.device(device)
        sb, ab = pool_bytes(desc)
        self._state_buf = torch.empty(sb // 4, dtype=torch.float32, device=self.device)
        self._aux_buf = torch.empty(ab, dtype=torch.uint8, device=self.device)
        h = ctypes.c_void_p()
        _check(lib.gdn_pool_create(ctypes.byref(desc), _ptr(self._state_buf), _ptr(self._aux_buf),
                                   _stream(stream), ctypes.byref(h)), "gdn_pool_create")
        self._h = h
        self.c_conv = 2 * desc.h_k * desc.d_k + desc.h_v * desc.d_v
        self.io_torch = _io_torch(desc.io_dtype)
        self._k_width, self._v_width = desc.h_k * desc.d_k, desc.h_v * desc.d_v
        self.state = self._state_buf.view(desc.n_slots, desc.n_layers, desc.h_v, desc.d_v, desc.d_k)
        io_size = 2 if desc.io_dtype == GDN_BF16 else 4
        nwin = desc.n_slots * desc.n_layers * (desc.conv_k - 1) * self.c_conv
        self.window = self._aux_buf[: nwin * io_size].view(self.io_torch).view(
            desc.n_slots, desc.n_layers, desc.conv_k - 1, self.c_conv)
        rl = ring_layout(desc)
        self.ring_count = self.ring_records = None
        if rl is not None:
            cnt, rec, stride = rl
            sl = desc.n_slots * desc.n_layers
            self.ring_count = self._aux_buf[cnt: cnt + 4 * sl].view(torch.int32).view(
                desc.n_slots, desc.n_layers)
            self.ring_records = self._aux_buf[rec: rec + 4 * sl * stride].view(torch.float32).view(
                desc.n_slots, desc.n_layers, stride)

    def close(self):
        if getattr(self, "_h", None):
            load_library().gdn_pool_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- argument checks (shapes follow include/gdn.h) ----------------------
    def _tokens(self, rows, q, k, v, a, b, conv_w):
        d, io = self.desc, self.io_torch
        _need(q, "q", rows * d.h_k * d.d_k, io)
        _need(k, "k", rows * d.h_k * d.d_k, io)
        _need(v, "v", rows * d.h_v * d.d_v, io)
        _need(a, "a", rows * d.h_v, torch.float32)
        _need(b, "b", rows * d.h_v, torch.float32)
        _need(conv_w, "conv_w", self.c_conv * d.conv_k if rows else 0, torch.float32)

    def _out(self, rows, out):
        _need(out, "out", rows * self.desc.h_v * self.desc.d_v, self.io_torch)

    # -- calls -------------------------------------------------------------
    def reset(self, slot_ids, stream=None):
        lib = load_library()
        _need(slot_ids, "slot_ids", slot_ids.numel(), torch.int32)
        _check(lib.gdn_slot_reset(self._h, int(slot_ids.numel()), _ptr(slot_ids), _stream(stream)),
               "gdn_slot_reset")

    def copy(self, src_ids, dst_ids, stream=None):
        lib = load_library()
        _need(src_ids, "src_ids", src_ids.numel(), torch.int32)
        _need(dst_ids, "dst_ids", src_ids.numel(), torch.int32)
        _check(lib.gdn_slot_copy(self._h, int(src_ids.numel()), _ptr(src_ids), _ptr(dst_ids),
                                 _stream(stream)), "gdn_slot_copy")

    def reorder(self, slots, parents, slots_out, stream=None):
        """gdn_slot_reorder: after beam selection, slot slots_out[r, i] holds
        what slot slots[r, parents[r, i]] held; slots_out [requests, width] is a
        permutation of slots and may be slots itself."""
        lib = _lib or load_library()
        if slots.dim() != 2 or slots.shape != parents.shape or slots.shape != slots_out.shape:
            raise ValueError("slots, parents and slots_out: expected [requests, width]")
        n_req, width = slots.shape
        n, dev = n_req * width, _current_device()
        _want(dev, slots, "slots", n, torch.int32)
        _want(dev, parents, "parents", n, torch.int32)
        _want(dev, slots_out, "slots_out", n, torch.int32)
        _check(lib.gdn_slot_reorder(self._h, n_req, width, slots.data_ptr(), parents.data_ptr(),
                                    slots_out.data_ptr(), _stream(stream)), "gdn_slot_reorder")
        return slots_out

    def batch_maps(self, lens, cu_seqlens, max_tokens=None, last_rows=None, token_seq=None, past=None,
                   token_pos=None, adapter_ids=None, n_adapters=0, token_adapter=None, ckpt_every=0,
                   free_slots=None, ckpt_offsets=None, ckpt_slots=None, stream=None):
        """gdn_batch_maps: from the lengths of a batch's requests, cu_seqlens
        and whichever of the other maps is given (all int32).  The per-token maps
        share one length, the tokens there is room for; without any, max_tokens
        says it."""
        lib = _lib or load_library()
        n, room, dev, i32 = lens.numel(), max_tokens, _current_device(), torch.int32
        for t, name in ((token_seq, "token_seq"), (token_pos, "token_pos"),
                        (token_adapter, "token_adapter")):
            if t is not None:
                if room is None:
                    room = t.numel()
                elif t.numel() != room:
                    raise ValueError(f"{name}: {t.numel()} elements, expected {room}")
                _want(dev, t, name, room, i32)
        if room is None:
            room = 2 ** 31 - 2
        if token_adapter is not None and adapter_ids is None:
            raise ValueError("token_adapter needs adapter_ids")
        _want(dev, lens, "lens", n, i32)
        _want(dev, cu_seqlens, "cu_seqlens", n + 1, i32)
        if last_rows is not None:
            _want(dev, last_rows, "last_rows", n, i32)
        if past is not None:
            _want(dev, past, "past", n, i32)
        if adapter_ids is not None:
            _want(dev, adapter_ids, "adapter_ids", n, i32)
        n_free = max_ckpt = 0
        if ckpt_every > 0:
            _want(dev, ckpt_offsets, "ckpt_offsets", n + 1, i32)
            n_free = 0 if free_slots is None else free_slots.numel()
            max_ckpt = 0 if ckpt_slots is None else ckpt_slots.numel()
            _want(dev, free_slots, "free_slots", n_free, i32)
            _want(dev, ckpt_slots, "ckpt_slots", max_ckpt, i32)
        _check(lib.gdn_batch_maps(self._h, n, _ptr(lens), room, cu_seqlens.data_ptr(), _ptr(last_rows),
                                  _ptr(token_seq), _ptr(past), _ptr(token_pos), _ptr(adapter_ids),
                                  n_adapters, _ptr(token_adapter), ckpt_every, _ptr(free_slots), n_free,
                                  _ptr(ckpt_offsets), _ptr(ckpt_slots), max_ckpt, _stream(stream)),
               "gdn_batch_maps")

    def decode(self, layer, slot_ids, q, k, v, a, b, conv_w, out, stream=None):
        lib = load_library()
        n = int(slot_ids.numel())
        _need(slot_ids, "slot_ids", n, torch.int32)
        self._tokens(n, q, k, v, a, b, conv_w)
        self._out(n, out)
        _check(lib.gdn_decode_step(self._h, layer, int(slot_ids.numel()), _ptr(slot_ids), _ptr(q),
                                   _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(conv_w), _ptr(out),
                                   _stream(stream)), "gdn_decode_step")
        return out

    def verify(self, layer, slot_ids, n_tok, q, k, v, a, b, conv_w, accept_len, out, stream=None):
        lib = load_library()
        n = int(slot_ids.numel())
        _need(slot_ids, "slot_ids", n, torch.int32)
        self._tokens(n * n_tok, q, k, v, a, b, conv_w)
        if accept_len is not None:
            _need(accept_len, "accept_len", n, torch.int32)
        if out is not None:   # None: commit only
            self._out(n * n_tok, out)
        _check(lib.gdn_verify_step(self._h, layer, int(slot_ids.numel()), _ptr(slot_ids), n_tok,
                                   _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(conv_w),
                                   _ptr(accept_len), _ptr(out), _stream(stream)),
               "gdn_verify_step")
        return out

    def ring_verify(self, layer, slot_ids, n_tok, q, k, v, a, b, conv_w, out, stream=None):
        lib = load_library()
        n = int(slot_ids.numel())
        _need(slot_ids, "slot_ids", n, torch.int32)
        self._tokens(n * n_tok, q, k, v, a, b, conv_w)
        self._out(n * n_tok, out)
        _check(lib.gdn_ring_verify(self._h, layer, int(slot_ids.numel()), _ptr(slot_ids), n_tok,
                                   _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(conv_w),
                                   _ptr(out), _stream(stream)), "gdn_ring_verify")
        return out

    def ring_commit(self, layer, slot_ids, n_tok, q, k, v, a, b, conv_w, accept_len, stream=None):
        lib = load_library()
        n = int(slot_ids.numel())
        _need(slot_ids, "slot_ids", n, torch.int32)
        self._tokens(n * n_tok, q, k, v, a, b, conv_w)
        _need(accept_len, "accept_len", n, torch.int32)
        _check(lib.gdn_ring_commit(self._h, layer, int(slot_ids.numel()), _ptr(slot_ids), n_tok,
                                   _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(conv_w),
                                   _ptr(accept_len), _stream(stream)), "gdn_ring_commit")

    def ring_flush(self, layer, slot_ids, stream=None):
        lib = load_library()
        _need(slot_ids, "slot_ids", slot_ids.numel(), torch.int32)
        _check(lib.gdn_ring_flush(self._h, layer, int(slot_ids.numel()), _ptr(slot_ids),
                                  _stream(stream)), "gdn_ring_flush")

    def in_proj_workspace_bytes(self, n_tok, hidden):
        lib = load_library()
        n = ctypes.c_size_t()
        _check(lib.gdn_in_proj_workspace_bytes(self._h, n_tok, hidden, ctypes.byref(n)),
               "gdn_in_proj_workspace_bytes")
        return n.value

    def in_proj(self, x, w, q, k, v, a, b, workspace=None, stream=None):
        """x [n_tok][hidden] bf16, w [C_conv + 2 h_v][hidden] bf16 -> q, k, v, a, b."""
        lib = load_library()
        n_tok, hidden = int(x.shape[0]), int(x.shape[1])
        d = self.desc
        _need(x, "x", n_tok * hidden, torch.bfloat16)
        _need(w, "w", (self.c_conv + 2 * d.h_v) * hidden if n_tok else 0, torch.bfloat16)
        _need(q, "q", n_tok * d.h_k * d.d_k, self.io_torch)
        _need(k, "k", n_tok * d.h_k * d.d_k, self.io_torch)
        _need(v, "v", n_tok * d.h_v * d.d_v, self.io_torch)
        _need(a, "a", n_tok * d.h_v, torch.float32)
        _need(b, "b", n_tok * d.h_v, torch.float32)
        ws_bytes = 0 if workspace is None else workspace.nbytes
        _check(lib.gdn_in_proj(self._h, n_tok, hidden, _ptr(x), _ptr(w), _ptr(q), _ptr(k), _ptr(v),
                               _ptr(a), _ptr(b), _ptr(workspace), ws_bytes, _stream(stream)),
               "gdn_in_proj")

    def prefill_workspace_bytes(self, n_seq, total_tokens, chunk):
        lib = load_library()
        n = ctypes.c_size_t()
        _check(lib.gdn_prefill_workspace_bytes(self._h, n_seq, total_tokens, chunk,
                                               ctypes.byref(n)), "gdn_prefill_workspace_bytes")
        return n.value

    def prefill(self, layer, cu_seqlens, slot_ids, total_tokens, chunk, q, k, v, a, b, conv_w,
                out, workspace=None, stream=None):
        lib = load_library()
        n_seq = int(slot_ids.numel())
        self._prefill_args(n_seq, cu_seqlens, slot_ids, total_tokens, q, k, v, a, b, conv_w, out)
        ws_bytes = 0 if workspace is None else workspace.nbytes
        _check(lib.gdn_prefill_chunked(self._h, layer, n_seq, _ptr(cu_seqlens), _ptr(slot_ids),
                                       total_tokens, chunk, _ptr(q), _ptr(k), _ptr(v), _ptr(a),
                                       _ptr(b), _ptr(conv_w), _ptr(out), _ptr(workspace), ws_bytes,
                                       _stream(stream)), "gdn_prefill_chunked")
        return out

    def prefill_static(self, layer, cu_seqlens, slot_ids, total_tokens, chunk, q, k, v, a, b,
                       conv_w, out, stream=None):
        """gdn_prefill_chunked_static: the workspace is the library's own
        device array (no allocation)."""
        lib = load_library()
        n_seq = int(slot_ids.numel())
        self._prefill_args(n_seq, cu_seqlens, slot_ids, total_tokens, q, k, v, a, b, conv_w, out)
        _check(lib.gdn_prefill_chunked_static(self._h, layer, n_seq, _ptr(cu_seqlens),
                                              _ptr(slot_ids), total_tokens, chunk, _ptr(q),
                                              _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(conv_w),
                                              _ptr(out), _stream(stream)),
               "gdn_prefill_chunked_static")
        return out

    def prefill_ckpt(self, layer, cu_seqlens, slot_ids, total_tokens, chunk, q, k, v, a, b,
                     conv_w, out, ckpt_every, ckpt_offsets, ckpt_slots, workspace=None,
                     stream=None):
        lib = load_library()
        n_seq = int(slot_ids.numel())
        self._prefill_args(n_seq, cu_seqlens, slot_ids, total_tokens, q, k, v, a, b, conv_w, out)
        if ckpt_every > 0:
            _need(ckpt_offsets, "ckpt_offsets", n_seq + 1, torch.int32)
            _need(ckpt_slots, "ckpt_slots", 0 if ckpt_slots is None else ckpt_slots.numel(),
                  torch.int32)
        ws_bytes = 0 if workspace is None else workspace.nbytes
        _check(lib.gdn_prefill_chunked_ckpt(self._h, layer, n_seq, _ptr(cu_seqlens),
                                            _ptr(slot_ids), total_tokens, chunk, _ptr(q), _ptr(k),
                                            _ptr(v), _ptr(a), _ptr(b), _ptr(conv_w), _ptr(out),
                                            ckpt_every, _ptr(ckpt_offsets), _ptr(ckpt_slots),
                                            _ptr(workspace), ws_bytes, _stream(stream)),
               "gdn_prefill_chunked_ckpt")
        return out

    def gated_norm(self, o, z, w, out, eps=1e-6, stream=None):
        """gdn_gated_norm: out [tokens, h_v, d_v] = the per-head norm of o times
        w times z * sigmoid(z).  out may be bfloat16 or float32."""
        lib = load_library()
        d = self.desc
        shape = (o.shape[0], d.h_v, d.d_v)
        if _dense(shape, self.io_torch, o, z):
            ld_o = ld_z = self._v_width
        else:
            ld_o = _rows(o, "o", shape, self.io_torch)
            ld_z = _rows(z, "z", shape, self.io_torch)
        ld_out = _rows(out, "out", shape, out.dtype)
        code = _dtype(out, "out")
        _need(w, "w", d.d_v, torch.float32)
        _check(lib.gdn_gated_norm(self._h, shape[0], _ptr(o), ld_o, _ptr(z), ld_z, _ptr(w), eps,
                                  code, _ptr(out), ld_out, _stream(stream)), "gdn_gated_norm")
        return out

    def mx_in_proj_workspace_bytes(self, n_tok, hidden, with_z=True):
        lib = load_library()
        n = ctypes.c_size_t()
        _check(lib.gdn_mx_in_proj_workspace_bytes(self._h, n_tok, hidden, int(with_z),
                                                  ctypes.byref(n)),
               "gdn_mx_in_proj_workspace_bytes")
        return n.value

    def mx_in_proj(self, x, codes, scales, q, k, v, a, b, z=None, workspace=None, stream=None):
        """gdn_mx_in_proj: x [n_tok, hidden] bf16 times the 4-bit weights whose
        rows are q | k | v | z | a | b (no z rows without z), into the raw
        q, k, v, the gate z and the activated gates a, b."""
        lib = load_library()
        n_tok, hidden = int(x.shape[0]), int(x.shape[1])
        d = self.desc
        h_v, kw, vw, io = d.h_v, self._k_width, self._v_width, self.io_torch
        n_out = self.c_conv + (0 if z is None else vw) + 2 * h_v
        _need(x, "x", n_tok * hidden, torch.bfloat16)
        _need(codes, "codes", n_out * hidden // 2, torch.uint8)
        _need(scales, "scales", n_out * hidden // GDN_MX_GROUP, torch.uint8)
        if not _hold(n_tok * kw, io, q, k):
            _need(q, "q", n_tok * kw, io)
            _need(k, "k", n_tok * kw, io)
        if not _hold(n_tok * vw, io, v, v if z is None else z):
            _need(v, "v", n_tok * vw, io)
            if z is not None:
                _need(z, "z", n_tok * vw, io)
        if not _hold(n_tok * h_v, torch.float32, a, b):
            _need(a, "a", n_tok * h_v, torch.float32)
            _need(b, "b", n_tok * h_v, torch.float32)
        ws_bytes = 0 if workspace is None else workspace.nbytes
        _check(lib.gdn_mx_in_proj(self._h, n_tok, hidden, _ptr(x), _ptr(codes), _ptr(scales),
                                  _ptr(q), _ptr(k), _ptr(v), _ptr(z), _ptr(a), _ptr(b),
                                  _ptr(workspace), ws_bytes, _stream(stream)), "gdn_mx_in_proj")

    def mx_in_proj_lora_workspace_bytes(self, n_tok, hidden, rank, with_z=True):
        lib = load_library()
        n = ctypes.c_size_t()
        _check(lib.gdn_mx_in_proj_lora_workspace_bytes(self._h, n_tok, hidden, rank, int(with_z),
                                                       ctypes.byref(n)),
               "gdn_mx_in_proj_lora_workspace_bytes")
        return n.value

    def mx_in_proj_lora(self, x, codes, scales, lora_a, lora_b, lora_scale, token_adapter, q, k, v, a,
                        b, z=None, workspace=None, stream=None):
        """gdn_mx_in_proj_lora: mx_in_proj with a low-rank adapter per token (see
        mx_proj_lora); the gates' logits get theirs before the activation."""
        lib = _lib or load_library()
        n_tok, hidden = x.shape
        h_v, kw, vw, io = self.desc.h_v, self._k_width, self._v_width, self.io_torch
        n_out, dev = self.c_conv + (0 if z is None else vw) + 2 * h_v, _current_device()
        _want(dev, x, "x", n_tok * hidden, torch.bfloat16)
        _want(dev, codes, "codes", n_out * hidden // 2, torch.uint8)
        _want(dev, scales, "scales", n_out * hidden // GDN_MX_GROUP, torch.uint8)
        if not _hold(n_tok * kw, io, q, k):
            _need(q, "q", n_tok * kw, io)
            _need(k, "k", n_tok * kw, io)
        if not _hold(n_tok * vw, io, v, v if z is None else z):
            _need(v, "v", n_tok * vw, io)
            if z is not None:
                _need(z, "z", n_tok * vw, io)
        if not _hold(n_tok * h_v, torch.float32, a, b):
            _need(a, "a", n_tok * h_v, torch.float32)
            _need(b, "b", n_tok * h_v, torch.float32)
        for t, name in ((q, "q"), (k, "k"), (v, "v"), (a, "a"), (b, "b"), (z, "z")):
            if t is not None:
                _here(dev, t, name)
        n, rank = _lora_args(dev, lora_a, lora_b, lora_scale, token_adapter, n_tok, hidden, n_out)
        ws, ws_bytes = _workspace(dev, workspace)
        _check(lib.gdn_mx_in_proj_lora(self._h, n_tok, hidden, x.data_ptr(), codes.data_ptr(),
                                       scales.data_ptr(), n, rank, _ptr(lora_a), _ptr(lora_b),
                                       _ptr(lora_scale), _ptr(token_adapter), _ptr(q), _ptr(k), _ptr(v),
                                       _ptr(z), _ptr(a), _ptr(b), ws, ws_bytes, _stream(stream)),
               "gdn_mx_in_proj_lora")

    def _prefill_args(self, n_seq, cu_seqlens, slot_ids, total_tokens, q, k, v, a, b, conv_w,
                      out):
        _need(slot_ids, "slot_ids", n_seq, torch.int32)
        _need(cu_seqlens, "cu_seqlens", n_seq + 1 if n_seq else 0, torch.int32)
        self._tokens(int(total_tokens), q, k, v, a, b, conv_w)
        self._out(int(total_tokens), out)

    def error(self, stream=None) -> int:
        lib = load_library()
        e = ctypes.c_int32()
        _check(lib.gdn_pool_error(self._h, _stream(stream), ctypes.byref(e)), "gdn_pool_error")
        return e.value
