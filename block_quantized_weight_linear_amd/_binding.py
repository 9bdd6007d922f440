"""ctypes binding of include/q8_linear.h.

Argument marshalling only: checks tensor dtypes/devices, allocates outputs with
torch when none are given, passes raw device pointers, sizes and torch's current
HIP stream, and turns a non-zero status into Q8Error.  Every step of the
computation runs in the HIP library; there is no fallback.  Importing raises if
the library has not been built.
"""

from __future__ import annotations

import ctypes
import os

# torch ships its own HIP runtime (libamdhip64.so.7).  The library links the same
# soname, and the first copy loaded serves the whole process; importing torch first
# makes that torch's copy, so tensors, streams and our kernels share one runtime.
import torch  # noqa: F401  (imported for its side effect on the loaded HIP runtime)

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libq8linear.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: the HIP library has not been built "
        "(python -m block_quantized_weight_linear_amd.build)")

lib = ctypes.CDLL(LIB_PATH)

_i64, _i32, _vp, _sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t

lib.q8_abi_version.restype = _i32
lib.q8_abi_version.argtypes = []
lib.q8_status_string.restype = ctypes.c_char_p
lib.q8_status_string.argtypes = [ctypes.c_int]
lib.q8_last_error.restype = ctypes.c_char_p
lib.q8_last_error.argtypes = []
lib.q8_linear.restype = ctypes.c_int
lib.q8_linear.argtypes = [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp]
lib.q8_linear_fused_gate_up_silu.restype = ctypes.c_int
lib.q8_linear_fused_gate_up_silu.argtypes = [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp]
lib.q4_0_linear.restype = ctypes.c_int
lib.q4_0_linear.argtypes = [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp]
lib.q4_0_linear_fused_gate_up_silu.restype = ctypes.c_int
lib.q4_0_linear_fused_gate_up_silu.argtypes = [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp]
for _name in ("q4_k_linear", "q4_k_linear_fused_gate_up_silu", "q5_k_linear", "q5_k_linear_fused_gate_up_silu",
              "q6_k_linear", "q6_k_linear_fused_gate_up_silu"):
    getattr(lib, _name).restype = ctypes.c_int
    getattr(lib, _name).argtypes = [_vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp]
lib.q8_quantize_act.restype = ctypes.c_int
lib.q8_quantize_act.argtypes = [_vp, _i64, _i64, _i64, _vp, _vp, _vp]
lib.q8_linear_q8act.restype = ctypes.c_int
lib.q8_linear_q8act.argtypes = [_vp, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _vp]
lib.q8_linear_fused_gate_up_silu_q8act.restype = ctypes.c_int
lib.q8_linear_fused_gate_up_silu_q8act.argtypes = [_vp, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _vp]
lib.moe_route_topk.restype = ctypes.c_int
lib.moe_route_topk.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _i32, _i32, _vp, _vp, _vp]
lib.moe_route_topk_top_p.restype = ctypes.c_int
lib.moe_route_topk_top_p.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _i32, _i32, ctypes.c_float, _vp, _vp, _vp]
lib.moe_route_workspace_bytes.restype = _sz
lib.moe_route_workspace_bytes.argtypes = [_i64, _i64]
lib.moe_route_topk_ws.restype = ctypes.c_int
lib.moe_route_topk_ws.argtypes = [_vp, _i64, _i64, _i64, _vp, _i64, _i32, _i32, ctypes.c_float, _vp, _vp, _vp, _sz,
                                  _vp]
lib.q8_moe_workspace_bytes.restype = _sz
lib.q8_moe_workspace_bytes.argtypes = [_i64, _i32, _i64, _i64, _i64]
lib.q8_moe_grouped_linear.restype = ctypes.c_int
lib.q8_moe_grouped_linear.argtypes = [_vp, _vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i32, _vp, _i64,
                                      _vp, _sz, _vp]

lib.q8_moe_grouped_linear_noalloc.restype = ctypes.c_int
lib.q8_moe_grouped_linear_noalloc.argtypes = [_vp, _vp, _i64, _i64, _i64, _vp, _i64, _i64, _vp, _vp, _i32, _vp,
                                              _i64, _vp]



class _Lora(ctypes.Structure):
    """struct q8_lora"""
    _fields_ = [("a", _vp), ("b", _vp), ("ranks", _vp), ("scale", _vp), ("adapter", _vp),
                ("section_rows", _i64 * 4), ("type", _i32), ("n_adapters", _i32), ("rank", _i32),
                ("n_sections", _i32)]


_lp = ctypes.POINTER(_Lora)
lib.q8_linear_lora_workspace_bytes.restype = _sz
lib.q8_linear_lora_workspace_bytes.argtypes = [_i64, _i64, _i64, _lp]
for _name in ("q8_linear_lora", "q8_linear_fused_gate_up_silu_lora"):
    getattr(lib, _name).restype = ctypes.c_int
    getattr(lib, _name).argtypes = [_vp, _i64, _i64, _vp, _i64, _i64, _lp, _vp, _i64, _vp, _sz, _vp]
lib.lora_workspace_bytes.restype = _sz
lib.lora_workspace_bytes.argtypes = [_i64, _lp]
for _name in ("lora_add", "lora_gate_up_silu"):
    getattr(lib, _name).restype = ctypes.c_int
    getattr(lib, _name).argtypes = [_vp, _i64, _i64, _vp, _i64, _i64, _i64, _lp, _vp, _i64, _vp, _sz, _vp]
lib.q8_moe_layer_workspace_bytes.restype = _sz
lib.q8_moe_layer_workspace_bytes.argtypes = [_i64, _i32, _i64, _i64, _i64]
lib.q8_moe_layer.restype = ctypes.c_int
lib.q8_moe_layer.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _i64, _i64, _i32, _i32, ctypes.c_float, _vp, _i64,
                             _vp, _sz, _vp]

for _name in ("f8_quantize_act", "f8_quantize_weight"):
    getattr(lib, _name).restype = ctypes.c_int
    getattr(lib, _name).argtypes = [_vp, _i32, _i64, _i64, _i64, _i32, _vp, _vp, _vp]
lib.f8_linear.restype = ctypes.c_int
lib.f8_linear.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _i32, _i64, _vp]
lib.f8_linear_fused_gate_up_silu.restype = ctypes.c_int
lib.f8_linear_fused_gate_up_silu.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _i32, _i64, _vp, _i64, _vp]
for _name in ("f8_linear_backward_workspace_bytes", "f8_linear_fused_gate_up_silu_backward_workspace_bytes"):
    getattr(lib, _name).restype = _sz
    getattr(lib, _name).argtypes = [_i64, _i64, _i64, _i32]
lib.f8_linear_backward.restype = ctypes.c_int
lib.f8_linear_backward.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _i32, _i64, _vp, _i64, _vp, _i64, _vp,
                                   _sz, _vp]
lib.f8_linear_fused_gate_up_silu_backward.restype = ctypes.c_int
lib.f8_linear_fused_gate_up_silu_backward.argtypes = [_vp, _vp, _i64, _i64, _vp, _vp, _i64, _vp, _i64, _vp, _i32, _i64,
                                                      _vp, _i64, _vp, _i64, _vp, _sz, _vp]

# measurement aids (include/q8_probe.h)
lib.q8_probe_shape_count.restype = _i32
lib.q8_probe_shape_count.argtypes = []
lib.q8_probe_sink_words.restype = _i64
lib.q8_probe_sink_words.argtypes = [_i32]
lib.q8_probe_stream_read.restype = ctypes.c_int
lib.q8_probe_stream_read.argtypes = [_vp, _i64, _i32, _vp, _i64, _vp]
lib.q8_probe_empty.restype = ctypes.c_int
lib.q8_probe_empty.argtypes = [_i64, _vp]

Q8_OK, Q8_ERR_NULL, Q8_ERR_SHAPE, Q8_ERR_ALIGN, Q8_ERR_WORKSPACE, Q8_ERR_DEVICE = range(6)


class Q8Error(RuntimeError):
    def __init__(self, status: int, detail: str):
        self.status = status
        super().__init__(f"{lib.q8_status_string(status).decode()} ({status}): {detail}")


def check(status: int) -> None:
    if status != Q8_OK:
        raise Q8Error(status, lib.q8_last_error().decode())


def abi_version() -> int:
    return int(lib.q8_abi_version())


def _stream(t):
    return ctypes.c_void_p(torch.cuda.current_stream(t.device).cuda_stream)


def _dev(t, dtype, name, device=None):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t


def _ld(x, width):
    """Leading dimension to pass for a 2-D tensor whose rows hold `width` used values."""
    if x.shape[0] <= 1:  # a single row: only its first `width` values are touched
        return width + (-width % 4)
    return x.stride(0)


def _rows_in(x, width, name):
    """A 2-D [m][width] input with unit column stride and rows that do not overlap."""
    if x.dim() != 2 or x.shape[1] != width:
        raise ValueError(f"{name} must be [m][{width}], got {tuple(x.shape)}")
    if x.numel() and (x.stride(1) != 1 or (x.shape[0] > 1 and x.stride(0) < width)):
        raise ValueError(f"{name} must have contiguous, non-overlapping rows")
    return x.shape[0]


def _rows_out(out, m, width, name, dtype, device):
    """A caller-supplied output: exactly [m][width], unit column stride, rows that do not
    overlap (the kernels write m rows of width values at the tensor's row stride)."""
    _dev(out, dtype, name, device)
    if out.dim() != 2 or tuple(out.shape) != (m, width):
        raise ValueError(f"{name} must be [{m}][{width}], got {tuple(out.shape)}")
    if out.numel() and (out.stride(1) != 1 or (m > 1 and out.stride(0) < width)):
        raise ValueError(f"{name} must have unit column stride and non-overlapping rows")
    return out


def _contig_out(t, shape, name, dtype, device):
    if (isinstance(t, torch.Tensor) and t.dtype == dtype and t.device == device and t.is_cuda and t.shape == shape
            and t.is_contiguous()):
        return t
    _dev(t, dtype, name, device)
    if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)} tensor, got {tuple(t.shape)}")
    return t


def _bytes(w, need, name, device):
    """A byte tensor (uint8, contiguous) holding at least `need` bytes."""
    _dev(w, torch.uint8, name, device)
    if not w.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if w.numel() < need:
        raise ValueError(f"{name} holds {w.numel()} bytes, the shape needs {need}")
    return w


# bytes per 256 weights of each packed format
Q8_0_BYTES, Q4_0_BYTES, Q4_K_BYTES, Q5_K_BYTES, Q6_K_BYTES = 272, 144, 144, 176, 210


def _quant_bytes(rows, k, bytes_256):
    if k <= 0 or k % 256 or rows < 0:
        return 0  # the library reports the shape error
    return rows * (k // 256) * bytes_256


def _call(device, fn, *args):
    # the library launches on the current device: make it the tensors' device
    if device.index == torch.cuda.current_device():
        check(fn(*args))
        return
    with torch.cuda.device(device):
        check(fn(*args))


def _dense(fn, w, n_w, n_out, k, x, out, bytes_256):
    """Shared marshalling of the dense linears: weight rows n_w, outputs n_out."""
    _dev(x, torch.float32, "x")
    dev = x.device
    m = _rows_in(x, k, "x")
    _bytes(w, _quant_bytes(n_w, k, bytes_256) if n_out and m else 0, "w", dev)
    if out is None:
        out = torch.empty((m, n_out), dtype=torch.float32, device=dev)
    _rows_out(out, m, n_out, "out", torch.float32, dev)
    _call(dev, fn, w.data_ptr(), n_out, k, x.data_ptr(), m, _ld(x, k), out.data_ptr(), _ld(out, n_out),
          _stream(x))
    return out


def q8_linear(w, n: int, k: int, x, out=None):
    """y = x . W^T for a Q8_0 weight W [n][k] (uint8 bytes) and float32 x [m][k]."""
    return _dense(lib.q8_linear, w, n, n, k, x, out, Q8_0_BYTES)


def q8_linear_fused_gate_up_silu(w, f: int, k: int, x, out=None):
    """h = SiLU(x . W_gate^T) * (x . W_up^T); W is Q8_0 [2f][k], gate rows first."""
    return _dense(lib.q8_linear_fused_gate_up_silu, w, 2 * f, f, k, x, out, Q8_0_BYTES)


def q4_0_linear(w, n: int, k: int, x, out=None):
    """y = x . W^T for a GGUF Q4_0 weight W [n][k] (uint8 bytes) and float32 x [m][k]."""
    return _dense(lib.q4_0_linear, w, n, n, k, x, out, Q4_0_BYTES)


def q4_0_linear_fused_gate_up_silu(w, f: int, k: int, x, out=None):
    """h = SiLU(x . W_gate^T) * (x . W_up^T); W is GGUF Q4_0 [2f][k], gate rows first."""
    return _dense(lib.q4_0_linear_fused_gate_up_silu, w, 2 * f, f, k, x, out, Q4_0_BYTES)


def q4_k_linear(w, n: int, k: int, x, out=None):
    """y = x . W^T for a GGUF Q4_K weight W [n][k] (uint8 bytes) and float32 x [m][k]."""
    return _dense(lib.q4_k_linear, w, n, n, k, x, out, Q4_K_BYTES)


def q4_k_linear_fused_gate_up_silu(w, f: int, k: int, x, out=None):
    """h = SiLU(x . W_gate^T) * (x . W_up^T); W is GGUF Q4_K [2f][k], gate rows first."""
    return _dense(lib.q4_k_linear_fused_gate_up_silu, w, 2 * f, f, k, x, out, Q4_K_BYTES)


def q5_k_linear(w, n: int, k: int, x, out=None):
    """y = x . W^T for a GGUF Q5_K weight W [n][k] (uint8 bytes) and float32 x [m][k]."""
    return _dense(lib.q5_k_linear, w, n, n, k, x, out, Q5_K_BYTES)


def q5_k_linear_fused_gate_up_silu(w, f: int, k: int, x, out=None):
    """h = SiLU(x . W_gate^T) * (x . W_up^T); W is GGUF Q5_K [2f][k], gate rows first."""
    return _dense(lib.q5_k_linear_fused_gate_up_silu, w, 2 * f, f, k, x, out, Q5_K_BYTES)


def q6_k_linear(w, n: int, k: int, x, out=None):
    """y = x . W^T for a GGUF Q6_K weight W [n][k] (uint8 bytes) and float32 x [m][k]."""
    return _dense(lib.q6_k_linear, w, n, n, k, x, out, Q6_K_BYTES)


def q6_k_linear_fused_gate_up_silu(w, f: int, k: int, x, out=None):
    """h = SiLU(x . W_gate^T) * (x . W_up^T); W is GGUF Q6_K [2f][k], gate rows first."""
    return _dense(lib.q6_k_linear_fused_gate_up_silu, w, 2 * f, f, k, x, out, Q6_K_BYTES)


def q8_quantize_act(x, xq=None, xd=None):
    """Int8 codes [m][k] and float32 scales [m][k/32] of float32 activation rows x [m][k]."""
    _dev(x, torch.float32, "x")
    if x.dim() != 2:
        raise ValueError("x must be [m][k]")
    m, k = x.shape
    _rows_in(x, k, "x")
    dev = x.device
    if xq is None:
        xq = torch.empty((m, k), dtype=torch.int8, device=dev)
    if xd is None:
        xd = torch.empty((m, k // 32), dtype=torch.float32, device=dev)
    _contig_out(xq, (m, k), "xq", torch.int8, dev)
    _contig_out(xd, (m, k // 32), "xd", torch.float32, dev)
    _call(dev, lib.q8_quantize_act, x.data_ptr(), m, k, _ld(x, k), xq.data_ptr(), xd.data_ptr(), _stream(x))
    return xq, xd


def _codes(xq, xd, k):
    _dev(xq, torch.int8, "xq")
    _dev(xd, torch.float32, "xd", xq.device)
    if xq.dim() != 2 or xq.shape[1] != k or not xq.is_contiguous():
        raise ValueError(f"xq must be a contiguous [m][{k}] tensor")
    m = xq.shape[0]
    if tuple(xd.shape) != (m, k // 32) or not xd.is_contiguous():
        raise ValueError(f"xd must be a contiguous [m][{k // 32}] tensor")
    return m


def _dense_codes(fn, w, n_w, n_out, k, xq, xd, out):
    m = _codes(xq, xd, k)
    dev = xq.device
    _bytes(w, _quant_bytes(n_w, k, Q8_0_BYTES) if n_out and m else 0, "w", dev)
    if out is None:
        out = torch.empty((m, n_out), dtype=torch.float32, device=dev)
    _rows_out(out, m, n_out, "out", torch.float32, dev)
    _call(dev, fn, w.data_ptr(), n_out, k, xq.data_ptr(), xd.data_ptr(), m, out.data_ptr(), _ld(out, n_out),
          _stream(xq))
    return out


def q8_linear_q8act(w, n: int, k: int, xq, xd, out=None):
    """y = the Q8_0 weight W [n][k] against int8 activation codes xq [m][k] with scales xd."""
    return _dense_codes(lib.q8_linear_q8act, w, n, n, k, xq, xd, out)


def q8_linear_fused_gate_up_silu_q8act(w, f: int, k: int, xq, xd, out=None):
    """h = SiLU(gate) * up from a fused Q8_0 gate_up matrix [2f][k] on int8 activation codes."""
    return _dense_codes(lib.q8_linear_fused_gate_up_silu_q8act, w, 2 * f, f, k, xq, xd, out)


def moe_route_topk(x, w_router, k: int, normalize: bool = True, idx_out=None, w_out=None, top_p=None,
                   workspace=None):
    """Softmax top-k routing; returns (topk_idx int32 [m][k], topk_w float32 [m][k]).

    With top_p (in (0, 1]) the adaptive expert top-p cut follows (moe_route_topk_top_p):
    dropped slots hold expert -1 and weight 0.  With a workspace (uint8 device tensor of
    at least moe_route_workspace_bytes(m, n_exp) bytes; True allocates one) the two-pass
    form runs (moe_route_topk_ws), bit-identical to the one-pass calls."""
    _dev(x, torch.float32, "x")
    dev = x.device
    _dev(w_router, torch.float32, "w_router", dev)
    if not w_router.is_contiguous() or w_router.dim() != 2:
        raise ValueError("w_router must be a contiguous [n_exp][h] tensor")
    n_exp, h = w_router.shape
    m = _rows_in(x, h, "x")
    if idx_out is None:
        idx_out = torch.empty((m, k), dtype=torch.int32, device=dev)
    if w_out is None:
        w_out = torch.empty((m, k), dtype=torch.float32, device=dev)
    _contig_out(idx_out, (m, k), "idx_out", torch.int32, dev)
    _contig_out(w_out, (m, k), "w_out", torch.float32, dev)
    norm = 1 if normalize else 0
    if workspace is not None:
        if workspace is True:
            workspace = torch.empty(max(moe_route_workspace_bytes(m, n_exp), 1), dtype=torch.uint8, device=dev)
        _bytes(workspace, 0, "workspace", dev)
        _call(dev, lib.moe_route_topk_ws, x.data_ptr(), m, h, _ld(x, h), w_router.data_ptr(), n_exp, k, norm,
              1.0 if top_p is None else float(top_p), idx_out.data_ptr(), w_out.data_ptr(), workspace.data_ptr(),
              workspace.numel(), _stream(x))
    elif top_p is None:
        _call(dev, lib.moe_route_topk, x.data_ptr(), m, h, _ld(x, h), w_router.data_ptr(), n_exp, k, norm,
              idx_out.data_ptr(), w_out.data_ptr(), _stream(x))
    else:
        _call(dev, lib.moe_route_topk_top_p, x.data_ptr(), m, h, _ld(x, h), w_router.data_ptr(), n_exp, k, norm,
              float(top_p), idx_out.data_ptr(), w_out.data_ptr(), _stream(x))
    return idx_out, w_out


def moe_route_workspace_bytes(m: int, n_exp: int) -> int:
    return int(lib.moe_route_workspace_bytes(m, n_exp))


def q8_moe_workspace_bytes(m: int, k: int, n_exp: int, f: int, h: int) -> int:
    return int(lib.q8_moe_workspace_bytes(m, k, n_exp, f, h))


def _moe_args(w_gate_up_exps, w_down_exps, n_exp, f, h, x, topk_idx, topk_w, out):
    _dev(x, torch.float32, "x")
    dev = x.device
    m = _rows_in(x, h, "x")
    _dev(topk_idx, torch.int32, "topk_idx", dev)
    _dev(topk_w, torch.float32, "topk_w", dev)
    if topk_idx.dim() != 2 or topk_idx.shape[0] != m or not topk_idx.is_contiguous():
        raise ValueError("topk_idx must be a contiguous [m][k] tensor")
    k = topk_idx.shape[1]
    _contig_out(topk_w, (m, k), "topk_w", torch.float32, dev)
    _bytes(w_gate_up_exps, _quant_bytes(n_exp * 2 * f, h, Q8_0_BYTES) if m else 0, "w_gate_up_exps", dev)
    _bytes(w_down_exps, _quant_bytes(n_exp * h, f, Q8_0_BYTES) if m else 0, "w_down_exps", dev)
    if out is None:
        out = torch.empty((m, h), dtype=torch.float32, device=dev)
    _rows_out(out, m, h, "out", torch.float32, dev)
    return dev, m, k, out


def q8_moe_grouped_linear(w_gate_up_exps, w_down_exps, n_exp: int, f: int, h: int, x, topk_idx, topk_w,
                          out=None, workspace=None):
    """Router-weighted SwiGLU expert mixture; returns y float32 [m][h]."""
    dev, m, k, out = _moe_args(w_gate_up_exps, w_down_exps, n_exp, f, h, x, topk_idx, topk_w, out)
    need = q8_moe_workspace_bytes(m, k, n_exp, f, h) if m else 0
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _bytes(workspace, 0, "workspace", dev)
    _call(dev, lib.q8_moe_grouped_linear, w_gate_up_exps.data_ptr(), w_down_exps.data_ptr(), n_exp, f, h,
          x.data_ptr(), m, _ld(x, h), topk_idx.data_ptr(), topk_w.data_ptr(), k, out.data_ptr(), _ld(out, h),
          workspace.data_ptr(), workspace.numel(), _stream(x))
    return out


def q8_moe_grouped_linear_noalloc(w_gate_up_exps, w_down_exps, n_exp: int, f: int, h: int, x, topk_idx, topk_w,
                                  out=None):
    """The same mixture with the library's fixed per-device scratch instead of a workspace
    (the C entry point allocates nothing; pass `out` to keep this wrapper allocation-free
    too).  Sizes whose workspace exceeds the scratch raise Q8Error."""
    dev, m, k, out = _moe_args(w_gate_up_exps, w_down_exps, n_exp, f, h, x, topk_idx, topk_w, out)
    _call(dev, lib.q8_moe_grouped_linear_noalloc, w_gate_up_exps.data_ptr(), w_down_exps.data_ptr(), n_exp, f, h,
          x.data_ptr(), m, _ld(x, h), topk_idx.data_ptr(), topk_w.data_ptr(), k, out.data_ptr(), _ld(out, h),
          _stream(x))
    return out


# ---------------------------------------------------------- low-rank adapters

_LORA_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


def _lora(a, b, adapter, scale, ranks, sections, n, k, m, device):
    """The q8_lora of one call (its tensors must stay alive until the call returns)."""
    if not isinstance(a, torch.Tensor) or a.dtype not in _LORA_TYPES:
        raise ValueError("a must be a float32, float16 or bfloat16 tensor")
    _dev(a, a.dtype, "a", device)
    _dev(b, a.dtype, "b", device)
    sections = (n,) if sections is None else tuple(sections)
    if not 1 <= len(sections) <= 4 or sum(sections) != n or min(sections) < 0:
        raise ValueError(f"sections must be 1 to 4 sizes that sum to {n}, got {sections}")
    if b.dim() != 3 or b.shape[1] != n or not b.is_contiguous():
        raise ValueError(f"b must be a contiguous [n_adapters][{n}][rank] tensor, got {tuple(b.shape)}")
    count, _, rank = b.shape
    _contig_out(a, (count, len(sections) * rank, k), "a", a.dtype, device)
    _contig_out(adapter, (m,), "adapter", torch.int32, device)
    if scale is not None:
        _contig_out(scale, (count,), "scale", torch.float32, device)
    if ranks is not None:
        _contig_out(ranks, (count,), "ranks", torch.int32, device)
    return _Lora(a.data_ptr(), b.data_ptr(), None if ranks is None else ranks.data_ptr(),
                 None if scale is None else scale.data_ptr(), adapter.data_ptr(), sections, _LORA_TYPES[a.dtype],
                 count, rank, len(sections))


def _workspace(workspace, need, device):
    if workspace is None:
        return torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    return _bytes(workspace, 0, "workspace", device)


def q8_linear_lora_workspace_bytes(m: int, n: int, k: int, rank: int, n_sections: int = 1) -> int:
    """Workspace bytes of q8_linear_lora (q8_linear_fused_gate_up_silu_lora: n = 2f); from
    256 rows on q8_linear_lora takes lora_workspace_bytes as well."""
    return int(lib.q8_linear_lora_workspace_bytes(m, n, k, _Lora(rank=rank, n_sections=n_sections)))


def lora_workspace_bytes(m: int, rank: int, n_sections: int = 1) -> int:
    """Workspace bytes of lora_add and lora_gate_up_silu."""
    return int(lib.lora_workspace_bytes(m, _Lora(rank=rank, n_sections=n_sections)))


def _linear_lora(fn, w, n_w, n_out, k, x, a, b, adapter, scale, ranks, sections, out, workspace):
    _dev(x, torch.float32, "x")
    dev = x.device
    m = _rows_in(x, k, "x")
    lo = _lora(a, b, adapter, scale, ranks, sections, n_w, k, m, dev)
    _bytes(w, _quant_bytes(n_w, k, Q8_0_BYTES) if n_out and m else 0, "w", dev)
    if out is None:
        out = torch.empty((m, n_out), dtype=torch.float32, device=dev)
    _rows_out(out, m, n_out, "out", torch.float32, dev)
    # from 256 rows on the plain call's product goes straight into out
    need = (lib.lora_workspace_bytes(m, lo) if n_out == n_w and m >= 256
            else lib.q8_linear_lora_workspace_bytes(m, n_w, k, lo))
    workspace = _workspace(workspace, need, dev)
    _call(dev, fn, w.data_ptr(), n_out, k, x.data_ptr(), m, _ld(x, k), lo, out.data_ptr(), _ld(out, n_out),
          workspace.data_ptr(), workspace.numel(), _stream(x))
    return out


def q8_linear_lora(w, n: int, k: int, x, a, b, adapter, scale=None, ranks=None, sections=None, out=None,
                   workspace=None):
    """y = x . W^T + D for a Q8_0 weight W [n][k]; D is each row's low-rank correction,
    D[t] = scale[e] * B[e] (A[e] x[t]) with e = adapter[t] (outside [0, n_adapters): none).

    a [n_adapters][len(sections) * rank][k] and b [n_adapters][n][rank] in float32, float16
    or bfloat16 (rank a multiple of 8), adapter int32 [m], scale float32 [n_adapters],
    ranks int32 [n_adapters] (each adapter's own rank, at most `rank`); sections: the row
    counts of a fused matrix's parts, each with its own `rank` rows of a."""
    return _linear_lora(lib.q8_linear_lora, w, n, n, k, x, a, b, adapter, scale, ranks, sections, out, workspace)


def q8_linear_fused_gate_up_silu_lora(w, f: int, k: int, x, a, b, adapter, scale=None, ranks=None, sections=None,
                                      out=None, workspace=None):
    """h = SiLU(g) * u with [g u] = x . W^T + D, W Q8_0 [2f][k], gate rows first; the
    adapters as for q8_linear_lora with n = 2f (sections (f, f): gate and up apart)."""
    return _linear_lora(lib.q8_linear_fused_gate_up_silu_lora, w, 2 * f, f, k, x, a, b, adapter, scale, ranks,
                        sections, out, workspace)


def _lora_beside(fn, y, n_in, n_out, x, a, b, adapter, scale, ranks, sections, out, workspace):
    _dev(x, torch.float32, "x")
    dev = x.device
    if x.dim() != 2:
        raise ValueError("x must be [m][k]")
    m, k = x.shape
    _rows_in(x, k, "x")
    _rows_out(y, m, n_in, "the product", torch.float32, dev)
    lo = _lora(a, b, adapter, scale, ranks, sections, n_in, k, m, dev)
    if out is None:
        out = torch.empty((m, n_out), dtype=torch.float32, device=dev)
    _rows_out(out, m, n_out, "out", torch.float32, dev)
    workspace = _workspace(workspace, lib.lora_workspace_bytes(m, lo), dev)
    _call(dev, fn, y.data_ptr(), n_out, y.stride(0) if m > 1 else n_in, x.data_ptr(), m, k, _ld(x, k), lo,
          out.data_ptr(), out.stride(0) if m > 1 else n_out, workspace.data_ptr(), workspace.numel(), _stream(x))
    return out


def lora_add(y, x, a, b, adapter, scale=None, ranks=None, sections=None, out=None, workspace=None):
    """y + D beside a product y float32 [m][n] of any format (out may be y itself); D, x
    float32 [m][k] and the adapters as for q8_linear_lora."""
    if not isinstance(y, torch.Tensor) or y.dim() != 2:
        raise ValueError("y must be an [m][n] tensor")
    n = y.shape[1]
    return _lora_beside(lib.lora_add, y, n, n, x, a, b, adapter, scale, ranks, sections, out, workspace)


def lora_gate_up_silu(gu, x, a, b, adapter, scale=None, ranks=None, sections=None, out=None, workspace=None):
    """SiLU(g) * u with [g u] = gu + D beside a fused gate_up product gu float32 [m][2f] of
    any format; the adapters as for q8_linear_lora with n = 2f."""
    if not isinstance(gu, torch.Tensor) or gu.dim() != 2 or gu.shape[1] % 2:
        raise ValueError("gu must be an [m][2f] tensor")
    n = gu.shape[1]
    return _lora_beside(lib.lora_gate_up_silu, gu, n, n // 2, x, a, b, adapter, scale, ranks, sections, out,
                        workspace)


# ------------------------------------------------- the whole mixture-of-experts layer


def q8_moe_layer_workspace_bytes(m: int, k: int, n_exp: int, f: int, h: int) -> int:
    return int(lib.q8_moe_layer_workspace_bytes(m, k, n_exp, f, h))


def q8_moe_layer(w_router, w_gate_up_exps, w_down_exps, n_exp: int, f: int, h: int, x, k: int,
                 normalize: bool = True, top_p=None, out=None, workspace=None):
    """The whole MoE layer: softmax top-k routing of x [m][h] (moe_route_topk) and the
    chosen experts' SwiGLU mixture (q8_moe_grouped_linear); returns y float32 [m][h]."""
    _dev(x, torch.float32, "x")
    dev = x.device
    m = _rows_in(x, h, "x")
    _contig_out(w_router, (n_exp, h), "w_router", torch.float32, dev)
    _bytes(w_gate_up_exps, _quant_bytes(n_exp * 2 * f, h, Q8_0_BYTES) if m else 0, "w_gate_up_exps", dev)
    _bytes(w_down_exps, _quant_bytes(n_exp * h, f, Q8_0_BYTES) if m else 0, "w_down_exps", dev)
    if out is None:
        out = torch.empty((m, h), dtype=torch.float32, device=dev)
    _rows_out(out, m, h, "out", torch.float32, dev)
    workspace = _workspace(workspace, q8_moe_layer_workspace_bytes(m, k, n_exp, f, h), dev)
    _call(dev, lib.q8_moe_layer, w_router.data_ptr(), w_gate_up_exps.data_ptr(), w_down_exps.data_ptr(), n_exp, f, h,
          x.data_ptr(), m, _ld(x, h), k, 1 if normalize else 0, 1.0 if top_p is None else float(top_p),
          out.data_ptr(), _ld(out, h), workspace.data_ptr(), workspace.numel(), _stream(x))
    return out


# ------------------------------------------------- block-scaled 8-bit floating point

_FLOAT_TYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}


def _float_type(dtype, name):
    if dtype not in _FLOAT_TYPES:
        raise ValueError(f"{name} must be float32, float16 or bfloat16, got {dtype}")
    return _FLOAT_TYPES[dtype]


def _float_rows(t, name, device=None):
    """A 2-D float tensor with contiguous, non-overlapping rows."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D tensor")
    _float_type(t.dtype, name)
    _dev(t, t.dtype, name, device)
    _rows_in(t, t.shape[1], name)
    return t


def _f8_ld(t, width):
    return t.stride(0) if t.shape[0] > 1 else width


def _f8_codes(q, d, name, device=None):
    """Codes [rows][k] with scales of unit stride on the same device."""
    if not isinstance(q, torch.Tensor) or q.dim() != 2 or q.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise ValueError(f"the codes of {name} must be a 2-D float8_e4m3fn (or uint8) tensor")
    _dev(q, q.dtype, name, device)
    if not q.is_contiguous():
        raise ValueError(f"the codes of {name} must be contiguous")
    _dev(d, torch.float32, f"the scales of {name}", q.device)
    return q.shape


def _f8_blocks(size):
    return (size + 127) // 128


def _f8_operands(wq, wd, xq, xd, parts):
    """(n of a part, k, m) of a product's codes and scales."""
    rows, k = _f8_codes(wq, wd, "w")
    m, kx = _f8_codes(xq, xd, "x", wq.device)
    if kx != k:
        raise ValueError(f"w has {k} inputs, x has {kx}")
    if rows % parts:
        raise ValueError(f"a gate_up matrix has an even number of rows, got {rows}")
    n = rows // parts
    _contig_out(wd, (parts * _f8_blocks(n), _f8_blocks(k)), "the scales of w", torch.float32, wq.device)
    _contig_out(xd, (m, _f8_blocks(k)), "the scales of x", torch.float32, wq.device)
    return n, k, m


def _f8_quantize(fn, x, name, block_rows, pow2, q, d):
    _float_rows(x, name)
    dev = x.device
    rows, k = x.shape
    if q is None:
        q = torch.empty((rows, k), dtype=torch.float8_e4m3fn, device=dev)
    shape = ((rows + block_rows - 1) // block_rows, _f8_blocks(k))
    if d is None:
        d = torch.empty(shape, dtype=torch.float32, device=dev)
    _contig_out(q, (rows, k), "q", torch.uint8 if getattr(q, "dtype", None) == torch.uint8 else torch.float8_e4m3fn, dev)
    _contig_out(d, shape, "d", torch.float32, dev)
    size = x.element_size()
    # a single row: only its k values are touched, so any leading dimension of whole 16 bytes does
    ld = x.stride(0) if rows > 1 else k + (-k % (16 // size))
    _call(dev, fn, x.data_ptr(), _FLOAT_TYPES[x.dtype], rows, k, ld, 1 if pow2 else 0, q.data_ptr(), d.data_ptr(),
          _stream(x))
    return q, d


def f8_quantize_act(x, pow2: bool = False, q=None, d=None):
    """e4m3 codes [m][k] and float32 scales [m][ceil(k/128)] of rows x [m][k] (float32,
    float16 or bfloat16): one scale for every 128 inputs, amax/448 or (pow2) the least power
    of two that is not below it.  Outside autograd, as all calls here: what requires a gradient
    gets it from the backward calls."""
    return _f8_quantize(lib.f8_quantize_act, x, "x", 1, pow2, q, d)


def f8_quantize_weight(w, pow2: bool = False, q=None, d=None):
    """e4m3 codes [n][k] and float32 scales [ceil(n/128)][ceil(k/128)] of a matrix w [n][k]: one
    scale for every block of 128 x 128.  The parts of a fused gate_up matrix are coded apart
    and their codes and scales put one under the other."""
    return _f8_quantize(lib.f8_quantize_weight, w, "w", 128, pow2, q, d)


def _f8_asked(want, name):
    """Whether an output that is asked for by True is: anything else that is no tensor is a caller's mistake."""
    if want not in (True, False, None):
        raise ValueError(f"{name} must be True, False or a device tensor, got {type(want).__name__}")
    return bool(want)


def f8_linear(wq, wd, xq, xd, dtype=torch.float32, out=None):
    """y = x . W^T [m][n] in `dtype` from e4m3 codes wq [n][k] and xq [m][k] and their scales
    (f8_quantize_weight, f8_quantize_act)."""
    n, k, m = _f8_operands(wq, wd, xq, xd, 1)
    dev = wq.device
    if out is None:
        out = torch.empty((m, n), dtype=dtype, device=dev)
    kind = _float_type(getattr(out, "dtype", None), "the output")
    _rows_out(out, m, n, "out", out.dtype, dev)
    _call(dev, lib.f8_linear, wq.data_ptr(), wd.data_ptr(), n, k, xq.data_ptr(), xd.data_ptr(), m, out.data_ptr(), kind,
          _f8_ld(out, n), _stream(wq))
    return out


def f8_linear_fused_gate_up_silu(wq, wd, xq, xd, dtype=torch.float32, keep_gate_up=False, out=None):
    """h = SiLU(g) * u [m][f] with [g u] = x . W^T; wq [2f][k] has gate rows first, wd gate's
    scales first.  keep_gate_up: True (or a tensor [m][2f] to write) returns (h, gu), gu the
    products g and u beside each other, as the backward call takes them."""
    f, k, m = _f8_operands(wq, wd, xq, xd, 2)
    dev = wq.device
    if out is None:
        out = torch.empty((m, f), dtype=dtype, device=dev)
    kind = _float_type(getattr(out, "dtype", None), "the output")
    _rows_out(out, m, f, "out", out.dtype, dev)
    gu = None
    if isinstance(keep_gate_up, torch.Tensor):
        gu = _rows_out(keep_gate_up, m, 2 * f, "keep_gate_up", out.dtype, dev)
    elif _f8_asked(keep_gate_up, "keep_gate_up"):
        gu = torch.empty((m, 2 * f), dtype=out.dtype, device=dev)
    _call(dev, lib.f8_linear_fused_gate_up_silu, wq.data_ptr(), wd.data_ptr(), f, k, xq.data_ptr(), xd.data_ptr(), m,
          out.data_ptr(), kind, _f8_ld(out, f), None if gu is None else gu.data_ptr(),
          0 if gu is None else _f8_ld(gu, 2 * f), _stream(wq))
    return out if gu is None else (out, gu)


def f8_linear_backward_workspace_bytes(m: int, n: int, k: int, dtype) -> int:
    """Workspace bytes of f8_linear_backward for gradients of `dtype`."""
    return int(lib.f8_linear_backward_workspace_bytes(m, n, k, _float_type(dtype, "dtype")))


def f8_linear_fused_gate_up_silu_backward_workspace_bytes(m: int, f: int, k: int, dtype) -> int:
    """Workspace bytes of f8_linear_fused_gate_up_silu_backward for gradients of `dtype`."""
    return int(lib.f8_linear_fused_gate_up_silu_backward_workspace_bytes(m, f, k, _float_type(dtype, "dtype")))


def _f8_gradient(want, m, width, name, dtype, device):
    """The tensor that a gradient goes to: new (True), the caller's, or none (False)."""
    if isinstance(want, torch.Tensor):
        return _rows_out(want, m, width, name, dtype, device)
    return torch.empty((m, width), dtype=dtype, device=device) if _f8_asked(want, name) else None


def _f8_backward(fn, parts, wq, wd, xq, xd, gu, d, dx, dw, workspace, need):
    n, k, m = _f8_operands(wq, wd, xq, xd, parts)
    dev = wq.device
    _float_rows(d, "the gradient", dev)
    if tuple(d.shape) != (m, n):
        raise ValueError(f"the gradient must be [{m}][{n}], got {tuple(d.shape)}")
    more = ()
    if parts == 2:
        _float_rows(gu, "gu", dev)
        if tuple(gu.shape) != (m, 2 * n) or gu.dtype != d.dtype:
            raise ValueError(f"gu must be [{m}][{2 * n}] of {d.dtype}, got {tuple(gu.shape)} of {gu.dtype}")
        more = (gu.data_ptr(), _f8_ld(gu, 2 * n))
    dx = _f8_gradient(dx, m, k, "dx", d.dtype, dev)
    dw = _f8_gradient(dw, parts * n, k, "dw", d.dtype, dev)
    kind = _FLOAT_TYPES[d.dtype]
    workspace = _workspace(workspace, need(m, n, k, kind), dev)
    _call(dev, fn, wq.data_ptr(), wd.data_ptr(), n, k, xq.data_ptr(), xd.data_ptr(), m, *more, d.data_ptr(), kind,
          _f8_ld(d, n), None if dx is None else dx.data_ptr(), k if dx is None else _f8_ld(dx, k),
          None if dw is None else dw.data_ptr(), k if dw is None else _f8_ld(dw, k), workspace.data_ptr(),
          workspace.numel(), _stream(wq))
    return dx, dw


def f8_linear_backward(wq, wd, xq, xd, dy, dx=True, dw=True, workspace=None):
    """The gradients of f8_linear's inputs, dx = dy . W [m][k] and dw = dy^T . x [n][k], in dy's
    type (float32, float16 or bfloat16); W and x are the values of their codes and scales.
    dx, dw: True, a tensor to write, or False to leave the gradient out (None is returned)."""
    return _f8_backward(lib.f8_linear_backward, 1, wq, wd, xq, xd, None, dy, dx, dw, workspace,
                        lib.f8_linear_backward_workspace_bytes)


def f8_linear_fused_gate_up_silu_backward(wq, wd, xq, xd, gu, dh, dx=True, dw=True, workspace=None):
    """The gradients of f8_linear_fused_gate_up_silu's inputs from dh [m][f] and the products
    gu [m][2f] that it kept: dx [m][k] and dw [2f][k], in dh's type; arguments as for
    f8_linear_backward."""
    return _f8_backward(lib.f8_linear_fused_gate_up_silu_backward, 2, wq, wd, xq, xd, gu, dh, dx, dw, workspace,
                        lib.f8_linear_fused_gate_up_silu_backward_workspace_bytes)


# ------------------------------------------------------------ measurement aids


def probe_shape_count() -> int:
    """Launch shapes of probe_stream_read (0 .. count-1)."""
    return int(lib.q8_probe_shape_count())


def probe_stream_read(buf, nbytes: int, shape: int, sink=None):
    """Plain streaming read of the first nbytes bytes of a device byte tensor in one
    launch (launch shape `shape`), for a benchmark's read ceiling; returns the sink
    tensor of per-lane xor words."""
    _bytes(buf, nbytes, "buf", None)
    with torch.cuda.device(buf.device):
        words = int(lib.q8_probe_sink_words(shape))
    if words < 0:
        raise ValueError(f"probe shape {shape} is out of range [0, {probe_shape_count()})")
    if sink is None:
        sink = torch.empty(words, dtype=torch.int32, device=buf.device)
    _contig_out(sink, (words,), "sink", torch.int32, buf.device)
    _call(buf.device, lib.q8_probe_stream_read, buf.data_ptr(), nbytes, shape, sink.data_ptr(), words, _stream(buf))
    return sink


def probe_empty(blocks: int, device=None):
    """One launch of `blocks` workgroups that do nothing, on the current stream."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        check(lib.q8_probe_empty(blocks, ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)))
