"""Thin Python binding of libbitlinear.so (C ABI in include/bitlinear.h).

Argument marshalling only: every step of the BitLinear forward runs in the library's
sm_100a kernels. PyTorch supplies device memory and the current stream. There is no
fallback: if the shared library is missing or no CUDA device is present, the calls raise.

stream= runs a call on that stream (of the tensors' device) instead of the current one; what it
allocates then belongs to that stream. As with any work put on another stream, the caller makes it
wait for the inputs, keeps them (and buffers it gives) until it is done, and waits for the outputs.
"""

from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libbitlinear.so")

BL_F32, BL_BF16, BL_I32 = 0, 1, 2
STATUS = {
    0: "BL_OK", 1: "BL_ERR_INVALID_ARG", 2: "BL_ERR_UNSUPPORTED_SHAPE", 3: "BL_ERR_MISALIGNED",
    4: "BL_ERR_CUDA", 5: "BL_ERR_TIMEOUT", 6: "BL_ERR_NONFINITE", 7: "BL_ERR_WORKSPACE",
}

# Every symbol declared in include/bitlinear.h.
EXPORTS = (
    "bitlinear_workspace_size", "bitlinear_quantize_weights", "bitlinear_quantize_acts",
    "bitlinear_weight_abssum", "bitlinear_quantize_weights_from_abssum", "bitlinear_act_absmax",
    "bitlinear_quantize_acts_absmax", "bitlinear_rescale", "bitlinear_chain_workspace_size",
    "bitlinear_chain_forward", "bitlinear_base3_row_bytes", "bitlinear_pack_base3",
    "bitlinear_forward_base3", "bitlinear_pack_transpose", "bitlinear_backward_workspace_size",
    "bitlinear_backward", "bitlinear_backward_quantized_workspace_size", "bitlinear_backward_quantized",
    "bitlinear_forward_quantized",
    "bitlinear_rmsnorm_quantize", "bitlinear_rmsnorm_backward_workspace_size",
    "bitlinear_rmsnorm_backward", "bitlinear_moe_workspace_size", "bitlinear_moe_forward",
    "bitlinear_forward", "bitlinear_forward_noalloc", "bitlinear_contract_i32",
    "bitlinear_get_device_status",
    "bitlinear_debug_timeout_probe", "bitlinear_debug_plan", "bitlinear_status_string",
)


class Layer(ctypes.Structure):
    """bl_layer of include/bitlinear.h: one layer of a chain."""
    _fields_ = [("packed", ctypes.c_void_p), ("gamma", ctypes.c_void_p), ("N", ctypes.c_int),
                ("K", ctypes.c_int), ("src", ctypes.c_int), ("out", ctypes.c_void_p)]


class Moe(ctypes.Structure):
    """bl_moe of include/bitlinear.h: a mixture-of-experts layer."""
    _fields_ = [(n, ctypes.c_void_p) for n in ("router", "gate", "up", "down", "gate_gamma",
                                               "up_gamma", "down_gamma")] + [
        (n, ctypes.c_int) for n in ("router_dtype", "E", "D", "F", "top_k", "act", "renormalize")]


class BitLinearError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}")
        self.status = status


_lib = None


def load_library() -> ctypes.CDLL:
    """Loads the in-tree libbitlinear.so (built by ternary_weight_linear_03_b200.build)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m ternary_weight_linear_03_b200.build`"
            " (or __graft_entry__.build()); there is no fallback implementation")
    lib = ctypes.CDLL(LIB_PATH)
    p, i, f, sz, u64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_uint64
    lib.bitlinear_workspace_size.argtypes = [i, i, i]
    lib.bitlinear_workspace_size.restype = sz
    lib.bitlinear_quantize_weights.argtypes = [p, i, i, i, f, p, p, p, sz, p]
    lib.bitlinear_quantize_weights.restype = i
    lib.bitlinear_quantize_acts.argtypes = [p, i, i, i, p, p, p]
    lib.bitlinear_quantize_acts.restype = i
    i64 = ctypes.c_longlong
    lib.bitlinear_weight_abssum.argtypes = [p, i, i, i, p, p, sz, p]
    lib.bitlinear_weight_abssum.restype = i
    lib.bitlinear_quantize_weights_from_abssum.argtypes = [p, i, i, i, i64, p, f, p, p, p]
    lib.bitlinear_quantize_weights_from_abssum.restype = i
    lib.bitlinear_act_absmax.argtypes = [p, i, i, i, p, p]
    lib.bitlinear_act_absmax.restype = i
    lib.bitlinear_quantize_acts_absmax.argtypes = [p, i, i, i, p, p, p, p]
    lib.bitlinear_quantize_acts_absmax.restype = i
    lib.bitlinear_rescale.argtypes = [p, p, p, p, i, i, i, p]
    lib.bitlinear_rescale.restype = i
    lib.bitlinear_chain_workspace_size.argtypes = [i, ctypes.POINTER(Layer), i]
    lib.bitlinear_chain_workspace_size.restype = sz
    lib.bitlinear_chain_forward.argtypes = [p, i, i, ctypes.POINTER(Layer), i, p, i, p, sz, p]
    lib.bitlinear_chain_forward.restype = i
    lib.bitlinear_base3_row_bytes.argtypes = [i]
    lib.bitlinear_base3_row_bytes.restype = sz
    lib.bitlinear_pack_base3.argtypes = [p, i, i, p, p]
    lib.bitlinear_pack_base3.restype = i
    lib.bitlinear_forward_base3.argtypes = [p, i, p, p, p, i, i, i, i, p]
    lib.bitlinear_forward_base3.restype = i
    lib.bitlinear_pack_transpose.argtypes = [p, i, i, p, p]
    lib.bitlinear_pack_transpose.restype = i
    lib.bitlinear_backward_workspace_size.argtypes = [i, i, i]
    lib.bitlinear_backward_workspace_size.restype = sz
    lib.bitlinear_backward.argtypes = [p, i, p, p, p, p, p, i, i, i, p, sz, p]
    lib.bitlinear_backward.restype = i
    lib.bitlinear_backward_quantized_workspace_size.argtypes = [i, i, i]
    lib.bitlinear_backward_quantized_workspace_size.restype = sz
    lib.bitlinear_backward_quantized.argtypes = [p, p, p, p, p, p, p, i, i, i, p, sz, p]
    lib.bitlinear_backward_quantized.restype = i
    lib.bitlinear_forward_quantized.argtypes = [p, p, p, p, p, i, i, i, i, p, sz, p]
    lib.bitlinear_forward_quantized.restype = i
    lib.bitlinear_rmsnorm_quantize.argtypes = [p, p, i, p, i, f, i, i, p, p, p, p, p, p]
    lib.bitlinear_rmsnorm_quantize.restype = i
    lib.bitlinear_rmsnorm_backward_workspace_size.argtypes = [i, i]
    lib.bitlinear_rmsnorm_backward_workspace_size.restype = sz
    lib.bitlinear_rmsnorm_backward.argtypes = [p, i, p, i, p, i, p, p, p, i, p, i, i, p, sz, p]
    lib.bitlinear_rmsnorm_backward.restype = i
    lib.bitlinear_moe_workspace_size.argtypes = [i, ctypes.POINTER(Moe)]
    lib.bitlinear_moe_workspace_size.restype = sz
    lib.bitlinear_moe_forward.argtypes = [p, i, i, ctypes.POINTER(Moe), p, i, p, sz, p]
    lib.bitlinear_moe_forward.restype = i
    lib.bitlinear_forward.argtypes = [p, i, p, p, p, i, i, i, i, p, sz, p]
    lib.bitlinear_forward.restype = i
    lib.bitlinear_forward_noalloc.argtypes = [p, i, p, p, p, i, i, i, i, p]
    lib.bitlinear_forward_noalloc.restype = i
    lib.bitlinear_contract_i32.argtypes = [p, p, p, i, i, i, p, sz, p]
    lib.bitlinear_contract_i32.restype = i
    lib.bitlinear_get_device_status.argtypes = [p]
    lib.bitlinear_get_device_status.restype = i
    lib.bitlinear_debug_timeout_probe.argtypes = [u64, p]
    lib.bitlinear_debug_timeout_probe.restype = i
    lib.bitlinear_debug_plan.argtypes = [i, i, i, i, p, p]
    lib.bitlinear_debug_plan.restype = i
    lib.bitlinear_status_string.argtypes = [i]
    lib.bitlinear_status_string.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(status: int, what: str) -> None:
    if status != 0:
        raise BitLinearError(status, what)


def _dev(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return BL_F32
    if t.dtype == torch.bfloat16:
        return BL_BF16
    raise TypeError(f"unsupported dtype {t.dtype} (fp32 or bf16)")


def _stream(stream=None) -> int:
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _on(stream, fn, *args):
    """fn(*args) with `stream` as the current one: what fn allocates then belongs to the stream its
    kernels run on, and not to one that may still use it, or hands it out again once fn has dropped
    it. New outputs are kept for the caller's stream too."""
    if args[0].device != stream.device:
        raise ValueError(f"stream (on {stream.device}) and tensors ({args[0].device}) must be on one device")
    if stream == torch.cuda.current_stream():
        return fn(*args)
    here = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        out = fn(*args)
    for t in out if isinstance(out, tuple) else (out,):
        if t is not None and not any(t is a for a in args):
            t.record_stream(here)
    return out


# The current stream's handle without a Stream object (3 us less per call), where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _run(fn, what: str, at: int, *args) -> None:
    """Calls fn(*args, stream) with device `at` current, on its current stream."""
    if at != torch.cuda.current_device():
        with torch.cuda.device(at):
            return _run(fn, what, at, *args)
    status = fn(*args, _raw_stream(at) if _raw_stream is not None else _stream())
    if status:
        _check(status, what)


def _take(t: torch.Tensor, name: str, shape, dtype, at: int) -> int:
    """Address of a contiguous tensor of this shape and type (one of them) on device `at`."""
    if t.get_device() != at:
        raise ValueError(f"{name} must be on cuda:{at}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.dtype is not dtype and (dtype is not _FLOATS or t.dtype not in _FLOATS):
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _take_ws(ws: torch.Tensor, at: int) -> int:
    if ws.get_device() != at or not ws.is_contiguous() or ws.dtype is not torch.uint8:
        raise ValueError(f"ws must be a contiguous uint8 tensor on cuda:{at}")
    return ws.data_ptr()


def _index(t: torch.Tensor, name: str) -> int:
    at = t.get_device()
    if at < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    return at


_FLOATS = (torch.float32, torch.bfloat16)


def _code(t: torch.Tensor) -> int:
    return BL_BF16 if t.dtype is torch.bfloat16 else BL_F32


def workspace_size(M: int, N: int, K: int) -> int:
    return int(load_library().bitlinear_workspace_size(M, N, K))


def workspace(M: int, N: int, K: int, device="cuda") -> torch.Tensor:
    """A caller-owned device workspace large enough for (M, N, K)."""
    n = workspace_size(M, N, K)
    if n == 0:
        raise BitLinearError(2, "workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def quantize_weights(W: torch.Tensor, eps: float = 1e-5, packed: torch.Tensor | None = None,
                     gamma: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                     stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Absmean ternary quantization of W [N][K] -> (packed uint8 [N][K/4], gamma fp32 [1])."""
    if stream is not None:
        return _on(stream, quantize_weights, W, eps, packed, gamma, ws)
    lib = load_library()
    N, K = W.shape
    if packed is None:
        packed = torch.empty((N, K // 4), dtype=torch.uint8, device=W.device)
    if gamma is None:
        gamma = torch.empty(1, dtype=torch.float32, device=W.device)
    if ws is None:
        ws = workspace(1, N, K, W.device)
    _check(lib.bitlinear_quantize_weights(
        _dev(W, "W"), _dtype_code(W), N, K, float(eps), _dev(packed, "packed"),
        _dev(gamma, "gamma"), _dev(ws, "ws"), ws.numel(), _stream()),
        "bitlinear_quantize_weights")
    return packed, gamma


def quantize_acts(x: torch.Tensor, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Per-token absmax int8: x [M][K] -> (xq int8 [M][K], scale fp32 [M])."""
    if stream is not None:
        return _on(stream, quantize_acts, x)
    lib = load_library()
    M, K = x.shape
    xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
    scale = torch.empty(M, dtype=torch.float32, device=x.device)
    _check(lib.bitlinear_quantize_acts(_dev(x, "x"), _dtype_code(x), M, K, _dev(xq, "xq"),
                                       _dev(scale, "scale"), _stream()),
           "bitlinear_quantize_acts")
    return xq, scale


ABSSUM_WORDS = 14


def weight_abssum(W: torch.Tensor, sums: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Exact sum of |w| over W (a shard of a matrix) as ABSSUM_WORDS int64 words (uint64
    bit patterns): the words of several shards add up exactly to those of their union."""
    if stream is not None:
        return _on(stream, weight_abssum, W, sums, ws)
    lib = load_library()
    N, K = W.shape
    if sums is None:
        sums = torch.empty(ABSSUM_WORDS, dtype=torch.int64, device=W.device)
    if ws is None:
        ws = workspace(1, N, K, W.device)
    _check(lib.bitlinear_weight_abssum(_dev(W, "W"), _dtype_code(W), N, K, _dev(sums, "sums"),
                                       _dev(ws, "ws"), ws.numel(), _stream()),
           "bitlinear_weight_abssum")
    return sums


def quantize_weights_from_abssum(W: torch.Tensor, n_total: int, sums: torch.Tensor,
                                 eps: float = 1e-5, packed: torch.Tensor | None = None,
                                 gamma: torch.Tensor | None = None,
                                 stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """gamma from the added words of every shard (over n_total weights), then this shard's
    packed codes."""
    if stream is not None:
        return _on(stream, quantize_weights_from_abssum, W, n_total, sums, eps, packed, gamma)
    lib = load_library()
    N, K = W.shape
    if packed is None:
        packed = torch.empty((N, K // 4), dtype=torch.uint8, device=W.device)
    if gamma is None:
        gamma = torch.empty(1, dtype=torch.float32, device=W.device)
    _check(lib.bitlinear_quantize_weights_from_abssum(
        _dev(W, "W"), _dtype_code(W), N, K, int(n_total), _dev(sums, "sums"), float(eps),
        _dev(packed, "packed"), _dev(gamma, "gamma"), _stream()),
        "bitlinear_quantize_weights_from_abssum")
    return packed, gamma


def act_absmax(x: torch.Tensor, amax: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Per-token max |x| (fp32 [M])."""
    if stream is not None:
        return _on(stream, act_absmax, x, amax)
    lib = load_library()
    M, K = x.shape
    if amax is None:
        amax = torch.empty(M, dtype=torch.float32, device=x.device)
    _check(lib.bitlinear_act_absmax(_dev(x, "x"), _dtype_code(x), M, K, _dev(amax, "amax"),
                                    _stream()), "bitlinear_act_absmax")
    return amax


def quantize_acts_absmax(x: torch.Tensor, amax: torch.Tensor,
                         stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Per-token int8 quantization with the absmax given (of the whole rows)."""
    if stream is not None:
        return _on(stream, quantize_acts_absmax, x, amax)
    lib = load_library()
    M, K = x.shape
    xq = torch.empty((M, K), dtype=torch.int8, device=x.device)
    scale = torch.empty(M, dtype=torch.float32, device=x.device)
    _check(lib.bitlinear_quantize_acts_absmax(_dev(x, "x"), _dtype_code(x), M, K,
                                              _dev(amax, "amax"), _dev(xq, "xq"),
                                              _dev(scale, "scale"), _stream()),
           "bitlinear_quantize_acts_absmax")
    return xq, scale


def rescale(acc: torch.Tensor, scale: torch.Tensor, gamma: torch.Tensor,
            out_dtype: torch.dtype = torch.bfloat16, y: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    """y = float(acc) * (scale_t * gamma) for an int32 product [M][N]."""
    if stream is not None:
        return _on(stream, rescale, acc, scale, gamma, out_dtype, y)
    lib = load_library()
    M, N = acc.shape
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=acc.device)
    _check(lib.bitlinear_rescale(_dev(acc, "acc"), _dev(scale, "scale"), _dev(gamma, "gamma"),
                                 _dev(y, "y"), _dtype_code(y), M, N, _stream()),
           "bitlinear_rescale")
    return y


def chain_layers(layers) -> ctypes.Array:
    """ctypes array of bl_layer from (packed, gamma, src[, out]) tuples (device tensors;
    out a bf16 [M][N] tensor or None)."""
    arr = (Layer * len(layers))()
    for i, ly in enumerate(layers):
        packed, gamma, src = ly[0], ly[1], ly[2]
        out = ly[3] if len(ly) > 3 else None
        arr[i] = Layer(_dev(packed, "packed"), _dev(gamma, "gamma"), packed.shape[0],
                       packed.shape[1] * 4, int(src), _dev(out, "out") if out is not None else None)
    return arr


def chain_workspace(M: int, layers, device="cuda") -> torch.Tensor:
    arr = chain_layers(layers)
    n = int(load_library().bitlinear_chain_workspace_size(M, arr, len(layers)))
    if n == 0:
        raise BitLinearError(1, "bitlinear_chain_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def chain_forward(x: torch.Tensor, layers, out_dtype: torch.dtype = torch.bfloat16,
                  y: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """A chain of BitLinear layers (bitlinear_chain_forward): layers are (packed, gamma,
    src[, out]) with src = -1 for x or the index of the layer whose output is the input."""
    if stream is not None:
        return _on(stream, chain_forward, x, layers, out_dtype, y, ws)
    lib = load_library()
    M = x.shape[0]
    arr = chain_layers(layers)
    if y is None:
        y = torch.empty((M, layers[-1][0].shape[0]), dtype=out_dtype, device=x.device)
    if ws is None:
        ws = chain_workspace(M, layers, x.device)
    _check(lib.bitlinear_chain_forward(_dev(x, "x"), _dtype_code(x), M, arr, len(layers),
                                       _dev(y, "y"), _dtype_code(y), _dev(ws, "ws"), ws.numel(),
                                       _stream()), "bitlinear_chain_forward")
    return y


def base3_row_bytes(K: int) -> int:
    return int(load_library().bitlinear_base3_row_bytes(K))


def pack_base3(packed: torch.Tensor, stream=None) -> torch.Tensor:
    """2-bit packed weights [N][K/4] -> base-3 [N][ceil(K/80)*16] (same codes)."""
    if stream is not None:
        return _on(stream, pack_base3, packed)
    lib = load_library()
    N, K = packed.shape[0], packed.shape[1] * 4
    out = torch.empty((N, base3_row_bytes(K)), dtype=torch.uint8, device=packed.device)
    _check(lib.bitlinear_pack_base3(_dev(packed, "packed"), N, K, _dev(out, "packed3"),
                                    _stream()), "bitlinear_pack_base3")
    return out


def forward_base3(x: torch.Tensor, packed3: torch.Tensor, gamma: torch.Tensor,
                  out_dtype: torch.dtype = torch.bfloat16, y: torch.Tensor | None = None,
                  stream=None) -> torch.Tensor:
    """BitLinear forward on base-3 weights (M <= 4 tokens)."""
    if stream is not None:
        return _on(stream, forward_base3, x, packed3, gamma, out_dtype, y)
    lib = load_library()
    M, K = x.shape
    N = packed3.shape[0]
    if packed3.shape[1] != base3_row_bytes(K):
        raise ValueError("packed3 must be [N][ceil(K/80)*16]")
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    _check(lib.bitlinear_forward_base3(
        _dev(x, "x"), _dtype_code(x), _dev(packed3, "packed3"), _dev(gamma, "gamma"),
        _dev(y, "y"), _dtype_code(y), M, N, K, _stream()), "bitlinear_forward_base3")
    return y


def pack_transpose(packed: torch.Tensor, stream=None) -> torch.Tensor:
    """2-bit weights [N][K/4] -> the transposed 2-bit weights [K][N/4] (N % 64 == 0)."""
    if stream is not None:
        return _on(stream, pack_transpose, packed)
    lib = load_library()
    N, K = packed.shape[0], packed.shape[1] * 4
    out = torch.empty((K, N // 4), dtype=torch.uint8, device=packed.device)
    _check(lib.bitlinear_pack_transpose(_dev(packed, "packed"), N, K, _dev(out, "packedT"),
                                        _stream()), "bitlinear_pack_transpose")
    return out


def backward(x: torch.Tensor, grad_y: torch.Tensor, packedT: torch.Tensor, gamma: torch.Tensor,
             need_x: bool = True, need_w: bool = True, ws: torch.Tensor | None = None,
             stream=None):
    """Straight-through BitLinear backward: (grad_x fp32 [M][K] or None, grad_w fp32 [N][K]
    or None) from the forward input x, grad_y bf16 [M][N] and the transposed weights."""
    if stream is not None:
        return _on(stream, backward, x, grad_y, packedT, gamma, need_x, need_w, ws)
    lib = load_library()
    M, K = x.shape
    N = grad_y.shape[1]
    if grad_y.dtype != torch.bfloat16:
        raise TypeError("grad_y must be bf16")
    gx = torch.empty((M, K), dtype=torch.float32, device=x.device) if need_x else None
    gw = torch.empty((N, K), dtype=torch.float32, device=x.device) if need_w else None
    if ws is None and need_w:
        n = int(lib.bitlinear_backward_workspace_size(M, N, K))
        if n == 0:
            raise BitLinearError(2, "bitlinear_backward_workspace_size")
        ws = torch.empty(n, dtype=torch.uint8, device=x.device)
    _check(lib.bitlinear_backward(
        _dev(x, "x"), _dtype_code(x), _dev(grad_y, "grad_y"), _dev(packedT, "packedT"),
        _dev(gamma, "gamma"), _dev(gx, "grad_x") if gx is not None else None,
        _dev(gw, "grad_w") if gw is not None else None, M, N, K,
        _dev(ws, "ws") if ws is not None else None, ws.numel() if ws is not None else 0,
        _stream()), "bitlinear_backward")
    return gx, gw


def backward_workspace(M: int, N: int, K: int, device="cuda") -> torch.Tensor:
    """A caller-owned device workspace for backward and backward_quantized."""
    lib = load_library()
    n = max(int(lib.bitlinear_backward_workspace_size(M, N, K)),
            int(lib.bitlinear_backward_quantized_workspace_size(M, N, K)))
    if n == 0:
        raise BitLinearError(2, "bitlinear_backward_quantized_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def backward_quantized(xq: torch.Tensor, scale: torch.Tensor, grad_y: torch.Tensor,
                       packedT: torch.Tensor, gamma: torch.Tensor, need_x: bool = True,
                       need_w: bool = True, ws: torch.Tensor | None = None, stream=None):
    """backward for a forward that ran on int8 activations xq [M][K] with scales [M]."""
    if stream is not None:
        return _on(stream, backward_quantized, xq, scale, grad_y, packedT, gamma, need_x, need_w,
                   ws)
    (M, K), N, at = xq.shape, grad_y.shape[1], _index(xq, "xq")
    gx = scale.new_empty((M, K)) if need_x else None
    gw = scale.new_empty((N, K)) if need_w else None
    if ws is None:
        ws = backward_workspace(M, N, K, xq.device)
    _run((_lib or load_library()).bitlinear_backward_quantized, "bitlinear_backward_quantized", at,
         _take(xq, "xq", (M, K), torch.int8, at), _take(scale, "scale", (M,), torch.float32, at),
         _take(grad_y, "grad_y", (M, N), torch.bfloat16, at),
         _take(packedT, "packedT", (K, N // 4), torch.uint8, at),
         _take(gamma, "gamma", (1,), torch.float32, at),
         gx.data_ptr() if need_x else None, gw.data_ptr() if need_w else None, M, N, K,
         _take_ws(ws, at), ws.numel())
    return gx, gw


def forward_quantized(xq: torch.Tensor, scale: torch.Tensor, packed: torch.Tensor,
                      gamma: torch.Tensor, out_dtype: torch.dtype = torch.bfloat16,
                      y: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """BitLinear forward of int8 activations xq [M][K] with scales [M] (rmsnorm_quantize,
    quantize_acts): y [M][N]."""
    if stream is not None:
        return _on(stream, forward_quantized, xq, scale, packed, gamma, out_dtype, y, ws)
    (M, K), N, at = xq.shape, packed.shape[0], _index(xq, "xq")
    if y is None:
        y = xq.new_empty((M, N), dtype=out_dtype)
    if ws is None and (M > FEW_TOKENS or K > 32768):
        ws = workspace(M, N, K, xq.device)
    _run((_lib or load_library()).bitlinear_forward_quantized, "bitlinear_forward_quantized", at,
         _take(xq, "xq", (M, K), torch.int8, at), _take(scale, "scale", (M,), torch.float32, at),
         _take(packed, "packed", (N, K // 4), torch.uint8, at),
         _take(gamma, "gamma", (1,), torch.float32, at), _take(y, "y", (M, N), _FLOATS, at),
         _code(y), M, N, K, None if ws is None else _take_ws(ws, at), 0 if ws is None else ws.numel())
    return y


FEW_TOKENS = 16  # forward_quantized needs no workspace up to here (with K <= 32768)


def rmsnorm_quantize(x: torch.Tensor, weight: torch.Tensor, residual: torch.Tensor | None = None,
                     eps: float = 1e-5, h: torch.Tensor | None = None,
                     xq: torch.Tensor | None = None, scale: torch.Tensor | None = None,
                     rstd: torch.Tensor | None = None, normed: torch.Tensor | None = None,
                     stream=None):
    """RMS norm of h = x + residual with gain weight [K], as int8 codes: (xq [M][K], scale [M],
    h [M][K], rstd [M]). h is x itself without a residual; it may be given as x or residual
    (added in place). normed, if given, receives the normalised rows themselves."""
    if stream is not None:
        return _on(stream, rmsnorm_quantize, x, weight, residual, eps, h, xq, scale, rstd, normed)
    (M, K), at, dt = x.shape, _index(x, "x"), x.dtype
    if residual is None:
        h = x
    elif h is None:
        h = x.new_empty((M, K))
    if xq is None:
        xq = x.new_empty((M, K), dtype=torch.int8)
    if scale is None:
        scale = x.new_empty(M, dtype=torch.float32)
    if rstd is None:
        rstd = x.new_empty(M, dtype=torch.float32)
    row = (M,)
    _run((_lib or load_library()).bitlinear_rmsnorm_quantize, "bitlinear_rmsnorm_quantize", at,
         _take(x, "x", (M, K), _FLOATS, at),
         None if residual is None else _take(residual, "residual", (M, K), dt, at), _code(x),
         _take(weight, "weight", (K,), _FLOATS, at), _code(weight), eps, M, K,
         None if residual is None else _take(h, "h", (M, K), dt, at),
         None if normed is None else _take(normed, "normed", (M, K), dt, at),
         _take(xq, "xq", (M, K), torch.int8, at), _take(scale, "scale", row, torch.float32, at),
         _take(rstd, "rstd", row, torch.float32, at))
    return xq, scale, h, rstd


def rmsnorm_backward_workspace(M: int, K: int, device="cuda") -> torch.Tensor:
    """A caller-owned device workspace for rmsnorm_backward."""
    device = torch.device(device)
    with torch.cuda.device(device):
        n = int(load_library().bitlinear_rmsnorm_backward_workspace_size(M, K))
    if n == 0:
        raise BitLinearError(2, "bitlinear_rmsnorm_backward_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def rmsnorm_backward(grad_n: torch.Tensor, h: torch.Tensor, weight: torch.Tensor,
                     rstd: torch.Tensor, grad_h: torch.Tensor | None = None,
                     out_dtype: torch.dtype = torch.float32, grad_x: torch.Tensor | None = None,
                     grad_weight: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                     stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """Gradient of rmsnorm_quantize (straight through the quantizer): (grad_x [M][K], for x and
    the residual alike, grad_weight fp32 [K]) from the gradient grad_n of the normalised rows
    and, if given, the gradient grad_h that reaches h past the norm (of grad_x's type; grad_x
    may be grad_h itself)."""
    if stream is not None:
        return _on(stream, rmsnorm_backward, grad_n, h, weight, rstd, grad_h, out_dtype, grad_x,
                   grad_weight, ws)
    (M, K), at = h.shape, _index(h, "h")
    if grad_x is None:
        grad_x = h.new_empty((M, K), dtype=out_dtype)
    if grad_weight is None:
        grad_weight = h.new_empty(K, dtype=torch.float32)
    if ws is None:
        ws = rmsnorm_backward_workspace(M, K, h.device)
    _run((_lib or load_library()).bitlinear_rmsnorm_backward, "bitlinear_rmsnorm_backward", at,
         _take(grad_n, "grad_n", (M, K), _FLOATS, at), _code(grad_n), _take(h, "h", (M, K), _FLOATS, at),
         _code(h), _take(weight, "weight", (K,), _FLOATS, at), _code(weight),
         _take(rstd, "rstd", (M,), torch.float32, at),
         None if grad_h is None else _take(grad_h, "grad_h", (M, K), grad_x.dtype, at),
         _take(grad_x, "grad_x", (M, K), _FLOATS, at), _code(grad_x),
         _take(grad_weight, "grad_weight", (K,), torch.float32, at), M, K, _take_ws(ws, at), ws.numel())
    return grad_x, grad_weight


ACTIVATIONS = {"silu": 0, "relu2": 1}


def quantize_expert_weights(W: torch.Tensor, eps: float = 1e-5,
                            stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """quantize_weights of every expert of W [E][N][K] -> (packed [E][N][K/4], gamma [E])."""
    if stream is not None:
        return _on(stream, quantize_expert_weights, W, eps)
    E, N, K = W.shape
    packed = torch.empty((E, N, K // 4), dtype=torch.uint8, device=W.device)
    one = torch.empty((E, 4), dtype=torch.float32, device=W.device)  # each gamma 16-byte aligned
    ws = workspace(1, N, K, W.device)
    with torch.cuda.device(W.device):
        for e in range(E):
            quantize_weights(W[e], eps, packed[e], one[e, :1], ws)
        return packed, one[:, 0].contiguous()


class MoeLayer:
    """The weights of a mixture-of-experts layer for moe_forward: router [E][D] (fp32 or bf16)
    and the packed experts gate, up [E][F][D/4] and down [E][D][F/4] with their gammas [E]
    (quantize_expert_weights). Keeps the tensors alive."""

    def __init__(self, router: torch.Tensor, gate: torch.Tensor, gate_gamma: torch.Tensor,
                 up: torch.Tensor, up_gamma: torch.Tensor, down: torch.Tensor,
                 down_gamma: torch.Tensor, top_k: int, activation: str = "silu",
                 renormalize: bool = True):
        if activation not in ACTIVATIONS:
            raise ValueError(f"activation must be one of {tuple(ACTIVATIONS)}")
        (E, D), F, at = router.shape, gate.shape[1], _index(router, "router")
        self.E, self.D, self.F, self.top_k, self.device = E, D, F, int(top_k), router.device
        self.tensors = (router, gate, up, down, gate_gamma, up_gamma, down_gamma)
        self.struct = Moe(
            _take(router, "router", (E, D), _FLOATS, at),
            _take(gate, "gate", (E, F, D // 4), torch.uint8, at),
            _take(up, "up", (E, F, D // 4), torch.uint8, at),
            _take(down, "down", (E, D, F // 4), torch.uint8, at),
            _take(gate_gamma, "gate_gamma", (E,), torch.float32, at),
            _take(up_gamma, "up_gamma", (E,), torch.float32, at),
            _take(down_gamma, "down_gamma", (E,), torch.float32, at),
            _code(router), E, D, F, int(top_k), ACTIVATIONS[activation], int(bool(renormalize)))
        self._ref = ctypes.byref(self.struct)


def moe_workspace(M: int, layer: MoeLayer) -> torch.Tensor:
    """A caller-owned device workspace for moe_forward of M tokens (or fewer)."""
    n = int(load_library().bitlinear_moe_workspace_size(M, layer._ref))
    if n == 0:
        raise BitLinearError(2, "bitlinear_moe_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=layer.device)


def moe_forward(x: torch.Tensor, layer: MoeLayer, out_dtype: torch.dtype = torch.bfloat16,
                y: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """A mixture-of-experts layer for a few tokens (up to 64): x [M][D] -> y [M][D]."""
    if stream is not None:
        return _on(stream, moe_forward, x, layer, out_dtype, y, ws)
    M, at, shape = x.shape[0], _index(layer.tensors[0], "router"), (x.shape[0], layer.D)
    if y is None:
        y = layer.tensors[0].new_empty(shape, dtype=out_dtype)
    if ws is None:
        ws = moe_workspace(M, layer)
    _run((_lib or load_library()).bitlinear_moe_forward, "bitlinear_moe_forward", at,
         _take(x, "x", shape, _FLOATS, at), _code(x), M, layer._ref, _take(y, "y", shape, _FLOATS, at), _code(y),
         _take_ws(ws, at), ws.numel())
    return y


def forward(x: torch.Tensor, packed: torch.Tensor, gamma: torch.Tensor,
            out_dtype: torch.dtype = torch.bfloat16, y: torch.Tensor | None = None,
            ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """BitLinear forward: y [M][N] = rescale(int32 contraction of quantized x with W)."""
    if stream is not None:
        return _on(stream, forward, x, packed, gamma, out_dtype, y, ws)
    lib = load_library()
    M, K = x.shape
    N = packed.shape[0]
    if packed.shape[1] * 4 != K:
        raise ValueError("packed must be [N][K/4]")
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    if ws is None:
        ws = workspace(M, N, K, x.device)
    _check(lib.bitlinear_forward(
        _dev(x, "x"), _dtype_code(x), _dev(packed, "packed"), _dev(gamma, "gamma"), _dev(y, "y"),
        _dtype_code(y), M, N, K, _dev(ws, "ws"), ws.numel(), _stream()),
        "bitlinear_forward")
    return y


def forward_noalloc(x: torch.Tensor, packed: torch.Tensor, gamma: torch.Tensor,
                    out_dtype: torch.dtype = torch.bfloat16, y: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """bitlinear_forward without a workspace: the library's built-in 16 MiB device scratch
    serves the tensor-core path (for callers that cannot allocate; calls must not overlap
    on the GPU)."""
    if stream is not None:
        return _on(stream, forward_noalloc, x, packed, gamma, out_dtype, y)
    lib = load_library()
    M, K = x.shape
    N = packed.shape[0]
    if packed.shape[1] * 4 != K:
        raise ValueError("packed must be [N][K/4]")
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    _check(lib.bitlinear_forward_noalloc(
        _dev(x, "x"), _dtype_code(x), _dev(packed, "packed"), _dev(gamma, "gamma"), _dev(y, "y"),
        _dtype_code(y), M, N, K, _stream()), "bitlinear_forward_noalloc")
    return y


def contract_i32(xq: torch.Tensor, packed: torch.Tensor, acc: torch.Tensor | None = None,
                 ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Integer stage only: acc [M][N] int32 = sum_k c[n,k] * xq[t,k]."""
    if stream is not None:
        return _on(stream, contract_i32, xq, packed, acc, ws)
    lib = load_library()
    M, K = xq.shape
    N = packed.shape[0]
    if acc is None:
        acc = torch.empty((M, N), dtype=torch.int32, device=xq.device)
    if ws is None:
        ws = workspace(M, N, K, xq.device)
    _check(lib.bitlinear_contract_i32(_dev(xq, "xq"), _dev(packed, "packed"), _dev(acc, "acc"),
                                      M, N, K, _dev(ws, "ws"), ws.numel(), _stream()),
           "bitlinear_contract_i32")
    return acc


def get_device_status(stream=None) -> int:
    """Synchronizes the stream, returns and clears the device status word (0 = BL_OK)."""
    return int(load_library().bitlinear_get_device_status(_stream(stream)))


def debug_timeout_probe(timeout_ns: int, stream=None) -> None:
    _check(load_library().bitlinear_debug_timeout_probe(int(timeout_ns), _stream(stream)),
           "bitlinear_debug_timeout_probe")


PATHS = ("gemv", "skinny", "prefill")


def debug_plan(M: int, N: int, K: int, sms: int = 148) -> tuple[str, int]:
    """The kernel a forward of this shape runs and its K splits (host only, no device)."""
    path, splits = ctypes.c_int(-1), ctypes.c_int(0)
    _check(load_library().bitlinear_debug_plan(M, N, K, sms, ctypes.byref(path),
                                               ctypes.byref(splits)), "bitlinear_debug_plan")
    return PATHS[path.value], splits.value


def status_string(status: int) -> str:
    return load_library().bitlinear_status_string(status).decode()
