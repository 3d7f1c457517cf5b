"""Python binding of libfg8 (the C ABI declared in include/fg8.h).

Argument marshalling only: every step of the path runs in the CUDA kernels of
libfg8.so.  PyTorch supplies device memory and streams.  There is no CPU
fallback: if the library is missing, or a tensor is not on a CUDA device,
these functions raise.

Two layers:
  * `fg8_*` functions with the C names and arguments (tensors or None in place
    of pointers), raising FG8Error on a non-OK status;
  * small helpers (`quantize_act`, `quantize_weight`, ...) that allocate the
    output tensors with torch, on the stream of the call, and call the former.
"""

from __future__ import annotations

import ctypes
import os
import re

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libfg8.so")
HEADER = os.path.join(os.path.dirname(HERE), "include", "fg8.h")

FG8_OK = 0
FG8_ERR_INVALID_ARG = 1
FG8_ERR_UNSUPPORTED = 2
FG8_ERR_CUDA = 3
FG8_ERR_BAD_EXPERT_ID = 4
FG8_ERR_TIMEOUT = 5
FG8_ERR_WORKSPACE_SHARED = 6
FG8_ROWWISE = 1
FG8_COLWISE = 2
FG8_OUT_BF16 = 0
FG8_OUT_F32 = 1
FG8_GROUP_M = 0
FG8_GROUP_K = 1
FG8_BSCALE_BLOCK128 = 0
FG8_BSCALE_ROW128 = 1
FG8_MOE_DECODE_HEAD = 4096 + 2 * 160 * 64 * 128 * 8


class FG8Error(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_name(status)} ({status})")
        self.status = status


_lib = None
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I = ctypes.c_int
_SZ = ctypes.c_size_t


def lib() -> ctypes.CDLL:
    """Load libfg8.so (built in-tree by fp8_fine_grained_permute_b200.build)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libfg8.so is not built ({LIB_PATH}); run "
                               "`python -m fp8_fine_grained_permute_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        L.fg8_quantize_act.restype = _I
        L.fg8_quantize_act.argtypes = [_P, _I64, _I64, _P, _I, _I, _P, _I, _P, _P, _P, _P, _P,
                                       _P, _P, _P, _SZ, _P, _P]
        L.fg8_route_quantize_act.restype = _I
        L.fg8_route_quantize_act.argtypes = [_P, _P, _P, _I64, _I64, _I, _I, _P, _P, _P, _P, _P,
                                             _P, _P, _P, _SZ, _P, _P]
        L.fg8_quantize_act_noalloc.restype = _I
        L.fg8_quantize_act_noalloc.argtypes = [_P, _I64, _I64, _P, _I, _I, _P, _P, _P, _P, _P,
                                               _P, _P]
        L.fg8_quantize_act_workspace.restype = _SZ
        L.fg8_quantize_act_workspace.argtypes = [_I64, _I, _I]
        L.fg8_colwise_capacity.restype = _I64
        L.fg8_colwise_capacity.argtypes = [_I64, _I]
        L.fg8_quantize_weight.restype = _I
        L.fg8_quantize_weight.argtypes = [_P, _I, _I, _I, _P, _P, _P, _P]
        L.fg8_quantize_weight_transposed.restype = _I
        L.fg8_quantize_weight_transposed.argtypes = [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P]
        L.fg8_transpose_blockq.restype = _I
        L.fg8_transpose_blockq.argtypes = [_P, _P, _I, _I, _I, _P, _P, _P]
        L.fg8_grouped_gemm.restype = _I
        L.fg8_grouped_gemm.argtypes = [_P, _P, _P, _P, _P, _I64, _I, _I, _I, _I, _I, _I, _P, _P,
                                       _SZ, _P, _P]
        L.fg8_grouped_gemm_workspace.restype = _SZ
        L.fg8_grouped_gemm_workspace.argtypes = [_I]
        L.fg8_grouped_gemm_swiglu_quant.restype = _I
        L.fg8_grouped_gemm_swiglu_quant.argtypes = [_P, _P, _P, _P, _P, _I64, _I, _I, _I, _P, _P,
                                                    _P, _P]
        L.fg8_grouped_gemm_swiglu_quant_save.restype = _I
        L.fg8_grouped_gemm_swiglu_quant_save.argtypes = [_P, _P, _P, _P, _P, _I64, _I, _I, _I, _P,
                                                         _P, _P, _P, _P, _P]
        L.fg8_swiglu_backward_quant.restype = _I
        L.fg8_swiglu_backward_quant.argtypes = [_P, _P, _P, _P, _P, _I64, _I, _I, _P, _P, _P, _P,
                                                _P, _P, _P, _P, _P, _P]
        L.fg8_requantize_colwise.restype = _I
        L.fg8_requantize_colwise.argtypes = [_P, _P, _I64, _I64, _P, _P, _I64, _I, _P, _P, _P, _P,
                                             _P]
        L.fg8_gate_weights.restype = _I
        L.fg8_gate_weights.argtypes = [_P, _P, _I64, _I, _I, _I64, _P, _P]
        L.fg8_gate_backward.restype = _I
        L.fg8_gate_backward.argtypes = [_P, _I, _I64, _P, _P, _P, _I64, _I, _I, _I, _P, _P, _P]
        L.fg8_route_topk.restype = _I
        L.fg8_route_topk.argtypes = [_P, _P, _I64, _I, _I, _P, _P, _P]
        L.fg8_unpermute_combine.restype = _I
        L.fg8_unpermute_combine.argtypes = [_P, _I64, _I, _P, _P, _I64, _I, _I, _I, _P, _P]
        L.fg8_grouped_gemm_combine_workspace.restype = _SZ
        L.fg8_grouped_gemm_combine_workspace.argtypes = [_I64]
        L.fg8_grouped_gemm_combine.restype = _I
        L.fg8_grouped_gemm_combine.argtypes = [_P, _P, _P, _P, _P, _I64, _I, _I, _I, _P, _P, _P,
                                               _I64, _I, _I, _P, _P, _SZ, _P, _P]
        L.fg8_moe_decode_workspace.restype = _SZ
        L.fg8_moe_decode_workspace.argtypes = [_I64, _I, _I64, _I64]
        L.fg8_moe_decode.restype = _I
        L.fg8_moe_decode.argtypes = [_P, _I64, _I, _P, _P, _P, _P, _I, _I, _P, _P, _I, _P, _P, _I,
                                     _I, _P, _P, _SZ, _P, _P]
        L.fg8_ep_pack_scales.restype = _I
        L.fg8_ep_pack_scales.argtypes = [_P, _I64, _I64, _P, _P]
        L.fg8_ep_unpack.restype = _I
        L.fg8_ep_unpack.argtypes = [_P, _P, _P, _I, _I, _I64, _I64, _P, _P, _P, _P, _P, _P]
        L.fg8_gather_rows.restype = _I
        L.fg8_gather_rows.argtypes = [_P, _I64, _I64, _P, _I64, _P, _P, _P]
        L.fg8_selftest_wait_timeout.restype = _I
        L.fg8_selftest_wait_timeout.argtypes = [_I, _P, _P, _P]
        L.fg8_status_string.restype = ctypes.c_char_p
        L.fg8_status_string.argtypes = [_I]
        _lib = L
    return _lib


def declared_symbols() -> list[str]:
    """Names of the functions include/fg8.h declares."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*(?:[\w\s\*]+?)\b(fg8_\w+)\s*\(", text, flags=re.M)))


def status_name(status: int) -> str:
    return lib().fg8_status_string(int(status)).decode()


def _check(status: int, what: str) -> None:
    if status != FG8_OK:
        raise FG8Error(status, what)


def _ptr(t):
    if t is None:
        return None
    try:
        if t.is_cuda and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor or None")
    if not t.is_cuda:
        raise ValueError("libfg8 takes CUDA tensors only (no CPU fallback)")
    raise ValueError("libfg8 takes contiguous tensors")


def _stream(stream) -> int:
    if stream is None:   # the current stream's handle, without building a Stream object
        device = _device()   # first: it raises where torch lacks the next line's function
        return torch._C._cuda_getCurrentRawStream(device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


# --------------------------------------------------------------------------
# C-named entry points
# --------------------------------------------------------------------------

def fg8_quantize_act(x, T, K, topk_ids, k, E, offsets_in, layout, xq, sa, row_token, token_row,
                     offsets_out, xqT, saT, workspace, ws_bytes, dev_status, stream=None):
    _check(lib().fg8_quantize_act(_ptr(x), T, K, _ptr(topk_ids), k, E, _ptr(offsets_in), layout,
                                  _ptr(xq), _ptr(sa), _ptr(row_token), _ptr(token_row),
                                  _ptr(offsets_out), _ptr(xqT), _ptr(saT), _ptr(workspace),
                                  ws_bytes, _ptr(dev_status), _stream(stream)),
           "fg8_quantize_act")


def fg8_route_quantize_act(logits, bias, x, T, K, k, E, topk_ids, affinity, xq, sa, row_token,
                           token_row, offsets_out, workspace, ws_bytes, dev_status, stream=None):
    _check(lib().fg8_route_quantize_act(_ptr(logits), _ptr(bias), _ptr(x), T, K, k, E,
                                        _ptr(topk_ids), _ptr(affinity), _ptr(xq), _ptr(sa),
                                        _ptr(row_token), _ptr(token_row), _ptr(offsets_out),
                                        _ptr(workspace), ws_bytes, _ptr(dev_status),
                                        _stream(stream)),
           "fg8_route_quantize_act")


def fg8_quantize_act_noalloc(x, T, K, topk_ids, k, E, xq, sa, row_token, token_row, offsets_out,
                             dev_status, stream=None):
    """Permute + 1x128 quantize using the library's built-in scratch (no
    workspace argument, nothing allocated; E <= 256)."""
    _check(lib().fg8_quantize_act_noalloc(_ptr(x), T, K, _ptr(topk_ids), k, E, _ptr(xq), _ptr(sa),
                                          _ptr(row_token), _ptr(token_row), _ptr(offsets_out),
                                          _ptr(dev_status), _stream(stream)),
           "fg8_quantize_act_noalloc")


def fg8_quantize_act_workspace(T: int, k: int, E: int) -> int:
    return lib().fg8_quantize_act_workspace(T, k, E)


def fg8_colwise_capacity(R: int, E: int) -> int:
    return lib().fg8_colwise_capacity(R, E)


def fg8_quantize_weight_transposed(w, E, N, K, wq, sw, wqT, swT, dev_status=None, stream=None):
    _check(lib().fg8_quantize_weight_transposed(_ptr(w), E, N, K, _ptr(wq), _ptr(sw), _ptr(wqT),
                                                _ptr(swT), _ptr(dev_status), _stream(stream)),
           "fg8_quantize_weight_transposed")


def fg8_quantize_weight(w, E, N, K, wq, sw, dev_status=None, stream=None):
    _check(lib().fg8_quantize_weight(_ptr(w), E, N, K, _ptr(wq), _ptr(sw), _ptr(dev_status),
                                     _stream(stream)),
           "fg8_quantize_weight")


def fg8_transpose_blockq(wq, sw, E, N, K, wqT, swT, stream=None):
    _check(lib().fg8_transpose_blockq(_ptr(wq), _ptr(sw), E, N, K, _ptr(wqT), _ptr(swT),
                                      _stream(stream)),
           "fg8_transpose_blockq")


def fg8_grouped_gemm(a, sa, b, sb, offsets, M_total, N, K, E, group_mode, bscale_mode,
                     out_dtype, out, workspace, ws_bytes, dev_status, stream=None):
    _check(lib().fg8_grouped_gemm(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(offsets), M_total,
                                  N, K, E, group_mode, bscale_mode, out_dtype, _ptr(out),
                                  _ptr(workspace), ws_bytes, _ptr(dev_status), _stream(stream)),
           "fg8_grouped_gemm")


def fg8_grouped_gemm_workspace(group_mode: int) -> int:
    return int(lib().fg8_grouped_gemm_workspace(group_mode))


def fg8_grouped_gemm_swiglu_quant(a, sa, b, sb, offsets, M_total, I, K, E, hq, sh, dev_status,
                                  stream=None):
    _check(lib().fg8_grouped_gemm_swiglu_quant(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(offsets),
                                               M_total, I, K, E, _ptr(hq), _ptr(sh),
                                               _ptr(dev_status), _stream(stream)),
           "fg8_grouped_gemm_swiglu_quant")


def fg8_grouped_gemm_swiglu_quant_save(a, sa, b, sb, offsets, M_total, I, K, E, hq, sh, guq, sgu,
                                       dev_status, stream=None):
    _check(lib().fg8_grouped_gemm_swiglu_quant_save(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb),
                                                    _ptr(offsets), M_total, I, K, E, _ptr(hq),
                                                    _ptr(sh), _ptr(guq), _ptr(sgu),
                                                    _ptr(dev_status), _stream(stream)),
           "fg8_grouped_gemm_swiglu_quant_save")


def fg8_swiglu_backward_quant(dh, guq, sgu, row_w, offsets, R, I, E, dq, sd, dqT, sdT, hqT, shT,
                              gate_dot, offsets_out, dev_status, stream=None):
    _check(lib().fg8_swiglu_backward_quant(_ptr(dh), _ptr(guq), _ptr(sgu), _ptr(row_w),
                                           _ptr(offsets), R, I, E, _ptr(dq), _ptr(sd), _ptr(dqT),
                                           _ptr(sdT), _ptr(hqT), _ptr(shT), _ptr(gate_dot),
                                           _ptr(offsets_out), _ptr(dev_status), _stream(stream)),
           "fg8_swiglu_backward_quant")


def fg8_requantize_colwise(xq, sx, T, K, row_token, offsets, R, E, xqT, saT, offsets_out,
                           dev_status, stream=None):
    _check(lib().fg8_requantize_colwise(_ptr(xq), _ptr(sx), T, K, _ptr(row_token), _ptr(offsets),
                                        R, E, _ptr(xqT), _ptr(saT), _ptr(offsets_out),
                                        _ptr(dev_status), _stream(stream)),
           "fg8_requantize_colwise")


def fg8_gate_weights(token_row, affinity, T, k, normalize, R, row_w, stream=None):
    _check(lib().fg8_gate_weights(_ptr(token_row), _ptr(affinity), T, k, normalize, R,
                                  _ptr(row_w), _stream(stream)),
           "fg8_gate_weights")


def fg8_gate_backward(gate_dot, nb, R, token_row, topk_ids, affinity, T, k, E, normalize,
                      daffinity, dlogits, stream=None):
    _check(lib().fg8_gate_backward(_ptr(gate_dot), nb, R, _ptr(token_row), _ptr(topk_ids),
                                   _ptr(affinity), T, k, E, normalize, _ptr(daffinity),
                                   _ptr(dlogits), _stream(stream)),
           "fg8_gate_backward")


def fg8_route_topk(logits, bias, T, E, k, ids, affinity, stream=None):
    _check(lib().fg8_route_topk(_ptr(logits), _ptr(bias), T, E, k, _ptr(ids), _ptr(affinity),
                                _stream(stream)),
           "fg8_route_topk")


def fg8_unpermute_combine(y, R, C, token_row, affinity, T, k, normalize, out_dtype, out,
                          stream=None):
    _check(lib().fg8_unpermute_combine(_ptr(y), R, C, _ptr(token_row), _ptr(affinity), T, k,
                                       normalize, out_dtype, _ptr(out), _stream(stream)),
           "fg8_unpermute_combine")


def fg8_grouped_gemm_combine_workspace(M_total: int) -> int:
    return int(lib().fg8_grouped_gemm_combine_workspace(M_total))


def fg8_grouped_gemm_combine(a, sa, b, sb, offsets, M_total, N, K, E, row_token, token_row,
                             affinity, T, k, normalize, out, workspace, ws_bytes, dev_status,
                             stream=None):
    _check(lib().fg8_grouped_gemm_combine(_ptr(a), _ptr(sa), _ptr(b), _ptr(sb), _ptr(offsets),
                                          M_total, N, K, E, _ptr(row_token), _ptr(token_row),
                                          _ptr(affinity), T, k, normalize, _ptr(out),
                                          _ptr(workspace), ws_bytes, _ptr(dev_status),
                                          _stream(stream)),
           "fg8_grouped_gemm_combine")


def fg8_moe_decode_workspace(T: int, k: int, C: int, I: int) -> int:
    return int(lib().fg8_moe_decode_workspace(T, k, C, I))


def fg8_moe_decode(x, T, C, logits, bias, topk_ids, affinity, k, E, wq_up, sw_up, I, wq_dn, sw_dn,
                   normalize, out_dtype, out, workspace, ws_bytes, dev_status, stream=None):
    _check(lib().fg8_moe_decode(_ptr(x), T, C, _ptr(logits), _ptr(bias), _ptr(topk_ids),
                                _ptr(affinity), k, E, _ptr(wq_up), _ptr(sw_up), I, _ptr(wq_dn),
                                _ptr(sw_dn), normalize, out_dtype, _ptr(out), _ptr(workspace),
                                ws_bytes, _ptr(dev_status), _stream(stream)),
           "fg8_moe_decode")


def fg8_ep_pack_scales(sa, R, K, sa_rows, stream=None):
    _check(lib().fg8_ep_pack_scales(_ptr(sa), R, K, _ptr(sa_rows), _stream(stream)),
           "fg8_ep_pack_scales")


def fg8_ep_unpack(recv_xq, recv_sa, counts, W, E_loc, R_recv, K, xq, sa, offsets, recv_to_local,
                  dev_status, stream=None):
    _check(lib().fg8_ep_unpack(_ptr(recv_xq), _ptr(recv_sa), _ptr(counts), W, E_loc, R_recv, K,
                               _ptr(xq), _ptr(sa), _ptr(offsets), _ptr(recv_to_local),
                               _ptr(dev_status), _stream(stream)),
           "fg8_ep_unpack")


def fg8_gather_rows(inp, n_in, row_bytes, map_, n, out, dev_status, stream=None):
    _check(lib().fg8_gather_rows(_ptr(inp), n_in, row_bytes, _ptr(map_), n, _ptr(out),
                                 _ptr(dev_status), _stream(stream)),
           "fg8_gather_rows")


def fg8_selftest_wait_timeout(which, scratch, dev_status, stream=None):
    _check(lib().fg8_selftest_wait_timeout(which, _ptr(scratch), _ptr(dev_status), _stream(stream)),
           "fg8_selftest_wait_timeout")


def fg8_status_string(status: int) -> str:
    return status_name(status)


# --------------------------------------------------------------------------
# allocate-and-call helpers
# --------------------------------------------------------------------------

def _u16(x: torch.Tensor) -> torch.Tensor:
    if x.dtype == torch.bfloat16:
        return x.view(torch.int16)
    if x.dtype in (torch.int16, torch.uint16):
        return x
    raise TypeError("expected bf16 data")


def _bf16(x):
    """bf16 data as it is (or its bit patterns): only the type is checked."""
    if x.dtype is not torch.bfloat16 and x.dtype not in (torch.int16, torch.uint16):
        raise TypeError("expected bf16 data")
    return x


def _no_cuda():
    raise RuntimeError("this torch has no CUDA")


_device = getattr(torch._C, "_cuda_getDevice", _no_cuda)   # the current device's number, without a lazy check


def _here():
    """The current device (-2 without one: no tensor is on it)."""
    try:
        return _device()
    except RuntimeError:
        return -2


def _at(t, here=None):
    """A tensor's pointer, or the tensor itself where it is not one the library
    takes (_call then says so, after all shapes and types were looked at).  The
    launch goes to the current device (`here`): a tensor of another one is refused."""
    d = t.get_device()
    if d == here and t.is_contiguous():
        return t.data_ptr()
    if d < 0 or not t.is_contiguous():
        return t
    if d != _device():
        raise ValueError(f"a tensor on cuda:{d}, current device cuda:{_device()}")
    return t.data_ptr()


def _raw(t, here=None):
    """_at of a tensor that may be left out."""
    return None if t is None else _at(t, here)


def _torch_stream(stream):
    """The torch stream of a stream argument: one already, or one's handle."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return torch.cuda.ExternalStream(0 if handle == 1 else handle)   # 1: the legacy default stream, as 0


def _new(shape, dtype, device, stream, make=None, scratch=False):
    """A tensor for a call on `stream` (None: the current one), taken from that
    stream's memory: a block of another stream's may still be in use there.  The
    current stream, where the caller usually goes on with it, is noted as a user;
    scratch is dropped at the end of the call and is not."""
    make = make or torch.empty
    if stream is None or torch.device(device).type != "cuda":
        return make(shape, dtype=dtype, device=device)
    here = torch.cuda.current_stream(device)
    with torch.cuda.stream(_torch_stream(stream)):
        t = make(shape, dtype=dtype, device=device)
    if not scratch:
        t.record_stream(here)
    return t


def _arg(what, t, shape, dtype, here=None):
    """_raw of a tensor that has to have this shape and type (one pass a tensor: a
    helper's checks cost host time on every call)."""
    if t.shape != shape or t.dtype is not dtype:
        raise ValueError(f"{what} of shape {tuple(t.shape)} {t.dtype}, expected {tuple(shape)} {dtype}")
    if t.get_device() == here and t.is_contiguous():
        return t.data_ptr()
    return _at(t)


def _arg_n(what, t, n, dtype, here=None):
    """As _arg, for a tensor of n elements of any shape."""
    if t.numel() != n or t.dtype is not dtype:
        raise ValueError(f"{what} of {t.numel()} {t.dtype}, expected {n} {dtype}")
    if t.get_device() == here and t.is_contiguous():
        return t.data_ptr()
    return _at(t)


def _call(name, stream, *args):
    """Call an entry point of the library with _arg results and the stream."""
    try:
        status = getattr(lib(), name)(*args, _stream(stream))
    except (ctypes.ArgumentError, RuntimeError):   # a tensor among them, or no GPU at all
        for a in args:
            if isinstance(a, torch.Tensor):
                _ptr(a)   # raises
        raise
    if status != FG8_OK:
        raise FG8Error(status, name)


def new_status(device=None, stream=None) -> torch.Tensor:
    """A cleared status word (cleared on `stream`, default: the current one)."""
    return _new(1, torch.int32, device or "cuda", stream, make=torch.zeros)


def quantize_act(x: torch.Tensor, topk_ids: torch.Tensor, E: int, dev_status=None,
                 workspace=None, stream=None):
    """Permute + 1x128 quantize.  Returns dict(xq, sa, row_token, token_row, offsets)."""
    T, K = x.shape
    k = topk_ids.shape[1]
    R = T * k
    dev = x.device
    out = dict(
        xq=_new((R, K), torch.uint8, dev, stream),
        sa=_new((K // 128, R), torch.float32, dev, stream),
        row_token=_new(R, torch.int32, dev, stream),
        token_row=_new(T * k, torch.int32, dev, stream),
        offsets=_new(E + 1, torch.int32, dev, stream),
    )
    ws_bytes = fg8_quantize_act_workspace(T, k, E)
    if workspace is None:
        workspace = _new(ws_bytes, torch.uint8, dev, stream, scratch=True)
    st = dev_status if dev_status is not None else new_status(dev, stream)
    fg8_quantize_act(_u16(x), T, K, topk_ids, k, E, None, FG8_ROWWISE, out["xq"], out["sa"],
                     out["row_token"], out["token_row"], out["offsets"], None, None, workspace,
                     ws_bytes, st, stream)
    out["status"] = st
    return out


def route_quantize_act(logits: torch.Tensor, bias: torch.Tensor, x: torch.Tensor, k: int,
                       dev_status=None, workspace=None, stream=None):
    """Routing (sigmoid + bias top-k) fused with permute + 1x128 quantize.
    Returns dict(ids, affinity, xq, sa, row_token, token_row, offsets, status)."""
    T, K = x.shape
    E = logits.shape[1]
    R = T * k
    dev = x.device
    out = dict(
        ids=_new((T, k), torch.int32, dev, stream),
        affinity=_new((T, k), torch.float32, dev, stream),
        xq=_new((R, K), torch.uint8, dev, stream),
        sa=_new((K // 128, R), torch.float32, dev, stream),
        row_token=_new(R, torch.int32, dev, stream),
        token_row=_new(T * k, torch.int32, dev, stream),
        offsets=_new(E + 1, torch.int32, dev, stream),
    )
    ws_bytes = fg8_quantize_act_workspace(T, k, E)
    if workspace is None:
        workspace = _new(ws_bytes, torch.uint8, dev, stream, scratch=True)
    st = dev_status if dev_status is not None else new_status(dev, stream)
    fg8_route_quantize_act(logits, bias, _u16(x), T, K, k, E, out["ids"], out["affinity"],
                           out["xq"], out["sa"], out["row_token"], out["token_row"],
                           out["offsets"], workspace, ws_bytes, st, stream)
    out["status"] = st
    return out


def quantize_act_rows(x: torch.Tensor, stream=None):
    """1x128 quantize of rows already in expert order -> (xq [R,K], sa [K/128,R])."""
    R, K = x.shape
    xq = _new((R, K), torch.uint8, x.device, stream)
    sa = _new((K // 128, R), torch.float32, x.device, stream)
    fg8_quantize_act(_u16(x), R, K, None, 1, 1, None, FG8_ROWWISE, xq, sa, None, None, None,
                     None, None, None, 0, None, stream)
    return xq, sa


def quantize_act_colwise(x: torch.Tensor, offsets: torch.Tensor, k: int = 1,
                         row_token: torch.Tensor | None = None, stream=None):
    """Token-axis 1x128 quantization per expert -> (xqT [C,P], saT [P/128,C], padded offsets)."""
    T, C = x.shape
    E = offsets.numel() - 1
    R = T * k
    P = fg8_colwise_capacity(R, E)
    xqT = _new((C, P), torch.uint8, x.device, stream)
    saT = _new((P // 128, C), torch.float32, x.device, stream)
    padoff = _new(E + 1, torch.int32, x.device, stream)
    fg8_quantize_act(_u16(x), T, C, None, k, E, offsets, FG8_COLWISE, None, None, row_token,
                     None, padoff, xqT, saT, None, 0, None, stream)
    return xqT, saT, padoff


def quantize_weight(w: torch.Tensor, status=None, stream=None):
    """128x128 block quantize of bf16 w [E,N,K] -> (wq, sw [E,N/128,K/128])."""
    E, N, K = w.shape
    wq = _new((E, N, K), torch.uint8, w.device, stream)
    sw = _new((E, N // 128, K // 128), torch.float32, w.device, stream)
    fg8_quantize_weight(_u16(w), E, N, K, wq, sw, status, stream)
    return wq, sw


def quantize_weight_transposed(w: torch.Tensor, status=None, stream=None):
    """128x128 block quantize of bf16 w [E,N,K] plus its block-transposed copy
    -> (wq, sw, wqT [E,K,N], swT [E,K/128,N/128])."""
    E, N, K = w.shape
    wq = _new((E, N, K), torch.uint8, w.device, stream)
    sw = _new((E, N // 128, K // 128), torch.float32, w.device, stream)
    wqT = _new((E, K, N), torch.uint8, w.device, stream)
    swT = _new((E, K // 128, N // 128), torch.float32, w.device, stream)
    fg8_quantize_weight_transposed(_u16(w), E, N, K, wq, sw, wqT, swT, status, stream)
    return wq, sw, wqT, swT


def transpose_blockq(wq: torch.Tensor, sw: torch.Tensor, stream=None):
    E, N, K = wq.shape
    wqT = _new((E, K, N), torch.uint8, wq.device, stream)
    swT = _new((E, K // 128, N // 128), torch.float32, wq.device, stream)
    fg8_transpose_blockq(wq, sw, E, N, K, wqT, swT, stream)
    return wqT, swT


def grouped_gemm(a, sa, b, sb, offsets, out_dtype=FG8_OUT_BF16, group_mode=FG8_GROUP_M,
                 dev_status=None, out=None, stream=None, workspace=None):
    """Row-grouped: a [M,K], b [E,N,K] -> out [M,N].  Contraction-grouped:
    a [M,P], b [N,P] -> out [E,M,N] (its tile counter lives in `workspace`,
    allocated here when not given)."""
    M_total, K = a.shape
    E = offsets.numel() - 1
    if group_mode == FG8_GROUP_M:
        N = b.shape[1]
        shape = (M_total, N)
        bmode = FG8_BSCALE_BLOCK128
    else:
        N = b.shape[0]
        shape = (E, M_total, N)
        bmode = FG8_BSCALE_ROW128
    if out is None:
        dt = torch.float32 if out_dtype == FG8_OUT_F32 else torch.bfloat16
        out = _new(shape, dt, a.device, stream)
    ws_bytes = fg8_grouped_gemm_workspace(group_mode)
    if workspace is None and ws_bytes:
        workspace = _new(ws_bytes, torch.uint8, a.device, stream, scratch=True)
    fg8_grouped_gemm(a, sa, b, sb, offsets, M_total, N, K, E, group_mode, bmode, out_dtype, out,
                     workspace, ws_bytes if workspace is not None else 0, dev_status, stream)
    return out


def grouped_gemm_swiglu_quant(a, sa, b, sb, offsets, dev_status=None, hq=None, sh=None,
                              stream=None):
    """a [M,K] E4M3, b [E,2I,K] E4M3 (gate rows then up rows) -> (hq [M,I]
    E4M3, sh [I/128,M] fp32): the 1x128 quantization of silu(gate) * up."""
    M_total, K = a.shape
    E = offsets.numel() - 1
    I = b.shape[1] // 2
    if hq is None:
        hq = _new((M_total, I), torch.uint8, a.device, stream)
    if sh is None:
        sh = _new((I // 128, M_total), torch.float32, a.device, stream)
    fg8_grouped_gemm_swiglu_quant(a, sa, b, sb, offsets, M_total, I, K, E, hq, sh, dev_status,
                                  stream)
    return hq, sh


def grouped_gemm_swiglu_quant_save(a, sa, b, sb, offsets, hq=None, sh=None, guq=None, sgu=None,
                                   dev_status=None, stream=None):
    """As grouped_gemm_swiglu_quant, keeping the gate and up projections in 8 bits
    for the backward: -> (hq [M, I] u8, sh [I/128, M], guq [M, 2I] u8, sgu [2I/128, M])."""
    M, K = a.shape
    E, I, dev = offsets.numel() - 1, b.shape[1] // 2, a.device
    u8, f32 = torch.uint8, torch.float32
    hq = _new((M, I), u8, dev, stream) if hq is None else hq
    sh = _new((I // 128, M), f32, dev, stream) if sh is None else sh
    guq = _new((M, 2 * I), u8, dev, stream) if guq is None else guq
    sgu = _new((2 * I // 128, M), f32, dev, stream) if sgu is None else sgu
    here = _here()
    _call("fg8_grouped_gemm_swiglu_quant_save", stream,
        _arg("a", a, (M, K), u8, here), _arg("sa", sa, (K // 128, M), f32, here),
        _arg("b", b, (E, 2 * I, K), u8, here), _arg("sb", sb, (E, 2 * I // 128, K // 128), f32, here),
        _arg("offsets", offsets, (E + 1,), torch.int32, here), M, I, K, E,
        _arg("hq", hq, (M, I), u8, here), _arg("sh", sh, (I // 128, M), f32, here),
        _arg("guq", guq, (M, 2 * I), u8, here), _arg("sgu", sgu, (2 * I // 128, M), f32, here),
        _raw(dev_status, here))
    return hq, sh, guq, sgu


def swiglu_backward_quant(dh, guq, sgu, offsets, row_w=None, dq=None, sd=None, dqT=None, sdT=None,
                          hqT=None, shT=None, gate_dot=None, offsets_out=None, dev_status=None,
                          stream=None, want_dots=True):
    """dh bf16 [R, I] (gradient of the activation's output), guq/sgu (the 8-bit
    gate and up) -> dict of the [dG dU] operand by rows (dq, sd) and by columns
    (dqT, sdT), the weighted activation by columns (hqT, shT), gate_dot
    [I/128, R] and the padded offsets_out.  want_dots=False (the gates are not
    trained): no gate_dot."""
    R, I = dh.shape
    E, dev = offsets.numel() - 1, dh.device
    P = fg8_colwise_capacity(R, E)
    u8, f32, i32 = torch.uint8, torch.float32, torch.int32
    dq = _new((R, 2 * I), u8, dev, stream) if dq is None else dq
    sd = _new((2 * I // 128, R), f32, dev, stream) if sd is None else sd
    dqT = _new((2 * I, P), u8, dev, stream) if dqT is None else dqT
    sdT = _new((P // 128, 2 * I), f32, dev, stream) if sdT is None else sdT
    hqT = _new((I, P), u8, dev, stream) if hqT is None else hqT
    shT = _new((P // 128, I), f32, dev, stream) if shT is None else shT
    gate_dot = _new((I // 128, R), f32, dev, stream) if gate_dot is None and want_dots else gate_dot
    offsets_out = _new((E + 1,), i32, dev, stream) if offsets_out is None else offsets_out
    here = _here()
    _call("fg8_swiglu_backward_quant", stream,
        _raw(_bf16(dh), here), _arg("guq", guq, (R, 2 * I), u8, here), _arg("sgu", sgu, (2 * I // 128, R), f32, here),
        None if row_w is None else _arg("row_w", row_w, (R,), f32, here),
        _arg("offsets", offsets, (E + 1,), i32, here), R, I, E,
        _arg("dq", dq, (R, 2 * I), u8, here), _arg("sd", sd, (2 * I // 128, R), f32, here),
        _arg("dqT", dqT, (2 * I, P), u8, here), _arg("sdT", sdT, (P // 128, 2 * I), f32, here),
        _arg("hqT", hqT, (I, P), u8, here), _arg("shT", shT, (P // 128, I), f32, here),
        None if gate_dot is None else _arg("gate_dot", gate_dot, (I // 128, R), f32, here),
        _arg("offsets_out", offsets_out, (E + 1,), i32, here), _raw(dev_status, here))
    return dict(dq=dq, sd=sd, dqT=dqT, sdT=sdT, hqT=hqT, shT=shT, gate_dot=gate_dot,
                offsets_out=offsets_out)


def requantize_colwise(xq, sx, offsets, row_token=None, xqT=None, saT=None, offsets_out=None,
                       dev_status=None, stream=None):
    """xq u8 [T, K], sx [K/128, T] (rows kept in 8 bits) -> (xqT [K, P] u8,
    saT [P/128, K], padded offsets): quantize_act_colwise from the checkpoint."""
    T, K = xq.shape
    R = T if row_token is None else row_token.numel()
    E, dev = offsets.numel() - 1, xq.device
    P = fg8_colwise_capacity(R, E)
    u8, f32, i32 = torch.uint8, torch.float32, torch.int32
    xqT = _new((K, P), u8, dev, stream) if xqT is None else xqT
    saT = _new((P // 128, K), f32, dev, stream) if saT is None else saT
    offsets_out = _new((E + 1,), i32, dev, stream) if offsets_out is None else offsets_out
    here = _here()
    _call("fg8_requantize_colwise", stream,
        _arg("xq", xq, (T, K), u8, here), _arg("sx", sx, (K // 128, T), f32, here), T, K,
        None if row_token is None else _arg("row_token", row_token, (R,), i32, here),
        _arg("offsets", offsets, (E + 1,), i32, here), R, E, _arg("xqT", xqT, (K, P), u8, here),
        _arg("saT", saT, (P // 128, K), f32, here), _arg("offsets_out", offsets_out, (E + 1,), i32, here),
        _raw(dev_status, here))
    return xqT, saT, offsets_out


def gate_weights(token_row, affinity, R, normalize=True, row_w=None, stream=None):
    """token_row int32 [T*k], affinity fp32 [T, k] -> row_w fp32 [R]: the combine's
    gate weight of every routed row (0 where no slot names the row)."""
    T, k = affinity.shape
    f32 = torch.float32
    row_w = _new(R, f32, affinity.device, stream, make=torch.zeros) if row_w is None else row_w
    here = _here()
    _call("fg8_gate_weights", stream, _arg_n("token_row", token_row, T * k, torch.int32, here),
                                  _arg("affinity", affinity, (T, k), f32, here), T, k,
                                  int(bool(normalize)), R, _arg("row_w", row_w, (R,), f32, here))
    return row_w


def gate_backward(gate_dot, token_row, topk_ids, affinity, E, normalize=True, daffinity=None,
                  dlogits=None, stream=None, want_dlogits=True):
    """gate_dot fp32 [I/128, R] (swiglu_backward_quant) -> (daffinity [T, k],
    dlogits [T, E]): the gradients of the chosen affinities and router logits.
    want_dlogits=False: (daffinity, None), and topk_ids may be None."""
    nb, R = gate_dot.shape
    T, k = affinity.shape
    f32, i32, dev = torch.float32, torch.int32, affinity.device
    daffinity = _new((T, k), f32, dev, stream) if daffinity is None else daffinity
    dlogits = _new((T, E), f32, dev, stream) if dlogits is None and want_dlogits else dlogits
    if dlogits is not None and topk_ids is None:
        raise ValueError("gate_backward needs topk_ids for dlogits")
    here = _here()
    _call("fg8_gate_backward", stream, _arg("gate_dot", gate_dot, (nb, R), f32, here), nb, R,
                                   _arg_n("token_row", token_row, T * k, i32, here),
                                   None if topk_ids is None and dlogits is None
                                   else _arg_n("topk_ids", topk_ids, T * k, i32, here),
                                   _arg("affinity", affinity, (T, k), f32, here), T, k, E,
                                   int(bool(normalize)), _arg("daffinity", daffinity, (T, k), f32, here),
                                   None if dlogits is None else _arg("dlogits", dlogits, (T, E), f32, here))
    return daffinity, dlogits


def grouped_gemm_combine(a, sa, b, sb, offsets, row_token, token_row, affinity, normalize=True,
                         dev_status=None, out=None, stream=None, workspace=None):
    """Row-grouped GEMM a [M,K] x b [E,N,K] with the combine in its epilogue:
    -> out fp32 [T, N], each token's rows weighted by its gate weights."""
    M_total, K = a.shape
    E, N = offsets.numel() - 1, b.shape[1]
    T, k = affinity.shape
    dev = a.device
    if out is None:
        out = _new((T, N), torch.float32, dev, stream)
    if workspace is None:
        workspace = _new(max(16, fg8_grouped_gemm_combine_workspace(M_total)), torch.uint8, dev, stream, scratch=True)
    st = dev_status if dev_status is not None else new_status(dev, stream)
    fg8_grouped_gemm_combine(a, sa, b, sb, offsets, M_total, N, K, E, row_token, token_row,
                             affinity, T, k, int(bool(normalize)), out, workspace,
                             workspace.numel(), st, stream)
    return out


def moe_decode_workspace(T, k, C, I, device=None, stream=None):
    """A zeroed workspace for moe_decode calls of up to T tokens (kept by the
    caller: a call leaves it ready for the next; zero it again after one that reported
    FG8_ERR_TIMEOUT or FG8_ERR_WORKSPACE_SHARED).  It is zeroed on `stream` (default:
    the current one)."""
    n = fg8_moe_decode_workspace(T, k, C, I)
    if n == 0:
        raise ValueError("moe_decode takes 1..64 tokens, 1..16 slots and I >= 128")
    return _new(n, torch.uint8, device or "cuda", stream, make=torch.zeros)


def moe_decode(x, wq_up, sw_up, wq_dn, sw_dn, k, logits=None, bias=None, ids=None, affinity=None,
               normalize=True, out_dtype=FG8_OUT_BF16, out=None, workspace=None, dev_status=None,
               stream=None):
    """The expert layer for a few tokens: x bf16 [T, C], the quantized weights
    (wq_up [E, 2I, C], wq_dn [E, C, I] and their scales) and either logits
    [T, E] and bias [E] (routing included; ids and affinity are then outputs) or
    ids int32 [T, k] and affinity fp32 [T, k] -> (out [T, C], ids, affinity).
    workspace: moe_decode_workspace(...), kept from call to call (without one each
    call zeroes its own); calls that overlap on the GPU need their own.  A call that
    reports FG8_ERR_WORKSPACE_SHARED or FG8_ERR_TIMEOUT in dev_status stopped early: `out`
    is unspecified and the workspace is to be zeroed before the next."""
    T, C = x.shape
    E, I, dev = wq_up.shape[0], wq_dn.shape[2], x.device
    f32, u8, i32 = torch.float32, torch.uint8, torch.int32
    if logits is None and (ids is None or affinity is None):
        raise ValueError("moe_decode needs logits and bias, or ids and affinity")
    out_t = f32 if out_dtype == FG8_OUT_F32 else torch.bfloat16
    ids = _new((T, k), i32, dev, stream) if ids is None else ids
    affinity = _new((T, k), f32, dev, stream) if affinity is None else affinity
    out = _new((T, C), out_t, dev, stream) if out is None else out
    if workspace is None and T > 0:
        workspace = moe_decode_workspace(T, k, C, I, dev, stream)
    here = _here()
    _call("fg8_moe_decode", stream,
        _raw(_bf16(x), here), T, C, None if logits is None else _arg("logits", logits, (T, E), f32, here),
        None if logits is None else _arg("bias", bias, (E,), f32, here), _arg("ids", ids, (T, k), i32, here),
        _arg("affinity", affinity, (T, k), f32, here), k, E, _arg("wq_up", wq_up, (E, 2 * I, C), u8, here),
        _arg("sw_up", sw_up, (E, 2 * I // 128, C // 128), f32, here), I,
        _arg("wq_dn", wq_dn, (E, C, I), u8, here),
        _arg("sw_dn", sw_dn, (E, C // 128, I // 128), f32, here), int(bool(normalize)), out_dtype,
        _arg("out", out, (T, C), out_t, here), _raw(workspace, here),
        0 if workspace is None else workspace.numel(), _raw(dev_status, here))
    return out, ids, affinity


def unpermute_combine(y, token_row, affinity, normalize=True, out_dtype=FG8_OUT_BF16, out=None,
                      stream=None):
    """y bf16 [R, C] (permuted rows), token_row int32 [T*k], affinity fp32 [T, k]
    -> out [T, C]: each token's rows summed with its (normalized) gate weights."""
    R, C = y.shape
    T, k = affinity.shape
    if out is None:
        dt = torch.float32 if out_dtype == FG8_OUT_F32 else torch.bfloat16
        out = _new((T, C), dt, affinity.device, stream)
    yv = y.view(torch.int16) if y.dtype == torch.bfloat16 else y
    fg8_unpermute_combine(yv, R, C, token_row, affinity, T, k, int(bool(normalize)), out_dtype,
                          out, stream)
    return out


def route_topk(logits, bias, k, ids=None, affinity=None, stream=None):
    """logits fp32 [T, E], bias fp32 [E] -> (ids int32 [T, k], affinity fp32 [T, k])."""
    T, E = logits.shape
    if ids is None:
        ids = _new((T, k), torch.int32, logits.device, stream)
    if affinity is None:
        affinity = _new((T, k), torch.float32, logits.device, stream)
    fg8_route_topk(logits, bias, T, E, k, ids, affinity, stream)
    return ids, affinity
