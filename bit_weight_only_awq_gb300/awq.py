"""ctypes binding over libawq.so (declared in include/awq.h), same entry-point names.

Argument marshalling only: every step of the computation runs in the library's
CUDA kernels.  PyTorch provides device memory (outputs and workspaces allocated
here when the caller passes none) and the current CUDA stream.  Importing this
module loads the library and raises ImportError when it has not been built;
there is no fallback path.

A call with `stream=` runs there: its operands are ready on that stream and stay until it is past
the call, and the current stream waits for it before it uses the results.
"""

from __future__ import annotations

import ctypes
import functools
import itertools
import os
import re
import threading

import torch

_LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libawq.so")
_HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "awq.h")

if not os.path.exists(_LIB_PATH):
    raise ImportError(f"{_LIB_PATH} is missing: build it with `python -m bit_weight_only_awq_gb300.build`")
lib = ctypes.CDLL(_LIB_PATH)

STATUS = {0: "AWQ_OK", -1: "AWQ_EINVAL", -2: "AWQ_EALIGN", -3: "AWQ_EARCH", -4: "AWQ_ECUDA",
          -5: "AWQ_ETIMEOUT", -6: "AWQ_EWORKSPACE", -7: "AWQ_ENULL"}
FP16, BF16 = 0, 1
OP_GEMV, OP_GEMM, OP_W4A8_GEMM, OP_GEMV_PREPACKED, OP_GEMV_BF16, OP_GEMM_BF16, OP_W4A8_GROUPED = 0, 1, 2, 3, 4, 5, 6
GROUP_SIZE = 128

_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_f32 = ctypes.c_float
_sz = ctypes.c_size_t

_SIGS = {
    "awq_status_string": (ctypes.c_char_p, [_i32]),
    "awq_pack": (_i32, [_p, _i64, _i64, _p, _p]),
    "awq_unpack": (_i32, [_p, _i64, _i64, _p, _p]),
    "awq_pack_order": (_i32, [_p, _i64, _i64, _i32, _p, _p]),
    "awq_unpack_order": (_i32, [_p, _i64, _i64, _i32, _p, _p]),
    "awq_dequant": (_i32, [_p, _p, _p, _i64, _i64, _i32, _p, _p]),
    "awq_workspace_bytes": (_sz, [_i32, _i64, _i64, _i64, _i32]),
    "awq_gemv": (_i32, [_p, _p, _p, _p, _p, _i64, _i64, _i64, _i32, _i32, _p, _sz, _p]),
    "awq_gemm": (_i32, [_p, _p, _p, _p, _p, _i64, _i64, _i64, _i32, _i32, _p, _sz, _p]),
    "awq_gemv_noalloc": (_i32, [_p, _p, _p, _p, _p, _i64, _i64, _i64, _i32, _i32, _p]),
    "w4a8_quant_act": (_i32, [_p, _p, _p, _i64, _i64, _p]),
    "w4a8_gemm": (_i32, [_p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _i32, _p, _sz, _p]),
    "w4a8_linear": (_i32, [_p, _p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _i32, _p, _sz, _p]),
    "awq_dequant_bf16": (_i32, [_p, _p, _p, _i64, _i64, _i32, _p, _p]),
    "awq_gemv_bf16": (_i32, [_p, _p, _p, _p, _p, _i64, _i64, _i64, _i32, _i32, _p, _sz, _p]),
    "awq_gemm_bf16": (_i32, [_p, _p, _p, _p, _p, _i64, _i64, _i64, _i32, _i32, _p, _sz, _p]),
    "awq_prepacked_bytes": (_sz, [_i64, _i64]),
    "awq_prepack_gemv": (_i32, [_p, _p, _p, _i64, _i64, _i32, _p, _sz, _p]),
    "awq_unprepack_gemv": (_i32, [_p, _i64, _i64, _p, _p, _p, _p]),
    "awq_gemv_prepacked": (_i32, [_p, _p, _p, _i64, _i64, _i64, _i32, _p, _sz, _p]),
    "w4a8_gemm_grouped": (_i32, [_p, _p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _i32, _i32, _p, _sz, _p]),
    "w4a8_linear_grouped": (_i32, [_p, _p, _p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _i32, _i32, _p, _sz, _p]),
    "w4a8_rmsnorm_quant": (_i32, [_p, _p, _p, _p, _p, _p, _p, _i64, _i64, _i64, _i64, _f32, _i32, _p]),
    "awq_rmsnorm": (_i32, [_p, _p, _p, _p, _p, _i64, _i64, _i64, _i64, _f32, _i32, _p]),
    "kv4_cache_bytes": (_sz, [_i64, _i32, _i32, _i32]),
    "kv4_append": (_i32, [_p, _p, _p, _i64, _i64, _i64, _p, _p, _p, _i64, _i32, _i32, _p, _i64, _p, _i64, _i64, _i32,
                          _i32, _i32, _i32, _i32, _p]),
    "kv4_gather": (_i32, [_p, _p, _p, _p, _i64, _i64, _i32, _i32, _i32, _i32, _p]),
    "kv4_attention_workspace_bytes": (_sz, [_i64, _i64, _i32, _i32, _i32, _i32]),
    "kv4_attention": (_i32, [_p, _i64, _p, _p, _i64, _p, _p, _p, _p, _i64, _i64, _i32, _i32, _i32, _i32, _i64, _i32,
                             _i32, _f32, _i32, _i32, _p, _sz, _p]),
    "awq_moe_plan": (_i32, [_p, _i64, _i32, _p, _p, _p, _p]),
    "awq_moe_route": (_i32, [_p, _i64, _i64, _i32, _i32, _i32, _i32, _p, _p, _p, _p, _p, _p]),
    "awq_moe_prepacked_bytes": (_sz, [_i32, _i64, _i64, _i32]),
    "awq_moe_prepack": (_i32, [_p, _p, _p, _i32, _i64, _i64, _i32, _i32, _p, _sz, _p]),
    "awq_moe_unprepack": (_i32, [_p, _i32, _i64, _i64, _i32, _p, _p, _p, _p]),
    "awq_moe_gemm_workspace_bytes": (_sz, [_i64, _i32, _i64, _i64, _i32]),
    "awq_moe_gemm": (_i32, [_p, _i64, _i64, _p, _p, _p, _i32, _p, _i32, _i64, _i32, _i64, _i64, _i32, _i32, _p, _sz, _p]),
    "awq_moe_combine": (_i32, [_p, _i32, _p, _p, _p, _i64, _p, _i64, _i32, _i64, _i64, _i32, _p]),
    "awq_moe_workspace_bytes": (_sz, [_i64, _i32, _i32, _i64, _i64, _i64]),
    "awq_moe": (_i32, [_p, _i64, _p, _p, _p, _p, _p, _p, _p, _i64, _p, _i64, _i32, _i32, _i64, _i64, _i64, _i32, _p, _sz, _p]),
    "awq_fp8_quant_act": (_i32, [_p, _i64, _p, _p, _i64, _i64, _i32, _p]),
    "awq_fp8_gemm_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "awq_fp8_gemm": (_i32, [_p, _p, _p, _p, _p, _i64, _i64, _i64, _i32, _p, _sz, _p]),
    "awq_fp8_linear_workspace_bytes": (_sz, [_i64, _i64, _i64]),
    "awq_fp8_linear": (_i32, [_p, _i64, _p, _p, _p, _i64, _i64, _i64, _i32, _p, _sz, _p]),
    "awq_last_device_error": (_i32, [ctypes.POINTER(_i32)]),
    "awq_selftest_wait_timeout": (_i32, [_i64, _p]),
}
for _name, (_res, _args) in _SIGS.items():
    _fn = getattr(lib, _name)
    _fn.restype = _res
    _fn.argtypes = _args


def header_functions() -> list[str]:
    """Names of the functions declared in include/awq.h."""
    with open(_HEADER) as fh:
        text = fh.read()
    return sorted(set(re.findall(r"^\s*(?:const\s+)?[a-z_0-9]+\s*\*?\s*((?:awq|w4a8|kv4)_[a-z0-9_]+)\s*\(", text, re.M)))


class AwqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        msg = lib.awq_status_string(status).decode()
        super().__init__(f"{fn}: {msg}")
        self.status = status


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise AwqError(fn, status)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


# A call may be several launches that hand data on through its workspace, and the interpreter runs other threads
# meanwhile: whoever takes a workspace that other calls share keeps its lock from the taking to the last launch.  A
# signal handler or finalizer that calls from within the taking has all its launches before the first of this call.
_locks: dict[tuple, threading.RLock] = {}


def _lock_of(*key) -> threading.RLock:
    lock = _locks.get(key)
    return lock if lock is not None else _locks.setdefault(key, threading.RLock())


# One zero-filled workspace per device, grown on demand.  The library leaves its tile
# counters at zero after every call, so reuse on one stream needs no re-zeroing.
_workspaces: dict[int, torch.Tensor] = {}


def device_workspace(nbytes: int, device: torch.device) -> torch.Tensor | None:
    if nbytes == 0:
        return None
    idx = device.index if device.index is not None else torch.cuda.current_device()
    ws = _workspaces.get(idx)
    if ws is None or ws.numel() < nbytes:
        ws = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
        _workspaces[idx] = ws
    return ws


def _call_with_workspace(name, fn, workspace, need: int, stream, device: torch.device, *args) -> None:
    """fn(*args, workspace, its bytes, stream); without a workspace the device's own, under its lock."""
    if workspace is not None:
        _check(name, fn(*args, _ptr(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
        return
    if need == 0:
        _check(name, fn(*args, None, 0, _stream(stream)))
        return
    with _lock_of("device", device.index):
        ws = device_workspace(need, device)
        _check(name, fn(*args, _ptr(ws), ws.numel(), _stream(stream)))


def awq_workspace_bytes(op: int, M: int, K: int, N: int, split_k: int = 0) -> int:
    return int(lib.awq_workspace_bytes(op, M, K, N, split_k))


# Workspace sizes by (op, M, K, N, split_k, device): the size depends only on these (the plan reads
# the device's SM count), and a decode loop repeats the same few shapes.
_ws_need: dict[tuple, int] = {}


def _workspace_need(op: int, M: int, K: int, N: int, split_k: int, device: torch.device) -> int:
    key = (op, M, K, N, split_k, device.index)
    need = _ws_need.get(key)
    if need is None:
        need = _ws_need[key] = awq_workspace_bytes(op, M, K, N, split_k)
    return need


def _empty(shape, dtype: torch.dtype, device: torch.device, stream) -> torch.Tensor:
    """Memory for a result that is written on `stream` (None: the current one).  It is that stream's, so that nothing queued
    elsewhere still reads what the memory held before, and stays until the current stream, which will use it, is past it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def awq_pack(q: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    rows, n = q.shape
    if out is None:
        out = _empty((rows, n // 8), torch.int32, q.device, stream)
    _check("awq_pack", lib.awq_pack(_ptr(q), rows, n, _ptr(out), _stream(stream)))
    return out


def awq_unpack(packed: torch.Tensor, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    rows, nw = packed.shape
    if out is None:
        out = _empty((rows, nw * 8), torch.uint8, packed.device, stream)
    _check("awq_unpack", lib.awq_unpack(_ptr(packed), rows, nw * 8, _ptr(out), _stream(stream)))
    return out


ORDER_OLD, ORDER_NEW = 0, 1


def awq_pack_order(q: torch.Tensor, order: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    rows, n = q.shape
    if out is None:
        out = _empty((rows, n // 8), torch.int32, q.device, stream)
    _check("awq_pack_order", lib.awq_pack_order(_ptr(q), rows, n, order, _ptr(out), _stream(stream)))
    return out


def awq_unpack_order(packed: torch.Tensor, order: int, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    rows, nw = packed.shape
    if out is None:
        out = _empty((rows, nw * 8), torch.uint8, packed.device, stream)
    _check("awq_unpack_order", lib.awq_unpack_order(_ptr(packed), rows, nw * 8, order, _ptr(out), _stream(stream)))
    return out


def awq_dequant(qweight, qzeros, scales, group_size: int = GROUP_SIZE, out=None, stream=None) -> torch.Tensor:
    K, nw = qweight.shape
    if out is None:
        out = _empty((K, nw * 8), torch.float16, qweight.device, stream)
    _check("awq_dequant", lib.awq_dequant(_ptr(qweight), _ptr(qzeros), _ptr(scales), K, nw * 8, group_size,
                                          _ptr(out), _stream(stream)))
    return out


def _gemm_like(name, op, x, qweight, qzeros, scales, group_size, split_k, out, ws, stream):
    M, K = x.shape
    N = qweight.shape[1] * 8
    if out is None:
        out = _empty((M, N), x.dtype, x.device, stream)
    need = 0 if ws is not None else _workspace_need(op, M, K, N, split_k, x.device)
    _call_with_workspace(name, getattr(lib, name), ws, need, stream, x.device, _ptr(x), _ptr(qweight), _ptr(qzeros),
                         _ptr(scales), _ptr(out), M, K, N, group_size, split_k)
    return out


def awq_gemv(x, qweight, qzeros, scales, group_size: int = GROUP_SIZE, split_k: int = 0, out=None,
             workspace=None, stream=None) -> torch.Tensor:
    return _gemm_like("awq_gemv", OP_GEMV, x, qweight, qzeros, scales, group_size, split_k, out, workspace, stream)


def awq_gemv_noalloc(x, qweight, qzeros, scales, group_size: int = GROUP_SIZE, split_k: int = 0, out=None,
                     stream=None) -> torch.Tensor:
    """awq_gemv without a caller workspace: the library's fixed per-device scratch array is used.

    The output tensor is the only memory this wrapper allocates (pass `out` to allocate nothing).
    """
    M, K = x.shape
    N = qweight.shape[1] * 8
    if out is None:
        out = _empty((M, N), torch.float16, x.device, stream)
    _check("awq_gemv_noalloc", lib.awq_gemv_noalloc(_ptr(x), _ptr(qweight), _ptr(qzeros), _ptr(scales), _ptr(out),
                                                    M, K, N, group_size, split_k, _stream(stream)))
    return out


class Prepacked:
    """A prepared decode copy of an AWQ layer (awq_prepack_gemv): the device bytes and the shape."""

    def __init__(self, data: torch.Tensor, K: int, N: int):
        self.data, self.K, self.N = data, K, N


def awq_prepack_gemv(qweight, qzeros, scales, group_size: int = GROUP_SIZE, stream=None) -> Prepacked:
    K, nw = qweight.shape
    N = nw * 8
    nbytes = int(lib.awq_prepacked_bytes(K, N))
    if nbytes == 0:
        raise AwqError("awq_prepack_gemv", -1)
    data = _empty(nbytes, torch.uint8, qweight.device, stream)
    _check("awq_prepack_gemv", lib.awq_prepack_gemv(_ptr(qweight), _ptr(qzeros), _ptr(scales), K, N, group_size,
                                                    _ptr(data), nbytes, _stream(stream)))
    return Prepacked(data, K, N)


def awq_unprepack_gemv(packed: Prepacked, with_zeros: bool = True, stream=None):
    """The AWQ (qweight, qzeros or None, scales) that `packed` was made from."""
    K, N = packed.K, packed.N
    dev = packed.data.device
    qweight = _empty((K, N // 8), torch.int32, dev, stream)
    qzeros = _empty((K // GROUP_SIZE, N // 8), torch.int32, dev, stream) if with_zeros else None
    scales = _empty((K // GROUP_SIZE, N), torch.float16, dev, stream)
    _check("awq_unprepack_gemv", lib.awq_unprepack_gemv(_ptr(packed.data), K, N, _ptr(qweight), _ptr(qzeros),
                                                        _ptr(scales), _stream(stream)))
    return qweight, qzeros, scales


def awq_gemv_prepacked(x, packed: Prepacked, split_k: int = 0, out=None, workspace=None, stream=None):
    M, K = x.shape
    N = packed.N
    if K != packed.K:
        raise ValueError("x has K columns different from the prepared layer's")
    if out is None:
        out = _empty((M, N), torch.float16, x.device, stream)
    need = 0 if workspace is not None else _workspace_need(OP_GEMV_PREPACKED, M, K, N, split_k, x.device)
    _call_with_workspace("awq_gemv_prepacked", lib.awq_gemv_prepacked, workspace, need, stream, x.device, _ptr(x),
                         _ptr(packed.data), _ptr(out), M, K, N, split_k)
    return out


def awq_gemm(x, qweight, qzeros, scales, group_size: int = GROUP_SIZE, split_k: int = 0, out=None,
             workspace=None, stream=None) -> torch.Tensor:
    return _gemm_like("awq_gemm", OP_GEMM, x, qweight, qzeros, scales, group_size, split_k, out, workspace, stream)


def _need_bf16(*tensors):
    for t in tensors:
        if t is not None and t.dtype != torch.bfloat16:
            raise TypeError("the bf16 entry points take bf16 activations and scales")


def awq_dequant_bf16(qweight, qzeros, scales, group_size: int = GROUP_SIZE, out=None, stream=None):
    _need_bf16(scales)
    K, nw = qweight.shape
    if out is None:
        out = _empty((K, nw * 8), torch.bfloat16, qweight.device, stream)
    _check("awq_dequant_bf16", lib.awq_dequant_bf16(_ptr(qweight), _ptr(qzeros), _ptr(scales), K, nw * 8,
                                                    group_size, _ptr(out), _stream(stream)))
    return out


def awq_gemv_bf16(x, qweight, qzeros, scales, group_size: int = GROUP_SIZE, split_k: int = 0, out=None,
                  workspace=None, stream=None) -> torch.Tensor:
    _need_bf16(x, scales)
    return _gemm_like("awq_gemv_bf16", OP_GEMV_BF16, x, qweight, qzeros, scales, group_size, split_k, out,
                      workspace, stream)


def awq_gemm_bf16(x, qweight, qzeros, scales, group_size: int = GROUP_SIZE, split_k: int = 0, out=None,
                  workspace=None, stream=None) -> torch.Tensor:
    _need_bf16(x, scales)
    return _gemm_like("awq_gemm_bf16", OP_GEMM_BF16, x, qweight, qzeros, scales, group_size, split_k, out,
                      workspace, stream)


GEMV_MAX_M = 16


def awq_linear(x, qweight, qzeros, scales, group_size: int = GROUP_SIZE, **kw) -> torch.Tensor:
    """The pages' dispatch by token count, with the threshold moved from 8 to 16: the GEMV kernel
    streams the weights once for up to 16 tokens (two 8-token halves) and was measured 1.3-2.9x
    faster than the tensor-core GEMM at 16 tokens; the GEMM above."""
    fn = awq_gemv if x.shape[0] <= GEMV_MAX_M else awq_gemm
    return fn(x, qweight, qzeros, scales, group_size, **kw)


def w4a8_quant_act(x, xq=None, s_tok=None, stream=None):
    M, K = x.shape
    if xq is None:
        xq = _empty((M, K), torch.int8, x.device, stream)
    if s_tok is None:
        s_tok = _empty((M,), torch.float32, x.device, stream)
    _check("w4a8_quant_act", lib.w4a8_quant_act(_ptr(x), _ptr(xq), _ptr(s_tok), M, K, _stream(stream)))
    return xq, s_tok


def w4a8_gemm(xq, s_tok, wq, s_ch, split_k: int = 0, out=None, acc_out=None, workspace=None, stream=None):
    M, K = xq.shape
    N = wq.shape[1] * 8
    if out is None:
        out = _empty((M, N), torch.float16, xq.device, stream)
    need = awq_workspace_bytes(OP_W4A8_GEMM, M, K, N, split_k)
    _call_with_workspace("w4a8_gemm", lib.w4a8_gemm, workspace, need, stream, xq.device, _ptr(xq), _ptr(s_tok),
                         _ptr(wq), _ptr(s_ch), _ptr(out), _ptr(acc_out), M, K, N, split_k)
    return out


def w4a8_linear(x, wq, s_ch, split_k: int = 0, out=None, acc_out=None, xq_out=None, s_tok=None, workspace=None,
                stream=None):
    """W4A8 from fp16 activations in one call (quantization fused); returns (y, s_tok)."""
    M, K = x.shape
    N = wq.shape[1] * 8
    if out is None:
        out = _empty((M, N), torch.float16, x.device, stream)
    if s_tok is None:
        s_tok = _empty((M,), torch.float32, x.device, stream)
    need = awq_workspace_bytes(OP_W4A8_GEMM, M, K, N, split_k)
    _call_with_workspace("w4a8_linear", lib.w4a8_linear, workspace, need, stream, x.device, _ptr(x), _ptr(wq),
                         _ptr(s_ch), _ptr(out), _ptr(acc_out), _ptr(xq_out), _ptr(s_tok), M, K, N, split_k)
    return out, s_tok


def w4a8_gemm_grouped(xq, s_tok, wq, s3, s2, split_k: int = 0, out=None, acc_out=None, workspace=None,
                      stream=None):
    """Per-group W4A8 from int8 codes (s3: integer group factors 1..16, s2: channel scales)."""
    M, K = xq.shape
    N = wq.shape[1] * 8
    if out is None:
        out = _empty((M, N), torch.float16, xq.device, stream)
    need = awq_workspace_bytes(OP_W4A8_GROUPED, M, K, N, split_k)
    _call_with_workspace("w4a8_gemm_grouped", lib.w4a8_gemm_grouped, workspace, need, stream, xq.device, _ptr(xq),
                         _ptr(s_tok), _ptr(wq), _ptr(s3), _ptr(s2), _ptr(out), _ptr(acc_out), M, K, N, GROUP_SIZE, split_k)
    return out


def w4a8_linear_grouped(x, wq, s3, s2, split_k: int = 0, out=None, acc_out=None, xq_out=None, s_tok=None,
                        workspace=None, stream=None):
    """Per-group W4A8 from fp16 activations in one call (quantization included); returns (y, s_tok)."""
    M, K = x.shape
    N = wq.shape[1] * 8
    if out is None:
        out = _empty((M, N), torch.float16, x.device, stream)
    if s_tok is None:
        s_tok = _empty((M,), torch.float32, x.device, stream)
    need = awq_workspace_bytes(OP_W4A8_GROUPED, M, K, N, split_k)
    _call_with_workspace("w4a8_linear_grouped", lib.w4a8_linear_grouped, workspace, need, stream, x.device, _ptr(x),
                         _ptr(wq), _ptr(s3), _ptr(s2), _ptr(out), _ptr(acc_out), _ptr(xq_out), _ptr(s_tok), M, K, N, GROUP_SIZE,
                         split_k)
    return out, s_tok


# ---- the operators between the linear layers of a decoder block

_DTYPES = {torch.float16: FP16, torch.bfloat16: BF16}


def _dtype16(name: str, first, *others) -> int:
    """The awq_dtype that all given tensors share; they are on a GPU."""
    dtype = first.dtype
    kind = _DTYPES.get(dtype)
    if kind is None or not first.is_cuda:
        raise TypeError(f"{name} takes fp16 or bf16 operands of one type on a GPU")
    for t in others:
        if t is not None and (t.dtype is not dtype or not t.is_cuda):
            raise TypeError(f"{name} takes fp16 or bf16 operands of one type on a GPU")
    return kind


def _raw_stream(stream, device: torch.device) -> int:
    """The handle of `stream`, or of the device's current stream (without building a Stream object)."""
    return torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream


_current_device = torch._C._cuda_getDevice


def _on_current_gpu(name: str, *tensors) -> None:
    """The library launches on the current device: all tensors, the caller's workspace among them, are there."""
    here = _current_device()
    for t in tensors:
        if t is not None and t.get_device() != here:
            raise ValueError(f"{name}: every tensor is on the current GPU (device {here})")


def _need(name: str, dtype, *tensors) -> None:
    for t in tensors:
        if t is not None and (t.dtype is not dtype or not t.is_cuda or not t.is_contiguous()):
            raise TypeError(f"{name}: expected a contiguous {dtype} tensor on a GPU")


def _row_stride(name: str, t, inner: int) -> int:
    """Elements from one row (token) to the next; the `inner` elements of a row are dense."""
    if t.is_contiguous():
        return inner
    shape, strides = t.shape, t.stride()
    if strides[-1] != 1 or (len(shape) == 3 and strides[1] != shape[2]):  # else dense, as it mostly is
        dense = 1
        for size, stride in zip(reversed(shape[1:]), reversed(strides[1:])):
            if size != 1 and stride != dense:
                raise ValueError(f"{name}: heads and channels of a token must be dense")
            dense *= size
    return max(strides[0], inner) if shape[0] <= 1 else strides[0]


def _rmsnorm_args(name, x, weight, residual, res_out, stream):
    M, K = x.shape
    dtype = _dtype16(name, x, weight, residual, res_out)
    if weight.shape != (K,) or (residual is not None and residual.shape != x.shape) or \
            (res_out is not None and res_out.shape != x.shape):
        raise ValueError(f"{name}: weight [K], residual and res_out [M, K] go with x [M, K]")
    _need(name, x.dtype, weight, res_out)
    if residual is None:
        rs = 0
    else:
        rs = _row_stride(name, residual, K)
        if res_out is None:
            res_out = _empty((M, K), x.dtype, x.device, stream)
    return M, K, dtype, res_out, _row_stride(name, x, K), rs


def w4a8_rmsnorm_quant(x, weight, residual=None, eps: float = 1e-6, res_out=None, y=None, xq=None, s_tok=None,
                       stream=None):
    """Residual addition, RMS norm and int8 codes of x [M, K]: (xq, s_tok, res_out), the first two as
    w4a8_gemm takes them; res_out (x + residual) is None without a residual.  `y`, when given, receives the
    normalized rows too.  res_out may be `x` or `residual` itself."""
    M, K, dtype, res_out, xs, rs = _rmsnorm_args("w4a8_rmsnorm_quant", x, weight, residual, res_out, stream)
    device = x.device
    if xq is not None or s_tok is not None or y is not None:
        _need("w4a8_rmsnorm_quant", torch.int8, xq)
        _need("w4a8_rmsnorm_quant", torch.float32, s_tok)
        _need("w4a8_rmsnorm_quant", x.dtype, y)
        if (xq is not None and xq.shape != (M, K)) or (s_tok is not None and s_tok.shape != (M,)) or \
                (y is not None and y.shape != (M, K)):
            raise ValueError("w4a8_rmsnorm_quant: xq and y are [M, K], s_tok is [M]")
    _on_current_gpu("w4a8_rmsnorm_quant", x, weight, residual, res_out, y, xq, s_tok)
    if xq is None:
        xq = _empty((M, K), torch.int8, device, stream)
    if s_tok is None:
        s_tok = _empty(M, torch.float32, device, stream)
    _check("w4a8_rmsnorm_quant", lib.w4a8_rmsnorm_quant(_ptr(x), _ptr(residual), _ptr(weight), _ptr(res_out), _ptr(y),
                                                        xq.data_ptr(), s_tok.data_ptr(), M, K, xs, rs, eps, dtype,
                                                        _raw_stream(stream, device)))
    return xq, s_tok, res_out


def awq_rmsnorm(x, weight, residual=None, eps: float = 1e-6, res_out=None, out=None, stream=None):
    """Residual addition and RMS norm of x [M, K] in its own type: (y, res_out), for the W4A16 layers."""
    M, K, dtype, res_out, xs, rs = _rmsnorm_args("awq_rmsnorm", x, weight, residual, res_out, stream)
    if out is None:
        out = _empty((M, K), x.dtype, x.device, stream)
    else:
        _need("awq_rmsnorm", x.dtype, out)
        if out.shape != (M, K):
            raise ValueError("awq_rmsnorm: out is [M, K]")
    _on_current_gpu("awq_rmsnorm", x, weight, residual, res_out, out)
    _check("awq_rmsnorm", lib.awq_rmsnorm(_ptr(x), _ptr(residual), _ptr(weight), _ptr(res_out), _ptr(out), M, K, xs,
                                          rs, eps, dtype, _raw_stream(stream, x.device)))
    return out, res_out


KV4_UNIT = 16  # tokens of a cache unit


def kv4_cache(num_pages: int, kv_heads: int, head_dim: int, page_size: int = 64, device="cuda") -> torch.Tensor:
    """A zeroed 4-bit cache of one layer: uint8 [num_pages, kv_heads, page_size / 16, 16 * head_dim + 128]
    (units as include/awq.h lays them out).  The kv4_* calls read their sizes from this shape."""
    if num_pages < 1 or lib.kv4_cache_bytes(num_pages, kv_heads, head_dim, page_size) == 0:
        raise AwqError("kv4_cache", -1)
    return torch.zeros((num_pages, kv_heads, page_size // KV4_UNIT, KV4_UNIT * head_dim + 128), dtype=torch.uint8,
                       device=device)


def _kv4_shape(name, cache):
    """(num_pages, kv_heads, head_dim, page_size) of a cache tensor."""
    shape = cache.shape
    if cache.dtype is not torch.uint8 or len(shape) != 4 or not cache.is_cuda or not cache.is_contiguous():
        raise TypeError(f"{name}: the cache is a contiguous uint8 tensor [pages, kv_heads, page_size / 16, unit] on a GPU")
    pages, kv_heads, units, unit = shape
    return pages, kv_heads, (unit - 128) // KV4_UNIT if unit % KV4_UNIT == 0 else 0, units * KV4_UNIT


def kv4_append(cache, k, v, positions, slots, table, q=None, interleaved: bool = False, q_out=None, stream=None):
    """Rotates q and k (table fp32 [max_pos, rot_dim]: cosines, then sines; None for no rotation) and writes k
    and v [T, kv_heads, D], quantized, to `slots` of the cache.  Returns the rotated queries (None without q)."""
    pages, kv_heads, dim, page = _kv4_shape("kv4_append", cache)
    dtype = _dtype16("kv4_append", k, v, q, q_out)
    T = k.shape[0]
    if k.shape != (T, kv_heads, dim) or v.shape != k.shape or slots.shape != (T,):
        raise ValueError("kv4_append: k, v [T, kv_heads, head_dim] and slots [T] go with the cache")
    _need("kv4_append", torch.int64, slots)
    heads, rot, max_pos, qs, qos = 0, 0, 0, 0, 0
    if q is not None:
        heads = q.shape[1]
        if q.shape != (T, heads, dim):
            raise ValueError("kv4_append: q is [T, heads, head_dim]")
        if q_out is None:
            q_out = _empty((T, heads, dim), q.dtype, q.device, stream)
        elif q_out.shape != q.shape:
            raise ValueError("kv4_append: q_out has another shape than q")
        inner = heads * dim
        qs, qos = _row_stride("kv4_append", q, inner), _row_stride("kv4_append", q_out, inner)
    if table is not None:
        max_pos, rot = table.shape
        _need("kv4_append", torch.float32, table)
        _need("kv4_append", torch.int32, positions)
        if positions is None or positions.shape != (T,):
            raise ValueError("kv4_append: positions is [T]")
        _on_current_gpu("kv4_append", positions, table)
    _on_current_gpu("kv4_append", cache, k, v, slots, q, q_out)
    _check("kv4_append", lib.kv4_append(
        _ptr(q), _ptr(k), _ptr(v), qs, _row_stride("kv4_append", k, kv_heads * dim),
        _row_stride("kv4_append", v, kv_heads * dim), _ptr(positions),
        _ptr(slots), _ptr(table), max_pos, rot, int(interleaved), _ptr(q_out), qos, _ptr(cache), pages, T, heads,
        kv_heads, dim, page, dtype, _raw_stream(stream, cache.device)))
    return q_out


def kv4_gather(cache, slots, dtype=torch.float16, k=None, v=None, stream=None):
    """The keys and values [T, kv_heads, head_dim] that the cache holds at `slots`."""
    pages, kv_heads, dim, page = _kv4_shape("kv4_gather", cache)
    shape = (slots.shape[0], kv_heads, dim)
    device = cache.device
    _need("kv4_gather", torch.int64, slots)
    given = k is not None or v is not None
    if k is None:
        k = _empty(shape, dtype, device, stream)
    if v is None:
        v = _empty(shape, dtype, device, stream)
    kind = _dtype16("kv4_gather", k, v)
    if given:
        _need("kv4_gather", k.dtype, k, v)
        if k.shape != shape or v.shape != shape:
            raise ValueError("kv4_gather: k and v are [T, kv_heads, head_dim]")
    _on_current_gpu("kv4_gather", cache, slots, k, v)
    _check("kv4_gather", lib.kv4_gather(cache.data_ptr(), slots.data_ptr(), k.data_ptr(), v.data_ptr(), pages, shape[0],
                                        kv_heads, dim, page, kind, _raw_stream(stream, device)))
    return k, v


def kv4_attention_workspace_bytes(T: int, B: int, max_q: int, heads: int, kv_heads: int, head_dim: int) -> int:
    """Bytes of a kv4_attention workspace on the current device."""
    return int(lib.kv4_attention_workspace_bytes(T, B, max_q, heads, kv_heads, head_dim))


@functools.lru_cache(maxsize=4096)
def _kv4_workspace_need(device: int, *shape) -> int:
    return kv4_attention_workspace_bytes(*shape)  # by the device's SM count


# One workspace of kv4_attention for each device and stream (calls on one stream may share it, under its lock), grown on
# demand, by half at least.  Outgrown ones stay.  A captured call never takes it: its graph may run on any stream, beside this
# one's calls or another graph that holds the same, and a workspace made in the capture would be the graph's memory.
_kv4_workspaces: dict[tuple, torch.Tensor] = {}
_kv4_outgrown: list[torch.Tensor] = []


class _Thread(threading.local):
    """A number for each thread.  That of one that has ended, whose stream may still be busy, is not given out again."""

    numbers = itertools.count()

    def __init__(self):
        self.number = next(_Thread.numbers)


_thread = _Thread()


def _stream_key(device: torch.device, handle: int) -> tuple:
    """What the calls that share a workspace have in common.  Handle 2 is each thread's own default stream."""
    return (device.index, handle) if handle != 2 else (device.index, handle, _thread.number)


def _call_on_stream(name, fn, workspace, shared, device: torch.device, handle: int, *args) -> None:
    """fn(*args, workspace, its bytes, handle); without a workspace the stream's own, shared(), under its lock."""
    if workspace is not None:
        _check(name, fn(*args, workspace.data_ptr(), workspace.numel() * workspace.element_size(), handle))
        return
    with _lock_of(*_stream_key(device, handle)):
        ws = shared()
        _check(name, fn(*args, ws.data_ptr(), ws.numel(), handle))


def _stream_workspace(pool: dict, name: str, handle: int, device: torch.device, nbytes: int, stream) -> torch.Tensor:
    """The workspace that `pool` has for the stream, made or grown where it is too small."""
    if stream is None:
        capturing = torch.cuda.is_current_stream_capturing()
    else:
        with torch.cuda.stream(stream):
            capturing = torch.cuda.is_current_stream_capturing()
    if capturing:
        raise RuntimeError(f"{name}: a captured call takes a workspace of its own")
    key = _stream_key(device, handle)
    ws = pool.get(key)
    if ws is None or ws.numel() < nbytes:
        with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream(device)):
            if ws is not None:
                nbytes = max(nbytes, ws.numel() + ws.numel() // 2)
            ws = pool[key] = torch.zeros(max(nbytes, 1 << 20), dtype=torch.uint8, device=device)
    return ws


def _kv4_workspace(handle: int, device: torch.device, nbytes: int, stream) -> torch.Tensor:
    before = _kv4_workspaces.get(_stream_key(device, handle))
    ws = _stream_workspace(_kv4_workspaces, "kv4_attention", handle, device, nbytes, stream)
    if before is not None and ws is not before:
        _kv4_outgrown.append(before)
    return ws


def kv4_attention(q, cache, block_table, kv_len, q_start=None, max_q: int | None = None, scale: float | None = None,
                  window: int = 0, out=None, lse=None, workspace=None, stream=None):
    """Causal attention of q [T, heads, D] over the cached tokens of each sequence.

    block_table int32 [B, max_pages], kv_len int32 [B] (new tokens included).  Without q_start every sequence
    has one query (T = B); with q_start int32 [B + 1] sequence b has the queries q_start[b] .. q_start[b + 1] - 1,
    at most max_q (T by default; a smaller one saves work), which are its last tokens.  scale: 1 / sqrt(D) by
    default; window: 0 or the number of keys a query looks back over, its own included.  `lse` fp32 [T, heads], when
    given, receives the log-sum-exp.
    Without `workspace` the calls of a stream share one that grows; a call to be captured in a graph needs one of
    its own (kv4_attention_workspace_bytes, zeroed once) and is refused without.  After awq_last_device_error reports a wait
    that expired, a workspace of one's own is zeroed again before its next use, as include/awq.h says of all of them.
    """
    pages, kv_heads, dim, page = _kv4_shape("kv4_attention", cache)
    shape = q.shape
    T, heads, qd = shape
    B, max_pages = block_table.shape
    dtype = _dtype16("kv4_attention", q, out)
    if qd != dim or kv_len.shape != (B,) or (q_start is not None and q_start.shape != (B + 1,)):
        raise ValueError("kv4_attention: q [T, heads, head_dim], kv_len [B] and q_start [B + 1] go with the cache and "
                         "block_table [B, pages]")
    _need("kv4_attention", torch.int32, kv_len, q_start)
    table_stride, inner = block_table.stride()
    if block_table.dtype is not torch.int32 or not block_table.is_cuda or (inner != 1 and max_pages > 1):
        raise TypeError("kv4_attention: block_table is int32 with dense rows, on a GPU")
    if B <= 1:  # no second row: the stride says nothing
        table_stride = max_pages
    elif table_stride < max_pages:
        raise ValueError("kv4_attention: the rows of block_table overlap (a table made with expand needs a copy)")
    if out is None:
        out = _empty(shape, q.dtype, q.device, stream)
    elif out.shape != shape or not out.is_contiguous():
        raise ValueError("kv4_attention: out is dense and has q's shape")
    if lse is not None:
        _need("kv4_attention", torch.float32, lse)
        if lse.shape != (T, heads):
            raise ValueError("kv4_attention: lse is [T, heads]")
    if scale is None:
        scale = dim ** -0.5
    if max_q is None:
        max_q = 1 if q_start is None else max(T, 1)
    _on_current_gpu("kv4_attention", q, cache, block_table, kv_len, q_start, out, lse, workspace)
    device = q.device
    handle = _raw_stream(stream, device)

    def shared():
        return _kv4_workspace(handle, device, _kv4_workspace_need(device.index, T, B, max_q, heads, kv_heads, dim), stream)

    _call_on_stream(
        "kv4_attention", lib.kv4_attention, workspace, shared, device, handle,
        q.data_ptr(), _row_stride("kv4_attention", q, heads * dim), cache.data_ptr(), block_table.data_ptr(),
        table_stride, kv_len.data_ptr(), _ptr(q_start), out.data_ptr(),
        _ptr(lse), T, B, max_q, heads, kv_heads, dim, pages, page, max_pages, scale, window, dtype)
    return out


# ---- the feed-forward layer with experts, fp8 linear layers

# Workspaces of the grouped product and the fp8 layers: one for each device and stream, under its lock, as for kv4_attention.
# An outgrown one goes back to its stream, whose calls alone have used it (a long prompt's are some hundred megabytes).
_layer_workspaces: dict[tuple, torch.Tensor] = {}


def _layer_workspace(name: str, handle: int, device: torch.device, nbytes: int, stream) -> torch.Tensor:
    return _stream_workspace(_layer_workspaces, name, handle, device, nbytes, stream)


@functools.lru_cache(maxsize=4096)
def _layer_workspace_need(device: int, query: str, *shape) -> int:
    return int(getattr(lib, query)(*shape))  # by the device's SM count


def _layer_share(name: str, handle: int, device: torch.device, stream, *shape):
    """The stream's workspace for a call of this shape, for _call_on_stream."""
    return lambda: _layer_workspace(name, handle, device, _layer_workspace_need(device.index, name + "_workspace_bytes", *shape),
                                    stream)


class MoePlan:
    """Rows of a layer with experts in the experts' order (awq_moe_plan): `offsets` int32 [experts + 1], `order` int32
    [R], `place` int32 [R], with R = tokens * top_k; the tensors that include/awq.h describes."""

    def __init__(self, offsets: torch.Tensor, order: torch.Tensor, place: torch.Tensor, top_k: int):
        for t in (offsets, order, place):
            if t.dtype is not torch.int32 or t.dim() != 1 or not t.is_contiguous():
                raise TypeError("MoePlan: offsets, order and place are dense vectors of int32")
        if offsets.shape[0] < 2 or place.shape != order.shape or top_k < 1 or order.shape[0] % top_k:
            raise ValueError("MoePlan: offsets [experts + 1], order and place [tokens * top_k]")
        self.offsets, self.order, self.place, self.top_k = offsets, order, place, top_k

    @classmethod
    def _of(cls, offsets, order, place, top_k) -> "MoePlan":
        """From tensors made here, which need no checks."""
        plan = cls.__new__(cls)
        plan.offsets, plan.order, plan.place, plan.top_k = offsets, order, place, top_k
        return plan

    @property
    def rows(self) -> int:
        return self.order.shape[0]

    @property
    def experts(self) -> int:
        return self.offsets.shape[0] - 1


def _plan_tensors(experts: int, rows: int, device, stream):
    # allocations of their own: parts of one cost the host more (a router's call 21 us against 15)
    return (_empty(experts + 1, torch.int32, device, stream), _empty(rows, torch.int32, device, stream),
            _empty(rows, torch.int32, device, stream))


def awq_moe_plan(ids: torch.Tensor, experts: int, stream=None) -> MoePlan:
    """The plan of a router of one's own: ids int32 [T, top_k], each in [0, experts) or a choice without a row."""
    if ids.dim() != 2:
        raise ValueError("awq_moe_plan: ids is [T, top_k]")
    _need("awq_moe_plan", torch.int32, ids)
    _on_current_gpu("awq_moe_plan", ids)
    T, top_k = ids.shape
    rows, device = T * top_k, ids.device
    if experts < 1:
        raise AwqError("awq_moe_plan", -1)
    offsets, order, place = _plan_tensors(experts, rows, device, stream)
    _check("awq_moe_plan", lib.awq_moe_plan(ids.data_ptr(), rows, experts, offsets.data_ptr(), order.data_ptr(), place.data_ptr(),
                                            _raw_stream(stream, device)))
    return MoePlan._of(offsets, order, place, top_k)


_LOGITS = {torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}


def awq_moe_route(logits: torch.Tensor, top_k: int, normalize: bool = True, stream=None):
    """Softmax and top_k of a router's logits [T, experts] (fp16, bf16 or fp32): (weights fp32 [T, top_k], ids int32
    [T, top_k], their MoePlan).  normalize: a token's weights sum to 1."""
    T, experts = logits.shape
    kind = _LOGITS.get(logits.dtype)
    if kind is None or not logits.is_cuda:
        raise TypeError("awq_moe_route takes fp16, bf16 or fp32 logits on a GPU")
    _on_current_gpu("awq_moe_route", logits)
    device = logits.device
    if not 1 <= top_k <= experts:
        raise AwqError("awq_moe_route", -1)
    rows = T * top_k
    weights = _empty((T, top_k), torch.float32, device, stream)
    ids = _empty((T, top_k), torch.int32, device, stream)
    offsets, order, place = _plan_tensors(experts, rows, device, stream)
    _check("awq_moe_route", lib.awq_moe_route(
        logits.data_ptr(), _row_stride("awq_moe_route", logits, experts), T, experts, top_k, int(normalize), kind, ids.data_ptr(),
        weights.data_ptr(), offsets.data_ptr(), order.data_ptr(), place.data_ptr(), _raw_stream(stream, device)))
    return weights, ids, MoePlan._of(offsets, order, place, top_k)


class MoeWeights:
    """Prepared weights of a layer's experts (awq_moe_prepack): the device bytes, the sizes and the scales' type."""

    def __init__(self, data: torch.Tensor, experts: int, K: int, N: int, gated: bool, dtype: torch.dtype):
        if data.dtype is not torch.uint8 or dtype not in _DTYPES or not data.is_contiguous():
            raise TypeError("MoeWeights: dense uint8 bytes, scales of fp16 or bf16")
        if data.numel() == 0 or data.numel() != lib.awq_moe_prepacked_bytes(experts, K, N, int(gated)):
            raise ValueError("MoeWeights: the bytes are not those of a prepared layer of this size")
        self.data, self.experts, self.K, self.N, self.gated, self.dtype = data, experts, K, N, gated, dtype

    @property
    def outputs(self) -> int:
        """Columns that awq_moe_gemm writes."""
        return self.N // 2 if self.gated else self.N


def awq_moe_prepack(qweight, qzeros, scales, gated: bool = False, group_size: int = GROUP_SIZE, stream=None) -> MoeWeights:
    """Lays the experts' AWQ weights out for awq_moe_gemm: qweight int32 [experts, K, N/8], qzeros int32 [experts,
    K/128, N/8] or None (symmetric), scales fp16 or bf16 [experts, K/128, N].  gated: the columns are gate's, then
    up's, and the product gives silu(gate) * up.  The originals are not needed afterwards (awq_moe_unprepack)."""
    experts, K, nw = qweight.shape
    N = nw * 8
    _dtype16("awq_moe_prepack", scales)
    _need("awq_moe_prepack", torch.int32, qweight, qzeros)
    _need("awq_moe_prepack", scales.dtype, scales)
    if scales.shape != (experts, K // GROUP_SIZE, N) or (qzeros is not None and qzeros.shape != (experts, K // GROUP_SIZE, nw)):
        raise ValueError("awq_moe_prepack: scales [experts, K / 128, N], qzeros [experts, K / 128, N / 8]")
    _on_current_gpu("awq_moe_prepack", qweight, qzeros, scales)
    nbytes = int(lib.awq_moe_prepacked_bytes(experts, K, N, int(gated)))
    if nbytes == 0:
        raise AwqError("awq_moe_prepack", -1)
    data = _empty(nbytes, torch.uint8, qweight.device, stream)
    _check("awq_moe_prepack", lib.awq_moe_prepack(_ptr(qweight), _ptr(qzeros), _ptr(scales), experts, K, N, group_size,
                                                  int(gated), _ptr(data), nbytes, _raw_stream(stream, qweight.device)))
    return MoeWeights(data, experts, K, N, bool(gated), scales.dtype)


def awq_moe_unprepack(weights: MoeWeights, with_zeros: bool = True, stream=None):
    """The AWQ (qweight, qzeros or None, scales) that `weights` was made from."""
    w, dev = weights, weights.data.device
    _on_current_gpu("awq_moe_unprepack", w.data)
    qweight = _empty((w.experts, w.K, w.N // 8), torch.int32, dev, stream)
    qzeros = _empty((w.experts, w.K // GROUP_SIZE, w.N // 8), torch.int32, dev, stream) if with_zeros else None
    scales = _empty((w.experts, w.K // GROUP_SIZE, w.N), w.dtype, dev, stream)
    _check("awq_moe_unprepack", lib.awq_moe_unprepack(_ptr(w.data), w.experts, w.K, w.N, int(w.gated), _ptr(qweight),
                                                      _ptr(qzeros), _ptr(scales), _raw_stream(stream, dev)))
    return qweight, qzeros, scales


def awq_moe_gemm_workspace_bytes(rows: int, weights: MoeWeights) -> int:
    """Bytes of an awq_moe_gemm workspace on the current device."""
    return int(lib.awq_moe_gemm_workspace_bytes(rows, weights.experts, weights.K, weights.N, int(weights.gated)))


def awq_moe_gemm(x, weights: MoeWeights, plan: MoePlan, gather: bool = False, out_dtype=None, out=None, workspace=None,
                 stream=None):
    """Every expert's rows times its weights: [plan.rows, weights.outputs] in x's type, or fp32 with out_dtype (or `out`) so.
    x holds the rows in the plan's order, or with `gather` the tokens that the plan was made for.  Rows that no expert
    has are not written.  Workspaces as for kv4_attention: the calls of a stream share one, from any thread, a captured call
    takes one of its own (awq_moe_gemm_workspace_bytes, zeroed once); a workspace that is passed serves one call at a time."""
    rows, K = plan.rows, weights.K
    dtype = _dtype16("awq_moe_gemm", x)
    if out_dtype is None:
        out_dtype = x.dtype if out is None else out.dtype
    if (out_dtype is not x.dtype and out_dtype is not torch.float32) or (out is not None and out.dtype is not out_dtype):
        raise TypeError("awq_moe_gemm: the output has x's type or is fp32")
    if x.dtype is not weights.dtype:
        raise TypeError("awq_moe_gemm: x and the weights' scales have one type")
    if x.dim() != 2 or x.shape[1] != K or plan.experts != weights.experts or \
            x.shape[0] * (plan.top_k if gather else 1) != rows:
        raise ValueError("awq_moe_gemm: x is [rows, K] ([tokens, K] with gather), plan and weights have the same experts")
    device = x.device
    if out is None:
        out = _empty((rows, weights.outputs), out_dtype, device, stream)
    elif out.shape != (rows, weights.outputs) or not out.is_contiguous():
        raise ValueError("awq_moe_gemm: out is dense, [rows, outputs]")
    _on_current_gpu("awq_moe_gemm", x, weights.data, plan.offsets, plan.order, out, workspace)
    handle = _raw_stream(stream, device)
    _call_on_stream(
        "awq_moe_gemm", lib.awq_moe_gemm, workspace,
        _layer_share("awq_moe_gemm", handle, device, stream, rows, weights.experts, K, weights.N, int(weights.gated)), device, handle,
        x.data_ptr(), _row_stride("awq_moe_gemm", x, K), x.shape[0], weights.data.data_ptr(), plan.offsets.data_ptr(),
        plan.order.data_ptr() if gather else None, plan.top_k, out.data_ptr(), int(out_dtype is torch.float32), rows,
        weights.experts, K, weights.N, int(weights.gated), dtype)
    return out


def awq_moe_combine(y, plan: MoePlan, weights, residual=None, dtype=None, out=None, stream=None):
    """Each token's rows of y [plan.rows, H], weighted (weights fp32 [T, top_k]) and added up, to `residual` [T, H] where
    one is given: [T, H] in `dtype`, that of out, residual or y by default (y may be fp32).  out may be residual itself."""
    T, top_k = weights.shape
    H = y.shape[1]
    if dtype is None:
        dtype = (out if out is not None else residual if residual is not None else y).dtype
    kind = _DTYPES.get(dtype)
    if kind is None or y.dtype not in (dtype, torch.float32) or (residual is not None and (residual.dtype is not dtype or not residual.is_cuda)):
        raise TypeError("awq_moe_combine: residual and output are fp16 or bf16, y is of their type or fp32, on a GPU")
    _need("awq_moe_combine", y.dtype, y)
    _need("awq_moe_combine", dtype, out)
    _need("awq_moe_combine", torch.float32, weights)
    if y.shape != (plan.rows, H) or top_k != plan.top_k or T * top_k != plan.rows or \
            (residual is not None and residual.shape != (T, H)) or (out is not None and out.shape != (T, H)):
        raise ValueError("awq_moe_combine: y [rows, H], weights [T, top_k], residual and out [T, H] go with the plan")
    _on_current_gpu("awq_moe_combine", y, plan.place, weights, residual, out)
    if out is None:
        out = _empty((T, H), dtype, y.device, stream)
    rs = 0 if residual is None else _row_stride("awq_moe_combine", residual, H)
    _check("awq_moe_combine", lib.awq_moe_combine(y.data_ptr(), int(y.dtype is torch.float32), plan.place.data_ptr(), weights.data_ptr(),
                                                  _ptr(residual), rs, out.data_ptr(), T, top_k, H, plan.rows, kind,
                                                  _raw_stream(stream, y.device)))
    return out


def awq_moe_workspace_bytes(tokens: int, top_k: int, up: MoeWeights, down: MoeWeights) -> int:
    """Bytes of an awq_moe workspace on the current device."""
    return int(lib.awq_moe_workspace_bytes(tokens, top_k, up.experts, up.K, down.K, down.N))


def awq_moe(x, up: MoeWeights, down: MoeWeights, weights, plan: MoePlan, residual=None, out=None, workspace=None, stream=None):
    """A sparse feed-forward layer: x [T, K] through every token's experts, down(silu(gate) * up), weighted and added up
    (to `residual` where one is given): awq_moe_gemm, awq_moe_gemm and awq_moe_combine.  `up` is gated, `down` plain;
    weights and plan from awq_moe_route.  Between the products the activations have x's type, between down and the sum they
    are fp32.  Workspaces as for awq_moe_gemm (awq_moe_workspace_bytes)."""
    name = "awq_moe"
    if not up.gated or down.gated or down.K != up.outputs:
        raise ValueError("awq_moe: up is gated, down is plain, and down takes up's outputs")
    dtype = _dtype16(name, x, residual, out)
    device, rows, experts, top_k = x.device, plan.rows, plan.experts, plan.top_k
    if x.dtype is not up.dtype or x.dtype is not down.dtype:
        raise TypeError("awq_moe: x and the weights' scales have one type")
    T, H = x.shape[0], down.N
    _need(name, torch.float32, weights)
    _need(name, x.dtype, out)
    if x.shape != (T, up.K) or weights.shape != (T, top_k) or T * top_k != rows or up.experts != experts or \
            down.experts != experts or (residual is not None and residual.shape != (T, H)) or \
            (out is not None and out.shape != (T, H)):
        raise ValueError("awq_moe: x [T, K], weights [T, top_k], residual and out [T, H] go with the layers and the plan")
    _on_current_gpu(name, x, up.data, down.data, weights, plan.offsets, plan.order, plan.place, residual, out, workspace)
    handle = _raw_stream(stream, device)
    if out is None:
        out = _empty((T, H), x.dtype, device, stream)
    _call_on_stream(
        name, lib.awq_moe, workspace, _layer_share(name, handle, device, stream, T, top_k, experts, up.K, down.K, H), device, handle,
        x.data_ptr(), _row_stride(name, x, up.K), up.data.data_ptr(), down.data.data_ptr(), plan.offsets.data_ptr(),
        plan.order.data_ptr(), plan.place.data_ptr(), weights.data_ptr(), _ptr(residual),
        0 if residual is None else _row_stride(name, residual, H), out.data_ptr(), T, top_k, experts, up.K, down.K, H, dtype)
    return out


FP8_BLOCK = 128


def _fp8_weights(name, wq, s_w):
    N, K = wq.shape
    _need(name, torch.float8_e4m3fn, wq)
    _need(name, torch.float32, s_w)
    if s_w.shape != (-(-N // FP8_BLOCK), -(-K // FP8_BLOCK)):
        raise ValueError(f"{name}: wq is [N, K], s_w [N / 128, K / 128] rounded up")
    return N, K


def awq_fp8_quant_act(x, xq=None, s_x=None, stream=None):
    """e4m3 codes [M, K] of 16-bit x [M, K] and their fp32 scales [K / 128, M], one for each token and 128 channels."""
    M, K = x.shape
    dtype = _dtype16("awq_fp8_quant_act", x)
    groups = -(-K // FP8_BLOCK)
    if xq is None:
        xq = _empty((M, K), torch.float8_e4m3fn, x.device, stream)
    if s_x is None:
        s_x = _empty((groups, M), torch.float32, x.device, stream)
    _need("awq_fp8_quant_act", torch.float8_e4m3fn, xq)
    _need("awq_fp8_quant_act", torch.float32, s_x)
    if xq.shape != (M, K) or s_x.shape != (groups, M):
        raise ValueError("awq_fp8_quant_act: xq is [M, K], s_x [K / 128, M]")
    _on_current_gpu("awq_fp8_quant_act", x, xq, s_x)
    _check("awq_fp8_quant_act", lib.awq_fp8_quant_act(x.data_ptr(), _row_stride("awq_fp8_quant_act", x, K), xq.data_ptr(),
                                                      s_x.data_ptr(), M, K, dtype, _raw_stream(stream, x.device)))
    return xq, s_x


def awq_fp8_gemm_workspace_bytes(M: int, K: int, N: int) -> int:
    """Bytes of an awq_fp8_gemm workspace on the current device."""
    return int(lib.awq_fp8_gemm_workspace_bytes(M, K, N))


def awq_fp8_linear_workspace_bytes(M: int, K: int, N: int) -> int:
    """Bytes of an awq_fp8_linear workspace on the current device."""
    return int(lib.awq_fp8_linear_workspace_bytes(M, K, N))


def _fp8_out(name, out, M, N, dtype, device, stream):
    if out is None:
        return _empty((M, N), dtype, device, stream)
    if out.shape != (M, N) or not out.is_contiguous() or out.dtype is not dtype or not out.is_cuda:
        raise ValueError(f"{name}: out is dense, [M, N], of the output's type")
    return out


def awq_fp8_gemm(xq, s_x, wq, s_w, dtype=torch.float16, out=None, workspace=None, stream=None):
    """e4m3 codes xq [M, K] with s_x [K / 128, M] times wq [N, K] with s_w [N / 128, K / 128]: [M, N] of `dtype` (fp16 or
    bf16).  Workspaces as for awq_moe_gemm."""
    M, K = xq.shape
    N, wk = _fp8_weights("awq_fp8_gemm", wq, s_w)
    _need("awq_fp8_gemm", torch.float8_e4m3fn, xq)
    _need("awq_fp8_gemm", torch.float32, s_x)
    kind = _DTYPES.get(dtype)
    if kind is None:
        raise TypeError("awq_fp8_gemm: outputs are fp16 or bf16")
    if wk != K or s_x.shape != (-(-K // FP8_BLOCK), M):
        raise ValueError("awq_fp8_gemm: xq [M, K] and s_x [K / 128, M] go with wq [N, K]")
    device = xq.device
    out = _fp8_out("awq_fp8_gemm", out, M, N, dtype, device, stream)
    _on_current_gpu("awq_fp8_gemm", xq, s_x, wq, s_w, out, workspace)
    handle = _raw_stream(stream, device)
    _call_on_stream("awq_fp8_gemm", lib.awq_fp8_gemm, workspace, _layer_share("awq_fp8_gemm", handle, device, stream, M, K, N),
                    device, handle, xq.data_ptr(), s_x.data_ptr(), wq.data_ptr(), s_w.data_ptr(), out.data_ptr(), M, K, N, kind)
    return out


def awq_fp8_linear(x, wq, s_w, out=None, workspace=None, stream=None):
    """16-bit x [M, K] through a layer of e4m3 weights wq [N, K], s_w [N / 128, K / 128]: quantization and product in one
    call, [M, N] in x's type; out may be x itself.  Workspaces as for awq_moe_gemm (awq_fp8_linear_workspace_bytes)."""
    M, K = x.shape
    kind = _dtype16("awq_fp8_linear", x)
    N, wk = _fp8_weights("awq_fp8_linear", wq, s_w)
    if wk != K:
        raise ValueError("awq_fp8_linear: x is [M, K], wq [N, K]")
    device = x.device
    out = _fp8_out("awq_fp8_linear", out, M, N, x.dtype, device, stream)
    _on_current_gpu("awq_fp8_linear", x, wq, s_w, out, workspace)
    handle = _raw_stream(stream, device)
    _call_on_stream("awq_fp8_linear", lib.awq_fp8_linear, workspace, _layer_share("awq_fp8_linear", handle, device, stream, M, K, N),
                    device, handle, x.data_ptr(), _row_stride("awq_fp8_linear", x, K), wq.data_ptr(), s_w.data_ptr(), out.data_ptr(),
                    M, K, N, kind)
    return out


def _renew_workspaces(device: int) -> None:
    """A call whose wait expired leaves its workspace's counters and flags as they were then.  Streams' workspaces are
    let go of (no graph holds them, and a call that has one still keeps it); the device's, which graphs may hold, is zeroed."""
    for pool in (_kv4_workspaces, _layer_workspaces):
        for key in [key for key in list(pool) if key[0] == device]:
            pool.pop(key, None)
    with _lock_of("device", device):
        if device in _workspaces:
            _workspaces[device].zero_()
            torch.cuda.current_stream(device).synchronize()


def awq_last_device_error() -> int:
    """The id of the last bounded wait that expired on the current device, 0 for none, and clears it; waits for the
    device.  After an id the results since the last reading may be wrong; the workspaces that the binding keeps are
    made anew, those of the caller's own are the caller's to zero."""
    code = _i32(0)
    status = lib.awq_last_device_error(ctypes.byref(code))
    if status not in (0, -5):
        raise AwqError("awq_last_device_error", status)
    if code.value:
        _renew_workspaces(_current_device())
    return int(code.value)


def awq_selftest_wait_timeout(limit_ns: int = 1_000_000, stream=None) -> None:
    """Run one bounded device wait that expires after `limit_ns` (see include/awq.h)."""
    _check("awq_selftest_wait_timeout", lib.awq_selftest_wait_timeout(int(limit_ns), _stream(stream)))
