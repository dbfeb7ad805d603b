"""Block-causal ReLU linear attention with a carried fp32 state, on B200.

Thin binding of the C-ABI library ``liblcla.so`` (declared in
``include/lcla.h``): it checks and marshals torch tensors (device memory and
the current CUDA stream) into its entry points -- the whole-sequence forward
(uniform or explicit blocks), the streaming step, the two halves of a
sequence-sharded forward, the Mix-FFN temporal convolution, and the gated
linear attention operators: rotary tables, the per-head norm of q and k with the
rotation, and the gated recurrence with its step and gradients.  No call records
anything for autograd: a result has no graph even where an input requires a
gradient, and a gradient is a call of its own (``*_backward``).  Every step of
the computation runs in the library's sm_100a kernels; there is no other path.
Importing this package fails if the library has not been built
(``python block_causal_relu_b200/build.py``).
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Tuple

import torch

__all__ = ["forward", "step", "forward_workspace_bytes", "step_workspace_bytes", "plan_info",
           "forward_blocks", "forward_blocks_workspace_bytes", "temporal_conv",
           "rotary_tables", "qk_norm_rope", "qk_norm_rope_backward",
           "gated_forward", "gated_step", "gated_backward", "gated_forward_workspace_bytes",
           "gated_backward_workspace_bytes",
           "shard_begin", "shard_end", "shard_workspace_bytes", "device_status", "selftest_bounded_wait",
           "LclaError", "LIB_PATH", "lib", "BF16", "F32", "D", "HEAD_DIMS"]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblcla.so")
BF16, F32 = 0, 1
D = 32                 # head dim of the tensor-core path
HEAD_DIMS = (32, 64)   # head dims the library serves
DEFAULT_EPS = 1e-8


class LclaError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"lcla status {status}: {msg}")
        self.status = status


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with "
                          "`python block_causal_relu_b200/build.py`")
    L = ctypes.CDLL(LIB_PATH)
    P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    L.lcla_forward_workspace_bytes.argtypes = [I, I, I, I, I, I]
    L.lcla_forward_workspace_bytes.restype = Z
    L.lcla_step_workspace_bytes.argtypes = [I, I, I, I, I]
    L.lcla_step_workspace_bytes.restype = Z
    L.lcla_forward.argtypes = [P, P, P, P, P, I, I, I, I, I, F, P, P, I, P, Z, P]
    L.lcla_forward.restype = I
    L.lcla_forward_timed.argtypes = [P, P, P, P, P, I, I, I, I, I, F, P, P, I, P, Z, P, P]
    L.lcla_forward_timed.restype = I
    L.lcla_step.argtypes = [P, P, P, P, P, I, I, I, I, F, P, I, P, I, P, Z, P]
    L.lcla_step.restype = I
    L.lcla_forward_blocks_workspace_bytes.argtypes = [I, I, I, I, I, I]
    L.lcla_forward_blocks_workspace_bytes.restype = Z
    L.lcla_forward_blocks.argtypes = [P, P, P, P, P, I, I, I, I, P, I, F, P, P, I, P, Z, P]
    L.lcla_forward_blocks.restype = I
    L.lcla_temporal_conv.argtypes = [P, I, I, I, I, P, P, P, I, P, I, P]
    L.lcla_temporal_conv.restype = I
    LL, DB = ctypes.c_longlong, ctypes.c_double
    L.lcla_rotary_tables.argtypes = [P, LL, I, I, P, P, DB, I, DB, DB, DB, DB, P, P, P]
    L.lcla_rotary_tables.restype = I
    L.lcla_qk_norm_rope.argtypes = [P, LL, P, LL, I, I, I, I, I, P, P, F, P, P, I, I, I, P, P, LL, P, LL, I, P]
    L.lcla_qk_norm_rope.restype = I
    L.lcla_qk_norm_rope_backward_workspace_bytes.argtypes = [I]
    L.lcla_qk_norm_rope_backward_workspace_bytes.restype = Z
    L.lcla_qk_norm_rope_backward.argtypes = [P, LL, P, LL, P, LL, P, LL, I, I, I, I, I, P, P, F, P, P, I, I, I, P,
                                             P, LL, P, LL, P, P, I, P, Z, P]
    L.lcla_qk_norm_rope_backward.restype = I
    for f in (L.lcla_gated_forward_workspace_bytes, L.lcla_gated_backward_workspace_bytes):
        f.argtypes, f.restype = [I, I, I, I, I], Z
    L.lcla_gated_forward.argtypes = [P, P, P, P, I, I, I, I, F, P, P, P, I, P, Z, P]
    L.lcla_gated_forward.restype = I
    L.lcla_gated_step.argtypes = [P, P, P, P, I, I, I, I, F, P, I, P, I, P, Z, P]
    L.lcla_gated_step.restype = I
    L.lcla_gated_backward.argtypes = [P, P, P, P, P, I, I, I, I, F, P, P, P, P, P, P, P, I, P, Z, P]
    L.lcla_gated_backward.restype = I
    L.lcla_shard_workspace_bytes.argtypes = [I, I, I, I, I, I]
    L.lcla_shard_workspace_bytes.restype = Z
    L.lcla_shard_begin.argtypes = [P, P, P, P, I, I, I, I, I, P, I, P, Z, P]
    L.lcla_shard_begin.restype = I
    L.lcla_shard_end.argtypes = [P, P, P, P, P, I, I, I, I, I, F, P, I, I, P, P, P, I, P, Z, P]
    L.lcla_shard_end.restype = I
    L.lcla_selftest_bounded_wait.argtypes = [I, P, P]
    L.lcla_selftest_bounded_wait.restype = I
    L.lcla_forward_plan_info.argtypes = [I, I, I, I, I, I, P]
    L.lcla_forward_plan_segments.argtypes = [I, I, I, I, I, I, P, P, P, I]
    L.lcla_forward_plan_segments.restype = I
    L.lcla_forward_plan_info.restype = I
    L.lcla_status_string.argtypes = [I]
    L.lcla_status_string.restype = ctypes.c_char_p
    L.lcla_version.restype = I
    return L


lib = _load()


def _check(rc: int) -> None:
    if rc != 0:
        raise LclaError(rc, lib.lcla_status_string(rc).decode())


def _ints(*sizes) -> None:
    """Sizes go to the library as C ints, which ctypes would cut to 32 bits."""
    for n in sizes:
        if not -0x80000000 <= n <= 0x7fffffff:
            raise LclaError(2, lib.lcla_status_string(2).decode())


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError(f"q, k, v must be bfloat16 or float32, got {t.dtype}")


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _workspace(workspace: Optional[torch.Tensor], need: int, device):
    """(workspace, its bytes): the given one, or one made of ``need`` bytes."""
    if workspace is None:
        if need > 0:
            workspace = torch.empty(need, dtype=torch.uint8, device=device)
            return workspace, need
        return None, 0
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda:
        raise TypeError("workspace must be a CUDA tensor")
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {device}")
    return workspace, workspace.numel() * workspace.element_size()


def _inputs(q, k, v, cos, sin):
    for name, t in (("q", q), ("k", k), ("v", v), ("cos", cos), ("sin", sin)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be a CUDA tensor")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if q.dim() != 4 or q.shape != k.shape or q.shape != v.shape:
        raise ValueError("q, k, v must share one [B, N, H, d] shape")
    if not (q.dtype == k.dtype == v.dtype):
        raise TypeError("q, k, v must share one dtype")
    B, N, H, d = q.shape
    if cos.dtype != torch.float32 or sin.dtype != torch.float32:
        raise TypeError("rope tables must be float32")
    if tuple(cos.shape) != (N, d // 2) or tuple(sin.shape) != (N, d // 2):
        raise ValueError("rope tables must be [N, d/2]")
    return B, N, H, d, _dtype_code(q)


def forward_workspace_bytes(B: int, H: int, N: int, d: int, block_len: int, dtype: int) -> int:
    return int(lib.lcla_forward_workspace_bytes(B, H, N, d, block_len, dtype))


def forward_blocks_workspace_bytes(B: int, H: int, N: int, d: int, nblocks: int, dtype: int) -> int:
    return int(lib.lcla_forward_blocks_workspace_bytes(B, H, N, d, nblocks, dtype))


def step_workspace_bytes(B: int, H: int, L: int, d: int, dtype: int) -> int:
    return int(lib.lcla_step_workspace_bytes(B, H, L, d, dtype))


def plan_info(B: int, H: int, N: int, d: int, block_len: int, dtype: int) -> dict:
    """The library's cut of a forward problem (see ``lcla_forward_plan_info``)."""
    info = (ctypes.c_int * 5)()
    _check(lib.lcla_forward_plan_info(B, H, N, d, block_len, dtype, info))
    return {"chunk_mode": bool(info[0]), "segments": info[1], "prefixes": info[2],
            "tile_tokens": info[3], "tensor_cores": bool(info[4])}


def plan_segments(B: int, H: int, N: int, d: int, block_len: int, dtype: int) -> list:
    """``lcla_forward_plan_segments``: [(t0, t1, block or -1), ...] per segment."""
    n = plan_info(B, H, N, d, block_len, dtype)["segments"]
    arr = [(ctypes.c_int * max(n, 1))() for _ in range(3)]
    _check(lib.lcla_forward_plan_segments(B, H, N, d, block_len, dtype, arr[0], arr[1], arr[2], n))
    return [(arr[0][i], arr[1][i], arr[2][i]) for i in range(n)]


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # current_stream without its wrapper


def _stream(stream, device) -> int:
    if stream is None:
        if _raw_stream is not None and isinstance(device, int):
            return _raw_stream(device)
        stream = torch.cuda.current_stream(device)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def _cuda_device(*candidates):
    """The device of the first CUDA tensor, or None: the call itself refuses what it gets then."""
    for t in candidates:
        if isinstance(t, torch.Tensor) and t.is_cuda:
            return t.device
    return None


def _on_stream(fn, stream, device, /, *args, **kw):
    """``fn`` with ``stream`` as the current stream, so that what it allocates is
    that stream's memory: a block that the caller's stream has freed, with work on
    it still queued there, is not written by another one.  The results are kept
    from reuse until both streams are done with them."""
    if device is None or torch.device(device).type != "cuda":
        return fn(*args, **kw)
    index = torch.device(device).index
    index = torch.cuda.current_device() if index is None else index
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), index) if int(stream) else torch.cuda.default_stream(index)
    if stream.device_index != index:
        raise ValueError(f"stream must be a stream of cuda:{index}")
    here = torch.cuda.current_stream(index)
    if stream.cuda_stream == here.cuda_stream:
        return fn(*args, **kw)
    with torch.cuda.stream(stream):
        result = fn(*args, **kw)
    for t in (*(result if isinstance(result, tuple) else (result,)), kw.get("workspace")):
        if t is not None:
            t.record_stream(stream)
            t.record_stream(here)
    return result


def forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, rope_cos: torch.Tensor,
            rope_sin: torch.Tensor, block_len: int, eps: float = DEFAULT_EPS, *,
            out: Optional[torch.Tensor] = None, state_out: Optional[torch.Tensor] = None,
            want_state: bool = True, workspace: Optional[torch.Tensor] = None,
            stream=None, events=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``lcla_forward``: whole-sequence block-causal attention.

    q, k, v [B, N, H, d] (bf16 or fp32), rope tables [N, d/2] fp32, all CUDA.
    Returns (out [B, N, H, d], state_out [B, H, d+1, d] fp32 or None).
    Buffers not passed in are allocated with torch on q's device.
    ``events``: optional 4 already-recorded ``torch.cuda.Event(enable_timing=True)``
    that the library re-records around its passes (``lcla_forward_timed``).
    """
    if stream is not None:
        return _on_stream(forward, stream, _cuda_device(q), q, k, v, rope_cos, rope_sin, block_len, eps, out=out,
                          state_out=state_out, want_state=want_state, workspace=workspace, events=events)
    B, N, H, d, code = _inputs(q, k, v, rope_cos, rope_sin)
    if out is None:
        out = torch.empty_like(q)
    if state_out is None and want_state:
        state_out = torch.empty((B, H, d + 1, d), dtype=torch.float32, device=q.device)
    workspace, size = _workspace(workspace, forward_workspace_bytes(B, H, N, d, block_len, code), q.device)
    evp = None
    if events is not None:
        if len(events) != 4:
            raise ValueError("events must hold 4 torch.cuda.Event")
        evp = (ctypes.c_void_p * 4)(*[e.cuda_event for e in events])
    _check(lib.lcla_forward_timed(_ptr(q), _ptr(k), _ptr(v), _ptr(rope_cos), _ptr(rope_sin),
                                  B, H, N, d, int(block_len), float(eps), _ptr(out),
                                  _ptr(state_out), code, _ptr(workspace), size, _stream(None, q.device), evp))
    return out, state_out


def forward_blocks(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, rope_cos: torch.Tensor,
                   rope_sin: torch.Tensor, block_offsets: torch.Tensor, eps: float = DEFAULT_EPS, *,
                   out: Optional[torch.Tensor] = None, state_out: Optional[torch.Tensor] = None,
                   want_state: bool = True, workspace: Optional[torch.Tensor] = None,
                   stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``lcla_forward_blocks``: as ``forward`` with explicit block boundaries,
    ``block_offsets`` an int32 CUDA tensor [nblocks + 1] rising from 0 to N."""
    if stream is not None:
        return _on_stream(forward_blocks, stream, _cuda_device(q), q, k, v, rope_cos, rope_sin, block_offsets, eps,
                          out=out, state_out=state_out, want_state=want_state, workspace=workspace)
    B, N, H, d, code = _inputs(q, k, v, rope_cos, rope_sin)
    if (not isinstance(block_offsets, torch.Tensor) or not block_offsets.is_cuda
            or block_offsets.dtype != torch.int32 or block_offsets.dim() != 1
            or not block_offsets.is_contiguous()):
        raise ValueError("block_offsets must be a contiguous int32 CUDA tensor [nblocks + 1]")
    nblocks = block_offsets.numel() - 1
    if out is None:
        out = torch.empty_like(q)
    if state_out is None and want_state:
        state_out = torch.empty((B, H, d + 1, d), dtype=torch.float32, device=q.device)
    workspace, size = _workspace(workspace, forward_blocks_workspace_bytes(B, H, N, d, nblocks, code), q.device)
    _check(lib.lcla_forward_blocks(_ptr(q), _ptr(k), _ptr(v), _ptr(rope_cos), _ptr(rope_sin),
                                   B, H, N, d, _ptr(block_offsets), nblocks, float(eps), _ptr(out),
                                   _ptr(state_out), code, _ptr(workspace), size, _stream(None, q.device)))
    return out, state_out


def shard_workspace_bytes(B: int, H: int, N: int, d: int, block_len: int, dtype: int) -> int:
    return int(lib.lcla_shard_workspace_bytes(B, H, N, d, block_len, dtype))


def _state_tensor(name: str, t: Optional[torch.Tensor], B: int, H: int, d: int, lead=()) -> None:
    if t is None:
        return
    if (not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != torch.float32
            or not t.is_contiguous() or tuple(t.shape) != (*lead, B, H, d + 1, d)):
        raise ValueError(f"{name} must be a contiguous float32 CUDA tensor {[*lead, B, H, d + 1, d]}")


def shard_begin(k: torch.Tensor, v: torch.Tensor, rope_cos: torch.Tensor, rope_sin: torch.Tensor,
                block_len: int, *, total_out: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None,
                stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``lcla_shard_begin``: this rank's state total over its tokens k, v
    [B, N, H, d] (whole blocks of the sequence, tables at their absolute
    positions).  Returns (total [B, H, d+1, d] fp32, workspace); pass the same
    workspace to ``shard_end``."""
    if stream is not None:
        return _on_stream(shard_begin, stream, _cuda_device(k), k, v, rope_cos, rope_sin, block_len,
                          total_out=total_out, workspace=workspace)
    B, N, H, d, code = _inputs(k, k, v, rope_cos, rope_sin)
    if total_out is None:
        total_out = torch.empty((B, H, d + 1, d), dtype=torch.float32, device=k.device)
    _state_tensor("total_out", total_out, B, H, d)
    workspace, size = _workspace(workspace, shard_workspace_bytes(B, H, N, d, block_len, code), k.device)
    _check(lib.lcla_shard_begin(_ptr(k), _ptr(v), _ptr(rope_cos), _ptr(rope_sin), B, H, N, d, int(block_len),
                                _ptr(total_out), code, _ptr(workspace), size, _stream(None, k.device)))
    return total_out, workspace


def shard_end(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, rope_cos: torch.Tensor,
              rope_sin: torch.Tensor, block_len: int, totals: torch.Tensor, rank: int,
              workspace: Optional[torch.Tensor], eps: float = DEFAULT_EPS, *,
              state_in: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
              state_out: Optional[torch.Tensor] = None, want_state: bool = True,
              stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``lcla_shard_end``: this rank's outputs from the gathered ``totals``
    [R, B, H, d+1, d] (every rank's ``shard_begin`` total, in rank order) and
    the workspace ``shard_begin`` filled.  Returns (out, state after the whole
    sequence, or None)."""
    if stream is not None:
        return _on_stream(shard_end, stream, _cuda_device(q), q, k, v, rope_cos, rope_sin, block_len, totals, rank,
                          workspace, eps, state_in=state_in, out=out, state_out=state_out, want_state=want_state)
    B, N, H, d, code = _inputs(q, k, v, rope_cos, rope_sin)
    if not isinstance(totals, torch.Tensor) or totals.dim() != 5:
        raise ValueError("totals must be [R, B, H, d+1, d]")
    nranks = totals.shape[0]
    _state_tensor("totals", totals, B, H, d, lead=(nranks,))
    _state_tensor("state_in", state_in, B, H, d)
    if out is None:
        out = torch.empty_like(q)
    if state_out is None and want_state:
        state_out = torch.empty((B, H, d + 1, d), dtype=torch.float32, device=q.device)
    _state_tensor("state_out", state_out, B, H, d)
    workspace, size = _workspace(workspace, 0, q.device)
    _check(lib.lcla_shard_end(_ptr(q), _ptr(k), _ptr(v), _ptr(rope_cos), _ptr(rope_sin), B, H, N, d,
                              int(block_len), float(eps), _ptr(totals), nranks, int(rank), _ptr(state_in),
                              _ptr(out), _ptr(state_out), code, _ptr(workspace), size, _stream(None, q.device)))
    return out, state_out


def device_status(workspace: Optional[torch.Tensor]) -> int:
    """The device status word a call left in ``workspace`` (0: every bounded
    wait completed; bit 0 / bit 1: pass A / pass C gave up).  Synchronises on
    the copy."""
    if workspace is None or workspace.numel() < 4:
        return 0
    return int(workspace[:4].view(torch.int32).item())


def selftest_bounded_wait(arrive_first: bool, stream=None) -> Tuple[bool, int, int]:
    """``lcla_selftest_bounded_wait``: (gave_up, nanoseconds waited, abort flag)."""
    res = torch.zeros(3, dtype=torch.int64, device="cuda")
    _check(lib.lcla_selftest_bounded_wait(int(bool(arrive_first)), _ptr(res), _stream(stream, res.device)))
    r = res.cpu().tolist()
    return bool(r[0]), int(r[1]), int(r[2])


def step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cos: torch.Tensor,
         sin: torch.Tensor, state: torch.Tensor, save: bool, eps: float = DEFAULT_EPS, *,
         out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
         stream=None) -> torch.Tensor:
    """``lcla_step``: one block [B, L, H, d] against ``state`` [B, H, d+1, d]
    fp32 (updated in place when ``save``).  Returns the block's outputs."""
    if stream is not None:
        return _on_stream(step, stream, _cuda_device(q), q, k, v, cos, sin, state, save, eps, out=out,
                          workspace=workspace)
    B, L, H, d, code = _inputs(q, k, v, cos, sin)
    if (not state.is_cuda or state.dtype != torch.float32 or not state.is_contiguous()
            or tuple(state.shape) != (B, H, d + 1, d)):
        raise ValueError("state must be a contiguous float32 CUDA tensor [B, H, d+1, d]")
    if out is None:
        out = torch.empty_like(q)
    workspace, size = _workspace(workspace, step_workspace_bytes(B, H, L, d, code), q.device)
    _check(lib.lcla_step(_ptr(q), _ptr(k), _ptr(v), _ptr(cos), _ptr(sin), B, H, L, d, float(eps),
                         _ptr(state), int(bool(save)), _ptr(out), code, _ptr(workspace), size, _stream(None, q.device)))
    return out


def temporal_conv(x: torch.Tensor, tokens_per_frame: int, weight: torch.Tensor,
                  bias: Optional[torch.Tensor] = None, cache: Optional[torch.Tensor] = None,
                  save: bool = False, *, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``lcla_temporal_conv``: causal size-2 depthwise convolution over latent
    frames of ``x`` [B, F * S, C] (S = ``tokens_per_frame``), with weight [2, C]
    and bias [C] fp32 and the previous frame from ``cache`` [B, S, C] (zeros
    when None); ``save`` overwrites the cache with x's last frame."""
    if stream is not None:
        return _on_stream(temporal_conv, stream, _cuda_device(x), x, tokens_per_frame, weight, bias, cache, save,
                          out=out)
    if not isinstance(x, torch.Tensor) or not x.is_cuda or not x.is_contiguous() or x.dim() != 3:
        raise ValueError("x must be a contiguous CUDA tensor [B, F * S, C]")
    B, N, C = x.shape
    S = int(tokens_per_frame)
    if S < 1 or N % S:
        raise ValueError("x's token count must be a whole number of frames")
    code = _dtype_code(x)
    for name, t, shape in (("weight", weight, (2, C)), ("bias", bias, (C,))):
        if t is None:
            continue
        if not t.is_cuda or t.dtype != torch.float32 or not t.is_contiguous() or tuple(t.shape) != shape:
            raise ValueError(f"{name} must be a contiguous float32 CUDA tensor {list(shape)}")
    if cache is not None and (not cache.is_cuda or cache.dtype != x.dtype or not cache.is_contiguous()
                              or tuple(cache.shape) != (B, S, C)):
        raise ValueError("cache must be a contiguous CUDA tensor [B, S, C] of x's dtype")
    if out is None:
        out = torch.empty_like(x)
    _check(lib.lcla_temporal_conv(_ptr(x), B, N // S, S, C, _ptr(weight), _ptr(bias), _ptr(cache),
                                  int(bool(save)), _ptr(out), code, _stream(None, x.device)))
    return out


def _run(device: int, fn, *args) -> None:
    """Calls the library with the tensors' device as the current one."""
    was = torch.cuda.current_device()
    if was == device:
        rc = fn(*args)
    else:
        torch.cuda.set_device(device)
        try:
            rc = fn(*args)
        finally:
            torch.cuda.set_device(was)
    if rc != 0:
        _check(rc)


def _array(name: str, t: Optional[torch.Tensor], shape: tuple, dtype: torch.dtype, device: int) -> Optional[int]:
    """The address of a contiguous CUDA tensor of this shape, dtype and device; None for None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor {list(shape)} on cuda:{device}")
    return t.data_ptr()


ROPE_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


def rotary_tables(n: int, dims, *, extents=None, first: int = 0, positions: Optional[torch.Tensor] = None,
                  theta: float = 10000.0, scaling: str = "none", factor: float = 1.0, original_len: float = 4096,
                  beta_fast: float = 32.0, beta_slow: float = 1.0, device="cuda",
                  out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                  stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """``lcla_rotary_tables``: (cos, sin) [n, sum(dims) / 2] fp32 of n tokens.

    ``dims`` holds the rotary dims of each axis (an int for one axis).  Tokens
    stand at ``positions`` [axes, n] ([n] for one axis) int64, or at indices
    ``first`` .. ``first + n - 1`` of a row-major grid whose inner axes have
    the sizes ``extents``, up to index 2^36 - 1.  ``scaling``: "none", "linear",
    "ntk" or "yarn"."""
    if stream is not None:
        return _on_stream(rotary_tables, stream, _cuda_device(positions, *(out or ())) or device, n, dims,
                          extents=extents, first=first, positions=positions, theta=theta, scaling=scaling,
                          factor=factor, original_len=original_len, beta_fast=beta_fast, beta_slow=beta_slow,
                          device=device, out=out)
    dims = [int(x) for x in ([dims] if isinstance(dims, int) else dims)]
    extents = None if extents is None else [int(x) for x in extents]
    n, first = int(n), int(first)
    _ints(n, *dims, *(extents or ()), first >> 32)
    if scaling not in ROPE_SCALING:
        raise ValueError(f"scaling must be one of {sorted(ROPE_SCALING)}")
    if not 1 <= len(dims) <= 3:
        raise ValueError("one to three axes")
    if n < 0 or min(dims) < 0:
        raise ValueError("negative sizes")
    if positions is None and len(dims) > 1 and (extents is None or len(extents) != len(dims) - 1):
        raise ValueError("extents must hold the sizes of the inner axes")
    pos = None
    if positions is not None:
        if not isinstance(positions, torch.Tensor) or not positions.is_cuda:
            raise TypeError("positions must be a CUDA tensor")
        index = positions.get_device()
        pos = _array("positions", positions, (n,) if positions.dim() == 1 and len(dims) == 1 else (len(dims), n),
                     torch.int64, index)
    elif out is not None:
        index = out[0].get_device()
    else:
        where = torch.device(device)
        if where.type != "cuda":
            raise ValueError(f"device must be a CUDA device, not {where}")
        index = torch.cuda.current_device() if where.index is None else where.index
    shape = (n, sum(dims) // 2)
    if out is None:
        cos = torch.empty(shape, dtype=torch.float32, device=f"cuda:{index}")
        out = (cos, torch.empty_like(cos))
        ptrs = [t.data_ptr() for t in out]
    else:
        ptrs = [_array(name, t, shape, torch.float32, index) for name, t in zip(("cos", "sin"), out)]
    ints = ctypes.c_int * 3
    _run(index, lib.lcla_rotary_tables, pos, first, n, len(dims), ints(*dims),
         None if extents is None else ints(*extents), float(theta), ROPE_SCALING[scaling], float(factor),
         float(original_len), float(beta_fast), float(beta_slow), *ptrs, _stream(None, index))
    return out[0], out[1]


def _rows(name: str, t: torch.Tensor, like: Optional[torch.Tensor] = None) -> int:
    """The distance between the tokens of ``t`` [B, N, H, d], in elements: heads
    lie side by side, tokens at one distance throughout."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dim() != 4:
        raise ValueError(f"{name} must be [B, N, H, d]")
    if like is not None and (t.shape != like.shape or t.dtype != like.dtype or t.get_device() != like.get_device()):
        raise ValueError(f"{name} must have the shape, dtype and device of its forward tensor")
    B, N, H, d = t.shape
    if t.is_contiguous() or t.numel() == 0:
        return H * d
    sb, sn, sh, sd = t.stride()
    if sd != 1 and d > 1 or sh != d and H > 1:
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    if N > 1:
        if B > 1 and sb != N * sn:
            raise ValueError(f"{name}: tokens must be evenly spaced over the batch")
        return sn
    return sb if B > 1 else H * d


def _norm_call(q, k, cos, sin, q_weight, k_weight, positions, eps, half_layout):
    """Checks the forward's inputs; what both entry points take of them, and the device."""
    ldq = _rows("q", q)
    B, N, H, d = q.shape
    code, device = _dtype_code(q), q.get_device()
    Hk, ldk, kp = 0, 0, None
    if k is not None:
        ldk = _rows("k", k)
        Bk, Nk, Hk, dk = k.shape
        if (Bk, Nk, dk) != (B, N, d) or k.dtype != q.dtype or k.get_device() != device:
            raise ValueError("k must be [B, N, Hk, d] of q's dtype on q's device")
        kp = k.data_ptr()
    elif k_weight is not None:
        raise ValueError("k_weight without k")
    if not isinstance(cos, torch.Tensor) or cos.dim() != 2:
        raise ValueError("rope tables must be [rows, rotary_dims / 2]")
    rows, pairs = table = cos.shape
    _ints(B, N, H, Hk, rows)
    f32 = torch.float32
    tail = (B, N, H, Hk, d, _array("q_weight", q_weight, (d,), f32, device),
            _array("k_weight", k_weight, (d,), f32, device), eps, _array("cos", cos, table, f32, device),
            _array("sin", sin, table, f32, device), rows, 2 * pairs, 1 if half_layout else 0,
            _array("positions", positions, (B, N), torch.int64, device))
    return (q.data_ptr(), ldq, kp, ldk), tail, code, device


def _norm_out(q, k, out):
    """Addresses and distances of the outputs, made unless they are given."""
    if out is None:
        form = torch.contiguous_format
        qo = torch.empty_like(q, memory_format=form)
        width = q.shape[2] * q.shape[3]
        if k is None:
            return (qo, None), (qo.data_ptr(), width, None, 0)
        ko = torch.empty_like(k, memory_format=form)
        return (qo, ko), (qo.data_ptr(), width, ko.data_ptr(), k.shape[2] * k.shape[3])
    qo, ko = out
    ldk = 0 if k is None else _rows("out k", ko, k)
    return (qo, ko), (_ptr(qo), _rows("out q", qo, q), None if k is None else _ptr(ko), ldk)


def qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], rope_cos: torch.Tensor, rope_sin: torch.Tensor, *,
                 q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None, eps: float = 1e-6,
                 positions: Optional[torch.Tensor] = None, half_layout: bool = False,
                 out: Optional[Tuple[torch.Tensor, Optional[torch.Tensor]]] = None,
                 stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``lcla_qk_norm_rope``: RMS norm of every head of q [B, N, H, d] and k
    [B, N, Hk, d] (or None), with weights [d], then the rotation of the first
    2 * rope_cos.shape[1] entries by the table rows at ``positions`` [B, N]
    int64 (token n's own row without).  q and k may be column windows of one
    projection; ``out`` = (q_out, k_out) may be (q, k) themselves.  No graph for
    autograd: the gradient is ``qk_norm_rope_backward``."""
    if stream is not None:
        return _on_stream(qk_norm_rope, stream, _cuda_device(q), q, k, rope_cos, rope_sin, q_weight=q_weight,
                          k_weight=k_weight, eps=eps, positions=positions, half_layout=half_layout, out=out)
    ins, tail, code, device = _norm_call(q, k, rope_cos, rope_sin, q_weight, k_weight, positions, eps, half_layout)
    out, to = _norm_out(q, k, out)
    _run(device, lib.lcla_qk_norm_rope, *ins, *tail, *to, code, _stream(None, device))
    return out


def qk_norm_rope_backward(dq_out: torch.Tensor, dk_out: Optional[torch.Tensor], q: torch.Tensor,
                          k: Optional[torch.Tensor], rope_cos: torch.Tensor, rope_sin: torch.Tensor, *,
                          q_weight: Optional[torch.Tensor] = None, k_weight: Optional[torch.Tensor] = None,
                          eps: float = 1e-6, positions: Optional[torch.Tensor] = None, half_layout: bool = False,
                          out: Optional[Tuple[torch.Tensor, Optional[torch.Tensor]]] = None,
                          workspace: Optional[torch.Tensor] = None, stream=None):
    """``lcla_qk_norm_rope_backward``: (dq, dk, dq_weight, dk_weight) from the
    gradients of ``qk_norm_rope``'s outputs and its inputs; a weight that was
    not given has no gradient (None)."""
    if stream is not None:
        return _on_stream(qk_norm_rope_backward, stream, _cuda_device(q), dq_out, dk_out, q, k, rope_cos, rope_sin,
                          q_weight=q_weight, k_weight=k_weight, eps=eps, positions=positions, half_layout=half_layout,
                          out=out, workspace=workspace)
    ins, tail, code, device = _norm_call(q, k, rope_cos, rope_sin, q_weight, k_weight, positions, eps, half_layout)
    ldgq = _rows("dq_out", dq_out, q)
    ldgk = 0 if k is None else _rows("dk_out", dk_out, k)
    out, to = _norm_out(q, k, out)
    dqw = None if q_weight is None else torch.empty_like(q_weight)
    dkw = None if k_weight is None else torch.empty_like(k_weight)
    workspace, size = _workspace(workspace, 0 if dqw is None and dkw is None else
                                 lib.lcla_qk_norm_rope_backward_workspace_bytes(q.shape[3]), q.device)
    _run(device, lib.lcla_qk_norm_rope_backward, dq_out.data_ptr(), ldgq, None if k is None else dk_out.data_ptr(),
         ldgk, *ins, *tail, *to, _ptr(dqw), _ptr(dkw), code, _ptr(workspace), size, _stream(None, device))
    return out[0], out[1], dqw, dkw


def _gated_inputs(q, k, v, g, scale):
    """(addresses of q, k, v, g), (B, H, N, d, scale), dtype code, device."""
    if not isinstance(q, torch.Tensor) or not q.is_cuda:
        raise TypeError("q must be a CUDA tensor")
    if q.dim() != 4:
        raise ValueError("q, k, v must share one [B, N, H, d] shape")
    if g is None or k is None or v is None:
        raise TypeError("k, v and g must be CUDA tensors")
    shape, dtype, device = q.shape, q.dtype, q.get_device()
    B, N, H, d = shape
    _ints(B, N, H)
    ptrs = (_array("q", q, shape, dtype, device), _array("k", k, shape, dtype, device),
            _array("v", v, shape, dtype, device), _array("g", g, (B, N, H), torch.float32, device))
    return ptrs, (B, H, N, d, float(d ** -0.5 if scale is None else scale)), _dtype_code(q), device


def _gated_need(B, H, N, d, code) -> int:
    # a block of one tile (32 tokens) needs none, and a serving step does not ask
    return 0 if N <= 32 else lib.lcla_gated_forward_workspace_bytes(B, H, N, d, code)


def gated_forward_workspace_bytes(B: int, H: int, N: int, d: int, dtype: int) -> int:
    return int(lib.lcla_gated_forward_workspace_bytes(B, H, N, d, dtype))


def gated_backward_workspace_bytes(B: int, H: int, N: int, d: int, dtype: int) -> int:
    return int(lib.lcla_gated_backward_workspace_bytes(B, H, N, d, dtype))


def gated_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, scale: Optional[float] = None, *,
                  state_in: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                  state_out: Optional[torch.Tensor] = None, want_state: bool = True,
                  workspace: Optional[torch.Tensor] = None,
                  stream=None) -> Tuple[torch.Tensor, Optional[torch.Tensor]]:
    """``lcla_gated_forward``: S_t = exp(g_t) S_{t-1} + v_t k_t^T, out_t =
    scale S_t q_t over q, k, v [B, N, H, d] with log decays g [B, N, H] fp32 and
    scale d^-1/2 unless given.  Returns (out, state after the last token
    [B, H, d, d] fp32 or None).  No graph for autograd: the gradient is
    ``gated_backward``."""
    if stream is not None:
        return _on_stream(gated_forward, stream, _cuda_device(q), q, k, v, g, scale, state_in=state_in, out=out,
                          state_out=state_out, want_state=want_state, workspace=workspace)
    ptrs, dims, code, device = _gated_inputs(q, k, v, g, scale)
    B, H, N, d, _ = dims
    st = (B, H, d, d)
    s0 = _array("state_in", state_in, st, torch.float32, device)
    if out is None:
        out = torch.empty_like(q)
        op = out.data_ptr()
    else:
        op = _array("out", out, q.shape, q.dtype, device)
    if state_out is None and want_state:
        state_out = torch.empty(st, dtype=torch.float32, device=q.device)
        s1 = state_out.data_ptr()
    else:
        s1 = _array("state_out", state_out, st, torch.float32, device)
    workspace, size = _workspace(workspace, _gated_need(B, H, N, d, code), q.device)
    _run(device, lib.lcla_gated_forward, *ptrs, *dims, s0, op, s1, code, _ptr(workspace), size,
         _stream(None, device))
    return out, state_out


def gated_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, state: torch.Tensor, save: bool,
               scale: Optional[float] = None, *, state_out: Optional[torch.Tensor] = None,
               out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               stream=None) -> torch.Tensor:
    """``lcla_gated_step``: one block [B, L, H, d] (one token, when serving)
    against ``state`` [B, H, d, d] fp32.  With ``save`` the state after the block
    goes to ``state_out``, or to ``state`` itself.  Returns the block's outputs."""
    if stream is not None:
        return _on_stream(gated_step, stream, _cuda_device(q), q, k, v, g, state, save, scale, state_out=state_out,
                          out=out, workspace=workspace)
    if state is None:
        raise TypeError("state must be a CUDA tensor")
    if state_out is not None:
        return gated_forward(q, k, v, g, scale, state_in=state, out=out, state_out=state_out if save else None,
                             want_state=False, workspace=workspace)[0]
    ptrs, dims, code, device = _gated_inputs(q, k, v, g, scale)
    B, H, L, d, _ = dims
    sp = _array("state", state, (B, H, d, d), torch.float32, device)
    if out is None:
        out = torch.empty_like(q)
        op = out.data_ptr()
    else:
        op = _array("out", out, q.shape, q.dtype, device)
    workspace, size = _workspace(workspace, _gated_need(B, H, L, d, code), q.device)
    _run(device, lib.lcla_gated_step, *ptrs, *dims, sp, 1 if save else 0, op, code, _ptr(workspace), size,
         _stream(None, device))
    return out


def gated_backward(dout: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor,
                   scale: Optional[float] = None, *, state_in: Optional[torch.Tensor] = None,
                   dstate_out: Optional[torch.Tensor] = None, want_dstate_in: bool = False,
                   out: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor, torch.Tensor]] = None,
                   workspace: Optional[torch.Tensor] = None, stream=None):
    """``lcla_gated_backward``: (dq, dk, dv, dg, dstate_in or None) from the
    gradients of ``gated_forward``'s outputs and its inputs; ``out`` gives the
    buffers of the first four."""
    if stream is not None:
        return _on_stream(gated_backward, stream, _cuda_device(q), dout, q, k, v, g, scale, state_in=state_in,
                          dstate_out=dstate_out, want_dstate_in=want_dstate_in, out=out, workspace=workspace)
    ptrs, dims, code, device = _gated_inputs(q, k, v, g, scale)
    B, H, N, d, _ = dims
    if dout is None:
        raise TypeError("dout must be a CUDA tensor")
    dp = _array("dout", dout, q.shape, q.dtype, device)
    st, f32 = (B, H, d, d), torch.float32
    s0 = _array("state_in", state_in, st, f32, device)
    ds1 = _array("dstate_out", dstate_out, st, f32, device)
    if out is None:
        out = (torch.empty_like(q), torch.empty_like(q), torch.empty_like(q), torch.empty_like(g))
        to = [t.data_ptr() for t in out]
    else:
        to = [_array(name, t, like.shape, like.dtype, device)
              for name, t, like in zip(("dq", "dk", "dv", "dg"), out, (q, q, q, g))]
    ds0 = torch.empty(st, dtype=f32, device=q.device) if want_dstate_in else None
    workspace, size = _workspace(workspace, lib.lcla_gated_backward_workspace_bytes(B, H, N, d, code), q.device)
    _run(device, lib.lcla_gated_backward, dp, *ptrs, *dims, s0, ds1, *to, _ptr(ds0), code, _ptr(workspace), size,
         _stream(None, device))
    return (*out, ds0)
