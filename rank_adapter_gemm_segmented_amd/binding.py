"""Thin ctypes binding of ``libmlora.so`` (the C ABI in ``include/mlora.h``).

Argument marshalling only: tensors become device pointers, the current torch
stream becomes the HIP stream, status codes become exceptions. Every step of
the layer runs in the library's HIP kernels; there is no Python or CPU
fallback, and importing this module fails loudly when the library is not
built.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmlora.so")

MLORA_F32, MLORA_BF16 = 0, 1
STATUS = {
    0: "MLORA_OK", 1: "MLORA_ERR_INVALID_ARG", 2: "MLORA_ERR_SHAPE", 3: "MLORA_ERR_DTYPE",
    4: "MLORA_ERR_RANK", 5: "MLORA_ERR_ADAPTER", 6: "MLORA_ERR_EXISTS",
    7: "MLORA_ERR_WORKSPACE", 8: "MLORA_ERR_METADATA", 9: "MLORA_ERR_HIP",
}
STATUS_CODE = {v: k for k, v in STATUS.items()}


# activations of an epilogue, by name
ACTS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "gelu_tanh": 4}
_GATED = 16


class _Epilogue(ctypes.Structure):
    """``mlora_epilogue_t``"""
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p), ("act", ctypes.c_int)]


class MloraError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        self.name = STATUS.get(code, f"status {code}")
        super().__init__(f"{what}: {self.name} ({_lib.mlora_status_string(code).decode()})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is not built: run `python rank_adapter_gemm_segmented_amd/build.py` "
            "(or __graft_entry__.build()) first. There is no fallback path.")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    sig = {
        "mlora_status_string": ([I], ctypes.c_char_p),
        "mlora_pool_bytes": ([I, I, I, I, I], SZ),
        "mlora_pool_create": ([P, SZ, I, I, I, I, I, P, ctypes.POINTER(P)], I),
        "mlora_pool_destroy": ([P], I),
        "mlora_register_adapter": ([P, I, I, P, P, P], I),
        "mlora_unregister_adapter": ([P, I, P], I),
        "mlora_adapter_rank": ([P, I], I),
        "mlora_workspace_bytes": ([P, I], SZ),
        "mlora_workspace_init": ([P, SZ, P], I),
        "mlora_linear": ([P, P, P, P, P, P, P, P, I, I, I, P, P, SZ, P], I),
        "mlora_build_segments": ([P, P, I, P, P, P, P, P, P, P, P], I),
        "mlora_linear_tokens": ([P, P, P, P, P, I, I, P, P, SZ, P], I),
        "mlora_token_map": ([P, P, I, I, P, P, P], I),
        "mlora_validate": ([P, P, P, P, P, I, I, P, SZ, P], I),
        "mlora_merge_adapter": ([P, P, P, I, ctypes.c_float, P], I),
        "mlora_register_adapter_fused": ([P, I, I, P, P, P, P, P], I),
        "mlora_linear_fp8w": ([P, P, P, P, P, P, P, P, P, I, I, I, P, P, SZ, P], I),
        "mlora_linear_noalloc": ([P, P, P, P, P, P, P, P, I, I, I, P, P], I),
        "mlora_linear_epilogue": ([P, P, P, P, P, P, P, P, I, I, I, P, P, P, SZ, P], I),
        "mlora_linear_tokens_epilogue": ([P, P, P, P, P, I, I, P, P, P, SZ, P], I),
        "mlora_linear_fp8w_epilogue": ([P, P, P, P, P, P, P, P, P, I, I, I, P, P, P, SZ, P], I),
        "mlora_route_workspace_bytes": ([I, I, I], SZ),
        "mlora_route": ([P, I, I, I, I, I, P, P, P, P, P, P, SZ, P], I),
        "mlora_experts_linear": ([P, P, P, I, I, I, I, I, P, P, I, P, P, P], I),
        "mlora_experts_workspace_bytes": ([I, I, I, I, I], SZ),
        "mlora_experts_combine": ([P, P, P, I, I, I, I, I, I, P, P, P, P, P, P, P, SZ, P], I),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


_lib = _load()


def library() -> ctypes.CDLL:
    return _lib


def _check(code: int, what: str):
    if code != 0:
        raise MloraError(code, what)


def _ptr(t: Optional[torch.Tensor]):
    # plain ints (ctypes passes them as void*): no wrapper object per argument
    return None if t is None else t.data_ptr()


_raw_stream = torch._C._cuda_getCurrentRawStream


def _stream():
    """The current torch stream of the current device as a raw HIP stream
    handle (also the capture stream inside torch.cuda.graph)."""
    return _raw_stream(torch.cuda.current_device())


def _dtype_code(dt: torch.dtype) -> int:
    if dt == torch.bfloat16:
        return MLORA_BF16
    if dt == torch.float32:
        return MLORA_F32
    raise TypeError(f"unsupported dtype {dt}")


def _i32(t, name):
    if t is None:
        return None
    if t.dtype != torch.int32 or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous int32 device tensor")
    return t


class Pool:
    """Fixed-slot device adapter pool (``mlora_pool_create``). The arena is a
    torch uint8 tensor, so torch's allocator owns every device byte."""

    def __init__(self, d_in: int, d_out: int, dtype: torch.dtype, max_rank: int, capacity: int,
                 device="cuda"):
        self.d_in, self.d_out, self.dtype = d_in, d_out, dtype
        self.max_rank, self.capacity = max_rank, capacity
        code = _dtype_code(dtype)
        nbytes = _lib.mlora_pool_bytes(d_in, d_out, code, max_rank, capacity)
        if nbytes == 0:
            raise MloraError(STATUS_CODE["MLORA_ERR_SHAPE"], "mlora_pool_bytes")
        self.arena = torch.empty(nbytes, dtype=torch.uint8, device=device)
        h = ctypes.c_void_p()
        _check(_lib.mlora_pool_create(_ptr(self.arena), nbytes, d_in, d_out, code, max_rank,
                                      capacity, _stream(), ctypes.byref(h)), "mlora_pool_create")
        self.handle = h

    def register(self, adapter_id: int, A: torch.Tensor, B: torch.Tensor):
        """Copy A [rank, d_in] and B [d_out, rank] into slot ``adapter_id``."""
        rank = int(A.shape[0])
        if A.dtype != self.dtype or B.dtype != self.dtype:
            raise TypeError("adapter dtype differs from the pool dtype")
        if tuple(A.shape) != (rank, self.d_in) or tuple(B.shape) != (self.d_out, rank):
            raise ValueError("adapter shapes must be A [rank, d_in], B [d_out, rank]")
        A = A.contiguous()
        B = B.contiguous()
        _check(_lib.mlora_register_adapter(self.handle, adapter_id, rank, _ptr(A), _ptr(B),
                                           _stream()), "mlora_register_adapter")
        # the copy is stream-ordered: keep the sources alive until it has run
        torch.cuda.current_stream().synchronize()

    def register_fused(self, adapter_id: int, slices):
        """``mlora_register_adapter_fused``: one adapter over stacked projections.
        ``slices`` is a list of (A_m [r_m, d_in], B_m [rows_m, r_m]) in the
        order the projections are stacked in W. A pool holds either plain or
        fused adapters, and all fused ones stack W the same way; segments
        name the adapter with the stacked rank sum(r_m)."""
        n = len(slices)
        rows = (ctypes.c_int * n)(*[int(B.shape[0]) for _, B in slices])
        ranks = (ctypes.c_int * n)(*[int(A.shape[0]) for A, _ in slices])
        keep = []
        for A, B in slices:
            if A.dtype != self.dtype or B.dtype != self.dtype:
                raise TypeError("adapter dtype differs from the pool dtype")
            if A.dim() != 2 or A.shape[1] != self.d_in or B.dim() != 2 or B.shape[1] != A.shape[0]:
                raise ValueError("slice shapes must be A [r, d_in], B [rows, r]")
            keep.append((A.contiguous(), B.contiguous()))
        pa = (ctypes.c_void_p * n)(*[A.data_ptr() for A, _ in keep])
        pb = (ctypes.c_void_p * n)(*[B.data_ptr() for _, B in keep])
        _check(_lib.mlora_register_adapter_fused(self.handle, adapter_id, n, rows, ranks, pa, pb,
                                                 _stream()), "mlora_register_adapter_fused")
        torch.cuda.current_stream().synchronize()

    def unregister(self, adapter_id: int):
        _check(_lib.mlora_unregister_adapter(self.handle, adapter_id, _stream()),
               "mlora_unregister_adapter")

    def rank(self, adapter_id: int) -> int:
        return int(_lib.mlora_adapter_rank(self.handle, adapter_id))

    def workspace_bytes(self, max_tokens: int) -> int:
        return int(_lib.mlora_workspace_bytes(self.handle, max_tokens))

    def workspace(self, max_tokens: int) -> torch.Tensor:
        n = self.workspace_bytes(max_tokens)
        ws = torch.empty(max(n, 256), dtype=torch.uint8, device=self.arena.device)
        _check(_lib.mlora_workspace_init(_ptr(ws), ws.numel(), _stream()), "mlora_workspace_init")
        return ws

    def __del__(self):
        h = getattr(self, "handle", None)
        if h is not None and h.value:
            _lib.mlora_pool_destroy(h)
            self.handle = None


def _check_xw(x, W, pool: Pool):
    if x.dtype != pool.dtype or W.dtype != pool.dtype:
        raise TypeError("x and W must have the pool's dtype")
    if x.dim() != 2 or x.shape[1] != pool.d_in or tuple(W.shape) != (pool.d_out, pool.d_in):
        raise ValueError("x must be [T, d_in] and W [d_out, d_in]")
    if not (x.is_contiguous() and W.is_contiguous()):
        raise ValueError("x and W must be contiguous")


def _segments(T: int, lora_on, seg_start, seg_adapter, seg_rank, seg_scale, token_index) -> int:
    """The number of segments, which seg_adapter gives; a call with adapters needs the other
    arrays as long (the kernels bound what they hold, and cannot bound how much)."""
    if seg_adapter is None:
        return 0
    n = seg_adapter.numel()
    if lora_on and T and n:   # (else none is read)
        if ((seg_start is not None and seg_start.numel() <= n) or (seg_rank is not None and seg_rank.numel() < n)
                or (seg_scale is not None and seg_scale.numel() < n)):
            raise ValueError("seg_start must be [n_seg + 1], seg_rank and seg_scale [n_seg], with n_seg that of seg_adapter")
        if token_index is not None and token_index.numel() < T:
            raise ValueError("token_index must be [T]")
    return n


def linear(x, W, pool: Pool, seg_start=None, seg_adapter=None, seg_rank=None, seg_scale=None,
           lora_on: int = 1, token_index=None, out=None, workspace=None):
    """``mlora_linear``: y = W x + per-segment adapter term (sorted metadata)."""
    _check_xw(x, W, pool)
    T = int(x.shape[0])
    y = out if out is not None else torch.empty((T, pool.d_out), dtype=pool.dtype, device=x.device)
    ws = workspace if workspace is not None else pool.workspace(T)
    n_seg = _segments(T, lora_on, seg_start, seg_adapter, seg_rank, seg_scale, token_index)
    if seg_scale is not None and (seg_scale.dtype != torch.float32 or not seg_scale.is_contiguous()):
        raise TypeError("seg_scale must be contiguous float32")
    _check(_lib.mlora_linear(_ptr(x), _ptr(W), pool.handle, _ptr(_i32(seg_start, "seg_start")),
                             _ptr(_i32(seg_adapter, "seg_adapter")), _ptr(_i32(seg_rank, "seg_rank")),
                             _ptr(seg_scale), _ptr(_i32(token_index, "token_index")), T, n_seg,
                             int(lora_on), _ptr(y), _ptr(ws), ws.numel(), _stream()),
           "mlora_linear")
    return y


def linear_noalloc(x, W, pool: Pool, seg_start=None, seg_adapter=None, seg_rank=None, seg_scale=None,
                   lora_on: int = 1, token_index=None, out=None):
    """``mlora_linear_noalloc``: ``linear`` with the library's own device
    scratch as the workspace (the call allocates nothing; ``out`` should be
    given by callers that cannot allocate either)."""
    _check_xw(x, W, pool)
    T = int(x.shape[0])
    y = out if out is not None else torch.empty((T, pool.d_out), dtype=pool.dtype, device=x.device)
    n_seg = _segments(T, lora_on, seg_start, seg_adapter, seg_rank, seg_scale, token_index)
    if seg_scale is not None and (seg_scale.dtype != torch.float32 or not seg_scale.is_contiguous()):
        raise TypeError("seg_scale must be contiguous float32")
    _check(_lib.mlora_linear_noalloc(_ptr(x), _ptr(W), pool.handle, _ptr(_i32(seg_start, "seg_start")),
                                     _ptr(_i32(seg_adapter, "seg_adapter")), _ptr(_i32(seg_rank, "seg_rank")),
                                     _ptr(seg_scale), _ptr(_i32(token_index, "token_index")), T, n_seg,
                                     int(lora_on), _ptr(y), _stream()), "mlora_linear_noalloc")
    return y


def linear_fp8w(x, W_fp8, w_scale, pool: Pool, seg_start=None, seg_adapter=None, seg_rank=None,
                seg_scale=None, lora_on: int = 1, token_index=None, out=None, workspace=None):
    """``mlora_linear_fp8w``: the layer with an FP8 (e4m3 codes, uint8 [d_out, d_in])
    base weight and float32 per-row scales; x, y and the pool in bf16."""
    if x.dtype != torch.bfloat16 or pool.dtype != torch.bfloat16:
        raise TypeError("x and the pool must be bf16")
    if W_fp8.dtype != torch.uint8 or tuple(W_fp8.shape) != (pool.d_out, pool.d_in) or not W_fp8.is_contiguous():
        raise ValueError("W_fp8 must be contiguous uint8 [d_out, d_in]")
    if w_scale.dtype != torch.float32 or w_scale.numel() != pool.d_out or not w_scale.is_contiguous():
        raise ValueError("w_scale must be contiguous float32 [d_out]")
    if x.dim() != 2 or x.shape[1] != pool.d_in or not x.is_contiguous():
        raise ValueError("x must be contiguous [T, d_in]")
    T = int(x.shape[0])
    y = out if out is not None else torch.empty((T, pool.d_out), dtype=pool.dtype, device=x.device)
    ws = workspace if workspace is not None else pool.workspace(T)
    n_seg = _segments(T, lora_on, seg_start, seg_adapter, seg_rank, seg_scale, token_index)
    _check(_lib.mlora_linear_fp8w(_ptr(x), _ptr(W_fp8), _ptr(w_scale), pool.handle,
                                  _ptr(_i32(seg_start, "seg_start")), _ptr(_i32(seg_adapter, "seg_adapter")),
                                  _ptr(_i32(seg_rank, "seg_rank")), _ptr(seg_scale),
                                  _ptr(_i32(token_index, "token_index")), T, n_seg, int(lora_on), _ptr(y),
                                  _ptr(ws), ws.numel(), _stream()), "mlora_linear_fp8w")
    return y


def linear_tokens(x, W, pool: Pool, token_adapter, adapter_scale, lora_on: int = 1, out=None,
                  workspace=None):
    """``mlora_linear_tokens``: the layer on an unsorted batch (library segments it)."""
    _check_xw(x, W, pool)
    T = int(x.shape[0])
    if lora_on and token_adapter is not None and token_adapter.numel() < T:
        raise ValueError("token_adapter must be [T]")
    y = out if out is not None else torch.empty((T, pool.d_out), dtype=pool.dtype, device=x.device)
    ws = workspace if workspace is not None else pool.workspace(T)
    _check(_lib.mlora_linear_tokens(_ptr(x), _ptr(W), pool.handle,
                                    _ptr(_i32(token_adapter, "token_adapter")), _ptr(adapter_scale),
                                    T, int(lora_on), _ptr(y), _ptr(ws), ws.numel(), _stream()),
           "mlora_linear_tokens")
    return y


def build_segments(token_adapter, adapter_scale, pool: Pool):
    """``mlora_build_segments``: canonical segments of an unsorted batch.
    Returns (token_index, seg_start, seg_adapter, seg_rank, seg_scale, n_seg) as
    device tensors sized for the worst case; n_seg is a 1-element tensor."""
    T = int(token_adapter.numel())
    dev = token_adapter.device
    ti = torch.empty(max(T, 1), dtype=torch.int32, device=dev)
    ss = torch.empty(T + 2, dtype=torch.int32, device=dev)
    sa = torch.empty(T + 1, dtype=torch.int32, device=dev)
    sr = torch.empty(T + 1, dtype=torch.int32, device=dev)
    sc = torch.empty(T + 1, dtype=torch.float32, device=dev)
    ns = torch.empty(1, dtype=torch.int32, device=dev)
    _check(_lib.mlora_build_segments(_ptr(_i32(token_adapter, "token_adapter")), _ptr(adapter_scale),
                                     T, pool.handle, _ptr(ti), _ptr(ss), _ptr(sa), _ptr(sr),
                                     _ptr(sc), _ptr(ns), _stream()), "mlora_build_segments")
    return ti[:T], ss, sa, sr, sc, ns


def token_map(seg_start, seg_adapter, n_tokens: int):
    """``mlora_token_map``: per sorted position, its segment and adapter id."""
    dev = seg_start.device
    ts = torch.empty(max(n_tokens, 1), dtype=torch.int32, device=dev)
    ta = torch.empty(max(n_tokens, 1), dtype=torch.int32, device=dev)
    n_seg = int(seg_adapter.numel())
    _check(_lib.mlora_token_map(_ptr(_i32(seg_start, "seg_start")), _ptr(_i32(seg_adapter, "seg_adapter")),
                                n_tokens, n_seg, _ptr(ts), _ptr(ta), _stream()), "mlora_token_map")
    return ts[:n_tokens], ta[:n_tokens]


def validate(pool: Pool, seg_start, seg_adapter, seg_rank=None, token_index=None, n_tokens=None,
             workspace=None) -> int:
    """``mlora_validate``: returns the status code (0 = valid); synchronizes."""
    T = int(n_tokens) if n_tokens is not None else int(seg_start[-1].item())
    ws = workspace if workspace is not None else pool.workspace(T)
    return int(_lib.mlora_validate(pool.handle, _ptr(_i32(seg_start, "seg_start")),
                                   _ptr(_i32(seg_adapter, "seg_adapter")),
                                   _ptr(_i32(seg_rank, "seg_rank")),
                                   _ptr(_i32(token_index, "token_index")), T,
                                   int(seg_adapter.numel()), _ptr(ws), ws.numel(), _stream()))


def merge_adapter(W, pool: Pool, adapter_id: int, scale: float, out=None):
    """``mlora_merge_adapter``: W + scale * B_a A_a into ``out`` (a new tensor
    if None; pass ``out=W`` to merge in place). A negative scale unmerges."""
    if W.dtype != pool.dtype or tuple(W.shape) != (pool.d_out, pool.d_in) or not W.is_contiguous():
        raise ValueError("W must be a contiguous [d_out, d_in] tensor of the pool's dtype")
    o = out if out is not None else torch.empty_like(W)
    if o.dtype != W.dtype or o.shape != W.shape or not o.is_contiguous():
        raise ValueError("out must match W")
    _check(_lib.mlora_merge_adapter(_ptr(W), _ptr(o), pool.handle, int(adapter_id), float(scale),
                                    _stream()), "mlora_merge_adapter")
    return o


# ---- the layer with what follows it -------------------------------------------
# These calls are short at small sizes: each tensor is looked at once, for its
# device, layout and pointer together.

_i32t, _f32t, _u8t, _bf16t = torch.int32, torch.float32, torch.uint8, torch.bfloat16
_device = torch._C._cuda_getDevice


def _refuse(t, dev, what):
    if t.get_device() != dev:
        raise ValueError(f"{what}: tensors must be on the current device")
    raise ValueError(f"{what}: tensors must be contiguous")


def _at(t, dev: int, what: str):
    """Pointer of a contiguous tensor of the current device (the call runs on
    that device's current stream), None for None."""
    if t is None:
        return None
    if t.get_device() != dev or not t.is_contiguous():
        _refuse(t, dev, what)
    return t.data_ptr()


def _at_i32(t, dev: int, what: str):
    if t is None:
        return None
    if t.dtype is not _i32t:
        raise TypeError(f"{what}: segment metadata must be int32")
    return _at(t, dev, what)


def _act_code(act: str, gated: bool) -> int:
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {sorted(ACTS)}")
    return code | _GATED if gated else code


def _epilogue_out(x, rows: int, d_out: int, gated: bool, bias, bias_shape, residual, out):
    """Checks an epilogue's tensors and returns y."""
    if gated:
        if d_out % 2:
            raise ValueError("a gated product needs an even number of weight rows")
        d_out //= 2
    shape, dt = (rows, d_out), x.dtype
    if bias is not None and (bias.dtype is not dt or bias.shape != bias_shape):
        raise ValueError(f"bias must be {list(bias_shape)} of x's dtype")
    if residual is not None and (residual.dtype is not dt or residual.shape != shape):
        raise ValueError(f"residual must be {list(shape)} of x's dtype")
    if out is None:
        return x.new_empty(shape)
    if out.dtype is not dt or out.shape != shape:
        raise ValueError(f"out must be {list(shape)} of x's dtype")
    return out


def linear_epilogue(x, W, pool: Pool, seg_start=None, seg_adapter=None, seg_rank=None, seg_scale=None,
                    lora_on: int = 1, token_index=None, bias=None, act: str = "none", gated: bool = False,
                    residual=None, w_scale=None, out=None, workspace=None):
    """``mlora_linear_epilogue``: act(W x + adapter term + bias) + residual; with
    ``gated``, W stacks gate over up rows and the result is act(gate) * up +
    residual. With ``w_scale``, W holds e4m3 codes (``mlora_linear_fp8w_epilogue``).
    ``residual`` may be ``out`` itself."""
    what, dev, d_out, d_in = "linear_epilogue", _device(), pool.d_out, pool.d_in
    if x.dtype is not pool.dtype or (w_scale is None and W.dtype is not pool.dtype):
        raise TypeError("x and W must have the pool's dtype")
    if x.dim() != 2 or x.shape[1] != d_in or W.shape != (d_out, d_in):
        raise ValueError("x must be [T, d_in] and W [d_out, d_in]")
    if w_scale is not None:
        if x.dtype is not _bf16t or W.dtype is not _u8t:
            raise TypeError("with w_scale, x and the pool must be bf16 and W uint8")
        if w_scale.dtype is not _f32t or w_scale.shape != (d_out,):
            raise ValueError("w_scale must be float32 [d_out]")
    if seg_scale is not None and seg_scale.dtype is not _f32t:
        raise TypeError("seg_scale must be float32")
    T = x.shape[0]
    n_seg = _segments(T, lora_on, seg_start, seg_adapter, seg_rank, seg_scale, token_index)
    code = _act_code(act, gated)
    y = _epilogue_out(x, T, d_out, gated, bias, (d_out,), residual, out)
    ws = workspace if workspace is not None else pool.workspace(T)
    epi = _Epilogue(_at(bias, dev, what), _at(residual, dev, what), code)
    rest = (pool.handle, _at_i32(seg_start, dev, what), _at_i32(seg_adapter, dev, what), _at_i32(seg_rank, dev, what),
            _at(seg_scale, dev, what), _at_i32(token_index, dev, what), T,
            n_seg, lora_on, ctypes.byref(epi), _at(y, dev, what),
            _at(ws, dev, what), ws.numel(), _raw_stream(dev))
    if w_scale is None:
        code = _lib.mlora_linear_epilogue(_at(x, dev, what), _at(W, dev, what), *rest)
    else:
        code = _lib.mlora_linear_fp8w_epilogue(_at(x, dev, what), _at(W, dev, what), _at(w_scale, dev, what), *rest)
    if code:
        raise MloraError(code, "mlora_linear_epilogue" if w_scale is None else "mlora_linear_fp8w_epilogue")
    return y


def linear_tokens_epilogue(x, W, pool: Pool, token_adapter, adapter_scale, lora_on: int = 1, bias=None,
                           act: str = "none", gated: bool = False, residual=None, out=None, workspace=None):
    """``mlora_linear_tokens_epilogue``: ``linear_epilogue`` on an unsorted batch."""
    what, dev, d_out = "linear_tokens_epilogue", _device(), pool.d_out
    _check_xw(x, W, pool)
    T = x.shape[0]
    code = _act_code(act, gated)
    y = _epilogue_out(x, T, d_out, gated, bias, (d_out,), residual, out)
    if adapter_scale is not None and (adapter_scale.dtype is not _f32t or adapter_scale.numel() != pool.capacity):
        raise TypeError("adapter_scale must be float32 [capacity]")
    if token_adapter is not None and token_adapter.numel() != T:
        raise ValueError("token_adapter must be [T]")
    ws = workspace if workspace is not None else pool.workspace(T)
    epi = _Epilogue(_at(bias, dev, what), _at(residual, dev, what), code)
    _check(_lib.mlora_linear_tokens_epilogue(_at(x, dev, what), _at(W, dev, what), pool.handle,
                                             _at_i32(token_adapter, dev, what), _at(adapter_scale, dev, what), T,
                                             int(lora_on), ctypes.byref(epi), _at(y, dev, what), _at(ws, dev, what),
                                             ws.numel(), _raw_stream(dev)), "mlora_linear_tokens_epilogue")
    return y


# ---- experts ---------------------------------------------------------------------

def route_workspace(n_tokens: int, n_experts: int, top_k: int, device="cuda") -> torch.Tensor:
    """A workspace for ``route`` on up to this many tokens."""
    n = _lib.mlora_route_workspace_bytes(n_tokens, n_experts, top_k)
    if n == 0:
        raise MloraError(STATUS_CODE["MLORA_ERR_SHAPE"], "mlora_route_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def route(logits, top_k: int, renormalize: bool = True, out=None, workspace=None):
    """``mlora_route``: top-k expert choice of logits [T, E] and its segments.
    Returns (expert [T, k], weight [T, k], token_index [T k], seg_start [E + 1],
    position [T, k]), views of one allocation, which any of them keeps; ``out`` is such a tuple
    to write into."""
    what, dev = "route", _device()
    if logits.dim() != 2:
        raise ValueError("logits must be [T, E]")
    code = _dtype_code(logits.dtype)
    T, E = logits.shape
    if not 1 <= top_k <= E:
        raise MloraError(STATUS_CODE["MLORA_ERR_SHAPE"], "mlora_route")
    at_logits, P = _at(logits, dev, what), T * top_k
    ws = workspace if workspace is not None else route_workspace(T, E, top_k, logits.device)
    if out is None:
        # one allocation, an output every `at` elements (16-byte aligned)
        at, slot, st = (P + 3) & ~3, (T, top_k), (top_k, 1)
        buf = logits.new_empty(4 * at + E + 1, dtype=_i32t)
        out = (buf.as_strided(slot, st, 0), buf.view(_f32t).as_strided(slot, st, at),
               buf.as_strided((P,), (1,), 2 * at), buf.as_strided((E + 1,), (1,), 4 * at),
               buf.as_strided(slot, st, 3 * at))
        p0 = buf.data_ptr()
        ptrs = (p0, p0 + 4 * at, p0 + 8 * at, p0 + 16 * at, p0 + 12 * at)
    else:
        want = ((P, _i32t), (P, _f32t), (P, _i32t), (E + 1, _i32t), (P, _i32t))
        if len(out) != len(want) or any(t.numel() != n or t.dtype is not dt for t, (n, dt) in zip(out, want)):
            raise ValueError("out must be (expert, weight, token_index, seg_start, position) of this batch")
        ptrs = [_at(t, dev, what) for t in out]
    code = _lib.mlora_route(at_logits, code, T, E, top_k, 1 if renormalize else 0, *ptrs, _at(ws, dev, what), ws.numel(),
                            _raw_stream(dev))
    if code:
        raise MloraError(code, "mlora_route")
    return out


def _check_experts(x, W, seg_start, w_scale):
    """Checks the operands of an expert product; returns (dtype code, E, d_out, d_in)."""
    dt = x.dtype
    code = _dtype_code(dt)
    if x.dim() != 2 or W.dim() != 3 or W.shape[2] != x.shape[1]:
        raise ValueError("x must be [rows, d_in] and W [E, d_out, d_in]")
    E, d_out, d_in = W.shape
    if w_scale is None:
        if W.dtype is not dt:
            raise TypeError("x and W must have one dtype")
    else:
        if W.dtype is not _u8t or dt is not _bf16t:
            raise TypeError("with w_scale, W must be uint8 and x bf16")
        if w_scale.dtype is not _f32t or w_scale.shape != (E, d_out):
            raise ValueError("w_scale must be float32 [E, d_out]")
    if seg_start.dtype is not _i32t or seg_start.numel() != E + 1:
        raise ValueError("seg_start must be int32 [E + 1]")
    return code, E, d_out, d_in


def experts_linear(x, W, seg_start, token_index=None, bias=None, act: str = "none", gated: bool = False,
                   w_scale=None, out=None):
    """``mlora_experts_linear``: act(W_e x[token_index[p]] + bias_e) for the sorted
    positions p of every expert e (``route``'s seg_start and token_index), gated as
    ``linear_epilogue``. Rows of the result behind seg_start[-1] are not written."""
    what, dev = "experts_linear", _device()
    code, E, d_out, d_in = _check_experts(x, W, seg_start, w_scale)
    n_rows = x.shape[0]
    n_pos = token_index.numel() if token_index is not None else n_rows
    epi = _Epilogue(_at(bias, dev, what), None, _act_code(act, gated))
    y = _epilogue_out(x, n_pos, d_out, gated, bias, (E, d_out), None, out)
    code = _lib.mlora_experts_linear(_at(x, dev, what), _at(W, dev, what), _at(w_scale, dev, what), code, n_rows, E, d_in,
                                     d_out, _at(seg_start, dev, what), _at_i32(token_index, dev, what), n_pos,
                                     ctypes.byref(epi), _at(y, dev, what), _raw_stream(dev))
    if code:
        raise MloraError(code, "mlora_experts_linear")
    return y


def experts_workspace(n_tokens: int, top_k: int, n_experts: int, d_out: int, dtype: torch.dtype,
                      device="cuda") -> torch.Tensor:
    """A workspace for ``experts_combine`` on up to this many tokens."""
    n = _lib.mlora_experts_workspace_bytes(n_tokens, top_k, n_experts, d_out, _dtype_code(dtype))
    if n == 0:
        raise MloraError(STATUS_CODE["MLORA_ERR_SHAPE"], "mlora_experts_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


def experts_combine(h, W, seg_start, position, weight, bias=None, residual=None, w_scale=None, out=None,
                    workspace=None):
    """``mlora_experts_combine``: residual[t] + sum_j weight[t, j] (W_e h[position[t, j]] + bias_e),
    with ``route``'s seg_start, position and weight. ``residual`` may be ``out`` itself."""
    what, dev = "experts_combine", _device()
    code, E, d_out, d_in = _check_experts(h, W, seg_start, w_scale)
    if position.dim() != 2 or position.dtype is not _i32t:
        raise ValueError("position must be int32 [T, k]")
    T, k = position.shape
    if weight.dtype is not _f32t or weight.shape != position.shape:
        raise ValueError("weight must be float32 [T, k]")
    if h.shape[0] != T * k:
        raise ValueError("h must hold a row per slot: [T k, d_in]")
    y = _epilogue_out(h, T, d_out, False, bias, (E, d_out), residual, out)
    ws = workspace if workspace is not None else experts_workspace(T, k, E, d_out, h.dtype, h.device)
    code = _lib.mlora_experts_combine(_at(h, dev, what), _at(W, dev, what), _at(w_scale, dev, what), code, T, k, E, d_in,
                                      d_out, _at(seg_start, dev, what), _at(position, dev, what), _at(weight, dev, what),
                                      _at(bias, dev, what), _at(residual, dev, what), _at(y, dev, what),
                                      _at(ws, dev, what), ws.numel(), _raw_stream(dev))
    if code:
        raise MloraError(code, "mlora_experts_combine")
    return y
