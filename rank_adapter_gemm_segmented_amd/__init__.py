"""MI355X (gfx950) multi-LoRA segmented linear layer.

``y_i = W x_i + scale_s * B_a (A_a x_i)`` over a batch partitioned into
per-adapter segments, with a ``lora_on`` switch for the LoRA-off drafter pass.
The layer also takes a bias, an activation, a gate and a residual (``*_epilogue``),
and a mixture of experts runs through ``route``, ``experts_linear`` and
``experts_combine``. The work runs in hand-written HIP kernels behind the C ABI of
``include/mlora.h`` (``csrc/``); this package is the thin Python binding.
"""
from .binding import (ACTS, LIB_PATH, MLORA_BF16, MLORA_F32, STATUS, STATUS_CODE, MloraError, Pool,
                      build_segments, experts_combine, experts_linear, experts_workspace, library,
                      linear, linear_epilogue, linear_fp8w, linear_noalloc, linear_tokens,
                      linear_tokens_epilogue, merge_adapter, route, route_workspace, token_map, validate)

__all__ = ["ACTS", "LIB_PATH", "MLORA_BF16", "MLORA_F32", "STATUS", "STATUS_CODE", "MloraError", "Pool",
           "build_segments", "experts_combine", "experts_linear", "experts_workspace", "library",
           "linear", "linear_epilogue", "linear_fp8w", "linear_noalloc", "linear_tokens",
           "linear_tokens_epilogue", "merge_adapter", "route", "route_workspace", "token_map", "validate"]
