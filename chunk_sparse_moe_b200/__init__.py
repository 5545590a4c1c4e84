"""BlockFFN chunk-union layer forward on B200 (sm_100a).

Python binding of libblockffn.so: ``route``, ``chunk_union``, ``forward``, top-k
routing with its gradient (``route_topk``, ``route_topk_backward``) and the products in
8-bit integers (``quantize_int8``, ``int8_linear``, ``forward_int8``) take CUDA torch tensors, check them, and pass raw device pointers and the current
CUDA stream to the C ABI (include/blockffn.h).  All arithmetic runs in the
library's kernels; PyTorch only provides device memory and streams.
"""
from .api import (BlockFFNError, Workspace, chunk_union, debug_set_trace, debug_skip_flag, device_status,
                  forward, forward_int8, int8_linear,
                  num_sms, quantize_int8, residual_layernorm, route, route_topk, route_topk_backward,
                  set_wait_limit_ns, version, workspace_bytes)

__all__ = ["BlockFFNError", "Workspace", "chunk_union", "debug_set_trace", "debug_skip_flag", "residual_layernorm",
           "device_status",
           "forward", "forward_int8", "int8_linear", "num_sms", "quantize_int8", "route", "route_topk", "route_topk_backward",
           "set_wait_limit_ns", "version", "workspace_bytes"]
