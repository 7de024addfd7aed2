"""B200-native routed-expert MoE feed-forward over 4-bit codebook weights.

The compute lives in ``libmoe_q4.so`` (hand-written sm_100a CUDA kernels
behind a C ABI, declared in ``include/moe_q4.h``); this package is a thin
binding.  Importing it does not load the library; the first call does, and
raises if the library was not built (there is no CPU fallback).
"""
from ._lib import (Layer, MlpI8, MoeQ4Error, Shared, add_norm, alloc_workspace, combine, dequant, forward, forward_ex,
                   forward_ex_workspace, forward_gated, forward_gated_workspace, forward_host, forward_host_async,
                   forward_host_workspace, forward_stages, forward_status, forward_workspace, i8_status, lib, linear_i8,
                   lloyd_fit, mlp_i8, mlp_i8_workspace, pack, quant_rows, route, router, router_workspace,
                   status_string)

__all__ = ["Layer", "MlpI8", "MoeQ4Error", "Shared", "add_norm", "alloc_workspace", "combine", "dequant", "forward",
           "forward_ex", "forward_ex_workspace", "forward_gated", "forward_gated_workspace", "forward_host",
           "forward_host_async", "forward_host_workspace", "forward_stages", "forward_status", "forward_workspace",
           "i8_status", "lib", "linear_i8", "lloyd_fit", "mlp_i8", "mlp_i8_workspace", "pack", "quant_rows", "route", "router",
           "router_workspace", "status_string"]
