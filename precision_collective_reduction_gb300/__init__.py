"""GB300-native low-precision (FP8) collective reduction and DDA flat / tree
allreduce, with N ranks emulated as N buffers in one GPU's HBM.

The compute path is liblpcoll.so (hand-written CUDA for sm_103a behind the C
ABI in include/lpcoll.h); this package is its binding (``_binding``, and
``layers`` for the operators around the collectives of a layer), an
in-place allreduce facade (``allreduce``), the build step (``build``) and the
seeded workload generators (``workloads``).
"""
from ._binding import (BF16, BLOCK, E4M3, E5M2, F32, MAX_RANKS, VARIANT_BLOCKS,
                       LpcollError, all_gather_sim, all_to_all_sim, dda_flat_sim,
                       dda_flat_sim_noalloc, dda_tree_sim, lib, lp_dequantize,
                       lp_dequantize_fmt, lp_quantize, lp_quantize_fmt, lp_reduce,
                       lp_reduce_fmt, lpcoll_host_allreduce,
                       lpcoll_host_workspace_bytes, nblocks, reduce_scatter_sim,
                       shard_len, status_string)
from .allreduce import Workspace, allreduce_sim, choose
from .layers import (GATE_CHANNEL, GATE_FULL, GATE_NONE, GATE_TOKEN, MAX_EXPERTS, MAX_HIDDEN,
                     MAX_TOPK, expert_balance, expert_balance_backward,
                     expert_balance_workspace_bytes, expert_combine, expert_combine_backward,
                     expert_dispatch, expert_dispatch_backward, expert_route,
                     expert_route_backward, expert_sort, expert_sort_workspace_bytes,
                     layer_norm, layer_norm_backward, layer_norm_backward_workspace_bytes,
                     residual_dropout, residual_dropout_backward,
                     residual_dropout_backward_workspace_bytes, residual_norm,
                     residual_norm_backward, residual_norm_backward_workspace_bytes,
                     token_embed, token_embed_backward, token_embed_backward_workspace_bytes)

__all__ = ["BF16", "BLOCK", "F32", "MAX_RANKS", "LpcollError", "Workspace",
           "all_gather_sim", "all_to_all_sim", "allreduce_sim", "choose",
           "dda_flat_sim", "dda_flat_sim_noalloc", "dda_tree_sim", "lib",
           "lp_dequantize", "lp_quantize", "lp_reduce", "nblocks", "E4M3", "E5M2",
           "VARIANT_BLOCKS", "lp_quantize_fmt", "lp_dequantize_fmt", "lp_reduce_fmt",
           "lpcoll_host_allreduce", "lpcoll_host_workspace_bytes",
           "reduce_scatter_sim", "shard_len", "status_string",
           "GATE_CHANNEL", "GATE_FULL", "GATE_NONE", "GATE_TOKEN", "MAX_EXPERTS",
           "MAX_HIDDEN", "MAX_TOPK", "expert_combine", "expert_combine_backward",
           "expert_dispatch", "expert_dispatch_backward", "expert_route",
           "expert_route_backward", "expert_sort", "expert_sort_workspace_bytes",
           "residual_norm", "residual_norm_backward",
           "residual_norm_backward_workspace_bytes", "expert_balance",
           "expert_balance_backward", "expert_balance_workspace_bytes", "layer_norm",
           "layer_norm_backward", "layer_norm_backward_workspace_bytes", "residual_dropout",
           "residual_dropout_backward", "residual_dropout_backward_workspace_bytes",
           "token_embed", "token_embed_backward", "token_embed_backward_workspace_bytes"]
