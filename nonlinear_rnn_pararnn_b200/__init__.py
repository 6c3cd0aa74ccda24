"""Newton-solved diag-mix sLSTM on NVIDIA B200 (sm_100a), and beside it a linear
attention with a decay for each head and the layer norm.

The compute lives in libslstm.so (CUDA, C ABI in include/slstm.h); this
package is its Python binding plus the seeded synthetic workloads.
"""
from .api import (layer_norm_backward, layer_norm_forward, linear_attention_backward,
                  linear_attention_backward_varlen, linear_attention_forward, linear_attention_forward_varlen,
                  linear_attention_step, linear_attention_workspace, newton_backward, newton_forward,
                  new_stats, preact_gemm, read_stats, scan_block4, sequential_step, workspace, workspace_size)

__all__ = ["layer_norm_backward", "layer_norm_forward", "linear_attention_backward",
           "linear_attention_backward_varlen", "linear_attention_forward", "linear_attention_forward_varlen",
           "linear_attention_step", "linear_attention_workspace", "newton_backward", "newton_forward",
           "new_stats", "preact_gemm", "read_stats", "scan_block4", "sequential_step", "workspace", "workspace_size"]
