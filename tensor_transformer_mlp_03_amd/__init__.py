"""libtpmlp: one tensor-parallel rank's share of the transformer MLP on MI355X (gfx950).

The compute path is the HIP library ``libtpmlp.so`` (C ABI in ``include/tpmlp.h``);
``_lib`` binds it with ctypes.  Importing the package does not load the library;
the first call does, and fails loudly if it has not been built.  ``block`` holds the
operators that stand around the MLP as objects (edge, expert route, gradient clipping), ``gated``
the gated MLP, dropout and products with 4-bit weights.
"""
from ._lib import (  # noqa: F401
    TpmlpError,
    lib,
    tpmlp_abi_version,
    tpmlp_bwd,
    tpmlp_bwd_workspace_bytes,
    tpmlp_clip_grad_norm,
    tpmlp_dropout_bwd,
    tpmlp_dropout_bwd_workspace_bytes,
    tpmlp_dropout_fwd,
    tpmlp_edge_bwd,
    tpmlp_edge_bwd_workspace_bytes,
    tpmlp_edge_fwd,
    tpmlp_edge_fwd_fp8,
    tpmlp_fp4_fwd,
    tpmlp_fp4_pack,
    tpmlp_fp4_packed_bytes,
    tpmlp_fp4_quantize,
    tpmlp_fwd,
    tpmlp_fwd_workspace_bytes,
    tpmlp_glu_bwd,
    tpmlp_glu_bwd_workspace_bytes,
    tpmlp_glu_fwd,
    tpmlp_glu_fwd_workspace_bytes,
    tpmlp_grad_clip,
    tpmlp_grad_sumsq,
    tpmlp_grad_workspace_bytes,
    tpmlp_kernel_name,
    tpmlp_route_combine,
    tpmlp_route_combine_bwd,
    tpmlp_route_dispatch,
    tpmlp_route_rows,
    tpmlp_route_sort,
    tpmlp_route_workspace_bytes,
    tpmlp_shard_sum,
    tpmlp_status_str,
    tpmlp_timing_begin,
    tpmlp_timing_end,
    tpmlp_timing_records,
    tpmlp_tp_bwd,
    tpmlp_tp_fwd,
    tpmlp_tp_workspace_bytes,
)
from .block import Edge, GradClip, Route  # noqa: F401
from .gated import Dropout, Fp4Linear, GatedMLP  # noqa: F401
