"""One data-parallel rank's sharded ZeRO/FSDP update on AMD MI355X (gfx950).

The compute lives in libzs.so (hand-written HIP kernels behind the C ABI of
include/zs.h); this package is its thin Python binding. Importing the package
does not load the library; the first call does, and fails loudly if it has
not been built.
"""
from .api import (  # noqa: F401
    Dim0Table,
    ParamTable,
    ShardedStep,
    ZsArgumentError,
    ZsError,
    zs_accumulate_grads,
    zs_accumulate_local,
    zs_activation_pack,
    zs_activation_unpack,
    zs_adamw_step,
    zs_cast_for_gather,
    zs_clip_coefficient,
    zs_copy_out,
    zs_copy_out_dim0,
    zs_dim0_layout,
    zs_embed_backward,
    zs_embed_forward,
    zs_embed_workspace_bytes,
    zs_flat_layout,
    zs_layer_norm_backward,
    zs_layer_norm_forward,
    zs_layer_norm_workspace_bytes,
    zs_linear_cross_entropy_backward,
    zs_linear_cross_entropy_forward,
    zs_linear_cross_entropy_workspace_bytes,
    zs_pack_shard,
    zs_pack_shard_dim0,
    zs_reduce_grads,
    zs_reduce_grads_noalloc,
    zs_rms_norm_backward,
    zs_rms_norm_forward,
    zs_rms_norm_workspace_bytes,
    zs_sharded_step,
    zs_version,
    zs_workspace_bytes,
)
from ._lib import LIB_PATH, load  # noqa: F401
