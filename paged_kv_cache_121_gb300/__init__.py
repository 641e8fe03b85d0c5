"""Paged KV cache hot path for NVIDIA GB300 (sm_103a).

The work happens in ``libpa.so`` (hand-written CUDA kernels and a C++ host
block manager, C ABI in ``include/pa.h``); this package is its binding.
"""
from .api import (  # noqa: F401
    PA_BF16, PA_ERR_CUDA, PA_ERR_INVALID_ARG, PA_ERR_NOT_FOUND, PA_ERR_OUT_OF_BLOCKS,
    PA_ERR_TIMEOUT, PA_ERR_UNSUPPORTED, PA_ERR_WORKSPACE, PA_F16, PA_F32, PA_OK, PA_ROPE_BANDS, PA_ROPE_HALF,
    PA_ROPE_INTERLEAVED, PA_ROPE_LINEAR, PA_ROPE_NTK, PA_ROPE_UNSCALED, PA_ROPE_YARN, BlockManager, PAError,
    pa_check_wait_timeout, pa_compute_slot_mapping, pa_copy_blocks, pa_cross_attention, pa_decode, pa_decode_append, pa_decode_contiguous, pa_decode_plan,
    pa_decode_shared_prefix,
    pa_decode_shared_prefix_workspace_size, pa_decode_splitk, pa_decode_static_scratch, pa_decode_weights,
    pa_decode_weights_workspace_size, pa_decode_workspace_size,
    pa_device_status, pa_evict, pa_lse_merge, pa_norm_rope, pa_norm_rope_and_cache, pa_norm_rope_backward,
    pa_norm_rope_backward_workspace_size, pa_prefill, pa_prefill_weights,
    pa_prefill_weights_workspace_size, pa_prefill_workspace_size, pa_reshape_and_cache, pa_rope, pa_rope_and_cache,
    pa_rope_frequencies, pa_swap_blocks,
)
from ._lib import library_path, load as load_library  # noqa: F401
