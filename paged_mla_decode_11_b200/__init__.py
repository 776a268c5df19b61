"""B200-native paged MLA decode: a C-ABI CUDA library (libpagedmla.so) and its binding.

The decode path -- split-KV scheduler, page-gather loader, fused QK^T / online softmax /
PV kernel and log-sum-exp combine -- runs in hand-written sm_100a kernels; ``ops`` only
marshals arguments.  So do the operators of a serving step around it: rotary positions, the
cache write and read-back, and the verification of drafted tokens.  ``workloads`` draws seeded
synthetic inputs.
"""

from .ops import (  # noqa: F401
    MlaError,
    device_sm_count,
    flash_mla_with_kvcache,
    get_mla_metadata,
    load_library,
    metadata_size,
    mla_cache_read,
    mla_cache_read_fp8,
    mla_cache_slots,
    mla_cache_write,
    mla_cache_write_fp8,
    mla_combine,
    mla_decode_paged,
    mla_decode_paged_fp8_rows,
    mla_rope,
    mla_verify_draft,
    new_workspace,
    num_parts_for,
    query_status,
    rope_frequencies,
    rope_magnitude,
    watchdog_selftest,
    workspace_size,
)
