"""Nexus Sampling eviction step for AMD Instinct MI355X (gfx950).

The work runs in libnexus.so (HIP kernels behind the C ABI of include/nexus.h);
this package is its build script and a thin torch-facing binding.  Importing
the binding fails loudly when the library has not been built.
"""

from ._lib import (  # noqa: F401
    NX_OK, NX_EINVAL, NX_EALIAS, NX_EWORKSPACE, NX_EUNSUPPORTED, NX_ENONFINITE, NX_EHIP,
    NX_BF16, NX_F32, NX_COMPACT_COPY, NX_COMPACT_INPLACE, NX_HEADS_UNIFORM, NX_HEADS_GIVEN,
    NX_HEADS_ALLOC, NX_MAX_ALLOC_HEADS, NX_SCRATCH_BYTES, NxDesc, NxUnit, NexusError, LIB_PATH,
    load, status_str, check, NX_CACHE_E4M3, NX_CACHE_I8, NX_CACHE_BLOCK, NX_ROPE_HALF, NX_ROPE_PAIRS,
    NxRows, NxRope, NxPaged,
)
from .api import (  # noqa: F401
    NexusConfig, TOPK, workspace_bytes, new_workspace, nx_evict_step, nx_evict_step_noalloc, nx_nexus_weights,
    nx_reservoir_select, nx_kv_compact, nx_head_budgets, make_units, nx_evict_batch,
    nx_read_device_status,
    profile_enable, profile_read,
)
from .paged import (  # noqa: F401
    PagedCache, Rope, rope_table, new_paged_cache, paged_workspace_bytes, new_paged_workspace,
    nx_qk_norm_rope, nx_paged_append, nx_paged_attn, nx_paged_gather,
)
from .decode import DecodeCache, EventBuffers  # noqa: F401
