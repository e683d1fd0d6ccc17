"""B200-native (sm_100a) hot path of the Orthrus dual-view diffusion decode step.

The compute lives in ``liborthrus.so`` (C ABI, include/orthrus.h); this package
holds its ctypes binding (``binding``), the in-tree build (``build``), the
seeded synthetic workloads (``workloads``) and a device-resident decode-step
driver (``step``).
"""
from .binding import (AR, BF16, DIFF, F16, F32, ROPE_HALF, ROPE_INTERLEAVED, ROPE_LINEAR,  # noqa: F401
                      ROPE_NTK, ROPE_PLAIN, ROPE_YARN, OrthrusError, orthrus_attn,
                      orthrus_attn_path, orthrus_attn_workspace_size, orthrus_consensus,
                      orthrus_consensus_workspace_size, orthrus_fp8_matmul, orthrus_kv_commit,
                      orthrus_paged_attn, orthrus_paged_attn_workspace_size, orthrus_quantize_fp8,
                      orthrus_rmsnorm, orthrus_rope, orthrus_rope_append, orthrus_rope_table,
                      orthrus_version, orthrus_write_block)
