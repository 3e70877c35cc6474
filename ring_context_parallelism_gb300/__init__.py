"""Blockwise exact attention walked in ring order, per-shard partials with a
row-indexed log-sum-exp merge, shared-prefix fan-out attention, and attention,
weights, eviction and upkeep of batches of paged sequences, for one NVIDIA GB300
(sm_103a).  The compute runs in libra.so (hand-written CUDA
kernels behind a C ABI, include/ra.h); this package is a thin binding."""
from .ra import (RAError, attn, attn_bwd, cache_append, cache_move, device_status, evict_select, fanout, fanout_noalloc, fanout_paged, fanout_plan, fanout_workspace_size, key_mass, layout_positions,  # noqa: F401
                 load, lse_merge, ring_partials, ring_shard_order, ring_walk, selftest_wait_timeout,
                 tile_launch_order, tree_attn, tree_attn_workspace_size)
