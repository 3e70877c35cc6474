"""Blockwise exact attention walked in ring order, per-shard partials with a
row-indexed log-sum-exp merge, shared-prefix fan-out attention, attention, weights,
eviction and upkeep of batches of paged sequences (in 8 bits too), and the norm and
rotation of the heads before it, for one NVIDIA GB300 (sm_103a).  The compute runs in libra.so (hand-written CUDA
kernels behind a C ABI, include/ra.h); this package is a thin binding."""
from .ra import (RAError, attn, attn_bwd, cache_append, cache_append_q8, cache_move, cache_read_q8, device_status, evict_select, fanout, fanout_noalloc, fanout_paged, fanout_plan, fanout_workspace_size, key_mass, layout_positions,  # noqa: F401
                 load, lse_merge, qk_norm_rope, qk_norm_rope_bwd, ring_partials, ring_shard_order, ring_walk, selftest_wait_timeout,
                 tile_launch_order, tree_attn, tree_attn_q8, tree_attn_q8_workspace_size, tree_attn_workspace_size)
