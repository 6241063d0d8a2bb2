"""Oracle: tree attention of a batch whose sequences share prefixes.

The pages verify one continuation a prompt ([JF] technical summary section 2, tree-causal mask; section 3, paged cache).
Reading for several: groups of consecutive sequences have their first shared_lens[g] tokens in common, and with S that
length rounded down to whole pages every sequence of the group reads slots [0, S) through the block-table row of the
group's first sequence; apart from where those slots are read it is the attention of :mod:`oracle.tree_attention`.

Pinned by tests/test_oracle_shared.py.
"""
from __future__ import annotations

import numpy as np

from .fp8_kv import tree_attention_fp8
from .tree_attention import PAGE_SIZE, tree_attention


def effective_table(block_table, group_offsets, shared_lens):
    """The block table with every group's shared entries taken from its first row."""
    bt = np.array(block_table, copy=True)
    for g, s in enumerate(shared_lens):
        first, n = int(group_offsets[g]), int(s) // PAGE_SIZE
        for b in range(first, int(group_offsets[g + 1])):
            bt[b, :n] = bt[first, :n]
    return bt


def tree_attention_shared(q, k_cache, v_cache, block_table, prefix_lens, tree_offsets, parent, group_offsets,
                          shared_lens, sm_scale, num_kv_heads=None, rows=None, scales=None):
    """(out, lse) in float64; with scales = (k_scale, v_scale) the caches are E4M3 codes."""
    bt = effective_table(block_table, group_offsets, shared_lens)
    if scales is not None:
        return tree_attention_fp8(q, k_cache, v_cache, *scales, bt, prefix_lens, tree_offsets, parent, sm_scale,
                                  num_kv_heads, rows)
    return tree_attention(q, k_cache, v_cache, bt, prefix_lens, tree_offsets, parent, sm_scale, num_kv_heads, rows)
