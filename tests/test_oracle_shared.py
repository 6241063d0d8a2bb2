"""Pins of the shared-prefix attention oracle (oracle/shared_prefix.py) against the attention of every sequence by
itself on a gathered, contiguous cache (torch's own attention for chain trees), and its group bookkeeping."""
import numpy as np
import torch

from oracle.shared_prefix import effective_table, tree_attention_shared
from oracle.tree_attention import tree_attention_inputs
from tests.shared_cases import shared_inputs, unused_slots
from tree_verify_attention_jf_b200 import synth


def run(inp, go, sl, **kw):
    return tree_attention_shared(inp.q, inp.k_cache, inp.v_cache, inp.block_table, inp.prefix_lens, inp.tree_offsets,
                                 inp.parent, go, sl, inp.sm_scale, inp.num_kv_heads, **kw)


def test_effective_table_by_hand():
    bt = np.array([[5, 6, 7, 1], [-1, -1, 8, 2], [9, 3, 4, 0], [-1, 10, 11, 12]])
    got = effective_table(bt, [0, 2, 4], [35, 16])
    assert got.tolist() == [[5, 6, 7, 1], [5, 6, 8, 2], [9, 3, 4, 0], [9, 10, 11, 12]]
    assert effective_table(bt, [0, 4], [15]).tolist() == bt.tolist()


def test_agreeing_tables_give_plain_tree_attention():
    inp, go, sl = shared_inputs(0, 4, 2, [(3, 70), (2, 16)], [3, 1, 5, 4, 2], [0, 20, 3, 40, 1], poison=False)
    out, lse = run(inp, go, sl)
    ref, lref = tree_attention_inputs(inp)
    assert np.array_equal(out, ref) and np.array_equal(lse, lref)


def test_chains_equal_causal_attention_on_prompt_plus_own_text():
    inp, go, sl = shared_inputs(1, 2, 1, [(2, 50), (1, 33)], [4, 3, 5], [10, 0, 7])
    inp.parent[:] = np.concatenate([synth.chain_tree(n) for n in (4, 3, 5)])
    out, _ = run(inp, go, sl)
    for b, first in ((0, 0), (1, 0), (2, 2)):
        n = int(inp.tree_offsets[b + 1] - inp.tree_offsets[b])
        P = int(inp.prefix_lens[b])
        w = int(sl[0 if b < 2 else 1]) // 16
        pages = np.concatenate([inp.block_table[first, :w], inp.block_table[b, w:(P + n + 15) // 16]])
        k = inp.k_cache[pages].reshape(-1, 1, 128)[:P + n, 0]
        v = inp.v_cache[pages].reshape(-1, 1, 128)[:P + n, 0]
        o0 = int(inp.tree_offsets[b])
        mask = torch.tril(torch.ones(n, P + n, dtype=torch.bool), diagonal=P)
        for h in range(2):
            ref = torch.nn.functional.scaled_dot_product_attention(
                torch.from_numpy(inp.q[o0:o0 + n, h]).double()[None, None], torch.from_numpy(k).double()[None, None],
                torch.from_numpy(v).double()[None, None], attn_mask=mask, scale=inp.sm_scale)[0, 0].numpy()
            assert np.allclose(out[o0:o0 + n, h], ref, atol=1e-12)


def test_slots_named_unused_do_not_matter():
    inp, go, sl = shared_inputs(2, 4, 2, [(3, 40), (1, 0), (2, 64)], [3, 0, 5, 2, 1, 7], [0, 9, 30, 4, 0, 0])
    out, _ = run(inp, go, sl)
    un = unused_slots(inp, go, sl)
    assert un.any()
    inp.k_cache[un] = 1e3
    inp.v_cache[un] = 1e3
    assert np.array_equal(run(inp, go, sl)[0], out)
