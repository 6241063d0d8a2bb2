"""Seeded inputs of shared-prefix tree attention, used by its CPU and GPU tests."""
import numpy as np

from tree_verify_attention_jf_b200 import synth

PAGE = 16


def shared_inputs(seed, hq, hkv, groups, nodes, suffixes, poison=True, scale=0.5):
    """groups: [(sequences, shared tokens)]; nodes and own tokens behind the shared ones per sequence.  Returns
    (AttentionInputs, group_offsets, shared_lens).  With `poison` the entries that must not be read (the shared part
    of every row but a group's first) are -1."""
    rng = np.random.default_rng(seed)
    count = [n for n, _ in groups]
    B = sum(count)
    offs = np.concatenate([[0], np.cumsum(count)]).astype(np.int32)
    shared = np.array([s for _, s in groups], np.int32)
    of = np.repeat(np.arange(len(groups)), count)
    prefix = [int(shared[of[b]]) + int(suffixes[b]) for b in range(B)]
    need = [(prefix[b] + nodes[b] + PAGE - 1) // PAGE for b in range(B)]
    whole = [int(s) // PAGE for s in shared]
    total = sum(w for w, n in zip(whole, count) if n) + sum(max(0, need[b] - whole[of[b]]) for b in range(B)) + 2
    ids = rng.permutation(total).astype(np.int32)
    bt = np.full((B, max(need + [1]) + 1), -1, np.int32)
    at = 0
    for g, w in enumerate(whole):
        if count[g] == 0:
            continue
        common = ids[at:at + w]
        at += w
        for b in range(offs[g], offs[g + 1]):
            if b == offs[g] or not poison:
                bt[b, :w] = common
            n = max(0, need[b] - w)
            bt[b, w:w + n] = ids[at:at + n]
            at += n
    parents = [synth.uniform_parent_tree(rng, n, 12) for n in nodes]
    to = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
    T = int(to[-1])
    draw = lambda *s: synth.bf16_round(rng.standard_normal(s, dtype=np.float32) * np.float32(scale))
    inp = synth.AttentionInputs(q=draw(T, hq, 128), k_cache=draw(total, PAGE, hkv, 128),
                                v_cache=draw(total, PAGE, hkv, 128), block_table=bt,
                                prefix_lens=np.array(prefix, np.int32), tree_offsets=to,
                                parent=np.concatenate(parents).astype(np.int32) if T else np.zeros(0, np.int32),
                                sm_scale=128 ** -0.5, num_q_heads=hq, num_kv_heads=hkv)
    return inp, offs, shared


def unused_slots(inp, group_offsets, shared_lens):
    """bool [pages, 16]: slots that no sequence reads."""
    unused = np.ones(inp.k_cache.shape[:2], bool)
    for g, s in enumerate(shared_lens):
        for b in range(group_offsets[g], group_offsets[g + 1]):
            n = int(inp.tree_offsets[b + 1] - inp.tree_offsets[b])
            if n == 0:
                continue
            w = int(s) // PAGE
            for t in range(int(inp.prefix_lens[b]) + n):
                row = group_offsets[g] if t // PAGE < w else b
                unused[inp.block_table[row, t // PAGE], t % PAGE] = False
    return unused
