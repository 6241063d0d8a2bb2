"""One decoding step of several sampled continuations of two prompts, as the calls are used together: the tree tokens'
K/V appended to the cache, tree attention over the shared prefixes, the sampled acceptance walk, the commit of the
accepted path, and a single-token step behind it with jf_sample; eager and replayed from one CUDA graph, each stage
against its oracle."""
import numpy as np
import pytest
import torch

from oracle.commit_kv import commit_kv as oracle_commit
from oracle.kv_append import tree_kv_append as oracle_append
from oracle.sampling import accept_sampled as oracle_accept, sample_row
from oracle.shared_prefix import tree_attention_shared as oracle_shared
from tests.gpu_util import compare
from tests.shared_cases import shared_inputs
from tree_verify_attention_jf_b200 import api, synth

pytestmark = pytest.mark.gpu
HQ, HKV, V, D, THETA = 8, 2, 5000, 6, 1e6


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def rooted_tree(rng, n):
    return np.array([-1] + [int(rng.integers(max(0, i - 4), i)) for i in range(1, n)], np.int32)


def test_a_step_of_sampled_continuations():
    rng = np.random.default_rng(0)
    B, N = 5, 12
    inp, go, sl = shared_inputs(50, HQ, HKV, [(3, 200), (2, 77)], [N] * B, [40, 0, 130, 9, 33])
    parent = np.stack([rooted_tree(rng, N) for _ in range(B)])
    token = rng.integers(0, V, (B, N)).astype(np.int32)
    depth = np.zeros((B, N), np.int64)
    for i in range(1, N):
        depth[:, i] = depth[np.arange(B), parent[:, i]] + 1
    logits = rng.standard_normal((B, N, V), dtype=np.float32) * np.float32(2)
    for b in range(B):
        for i in range(1, N):
            row = logits[b, parent[b, i]]
            row[token[b, i]] = row.max() + 3
    u = rng.random((B, D + 1), dtype=np.float32)
    par = (np.full(B, 0.8, np.float32), np.full(B, 40, np.int32), np.full(B, 0.95, np.float32),
           np.full(B, 0.02, np.float32))
    draw = lambda *s: synth.to_bf16_tensor(rng.standard_normal(s, dtype=np.float32) * np.float32(0.5)).cuda()
    T = B * N
    kn, vn, q0 = draw(T, HKV, 128), draw(T, HKV, 128), draw(T, HQ, 128)
    kc0, vc0 = (synth.to_bf16_tensor(c).cuda() for c in (inp.k_cache, inp.v_cache))
    # the append and the commit take block tables that agree on the shared pages
    bt_full = inp.block_table.copy()
    for g in range(2):
        bt_full[go[g]:go[g + 1], :sl[g] // 16] = bt_full[go[g], :sl[g] // 16]
    bt, pl, to = i32(np.maximum(bt_full, 0)), i32(inp.prefix_lens), i32(inp.tree_offsets)
    dpar, dtok, ddep = i32(parent), i32(token), i32(depth.reshape(-1))
    dgo, dsl, dlog, du = i32(go), i32(sl), torch.from_numpy(logits).cuda(), torch.from_numpy(u).cuda()
    how = [torch.from_numpy(a).cuda() for a in par]
    k, v, q = kc0.clone(), vc0.clone(), q0.clone()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = api.SharedAttentionWorkspace(T, HQ, k.device)
    out, lse = torch.empty_like(q), torch.empty(T, HQ, device="cuda")
    walk = dict(accepted_len=torch.empty(B, dtype=torch.int32, device="cuda"),
                path=torch.empty(B, D + 1, dtype=torch.int32, device="cuda"),
                bonus=torch.empty(B, dtype=torch.int32, device="cuda"), logprob=torch.empty(B, D + 1, device="cuda"))
    newp = torch.empty(B, dtype=torch.int32, device="cuda")
    nxt = dict(token=torch.empty(B, dtype=torch.int32, device="cuda"), logprob=torch.empty(B, device="cuda"))

    def step():
        api.tree_kv_append(kn, vn, k, v, bt, pl, to, ddep, THETA, q=q, dev_status=status)
        api.tree_attention_shared(q, k, v, bt, pl, to, dpar.view(-1), dgo, dsl, inp.sm_scale, out=out, lse=lse,
                                  workspace=ws, dev_status=status)
        api.accept_sampled(dtok, dpar, dlog, du, how[0], D, *how[1:], out=walk, dev_status=status)
        api.commit_kv(k, v, bt, pl, to, walk["path"], walk["accepted_len"], new_prefix_lens=newp, dev_status=status)
        api.sample(dlog[:, 0], du[:, 0].contiguous(), *how, out=nxt, dev_status=status)

    def check():
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        rk, rv, rq = oracle_append(f64(kn), f64(vn), f64(q0), f64(kc0), f64(vc0), bt.cpu().numpy(), inp.prefix_lens,
                                   inp.tree_offsets, depth.reshape(-1), THETA)
        b16 = lambda x: synth.bf16_round(x.astype(np.float32))
        ref, lref = oracle_shared(b16(rq), b16(rk), b16(rv), bt.cpu().numpy(), inp.prefix_lens, inp.tree_offsets,
                                  parent.reshape(-1), go, sl, inp.sm_scale)
        compare(out.float().cpu().numpy(), ref, lse.cpu().numpy(), lref)
        acc, path, bonus, _ = oracle_accept(token, parent, logits, u, D, *par)
        assert np.array_equal(walk["accepted_len"].cpu().numpy(), acc) and acc.max() > 0
        assert np.array_equal(walk["path"].cpu().numpy(), path)
        assert np.array_equal(walk["bonus"].cpu().numpy(), bonus)
        ck, cv, cp = oracle_commit(b16(rk), b16(rv), bt.cpu().numpy(), inp.prefix_lens, inp.tree_offsets, path, acc)
        assert np.array_equal(newp.cpu().numpy(), cp)
        # the accepted slots; a rotated K may differ from the oracle's by the rounding of a tie
        for b in range(B):
            for s in range(int(inp.prefix_lens[b]), int(cp[b])):
                pg, off = int(bt_full[b, s // 16]), s % 16
                assert np.allclose(f64(k)[pg, off], ck[pg, off], rtol=2 ** -7, atol=1e-6)
                assert np.array_equal(f64(v)[pg, off], cv[pg, off])
        for b in range(B):
            want, lp = sample_row(logits[b, 0], float(u[b, 0]), *(float(a[b]) if a.dtype != np.int32 else int(a[b])
                                                                  for a in par))
            assert int(nxt["token"][b]) == want and abs(float(nxt["logprob"][b]) - lp) <= 2 ** -20

    step()
    check()
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        step()
    for _ in range(2):
        k.copy_(kc0)
        v.copy_(vc0)
        q.copy_(q0)
        out.fill_(float("nan"))
        g.replay()
        check()
