"""GPU parity of jf_tree_attention_shared (bf16 and 8-bit caches) against the float64 oracle, with the bounds of the
other attention tests (tests/gpu_util.py: the kernel rounds at the same two places)."""
import dataclasses

import numpy as np
import pytest
import torch

from oracle.shared_prefix import tree_attention_shared as oracle_shared
from tests.gpu_util import compare, to_dev
from tests.shared_cases import shared_inputs, unused_slots
from tree_verify_attention_jf_b200 import _lib, api, synth

pytestmark = pytest.mark.gpu
SCALES = (1.0 / 128, 1.0 / 64)


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def run(case, ws=None, status=None, fp8=False, d=None, out=None, stream=None):
    inp, go, sl = case
    d = d or to_dev(inp)
    T, Hq = inp.q.shape[:2]
    lse = torch.full((T, Hq), float("nan"), device="cuda")
    out = torch.full_like(d["q"], float("nan")) if out is None else out
    kw = dict(out=out, lse=lse, workspace=ws, dev_status=status, stream=stream)
    rest = (d["block_table"], d["prefix_lens"], d["tree_offsets"], d["parent"], i32(go), i32(sl), inp.sm_scale)
    if fp8:
        codes = [torch.from_numpy(synth.e4m3_cache(c, s)).cuda() for c, s in zip((inp.k_cache, inp.v_cache), SCALES)]
        api.tree_attention_shared_fp8(d["q"], *codes, *SCALES, *rest, **kw)
    else:
        api.tree_attention_shared(d["q"], d["k_cache"], d["v_cache"], *rest, **kw)
    torch.cuda.synchronize()
    return out.float().cpu().numpy(), lse.cpu().numpy()


def oracle(case, fp8=False, rows=None):
    inp, go, sl = case
    k, v = inp.k_cache, inp.v_cache
    if fp8:
        k, v = synth.e4m3_cache(k, SCALES[0]), synth.e4m3_cache(v, SCALES[1])
    return oracle_shared(inp.q, k, v, inp.block_table, inp.prefix_lens, inp.tree_offsets, inp.parent, go, sl,
                         inp.sm_scale, inp.num_kv_heads, rows=rows, scales=SCALES if fp8 else None)


def check(case, fp8=False, **kw):
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out, lse = run(case, status=st, fp8=fp8, **kw)
    assert int(st.item()) == 0
    ref, lref = oracle(case, fp8)
    return compare(out, ref, lse, lref)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("group", [1, 2, 4, 8, 16])
@pytest.mark.parametrize("shared", [0, 1, 15, 16, 17, 128, 144, 1000])
def test_head_groups_and_shared_lengths(fp8, group, shared):
    rng = np.random.default_rng(shared * 31 + group)
    nodes = rng.integers(1, 20, 5)
    case = shared_inputs(shared + group, 2 * group, 2, [(3, shared), (2, shared // 2)], nodes,
                         rng.integers(0, 200, 5))
    check(case, fp8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,shared,suffix", [(1, 300, 0), (2, 64, 1), (33, 4096, 40), (64, 700, 300)])
def test_single_tokens(fp8, B, shared, suffix):
    rng = np.random.default_rng(B)
    check(shared_inputs(B, 8, 2, [(B, shared)], [1] * B, rng.integers(0, suffix + 1, B)), fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_few_rows_at_the_edges_of_their_kernel(fp8):
    # 16 and 17 rows, 1024 and 1025 own keys (nodes included), the last page full, begun and empty but for one slot
    suffix = [1023, 1024, 1008 - 3, 15, 0, 14, 1019, 1000]
    nodes = [1, 1, 3, 1, 4, 2, 4, 5]
    check(shared_inputs(40, 8, 2, [(5, 48), (3, 33)], nodes, suffix), fp8)
    check(shared_inputs(41, 16, 1, [(2, 0), (6, 160)], [1] * 8, suffix), fp8)
    check(shared_inputs(42, 2, 2, [(8, 7)], [16, 17, 1, 15, 0, 16, 2, 16], suffix), fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_large_trees_ragged_groups_and_empty_sequences(fp8):
    nodes = [256, 0, 1, 255, 130, 0, 17, 64, 0]
    suffix = [0, 5, 130, 16, 1, 0, 333, 48, 7]
    check(shared_inputs(5, 16, 4, [(4, 513), (1, 200), (1, 64), (0, 0), (2, 96), (1, 32)], nodes, suffix), fp8)


def test_long_prefix_cut_over_every_block():
    # one unit of 1 kv head: its shared keys are cut over all SMs
    check(shared_inputs(6, 8, 1, [(4, 40000)], [7, 7, 7, 7], [3, 0, 100, 16]))


def test_many_groups_and_many_sequences():
    rng = np.random.default_rng(7)
    check(shared_inputs(7, 2, 1, [(2, int(s)) for s in rng.integers(0, 90, 340)], rng.integers(0, 4, 680),
                        rng.integers(0, 40, 680)))
    check(shared_inputs(8, 2, 1, [(1023, 48)], rng.integers(0, 3, 1023), rng.integers(0, 20, 1023)))


def test_nothing_shared_equals_tree_attention():
    case = shared_inputs(9, 8, 2, [(1, 0)] * 4, [20, 3, 70, 1], [100, 37, 500, 0])
    inp = case[0]
    got, lse = run(case)
    d = to_dev(inp)
    ref = api.tree_attention(d["q"], d["k_cache"], d["v_cache"], d["block_table"], d["prefix_lens"], d["tree_offsets"],
                             d["parent"], inp.sm_scale).float().cpu().numpy()
    # the same float32 states, split at other places and rounded once more or less: a bf16 step either way
    assert np.abs(got - ref).max() <= 2 ** -7 * np.abs(ref).max()


@pytest.mark.parametrize("fp8", [False, True])
def test_uniform_weights_give_the_exact_mean(fp8):
    # q = 0: every visible key weighs the same; V = its slot's share of a count that bf16 holds exactly
    case = shared_inputs(10, 4, 1, [(3, 64), (2, 32)], [1] * 5, [63, 191, 31, 95, 223])
    inp, go, sl = case
    q = np.zeros_like(inp.q)
    v = np.ones_like(inp.v_cache)
    case = (dataclasses.replace(inp, q=q, v_cache=v), go, sl)
    out, lse = run(case, fp8=fp8)
    assert np.array_equal(out, np.ones_like(out))
    n = np.asarray(inp.prefix_lens, np.float64) + 1
    assert np.abs(lse - np.log(n)[:, None]).max() <= 2 ** -20  # log2 and a product in float32, values below 6


def test_nan_in_unused_slots_and_page_permutation():
    case = shared_inputs(11, 8, 2, [(3, 200), (2, 77)], [5, 1, 40, 9, 3], [0, 33, 150, 2, 60])
    inp, go, sl = case
    ref, lref = run(case)
    un = unused_slots(inp, go, sl)
    k, v = inp.k_cache.copy(), inp.v_cache.copy()
    k[un] = np.nan
    v[un] = np.nan
    out, lse = run((dataclasses.replace(inp, k_cache=k, v_cache=v), go, sl))
    assert np.array_equal(out, ref) and np.array_equal(lse, lref)
    perm = np.random.default_rng(0).permutation(inp.k_cache.shape[0])
    k, v = np.empty_like(inp.k_cache), np.empty_like(inp.v_cache)
    k[perm], v[perm] = inp.k_cache, inp.v_cache
    bt = np.where(inp.block_table >= 0, perm[inp.block_table], -1).astype(np.int32)
    out, lse = run((dataclasses.replace(inp, k_cache=k, v_cache=v, block_table=bt), go, sl))
    assert np.array_equal(out, ref) and np.array_equal(lse, lref)


def test_large_scores_stay_apart():
    # the two parts' maxima lie far from each other, either way round
    for k_scale in (30.0, 0.01):
        inp, go, sl = shared_inputs(12, 4, 1, [(3, 160)], [3, 1, 6], [40, 0, 9])
        k = inp.k_cache.copy()
        k[inp.block_table[0, :10]] = synth.bf16_round(k[inp.block_table[0, :10]] * k_scale)
        check((dataclasses.replace(inp, k_cache=k), go, sl))


def test_device_checks():
    base = shared_inputs(13, 4, 1, [(3, 64), (2, 48)], [4, 3, 5, 2, 6], [20, 40, 3, 9, 1])
    inp, go, sl = base
    ref, _ = run(base)
    rows = lambda *bs: np.concatenate([np.arange(inp.tree_offsets[b], inp.tree_offsets[b + 1]) for b in bs])

    def expect(case, bad):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = run(case, status=st)
        assert int(st.item()) == _lib.JF_ERR_DEVICE_CHECK
        hit = np.zeros(len(out), bool)
        hit[rows(*bad)] = True
        assert np.isnan(out[hit]).all() and np.isnan(lse[hit]).all()
        assert np.array_equal(out[~hit], ref[~hit])

    def table(b, i, v):
        bt = inp.block_table.copy()
        bt[b, i] = v
        return dataclasses.replace(inp, block_table=bt), go, sl

    expect(table(0, 1, -1), [0, 1, 2])                       # a shared page: its whole group
    expect(table(0, 1, inp.k_cache.shape[0]), [0, 1, 2])
    expect(table(1, 4, -1), [1])                             # an own page: that sequence
    par = inp.parent.copy()
    par[inp.tree_offsets[2] + 1] = 1
    expect((dataclasses.replace(inp, parent=par), go, sl), [2])
    pl = inp.prefix_lens.copy()
    pl[4] = 47                                               # shorter than the 48 shared
    expect((dataclasses.replace(inp, prefix_lens=pl), go, sl), [4])
    every = range(5)
    expect((inp, np.array([0, 3, 4], np.int32), sl), every)  # groups that do not cover the batch
    expect((inp, np.array([0, 6, 5], np.int32), sl), every)
    expect((inp, np.array([1, 3, 5], np.int32), sl), every)
    expect((inp, go, np.array([64, -1], np.int32)), every)
    sl2 = np.array([64, 100000], np.int32)                   # more than the prefixes and the table hold
    expect((inp, go, sl2), [3, 4])
    expect((inp, go, np.array([64, 2 ** 31 - 1], np.int32)), [3, 4])
    pl = inp.prefix_lens.copy()
    pl[1] = 2 ** 31 - 1                                      # more than its table holds
    expect((dataclasses.replace(inp, prefix_lens=pl), go, sl), [1])


def test_malformed_lengths_of_one_sequence_leave_the_batch_unwritten():
    # found by the plan's second check, each by one thread of few: all others must agree to leave
    rng = np.random.default_rng(14)
    B = 600
    nodes = rng.integers(0, 4, B)
    nodes[[0, 299, 300, B - 1]] = [2, 200, 200, 2]
    inp, go, sl = shared_inputs(14, 4, 1, [(300, 48), (299, 16), (1, 0)], nodes, rng.integers(0, 40, B))
    ws = api.SharedAttentionWorkspace(inp.q.shape[0], 4, torch.device("cuda"))
    ref, lref = run((inp, go, sl), ws=ws)
    lengths = []
    for b in (0, 299, 301, B - 1):
        pl = inp.prefix_lens.copy()
        pl[b] = -1
        lengths.append(dict(prefix_lens=pl))
    for b, to in ((300, inp.tree_offsets[299]), (300, inp.tree_offsets[301])):
        off = inp.tree_offsets.copy()
        off[b] = to                       # 400 nodes in one tree, none in the other
        lengths.append(dict(tree_offsets=off))
    off = inp.tree_offsets.copy()
    off[1] = off[2] + 1                   # decreasing
    lengths.append(dict(tree_offsets=off))
    for bad in lengths:
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        out, lse = run((dataclasses.replace(inp, **bad), go, sl), ws=ws, status=st)
        assert int(st.item()) == _lib.JF_ERR_DEVICE_CHECK
        assert np.isnan(out).all() and np.isnan(lse).all()
    out, lse = run((inp, go, sl), ws=ws)
    assert np.array_equal(out, ref) and np.array_equal(lse, lref)


def test_workspace_is_reusable_and_graphs_replay():
    cases = [shared_inputs(20, 8, 2, [(3, 300)], [30, 2, 9], [5, 70, 0]),
             shared_inputs(21, 8, 2, [(1, 16), (2, 900)], [1, 1, 1], [1, 2, 3]),
             shared_inputs(22, 8, 2, [(2, 0)], [256, 5], [400, 0])]
    T = max(c[0].q.shape[0] for c in cases)
    ws = api.SharedAttentionWorkspace(T, 8, torch.device("cuda"))
    refs = [run(c, ws=ws) for c in cases]
    for c, r in zip(cases, refs):
        check(c, ws=ws)
        again = run(c, ws=ws)
        assert np.array_equal(again[0], r[0]) and np.array_equal(again[1], r[1])
    inp, go, sl = cases[0]
    d, g32, s32 = to_dev(inp), i32(go), i32(sl)
    out = torch.empty_like(d["q"])
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        api.tree_attention_shared(d["q"], d["k_cache"], d["v_cache"], d["block_table"], d["prefix_lens"],
                                  d["tree_offsets"], d["parent"], g32, s32, inp.sm_scale, out=out, workspace=ws)
    for _ in range(2):
        out.fill_(float("nan"))
        run(cases[1], ws=ws)  # leaves other contents in the workspace
        g.replay()
        torch.cuda.synchronize()
        assert np.array_equal(out.float().cpu().numpy(), refs[0][0])


def test_two_streams_with_workspaces_of_their_own():
    case = shared_inputs(30, 8, 2, [(6, 2000)], [20] * 6, [50] * 6)
    ref, _ = run(case)
    inp, go, sl = case
    d, g32, s32 = to_dev(inp), i32(go), i32(sl)
    args = (d["q"], d["k_cache"], d["v_cache"], d["block_table"], d["prefix_lens"], d["tree_offsets"], d["parent"], g32,
            s32, inp.sm_scale)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [api.tree_attention_shared(*args, stream=streams[i % 2]) for i in range(6)]  # scratch allocated per call
    torch.cuda.synchronize()
    assert all(np.array_equal(o.float().cpu().numpy(), ref) for o in outs)


def test_wait_that_runs_out_reports_timeout_and_writes_nothing():
    L = _lib.debug_lib()
    case = shared_inputs(31, 4, 1, [(3, 300)], [5, 1, 9], [0, 40, 3])
    inp, go, sl = case
    d, g32, s32 = to_dev(inp), i32(go), i32(sl)
    T, Hq = inp.q.shape[:2]
    ws = torch.empty(L.jf_tree_attention_shared_workspace_size(T, Hq), dtype=torch.uint8, device="cuda")
    out, status = torch.full_like(d["q"], float("nan")), torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        code = L.jf_tree_attention_shared(
            *(d[k].data_ptr() for k in ("q", "k_cache", "v_cache", "block_table")), inp.block_table.shape[1],
            *(t.data_ptr() for t in (d["prefix_lens"], d["tree_offsets"], d["parent"], g32, s32)), 1, 3, T, Hq, 1, 128,
            16, inp.k_cache.shape[0], inp.sm_scale, out.data_ptr(), None, ws.data_ptr(), ws.numel(), status.data_ptr(),
            torch.cuda.current_stream().cuda_stream)
        assert code == _lib.JF_OK
        torch.cuda.synchronize()

    call()
    good = out.clone()
    out.fill_(float("nan"))
    assert L.jf_debug_hold(1) == _lib.JF_OK
    try:
        call()
    finally:
        assert L.jf_debug_hold(0) == _lib.JF_OK
    assert int(status.item()) == _lib.JF_ERR_TIMEOUT
    assert torch.isnan(out.float()).all()
    status.zero_()
    call()
    assert int(status.item()) == 0 and torch.equal(out, good)


def test_refusals():
    case = shared_inputs(32, 4, 1, [(2, 32)], [3, 2], [0, 4])
    inp, go, sl = case
    d = to_dev(inp)
    a = dict(q=d["q"], k_cache=d["k_cache"], v_cache=d["v_cache"], block_table=d["block_table"],
             prefix_lens=d["prefix_lens"], tree_offsets=d["tree_offsets"], parent=d["parent"], group_offsets=i32(go),
             shared_lens=i32(sl), sm_scale=inp.sm_scale)
    call = lambda **o: api.tree_attention_shared(**{**a, **o})
    for bad in (dict(q=a["q"].float()), dict(k_cache=a["k_cache"].half()), dict(shared_lens=a["shared_lens"].long())):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(group_offsets=a["group_offsets"][:1]), dict(block_table=a["block_table"][:1]),
                dict(tree_offsets=a["tree_offsets"][:2]), dict(parent=a["parent"][:4]),
                dict(out=torch.empty_like(a["q"][:2])), dict(v_cache=a["v_cache"][1:]),
                dict(group_offsets=a["group_offsets"].cpu()), dict(q=a["q"].transpose(0, 1))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(_lib.JFError):
        call(sm_scale=0.0)
    with pytest.raises(_lib.JFError):
        call(workspace=api.SharedAttentionWorkspace(1, 1, torch.device("cuda")))
    with pytest.raises(_lib.JFError):
        call(group_offsets=i32([0, 1, 2, 2]), shared_lens=i32([0, 0, 0]))  # more groups than sequences


def test_workspace_of_another_device_is_refused():
    inp, go, sl = shared_inputs(33, 4, 1, [(2, 32)], [3, 2], [0, 4])
    ws = api.SharedAttentionWorkspace(5, 4, torch.device("cpu"))
    with pytest.raises(ValueError, match="workspace"):
        run((inp, go, sl), ws=ws)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("nodes", [[1, 1, 2], [40, 1, 30]])
def test_pages_behind_two_to_the_31_entries(fp8, nodes):
    hkv = 8
    inp, go, sl = shared_inputs(34, 2 * hkv, hkv, [(2, 144), (1, 0)], nodes, [5, 40, 33])
    first = 2 ** 31 // (16 * hkv * 128)  # the pages move up by 2^31 entries
    d = to_dev(inp)
    d["block_table"] = torch.where(d["block_table"] >= 0, d["block_table"] + first, d["block_table"])
    pages, st = inp.k_cache.shape[0], torch.zeros(1, dtype=torch.int32, device="cuda")
    caches = []
    for c, s in zip((inp.k_cache, inp.v_cache), SCALES):
        c = torch.from_numpy(synth.e4m3_cache(c, s)).cuda() if fp8 else torch.from_numpy(c).cuda().bfloat16()
        big = torch.zeros((first + pages, *c.shape[1:]), dtype=c.dtype, device="cuda")
        big[first:] = c
        caches.append(big)
    rest = (d["block_table"], d["prefix_lens"], d["tree_offsets"], d["parent"], i32(go), i32(sl), inp.sm_scale)
    lse = torch.full(inp.q.shape[:2], float("nan"), device="cuda")
    if fp8:
        out = api.tree_attention_shared_fp8(d["q"], *caches, *SCALES, *rest, lse=lse, dev_status=st)
    else:
        out = api.tree_attention_shared(d["q"], *caches, *rest, lse=lse, dev_status=st)
    assert int(st.item()) == 0
    ref, lref = oracle((inp, go, sl), fp8)
    compare(out.float().cpu().numpy(), ref, lse.cpu().numpy(), lref)
