"""GPU parity of jf_sample and jf_accept_sampled against the float64 oracle: tokens and paths exactly, log-probabilities
to float32 rounding."""
import numpy as np
import pytest
import torch

from oracle.sampling import accept_sampled as oracle_accept, sample_row
from tree_verify_attention_jf_b200 import _lib, api

pytestmark = pytest.mark.gpu

# One rounding to float32 of the log-probability (half a step, 2^-24 relative), of which the oracle's own float64
# sums take nothing visible; 2^-23 with an absolute floor for log-probabilities near 0, where ln(1 - tiny) carries the
# float64 rounding of a sum of up to 2^19 terms (2^19 * 2^-53 = 2^-34).
LP_REL, LP_ABS = 2.0 ** -23, 2.0 ** -33


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def make_rows(seed, R, V, sigma=2.0, plant=8):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((R, V), dtype=np.float32) * np.float32(sigma)
    for r in range(R):
        n = min(plant, V)
        x[r, rng.choice(V, n, replace=False)] = x[r].max() + rng.uniform(0, 5) - np.log(np.arange(1, n + 1))
    return x.astype(np.float32), rng


def params(rng, R, kind):
    f = lambda a: np.asarray(a, np.float32)
    t, k, p, m = f(rng.uniform(0.4, 1.4, R)), np.zeros(R, np.int32), np.ones(R, np.float32), np.zeros(R, np.float32)
    if kind in ("top_k", "all"):
        k = rng.integers(1, 60, R).astype(np.int32)
    if kind in ("top_p", "all"):
        p = f(rng.uniform(0.3, 0.995, R))
    if kind in ("min_p", "all"):
        m = f(rng.uniform(0.001, 0.3, R))
    if kind == "mixed":
        t[rng.random(R) < 0.2] = 0
        k = np.where(rng.random(R) < 0.5, rng.integers(1, 3000, R), 0).astype(np.int32)
        p = np.where(rng.random(R) < 0.5, f(rng.uniform(0, 1, R)), np.float32(1)).astype(np.float32)
        m = np.where(rng.random(R) < 0.4, f(rng.uniform(0, 1, R)), np.float32(0)).astype(np.float32)
    return t, k, p, m


def run(x, u, par, dtype=torch.float32, pad=0, **kw):
    """x float32 rows (bf16-representable for bf16); returns numpy (token, logprob)."""
    R, V = x.shape
    big = torch.full((R, V + pad), float("nan"), dtype=dtype, device="cuda")
    big[:, :V] = dev(x, dtype)
    got = api.sample(big[:, :V], dev(u), *(dev(a) for a in par), **kw)
    torch.cuda.synchronize()
    return got["token"].cpu().numpy(), got["logprob"].cpu().numpy()


def check(x, u, par, got):
    tok, lp = got
    for r in range(x.shape[0]):
        want, wlp = sample_row(x[r], float(u[r]), float(par[0][r]), int(par[1][r]), float(par[2][r]), float(par[3][r]))
        assert tok[r] == want, (r, tok[r], want, [a[r] for a in par], u[r])
        if np.isinf(wlp):
            assert lp[r] == wlp
        else:
            assert abs(lp[r] - wlp) <= LP_REL * abs(wlp) + LP_ABS, (r, lp[r], wlp)


def bf16(x):
    return torch.from_numpy(x).to(torch.bfloat16).float().numpy()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V", [(3, 1), (5, 2), (4, 7), (33, 31), (17, 1000), (9, 4099), (20, 32003), (6, 151936)])
@pytest.mark.parametrize("kind", ["none", "top_k", "top_p", "min_p", "all", "mixed"])
def test_matches_oracle(dtype, R, V, kind):
    x, rng = make_rows(1000 + V, R, V)
    if dtype == torch.bfloat16:
        x = bf16(x)  # coarse values: many equal logits, ordered by id
    par, u = params(rng, R, kind), rng.random(R, dtype=np.float32)
    u[0] = 0.0
    u[-1] = np.float32(1 - 2.0 ** -24)
    check(x, u, par, run(x, u, par, dtype, pad=(V * 5) % 13))


def test_largest_vocabulary():
    V = 524288
    x, rng = make_rows(7, 3, V)
    par, u = params(rng, 3, "all"), rng.random(3, dtype=np.float32)
    check(x, u, par, run(x, u, par))
    par = params(rng, 3, "top_p")
    check(x, u, par, run(x, u, par))


@pytest.mark.parametrize("V", [50, 5000, 151936])
def test_equal_logits_are_taken_in_id_order(V):
    # a uniform row: every sum is exact on both sides
    x = np.full((8, V), -7.25, np.float32)
    u = np.array([0, 1 / 16, 0.25, 0.5, 0.75, 0.875, 15 / 16, 1 - 2.0 ** -24], np.float32)
    one = np.ones(8, np.float32)
    for k, p, m in ((0, 1, 0), (17, 1, 0), (0, 0.5, 0), (40, 0.25, 1), (V, 1, 1), (0, 0, 0)):
        par = (one * np.float32(0.7), np.full(8, k, np.int32), np.full(8, p, np.float32), np.full(8, m, np.float32))
        check(x, u, par, run(x, u, par))


@pytest.mark.parametrize("levels", [2, 3, 40])
def test_few_distinct_values(levels):
    # heavy ties across the cut, both signs and both zeros
    rng = np.random.default_rng(levels)
    vals = np.concatenate([[0.0, -0.0], np.linspace(-1, 1, max(0, levels - 1))]).astype(np.float32)
    x = vals[rng.integers(0, len(vals), (24, 20011))]
    par = params(rng, 24, "mixed")
    u = rng.random(24, dtype=np.float32)
    check(x, u, par, run(x, u, par))
    check(bf16(x), u, par, run(bf16(x), u, par, torch.bfloat16, pad=3))


def test_masked_infinite_and_nan_logits():
    V = 3001
    x, rng = make_rows(3, 12, V)
    inf = np.float32(np.inf)
    x[0] = -inf                                  # nothing left
    x[1] = np.nan
    x[2] = -inf
    x[2, 1234] = -5                              # one token left
    x[3, rng.random(V) < 0.9] = -inf
    x[4, rng.random(V) < 0.5] = np.nan
    x[5, [10, 2000]] = inf                       # +inf shares the weight
    x[6] = np.finfo(np.float32).min              # a mask of the type's lowest value over the whole row
    x[7, rng.random(V) < 0.9] = np.finfo(np.float32).min
    x[8] = -inf
    x[8, 7] = np.finfo(np.float32).min
    x[9, 5] = np.finfo(np.float32).max
    x[10, :] = 0
    x[10, 100] = -inf
    x[11, 0] = np.nan
    for kind in ("none", "all", "top_p", "mixed"):
        par, u = params(rng, 12, kind), rng.random(12, dtype=np.float32)
        check(x, u, par, run(x, u, par))


def test_temperatures_from_tiny_to_huge():
    x, rng = make_rows(4, 8, 9001)
    t = np.array([1e-38, 1e-6, 1e-2, 0.1, 1.0, 10.0, 1e4, 1e38], np.float32)
    u = rng.random(8, dtype=np.float32)
    for k, p, m in ((0, 1, 0), (500, 1, 0), (0, 0.9, 0), (0, 1, 0.5), (100, 0.7, 0.01)):
        par = (t, np.full(8, k, np.int32), np.full(8, p, np.float32), np.full(8, m, np.float32))
        check(x, u, par, run(x, u, par))


# (m, T) where one float32 step below m is about 954, 977, 1024 and 60 times T
STEPS = [(10.0, 1e-9), (1e4, 1e-6), (1e10, 1.0), (-3e38, 3.4e29), (2.0, 2e-9)]


def step_rows(rng, V, dtype):
    """A row per entry of STEPS: the maximum at two places and its neighbours, one to four steps below, at many."""
    x = np.empty((len(STEPS), V), np.float32)
    for r, (m, _) in enumerate(STEPS):
        v = [torch.tensor(m, dtype=dtype)]
        for _ in range(4):
            v.append(torch.nextafter(v[-1], torch.tensor(-np.inf, dtype=dtype)))
        v = torch.stack(v).float().numpy()
        x[r] = v[rng.integers(1, 5, V)]
        x[r, rng.choice(V, 2, replace=False)] = v[0]
    return x


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [40, 4099, 120001])
def test_logits_one_step_below_the_largest_at_tiny_temperatures(dtype, V):
    rng = np.random.default_rng(V)
    x, R = step_rows(rng, V, dtype), len(STEPS)
    t = np.array([T for _, T in STEPS], np.float32)
    for k, p, m in ((0, 1, 0), (0, 0.9, 0), (20, 1, 0), (V // 2, 1, 0), (V // 2, 0.8, 0), (0, 1, 0.3)):
        par = (t, np.full(R, k, np.int32), np.full(R, p, np.float32), np.full(R, m, np.float32))
        u = rng.uniform(0.02, 0.98, R).astype(np.float32)  # u = 0 may draw what weighs less than the sums resolve
        check(x, u, par, run(x, u, par, dtype, pad=3))


@pytest.mark.parametrize("V", [1, 2, 100, 5000, 151936, 524288])
def test_log_probabilities_are_never_positive(V):
    rng = np.random.default_rng(V)
    x = np.full((24, V), -3, np.float32)
    x[np.arange(24), rng.integers(0, V, 24)] = 60
    x[16:] = rng.standard_normal((8, V), dtype=np.float32)
    k = np.where(np.arange(24) % 3 == 0, 1, 0).astype(np.int32)
    t = np.linspace(0.1, 1.0, 24, dtype=np.float32)
    par, u = (t, k, np.ones(24, np.float32), np.zeros(24, np.float32)), rng.random(24, dtype=np.float32)
    tok, lp = run(x, u, par)
    assert (lp <= 0).all()
    alone = (k == 1) | (np.arange(24) < 16)   # e^-63 and less is below what the sums resolve: the rest weighs nothing
    assert (lp[alone] == 0).all() and (tok[alone] == x.argmax(1)[alone]).all()


def test_parameters_left_out_are_off():
    x, rng = make_rows(5, 4, 700)
    t, u = rng.uniform(0.5, 1, 4).astype(np.float32), rng.random(4, dtype=np.float32)
    off = (t, np.zeros(4, np.int32), np.ones(4, np.float32), np.zeros(4, np.float32))
    got = api.sample(dev(x), dev(u), dev(t))
    check(x, u, off, (got["token"].cpu().numpy(), got["logprob"].cpu().numpy()))
    only = api.sample(dev(x), dev(u), dev(t), out=dict(token=got["token"].clone().fill_(-9)))
    assert torch.equal(only["token"], got["token"]) and "logprob" not in only


def test_bad_parameters_leave_their_row_unwritten():
    x, rng = make_rows(6, 12, 500)
    par, u = params(rng, 12, "all"), rng.random(12, dtype=np.float32)
    t, k, p, m = (a.copy() for a in par)
    t[0], t[1], t[2], k[3], p[4], p[5], m[6], m[7], u[8], u[9], u[10] = (
        -1, np.nan, np.inf, -1, -0.1, 1.1, np.nan, 1.5, 1.0, -0.1, np.nan)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = dict(token=torch.full((12,), -77, dtype=torch.int32, device="cuda"),
               logprob=torch.full((12,), 5.0, device="cuda"))
    tok, lp = run(x, u, (t, k, p, m), out=out, dev_status=st)
    assert int(st.item()) == _lib.JF_ERR_DEVICE_CHECK
    assert (tok[:11] == -77).all() and (lp[:11] == 5.0).all()
    check(x[11:], u[11:], [a[11:] for a in (t, k, p, m)], (tok[11:], lp[11:]))


def test_greedy_rows_take_any_other_parameters():
    x, rng = make_rows(16, 9, 700)
    x[8, 3] = np.inf
    nan, big = np.float32(np.nan), np.int32(2 ** 31 - 1)
    u = np.array([1, -1, nan, np.inf, 0.5, 0.5, 0.5, 0.5, nan], np.float32)
    t = np.zeros(9, np.float32)
    t[1] = -0.0
    k = np.array([-1, 0, -big - 1, big, -5, 1, 0, 0, -2], np.int32)
    p = np.array([1, 2, nan, -1, np.inf, nan, 1, 0, -nan], np.float32)
    m = np.array([0, 0, nan, 7, -1, np.inf, nan, 2, nan], np.float32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    check(x, u, (t, k, p, m), run(x, u, (t, k, p, m), dev_status=st))
    assert int(st.item()) == 0
    # the same in the walk, beside a sequence that draws and one that must not be written
    token, parent, x, _, rng = walk_case(17, 3, 40, 900, 6)
    u = np.full((3, 7), nan, np.float32)
    u[1] = rng.random(7, dtype=np.float32)
    t = np.array([0, 0.5, 0.5], np.float32)
    k, p, m = (np.array([bad, good, good], dt) for bad, good, dt in ((-3, 0, np.int32), (nan, 1, np.float32),
                                                                     (5, 0, np.float32)))
    out = dict(accepted_len=torch.full((3,), -9, dtype=torch.int32, device="cuda"),
               path=torch.full((3, 7), -9, dtype=torch.int32, device="cuda"),
               bonus=torch.full((3,), -9, dtype=torch.int32, device="cuda"),
               logprob=torch.full((3, 7), 3.0, device="cuda"))
    api.accept_sampled(dev(token), dev(parent), dev(x), dev(u), dev(t), 6, dev(k), dev(p), dev(m), out=out,
                       dev_status=st)
    assert int(st.item()) == _lib.JF_ERR_DEVICE_CHECK and int(out["accepted_len"][2]) == -9
    check_walk((token[:2], parent[:2], x[:2], u[:2]), [a[:2] for a in (t, k, p, m)], 6,
               {n: v[:2] for n, v in out.items()})


def test_repeats_graph_replays_and_streams_agree_bit_for_bit():
    x, rng = make_rows(8, 40, 50021)
    par, u = params(rng, 40, "mixed"), rng.random(40, dtype=np.float32)
    d = [dev(x), dev(u)] + [dev(a) for a in par]
    ref = api.sample(*d)
    torch.cuda.synchronize()
    out = {k: torch.empty_like(v) for k, v in ref.items()}
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        api.sample(*d, out=out)
    for _ in range(3):
        for v in out.values():
            v.fill_(-5)
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[k], ref[k]) for k in ref)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    ra = [api.sample(*d, stream=a) for _ in range(4)]
    rb = [api.sample(*d, stream=b) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(r[k], ref[k]) for r in ra + rb for k in ref)


def test_refusals():
    x, u, t = torch.zeros(2, 8, device="cuda"), torch.zeros(2, device="cuda"), torch.ones(2, device="cuda")
    with pytest.raises(TypeError):
        api.sample(x.half(), u, t)
    with pytest.raises(TypeError):
        api.sample(x, u.double(), t)
    with pytest.raises(ValueError):
        api.sample(x[0], u, t)
    with pytest.raises(ValueError):
        api.sample(x.t(), u, t)
    with pytest.raises(ValueError):
        api.sample(x, u[:1], t)
    with pytest.raises(ValueError):
        api.sample(x, u, t, top_k=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        api.sample(x, u.cpu(), t)
    with pytest.raises(_lib.JFError):
        api.sample(x[:, 1:], u, t)  # not 16-byte aligned
    with pytest.raises(_lib.JFError):
        api.sample(x[:1].expand(2, 8), u, t)  # rows on top of each other
    assert api.sample(x[:0], u[:0], t[:0])["token"].shape == (0,)


# ---------------------------------------------------------------------------------------------- the walk
def walk_case(seed, B, N, V, D, lift=4.0, sigma=2.0):
    rng = np.random.default_rng(seed)
    parent = np.array([[-1] + [int(rng.integers(max(0, i - 6), i)) for i in range(1, N)] for _ in range(B)], np.int32)
    token = rng.integers(0, V, (B, N)).astype(np.int32)
    x = rng.standard_normal((B, N, V), dtype=np.float32) * np.float32(sigma)
    for b in range(B):
        for i in range(1, N):  # every child's token stands out at its parent
            row = x[b, parent[b, i]]
            row[token[b, i]] = row.max() + rng.uniform(0, lift)
    return token, parent, x, rng.random((B, D + 1), dtype=np.float32), rng


def check_walk(case, par, D, got):
    token, parent, x, u = case[:4]
    acc, path, bonus, lp = oracle_accept(token, parent, x, u, D, *par)
    assert np.array_equal(got["accepted_len"].cpu().numpy(), acc)
    assert np.array_equal(got["path"].cpu().numpy(), path)
    assert np.array_equal(got["bonus"].cpu().numpy(), bonus)
    g = got["logprob"].cpu().numpy()
    fin = np.isfinite(lp)
    assert np.array_equal(g[~fin], lp[~fin])
    assert (np.abs(g[fin] - lp[fin]) <= LP_REL * np.abs(lp[fin]) + LP_ABS).all()
    return acc


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,N,V,D", [(1, 1, 5, 0), (1, 1, 40, 3), (4, 12, 9, 6), (3, 200, 4001, 16), (2, 1024, 301, 20),
                                     (2, 40, 151936, 12), (150, 5, 333, 4)])
@pytest.mark.parametrize("kind", ["none", "mixed"])
def test_walk_matches_oracle(dtype, B, N, V, D, kind):
    case = walk_case(31 * V + N, B, N, V, D)
    if dtype == torch.bfloat16:
        case = case[:2] + (bf16(case[2]),) + case[3:]
    par = params(case[4], B, kind)
    got = api.accept_sampled(dev(case[0]), dev(case[1]), dev(case[2], dtype), dev(case[3]), dev(par[0]), D,
                             *(dev(a) for a in par[1:]))
    acc = check_walk(case, par, D, got)
    if N >= 12 and B > 1:
        assert acc.max() > 0  # the case is no test of walks that end at the root only


def test_walk_with_temperature_zero_is_jf_accept():
    token, parent, x, u, rng = walk_case(5, 6, 64, 3000, 10)
    t = torch.zeros(6, device="cuda")
    got = api.accept_sampled(dev(token), dev(parent), dev(x), dev(u), t, 10)
    ref = api.accept(dev(token), dev(parent), dev(x), 10)
    for k in ref:
        assert torch.equal(got[k], ref[k]), k


def test_walk_stops_at_a_row_without_candidates():
    token, parent, x, u, rng = walk_case(6, 3, 20, 100, 8)
    x[1, 0] = -np.inf
    par = params(rng, 3, "none")
    got = api.accept_sampled(dev(token), dev(parent), dev(x), dev(u), dev(par[0]), 8)
    check_walk((token, parent, x, u), par, 8, got)
    assert int(got["bonus"][1]) == -1 and int(got["accepted_len"][1]) == 0


@pytest.mark.parametrize("kind", ["none", "top_p", "top_k"])
def test_walk_over_logits_one_step_below_the_largest(kind):
    rng = np.random.default_rng(10)
    B, N, V, D = len(STEPS), 12, 2003, 6
    x = np.stack([step_rows(rng, V, torch.float32) for _ in range(N)], 1)
    par = list(params(rng, B, kind))
    par[0] = np.array([T for _, T in STEPS], np.float32)
    parent = np.tile(np.arange(-1, N - 1, dtype=np.int32), (B, 1))  # a chain that carries one of the two maxima
    token = np.zeros((B, N), np.int32)
    token[:, 1:] = x[:, :-1].argmax(-1)
    u = rng.uniform(0.02, 0.98, (B, D + 1)).astype(np.float32)
    got = api.accept_sampled(dev(token), dev(parent), dev(x), dev(u), dev(par[0]), D, *(dev(a) for a in par[1:]))
    assert check_walk((token, parent, x, u), par, D, got).max() > 0


def test_walk_device_checks_leave_the_sequence_unwritten():
    token, parent, x, u, rng = walk_case(8, 5, 20, 100, 8)
    par = params(rng, 5, "none")
    par[0][1] = -2                     # temperature
    parent[2, 4] = 4                   # parent not before its node
    u[3, 0] = 1.0                      # the first random number
    u[4, 8] = np.nan                   # one that the walk does not come to (checked below)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = dict(accepted_len=torch.full((5,), -9, dtype=torch.int32, device="cuda"),
               path=torch.full((5, 9), -9, dtype=torch.int32, device="cuda"),
               bonus=torch.full((5,), -9, dtype=torch.int32, device="cuda"),
               logprob=torch.full((5, 9), 3.0, device="cuda"))
    api.accept_sampled(dev(token), dev(parent), dev(x), dev(u), dev(par[0]), 8, out=out, dev_status=st)
    assert int(st.item()) == _lib.JF_ERR_DEVICE_CHECK
    for b in (1, 2, 3):
        assert int(out["accepted_len"][b]) == -9 and int(out["bonus"][b]) == -9
        assert (out["path"][b] == -9).all() and (out["logprob"][b] == 3.0).all()
    for b in (0, 4):
        one = [a[b:b + 1] for a in (token, parent, x, u)]
        ref = oracle_accept(*one, 8, par[0][b:b + 1])
        assert ref[0][0] < 8
        assert int(out["accepted_len"][b]) == ref[0][0] and out["path"][b].cpu().tolist() == ref[1][0].tolist()


def test_walk_replays_in_a_cuda_graph():
    token, parent, x, u, rng = walk_case(9, 4, 64, 20000, 10)
    par = params(rng, 4, "all")
    d = [dev(a) for a in (token, parent, x, u)]
    p = [dev(a) for a in par]
    out = dict(accepted_len=torch.empty(4, dtype=torch.int32, device="cuda"),
               path=torch.empty(4, 11, dtype=torch.int32, device="cuda"),
               bonus=torch.empty(4, dtype=torch.int32, device="cuda"), logprob=torch.empty(4, 11, device="cuda"))
    g, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        api.accept_sampled(*d, p[0], 10, *p[1:], out=out)
    for seed in (1, 2):  # new random numbers between the replays
        case = (token, parent, x, np.random.default_rng(seed).random((4, 11), dtype=np.float32))
        d[3].copy_(dev(case[3]))
        g.replay()
        torch.cuda.synchronize()
        check_walk(case, par, 10, out)


def test_walk_refusals():
    z = lambda *s, dt=torch.float32: torch.zeros(*s, dtype=dt, device="cuda")
    tok, par, x, u, t = z(2, 4, dt=torch.int32), z(2, 4, dt=torch.int32), z(2, 4, 8), z(2, 3), z(2)
    with pytest.raises(TypeError):
        api.accept_sampled(tok, par, x.double(), u, t, 2)
    with pytest.raises(ValueError):
        api.accept_sampled(tok[:, :3], par, x, u, t, 2)
    with pytest.raises(ValueError):
        api.accept_sampled(tok, par, x, u, t, 3)
    with pytest.raises(ValueError):
        api.accept_sampled(tok, par, x, u, t[:1], 2)
    with pytest.raises(ValueError):
        api.accept_sampled(tok, par, x[:, :, :7], u, t, 2)
    with pytest.raises(ValueError):
        i = torch.int32
        out = dict(accepted_len=z(2, dt=i), path=z(2, 4, dt=i), bonus=z(2, dt=i))
        api.accept_sampled(tok, par, x, u, t, 2, out=out)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["none", "top_p", "all"])
def test_rows_behind_two_to_the_31_entries(dtype, kind):
    R, V, stride = 3, 5000, 2 ** 30 + 3
    x, rng = make_rows(41, R, V)
    if dtype == torch.bfloat16:
        x = bf16(x)
    par, u = params(rng, R, kind), rng.random(R, dtype=np.float32)
    rows = torch.empty(2 * stride + V, dtype=dtype, device="cuda").as_strided((R, V), (stride, 1))
    rows.copy_(dev(x, dtype))
    got = api.sample(rows, dev(u), *(dev(a) for a in par))
    check(x, u, par, (got["token"].cpu().numpy(), got["logprob"].cpu().numpy()))


def test_walk_behind_two_to_the_31_entries():
    B, N, V, D = 5, 1024, 524288, 2
    rng = np.random.default_rng(42)
    x, u = bf16(make_rows(43, 1, V)[0]), rng.random((B, D + 1), dtype=np.float32)
    par = [np.ones(B, np.float32), np.full(B, 50, np.int32)]
    logits = torch.zeros(B, N, V, dtype=torch.bfloat16, device="cuda")
    logits[B - 1] = dev(x, torch.bfloat16)
    token, parent = np.zeros((B, N), np.int32), np.zeros((B, N), np.int32)
    want = [sample_row(x[0], float(u[B - 1, i]), 1.0, 50, 1.0, 0.0) for i in range(D + 1)]
    parent[:, 0] = -1
    parent[:, N - 1] = N - 2  # root, node N - 2, node N - 1
    token[B - 1, N - 2:] = [want[0][0], want[1][0]]
    token[B - 1, 1:N - 2] = -1
    got = api.accept_sampled(dev(token), dev(parent), logits, dev(u), dev(par[0]), D, top_k=dev(par[1]))
    assert int(got["accepted_len"][B - 1]) == D and got["path"][B - 1].tolist()[1:] == [N - 2, N - 1]
    assert int(got["bonus"][B - 1]) == want[D][0]
    lp = got["logprob"][B - 1].cpu().numpy()
    assert all(abs(lp[i] - want[i][1]) <= LP_REL * abs(want[i][1]) + LP_ABS for i in range(D + 1))


# Batches whose slices do not fit the shared memory that their CTAs may take, so that every pass reads the rows from
# memory again: one CTA a row from 149 rows on and about 70 KB a row, or clusters of a few CTAs for longer rows of
# fewer.  Odd lengths, and rows that start at every place of a 16-byte granule.
@pytest.mark.parametrize("dtype,R,V,pad", [(torch.float32, 40, 151936, 1), (torch.float32, 80, 50003, 2),
                                           (torch.float32, 160, 20011, 3), (torch.bfloat16, 80, 90001, 4),
                                           (torch.bfloat16, 160, 40003, 7)])
@pytest.mark.parametrize("kind", ["none", "top_p", "all", "mixed"])
def test_rows_read_from_memory_in_each_pass(dtype, R, V, pad, kind):
    x, rng = make_rows(V + R, R, V)
    x[1, :9] = -np.inf
    x[2, -9:] = np.nan
    x[3] = -np.inf
    x[4, rng.random(V) < 0.9] = -np.inf
    x[5] = x[5].max()                            # ties throughout
    x[6] = np.where(rng.random(V) < 0.5, np.float32(1.5), np.float32(1.25))
    if dtype == torch.bfloat16:
        x = bf16(x)
    par, u = params(rng, R, kind), rng.random(R, dtype=np.float32)
    u[0], u[-1] = 0.0, np.float32(1 - 2.0 ** -24)
    if kind == "mixed":
        par[1][7], par[2][7] = V // 2, 0.9       # a large top-k with a top-p
    check(x, u, par, run(x, u, par, dtype, pad=pad))


# More sequences than the SMs hold clusters of the width that keeps a row in shared memory.
@pytest.mark.parametrize("dtype,B,N,V", [(torch.float32, 40, 3, 151936), (torch.float32, 80, 4, 45001),
                                         (torch.bfloat16, 80, 4, 90001), (torch.float32, 12, 3, 524288)])
@pytest.mark.parametrize("kind", ["none", "top_p", "mixed"])
def test_walk_of_many_sequences_over_long_rows(dtype, B, N, V, kind):
    case = walk_case(V + B, B, N, V, 3, lift=6.0)
    if dtype == torch.bfloat16:
        case = case[:2] + (bf16(case[2]),) + case[3:]
    par = params(case[4], B, kind)
    if kind == "mixed":
        par[1][3], par[2][3], par[0][3] = V // 2, 0.9, 1.0
    got = api.accept_sampled(dev(case[0]), dev(case[1]), dev(case[2], dtype), dev(case[3]), dev(par[0]), 3,
                             *(dev(a) for a in par[1:]))
    acc, path, bonus, lp = oracle_accept(*case[:4], 3, *par)
    assert acc.max() > 0
    for name, want in (("accepted_len", acc), ("path", path), ("bonus", bonus)):
        assert np.array_equal(got[name].cpu().numpy(), want), name
    # Each of at most V weights is off by half a step of 2^-f of the largest, so the sum, which is at least the largest,
    # is off by V 2^-(f+1) relative, and its logarithm by as much; beside that the rounding to float32.
    f = min(48, 62 - int(np.ceil(np.log2(V))))
    assert (np.abs(got["logprob"].cpu().numpy() - lp) <= LP_REL * np.abs(lp) + V * 2.0 ** -(f + 1)).all()


def test_waits_that_run_out_report_timeout_and_write_nothing():
    # the debug build leaves out the copies of the rows and gives up after 50 ms; nothing faults and the next call works
    L = _lib.debug_lib()
    R, V, N, D = 3, 5000, 4, 2
    x, rng = make_rows(50, R, V)
    par, u = params(rng, R, "all"), rng.random(R, dtype=np.float32)
    rows, st = dev(x), torch.zeros(1, dtype=torch.int32, device="cuda")
    p = [dev(a) for a in par]
    ptr = lambda *ts: [t.data_ptr() for t in ts]
    token = torch.full((R,), -77, dtype=torch.int32, device="cuda")
    lp, du = torch.full((R,), 5.0, device="cuda"), dev(u)
    case = walk_case(51, 2, N, V, D)
    w = [dev(a) for a in case[:4]]
    i32 = lambda *s: torch.full(s, -9, dtype=torch.int32, device="cuda")
    acc, path, bonus, wlp = i32(2), i32(2, D + 1), i32(2), torch.full((2, D + 1), 3.0, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream

    def sample():
        assert L.jf_sample(*ptr(rows), 0, V, R, V, *ptr(du, *p, token, lp, st), stream) == _lib.JF_OK
        torch.cuda.synchronize()

    def walk():
        assert L.jf_accept_sampled(*ptr(*w[:3]), 0, *ptr(w[3], *p), 2, N, V, D, *ptr(acc, path, bonus, wlp, st),
                                   stream) == _lib.JF_OK
        torch.cuda.synchronize()

    for call in (sample, walk):
        st.zero_()
        assert L.jf_debug_hold(1) == _lib.JF_OK
        try:
            call()
        finally:
            assert L.jf_debug_hold(0) == _lib.JF_OK
        assert int(st.item()) == _lib.JF_ERR_TIMEOUT
    assert (token == -77).all() and (lp == 5.0).all()
    assert all((t == -9).all() for t in (acc, path, bonus)) and (wlp == 3.0).all()
    st.zero_()
    sample()
    walk()
    assert int(st.item()) == 0
    check(x, u, par, (token.cpu().numpy(), lp.cpu().numpy()))
    check_walk(case, [a[:2] for a in par], D, dict(accepted_len=acc, path=path, bonus=bonus, logprob=wlp))
