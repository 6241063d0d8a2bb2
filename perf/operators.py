"""Measured cases of the operators that serve several sampled continuations of one prompt: attention of draft trees
whose sequences share a long prefix, token sampling from given random numbers, and the sampled acceptance walk.

Every case runs either through the library's public calls (``own``) or through the operator's plain form, elementary
torch operations written from the definition.  Inputs are seeded and synthetic.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
VOCAB = 151936   # the vocabulary of the library's draft and target logits
HEAD_DIM = 128
PAGE = 16


# ----------------------------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------------------------
def _sample(name, rows, vocab, dtype, filters, pad=0):
    return dict(name=name, op="sample", rows=rows, vocab=vocab, dtype=dtype, filters=filters, pad=pad)


def _accept(name, batch, nodes, vocab, dtype, filters, path, max_depth):
    return dict(name=name, op="accept", batch=batch, nodes=nodes, vocab=vocab, dtype=dtype, filters=filters, path=path,
                max_depth=max_depth)


def _shared(name, batch, groups, nodes, ragged, hq, hkv, shared, suffix, fp8, lens=1):
    return dict(name=name, op="shared", batch=batch, groups=groups, nodes=nodes, ragged=ragged, hq=hq, hkv=hkv,
                shared=shared, suffix=suffix, fp8=fp8, lens=lens)


def listed():
    return [
        # one sequence decoding: the smallest call of every step, latency counts
        _sample("sample one row", 1, VOCAB, "f32", "all"),
        # a decode batch with nucleus sampling over the whole vocabulary
        _sample("sample nucleus batch", 64, VOCAB, "f32", "top_p"),
        # many rollouts of a few prompts at once, no truncation, 16-bit logits
        _sample("sample rollouts bf16", 512, VOCAB, "bf16", "none"),
        # a mixed batch: every row with filters of its own, an odd vocabulary, rows of a padded matrix
        _sample("sample mixed odd", 257, 32003, "f32", "mixed", 61),
        # one sequence with a small tree: latency
        _accept("accept small tree", 1, 16, VOCAB, "f32", "all", 5, 8),
        # the library's build-and-accept batch (8 sequences, 256 nodes, 16 levels), sampled
        _accept("accept batch", 8, 256, VOCAB, "f32", "top_p", 10, 16),
        # a serving batch of small trees with 16-bit logits and mixed filters
        _accept("accept serving bf16", 32, 64, VOCAB, "bf16", "mixed", 6, 12),
        # four short continuations of one prompt, one new token each: the smallest call
        _shared("shared decode small", 4, 1, 1, False, 4, 1, 1024, 64, False),
        # single-token decode of 64 continuations of one prompt
        _shared("shared decode batch", 64, 1, 1, False, 32, 8, 16384, 256, False),
        # small ragged trees over two system prompts
        _shared("shared trees two prompts", 32, 2, 64, True, 32, 8, 8192, 1000, False),
        # the largest: 256-node trees on eight continuations of one 32768-token prompt
        _shared("shared trees long prompt", 8, 1, 256, False, 32, 4, 32768, 500, False),
        # the 8-bit cache under the serving shape
        _shared("shared trees 8-bit cache", 32, 1, 16, True, 32, 8, 8192, 1000, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["sample", "sample", "accept", "shared", "shared"])
    if op == "sample":
        case = _sample("", _log_int(rng, 1, 400), _log_int(rng, 1000, VOCAB), rng.choice(["f32", "bf16"]),
                       rng.choice(["none", "top_p", "all", "mixed"]), rng.choice([0, 0, 1, 8, 37]))
    elif op == "accept":
        depth = rng.randint(4, 16)
        case = _accept("", _log_int(rng, 1, 14), rng.randint(depth + 1, 200), _log_int(rng, 1000, VOCAB),
                       rng.choice(["f32", "bf16"]), rng.choice(["none", "top_p", "all", "mixed"]),
                       rng.randint(1, depth), depth)
    else:
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([r for r in (1, 2, 4, 8, 16) if hkv * r <= 32])
        batch, shared = _log_int(rng, 2, 48), _log_int(rng, 64, 16384)
        groups = rng.randint(1, max(1, min(4, batch // 3)))
        most = max(1, (1 << 30) // (groups * batch * hq * shared))  # the plain form's scores are held in memory
        case = _shared("", batch, groups, min(most, _log_int(rng, 1, 100)), rng.random() < 0.7, hq, hkv, shared,
                       _log_int(rng, 1, 2000), rng.random() < 0.3, rng.randint(1, 1 << 20))
    del case["name"]
    return case


# ----------------------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _params(case, g, n):
    """Sampling parameters of n rows: temperature, top_k (0 = off), top_p (1 = off), min_p (0 = off)."""
    uni = lambda lo, hi: lo + (hi - lo) * torch.rand(n, device=DEV, generator=g)
    t = uni(0.5, 1.3)
    k = torch.zeros(n, dtype=torch.int32, device=DEV)
    p = torch.ones(n, device=DEV)
    m = torch.zeros(n, device=DEV)
    f = case["filters"]
    if f == "top_p":
        p = uni(0.8, 0.99)
    elif f == "all":
        k, p, m = torch.full_like(k, 50), uni(0.85, 0.98), uni(0.01, 0.1)
    elif f == "mixed":
        on = lambda share: torch.rand(n, device=DEV, generator=g) < share
        t = torch.where(on(0.15), 0.0, t)  # greedy rows
        k = torch.where(on(0.5), torch.randint(1, 2000, (n,), device=DEV, generator=g), 0).to(torch.int32)
        p = torch.where(on(0.5), uni(0.3, 0.99), p)
        m = torch.where(on(0.3), uni(0.0, 0.2), m)
    return dict(temperature=t, top_k=k, top_p=p, min_p=m)


def _logits(g, shape, dtype, pad):
    """N(0, 2^2) with 8 tokens a row lifted to rowmax + c - s ln r, as draft and target heads peak; rows of a matrix
    that is `pad` entries wider."""
    x = torch.randn(*shape[:-1], shape[-1] + pad, device=DEV, generator=g).mul_(2.0)[..., :shape[-1]]
    lead = shape[:-1] + (8,)
    top = x.max(-1, keepdim=True).values
    c = 1.0 + 4.0 * torch.rand(*shape[:-1], 1, device=DEV, generator=g)
    s = 0.8 + 0.7 * torch.rand(*shape[:-1], 1, device=DEV, generator=g)
    lift = top + c - s * torch.arange(1, 9, device=DEV, dtype=torch.float32).log()
    x.scatter_(-1, torch.randint(0, shape[-1], lead, device=DEV, generator=g), lift)
    if dtype == "bf16":
        wide = torch.empty(*shape[:-1], shape[-1] + pad, device=DEV, dtype=torch.bfloat16)
        return wide[..., :shape[-1]].copy_(x)
    return x


def _tree_parents(r, n, levels=16):
    """A rooted tree in topological order: node 0 on the prefix, the others below random earlier nodes."""
    par, level = [-1], [0]
    while len(par) < n:
        p = r.randrange(max(0, len(par) - 40), len(par))
        if level[p] < levels:
            par.append(p)
            level.append(level[p] + 1)
    return par, level


def _shapes(case):
    """Lengths and trees of a shared-prefix case; they are the case's own, whatever the seed of the values."""
    r = random.Random(case["lens"])
    B, G = case["batch"], case["groups"]
    cuts = sorted(r.sample(range(1, B), G - 1)) if G > 1 else []
    groups = [0] + cuts + [B]
    shared = [max(1, case["shared"] - (r.randrange(case["shared"] // 4 + 1) if g else 0)) for g in range(G)]
    nodes = [r.randint(1, case["nodes"]) if case["ragged"] else case["nodes"] for _ in range(B)]
    prefix = [shared[g] + r.randint(0, case["suffix"]) for g in range(G) for _ in range(groups[g], groups[g + 1])]
    trees = [_tree_parents(r, n) for n in nodes]
    return dict(groups=groups, shared=shared, nodes=nodes, prefix=prefix, trees=trees)


def _prepare_shared(case, seed):
    g = _generator(seed)
    sh = _shapes(case)
    B, H = case["batch"], case["hkv"]
    of = [k for k in range(case["groups"]) for _ in range(sh["groups"][k], sh["groups"][k + 1])]
    whole = [s // PAGE for s in sh["shared"]]  # pages that a group's sequences have in common
    need = [-(-(p + n) // PAGE) for p, n in zip(sh["prefix"], sh["nodes"])]
    pages = sum(whole) + sum(n - whole[k] for n, k in zip(need, of))
    ids = torch.randperm(pages, device=DEV, generator=g).cpu().numpy().astype(np.int32)
    table = np.zeros((B, max(need)), np.int32)
    at, common = 0, []
    for w in whole:
        common.append(ids[at:at + w])
        at += w
    for b in range(B):
        own_pages = need[b] - whole[of[b]]
        table[b, :need[b]] = np.concatenate([common[of[b]], ids[at:at + own_pages]])
        at += own_pages
    T = sum(sh["nodes"])
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).to(DEV)
    cache = lambda: torch.randn(pages, PAGE, H, HEAD_DIM, device=DEV, generator=g).mul_(0.5)
    k, v = cache(), cache()
    s = dict(op="shared", q=torch.randn(T, case["hq"], HEAD_DIM, device=DEV, generator=g).to(torch.bfloat16),
             block_table=i32(table), prefix_lens=i32(sh["prefix"]),
             tree_offsets=i32(np.concatenate([[0], np.cumsum(sh["nodes"])])),
             parent=i32(np.concatenate([t[0] for t in sh["trees"]])), group_offsets=i32(sh["groups"]),
             shared_lens=i32(sh["shared"]), sm_scale=HEAD_DIM ** -0.5, fp8=case["fp8"], k_scale=1.0, v_scale=1.0,
             # sizes that the host of a serving engine knows without asking the device
             max_nodes=max(sh["nodes"]), max_shared=max(sh["shared"]),
             max_group=max(sum(sh["nodes"][a:b]) for a, b in zip(sh["groups"], sh["groups"][1:])),
             max_suffix=max(p + n - whole[k] * PAGE for p, n, k in zip(sh["prefix"], sh["nodes"], of)))
    if case["fp8"]:
        s["k_scale"], s["v_scale"] = 1 / 128, 1 / 64
        k = (k * 128).to(torch.float8_e4m3fn).view(torch.uint8)
        v = (v * 64).to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        k, v = k.to(torch.bfloat16), v.to(torch.bfloat16)
    s["k_cache"], s["v_cache"] = k, v
    return s


def _prepare_accept(case, seed):
    g = _generator(seed)
    B, N, V, L = case["batch"], case["nodes"], case["vocab"], case["path"]
    i = torch.arange(N, device=DEV)
    parent = (torch.rand(B, N, device=DEV, generator=g) * i).long()
    parent = torch.where(i <= L, i - 1, parent)  # nodes 0 .. L are a chain, the path that the target mostly agrees with
    token = torch.randint(0, V, (B, N), device=DEV, generator=g)
    x = _logits(g, (B, N, V), case["dtype"], 0)
    rows = x[:, :L].float()
    x[:, :L].scatter_(-1, token[:, 1:L + 1, None], (rows.max(-1, keepdim=True).values + 5.0).to(x.dtype))
    return dict(op="accept", token=token.int(), parent=parent.int(), logits=x, max_depth=case["max_depth"],
                u=torch.rand(B, case["max_depth"] + 1, device=DEV, generator=g), **_params(case, g, B))


def prepare(case, seed):
    if case["op"] == "shared":
        return _prepare_shared(case, seed)
    if case["op"] == "accept":
        return _prepare_accept(case, seed)
    g = _generator(seed)
    R = case["rows"]
    x = _logits(g, (R, case["vocab"]), case["dtype"], case["pad"])
    return dict(op="sample", logits=x, u=torch.rand(R, device=DEV, generator=g), **_params(case, g, R))


# ----------------------------------------------------------------------------------------------
# The plain forms
# ----------------------------------------------------------------------------------------------
def _plain_sample(x, u, temperature, top_k, top_p, min_p):
    """Token and log-probability per row.  In 64 bits: the cut and the drawn token lie at borders of long sums."""
    x, t = x.double(), temperature.double()[:, None]
    greedy = t == 0
    t = torch.where(greedy, 1.0, t)
    m = x.max(-1, keepdim=True).values
    k = torch.where(greedy[:, 0], 1, torch.where(top_k == 0, x.shape[1], top_k))[:, None]
    y = torch.where(x - m >= t * min_p.double()[:, None].log(), x, -torch.inf)
    y, order = y.sort(dim=-1, descending=True, stable=True)  # by value, the lowest id first among equals
    w = ((y - m) / t).exp() * (torch.arange(x.shape[1], device=x.device) < k)
    before = w.cumsum(-1) - w
    p = top_p.double()[:, None]
    w = torch.where((p >= 1) | (before < p * w.sum(-1, keepdim=True)), w, 0.0)
    w = torch.zeros_like(w).scatter_(-1, order, w)  # back to the order of the ids
    c = w.cumsum(-1)
    token = (c <= u.double()[:, None] * c[:, -1:]).sum(-1, keepdim=True)
    return token[:, 0].int(), (w.gather(-1, token) / c[:, -1:]).log()[:, 0].float()


def _plain_accept(s):
    """The walk, all sequences at once: sample at the current node, go to the child that carries the token."""
    B, N, V = s["logits"].shape
    b = torch.arange(B, device=s["token"].device)
    cur, going = torch.zeros_like(b), torch.ones_like(b, dtype=torch.bool)
    length, bonus = torch.zeros_like(s["token"][:, 0]), torch.zeros_like(s["token"][:, 0])
    path = torch.full((B, s["max_depth"] + 1), -1, dtype=torch.int32, device=b.device)
    logprob = torch.zeros(B, s["max_depth"] + 1, device=b.device)
    path[:, 0] = 0
    for step in range(s["max_depth"] + 1):
        tok, lp = _plain_sample(s["logits"][b, cur], s["u"][:, step], s["temperature"], s["top_k"], s["top_p"],
                                s["min_p"])
        bonus = torch.where(going, tok, bonus)
        logprob[:, step] = torch.where(going, lp, 0.0)
        if step == s["max_depth"]:
            break
        child = (s["parent"] == cur[:, None]) & (s["token"] == tok[:, None])
        going = going & child.any(-1)
        cur = torch.where(going, child.int().argmax(-1), cur)
        path[:, step + 1] = torch.where(going, cur, -1).int()
        length = length + going.int()
    return dict(accepted_len=length, path=path, bonus=bonus, logprob=logprob)


def _plain_shared(s):
    """Scores against the group's prefix, read once, and against each sequence's own slots, one softmax over both."""
    off, dev = s["tree_offsets"].long(), s["q"].device
    T, Hq, D = s["q"].shape
    H = s["k_cache"].shape[2]
    seq = torch.searchsorted(off[1:], torch.arange(T, device=dev), right=True)     # sequence of every node
    group = torch.searchsorted(s["group_offsets"].long()[1:], seq, right=True)
    node = torch.arange(T, device=dev) - off[seq]
    start = s["shared_lens"].long() // PAGE * PAGE
    B, G, N = s["prefix_lens"].numel(), s["shared_lens"].numel(), s["max_nodes"]
    read = (lambda c: c.view(torch.float8_e4m3fn).float()) if s["fp8"] else (lambda c: c.float())

    def gather(rows, first, count):
        slot = first[:, None] + torch.arange(count, device=dev)
        page = s["block_table"].long()[rows].gather(1, (slot // PAGE).clamp(max=s["block_table"].shape[1] - 1))
        return [read(c[page, slot % PAGE]) * f for c, f in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"]))]

    q = s["q"].float() * s["sm_scale"]
    # the common prefix of every group: all its nodes at once
    most, S = s["max_group"], s["max_shared"]
    inside = torch.arange(T, device=dev) - off[s["group_offsets"].long()[:-1]][group]
    qg = torch.zeros(G, most, H, Hq // H, D, device=dev)
    qg[group, inside] = q.view(T, H, Hq // H, D)
    kg, vg = gather(s["group_offsets"].long()[:-1], torch.zeros(G, dtype=torch.long, device=dev), S)
    a = torch.einsum("gnhrd,gshd->ghrns", qg, kg)
    a.masked_fill_(torch.arange(S, device=dev) >= start[:, None, None, None, None], -torch.inf)
    # each sequence's own slots: the rest of its prefix and its tree
    qs = torch.zeros(B, N, H, Hq // H, D, device=dev)
    qs[seq, node] = q.view(T, H, Hq // H, D)
    first = start[torch.searchsorted(s["group_offsets"].long()[1:], torch.arange(B, device=dev), right=True)]
    E = s["max_suffix"]
    ks, vs = gather(torch.arange(B, device=dev), first, E)
    below = torch.zeros(B, N, N, dtype=torch.bool, device=dev)
    up, at = s["parent"].long(), node.clone()
    for _ in range(18):  # the root path of every node (levels 0 .. 16, then nothing)
        below[seq, node, at.clamp(min=0)] |= at >= 0
        at = torch.where(at >= 0, up[off[seq] + at.clamp(min=0)], at)
    slot = torch.arange(E, device=dev) + first[:, None]
    tree = slot - s["prefix_lens"].long()[:, None]
    seen = (tree < 0)[:, None, :] | ((tree >= 0) & (tree < N))[:, None, :] & below.gather(
        2, tree.clamp(0, N - 1)[:, None, :].expand(B, N, E))
    e = torch.einsum("bnhrd,bshd->bnhrs", qs, ks).masked_fill(~seen[:, :, None, None, :], -torch.inf)
    e = e[seq, node].reshape(T, Hq, E)
    vis = torch.isfinite(e)
    top = torch.maximum(e.max(-1).values,
                        a.amax(-1).permute(0, 3, 1, 2)[group, inside].reshape(T, Hq))
    e = (e - top[..., None]).exp()
    tg = torch.zeros(G, most, H, Hq // H, device=dev)
    tg[group, inside] = top.view(T, H, Hq // H)
    a.sub_(tg.permute(0, 2, 3, 1)[..., None]).exp_()
    total = e.sum(-1) + a.sum(-1).permute(0, 3, 1, 2)[group, inside].reshape(T, Hq)
    vg.masked_fill_((torch.arange(S, device=dev) >= start[:, None])[..., None, None], 0.0)
    o = torch.einsum("ghrns,gshd->gnhrd", a, vg)[group, inside].reshape(T, Hq, D)
    es = torch.zeros(B, N, H, Hq // H, E, device=dev)
    es[seq, node] = torch.where(vis, e, 0.0).view(T, H, Hq // H, E)
    o = o + torch.einsum("bnhrs,bshd->bnhrd", es, vs)[seq, node].reshape(T, Hq, D)
    return (o / total[..., None]).to(torch.bfloat16), top + total.log()


# ----------------------------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------------------------
def run(s):
    if not own:
        if s["op"] == "sample":
            tok, lp = _plain_sample(*(s[k] for k in ("logits", "u", "temperature", "top_k", "top_p", "min_p")))
            return dict(token=tok, logprob=lp)
        if s["op"] == "accept":
            return _plain_accept(s)
        out, lse = _plain_shared(s)
        return dict(out=out, lse=lse)
    from tree_verify_attention_jf_b200 import api

    how = {k: s[k] for k in ("temperature", "top_k", "top_p", "min_p") if k in s}
    if s["op"] == "sample":
        return api.sample(s["logits"], s["u"], **how)
    if s["op"] == "accept":
        return api.accept_sampled(s["token"], s["parent"], s["logits"], s["u"], max_depth=s["max_depth"], **how)
    T, Hq, _ = s["q"].shape
    if "workspace" not in s:  # a serving loop keeps it
        s["workspace"] = api.SharedAttentionWorkspace(T, Hq, s["q"].device)
    lse = torch.empty(T, Hq, device=s["q"].device)
    args = [s[k] for k in ("block_table", "prefix_lens", "tree_offsets", "parent", "group_offsets", "shared_lens",
                           "sm_scale")]
    if s["fp8"]:
        out = api.tree_attention_shared_fp8(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], *args,
                                            lse=lse, workspace=s["workspace"])
    else:
        out = api.tree_attention_shared(s["q"], s["k_cache"], s["v_cache"], *args, lse=lse, workspace=s["workspace"])
    return dict(out=out, lse=lse)


def work(case):
    """Bytes and operations that one pass cannot do without."""
    if case["op"] == "shared":
        sh = _shapes(case)
        whole = [s // PAGE * PAGE for s in sh["shared"]]
        of = [k for k in range(case["groups"]) for _ in range(sh["groups"][k], sh["groups"][k + 1])]
        T = sum(sh["nodes"])
        slots = sum(whole) + sum(p + n - whole[k] for p, n, k in zip(sh["prefix"], sh["nodes"], of))
        pairs = sum(p * n + sum(x + 1 for x in t[1]) for p, n, t in zip(sh["prefix"], sh["nodes"], sh["trees"]))
        kv = 2 * HEAD_DIM * case["hkv"] * (1 if case["fp8"] else 2)
        return dict(bytes=slots * kv + T * case["hq"] * (HEAD_DIM * 4 + 4) + slots // PAGE * 4 + 4 * T,
                    flops=4.0 * HEAD_DIM * case["hq"] * pairs)
    size = 4 if case["dtype"] == "f32" else 2
    # a sampled row is read once; an exponential and a running sum are a few operations an entry.  The walk reads
    # one row a step: the planted path and the row where it ends
    rows = case["rows"] if case["op"] == "sample" else case["batch"] * (min(case["path"], case["max_depth"]) + 1)
    extra = 28 * rows if case["op"] == "sample" else case["batch"] * (8 * case["nodes"] + 12 * case["max_depth"] + 30)
    return dict(bytes=rows * case["vocab"] * size + extra, flops=4.0 * rows * case["vocab"])


# ----------------------------------------------------------------------------------------------
# The definition in 64 bits
# ----------------------------------------------------------------------------------------------
def _exact_row(x, u, t, k, p, m):
    """The definition for one row, in numpy: (token, log-probability)."""
    if t == 0:
        return int(np.argmax(x)), 0.0
    z = (x - x.max()) / t
    ids = np.flatnonzero(z >= np.log(m)) if m > 0 else np.arange(x.size)
    ids = ids[np.argsort(-x[ids], kind="stable")]
    if k > 0:
        ids = ids[:k]
    if p < 1:
        c = np.cumsum(np.exp(z[ids]))
        ids = ids[:1 + np.searchsorted(c, p * c[-1], side="left")]
    ids = np.sort(ids)
    w = np.exp(z[ids])
    c = np.cumsum(w)
    j = int(np.searchsorted(c, u * c[-1], side="right"))
    return int(ids[j]), float(np.log(w[j] / c[-1]))


def exact(case, seed):
    s = prepare(case, seed)
    f64 = lambda t: t.double().cpu().numpy()
    if case["op"] == "shared":
        return _exact_shared(s)
    par = [f64(s[k]) for k in ("temperature", "top_k", "top_p", "min_p")]
    u = f64(s["u"])
    if case["op"] == "sample":
        rows = [_exact_row(f64(s["logits"][r]), u[r], par[0][r], int(par[1][r]), par[2][r], par[3][r])
                for r in range(case["rows"])]
        return dict(token=np.array([r[0] for r in rows]), logprob=np.array([r[1] for r in rows]))
    B, D = case["batch"], case["max_depth"]
    parent, token = s["parent"].cpu().numpy(), s["token"].cpu().numpy()
    out = dict(accepted_len=np.zeros(B, np.int64), path=np.full((B, D + 1), -1), bonus=np.zeros(B, np.int64),
               logprob=np.zeros((B, D + 1)))
    for b in range(B):
        cur = length = out["path"][b, 0] = 0
        while True:
            tok, out["logprob"][b, length] = _exact_row(f64(s["logits"][b, cur]), u[b, length], par[0][b],
                                                        int(par[1][b]), par[2][b], par[3][b])
            kids = np.flatnonzero((parent[b] == cur) & (token[b] == tok))
            if length == D or kids.size == 0:
                break
            length, cur = length + 1, int(kids[0])
            out["path"][b, length] = cur
        out["accepted_len"][b], out["bonus"][b] = length, tok
    return out


def _exact_shared(s):
    """Every sequence for itself: all its slots through the block table (the shared ones through its group's first
    row), a dense mask, a softmax in 64 bits."""
    off, gro = s["tree_offsets"].tolist(), s["group_offsets"].tolist()
    pre, sha, par = s["prefix_lens"].tolist(), s["shared_lens"].tolist(), s["parent"].tolist()
    H = s["k_cache"].shape[2]
    outs, lses = [], []
    dec = (lambda c: c.view(torch.float8_e4m3fn).double()) if s["fp8"] else (lambda c: c.double())
    for g in range(len(sha)):
        for b in range(gro[g], gro[g + 1]):
            N, P = off[b + 1] - off[b], pre[b]
            pages = s["block_table"][b].long().clone()
            pages[:sha[g] // PAGE] = s["block_table"][gro[g], :sha[g] // PAGE].long()
            pages = pages[:-(-(P + N) // PAGE)]
            k, v = (dec(c[pages]).reshape(-1, H, HEAD_DIM)[:P + N] * f
                    for c, f in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
            mask = np.zeros((N, P + N), bool)
            mask[:, :P] = True
            for n in range(N):
                j = n
                while j >= 0:
                    mask[n, P + j] = True
                    j = par[off[b] + j]
            mask = torch.from_numpy(mask).to(k.device)
            q = s["q"][off[b]:off[b + 1]].double()
            r = q.shape[1] // H
            o, l = [], []
            for h in range(H):
                z = torch.einsum("nrd,sd->nrs", q[:, h * r:(h + 1) * r], k[:, h]) * s["sm_scale"]
                z = z.masked_fill(~mask[:, None], -torch.inf)
                l.append(torch.logsumexp(z, -1))
                o.append(torch.einsum("nrs,sd->nrd", (z - l[-1][..., None]).exp(), v[:, h]))
            outs.append(torch.cat(o, 1))
            lses.append(torch.cat(l, 1))
    return dict(out=torch.cat(outs), lse=torch.cat(lses))
