"""Torch-facing calls of the tree-verify hot path.  PyTorch only supplies device memory and the stream;
each function checks dtypes/shapes/devices, passes raw pointers to libjf.so (:mod:`._lib`) and returns.
Nothing here computes any part of the method."""
from __future__ import annotations

import contextlib
from typing import Optional

import torch

from . import _lib

PAGE_SIZE = 16
HEAD_DIM = 128


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, device: torch.device) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} must live on {device}, got {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


class AttentionWorkspace:
    """Scratch for :func:`tree_attention` (partial results of split work units).  One per stream;
    needs no initialisation and is reusable across calls."""

    def __init__(self, device: torch.device):
        n = _lib.lib().jf_tree_attention_workspace_size(0, 0, 0, 0)
        self.buf = torch.empty(n, dtype=torch.uint8, device=device)

    @property
    def nbytes(self) -> int:
        return self.buf.numel()


def tree_attention(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                   prefix_lens: torch.Tensor, tree_offsets: torch.Tensor, parent: torch.Tensor, sm_scale: float,
                   out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                   workspace: Optional[AttentionWorkspace] = None, dev_status: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """jf_tree_attention: q bf16 [T, Hq, 128]; k/v_cache bf16 [pages, 16, Hkv, 128]; block_table int32
    [B, max_pages]; prefix_lens int32 [B]; tree_offsets int32 [B+1]; parent int32 [T].  Returns out."""
    dev = q.device
    T, Hq, D = q.shape
    num_pages, page, Hkv, D2 = k_cache.shape
    _need(q, "q", torch.bfloat16, dev)
    _need(k_cache, "k_cache", torch.bfloat16, dev)
    _need(v_cache, "v_cache", torch.bfloat16, dev)
    for name, t in (("block_table", block_table), ("prefix_lens", prefix_lens), ("tree_offsets", tree_offsets),
                    ("parent", parent)):
        _need(t, name, torch.int32, dev)
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    B = prefix_lens.numel()
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, dev)
    if lse is not None:
        _need(lse, "lse", torch.float32, dev)
    if workspace is None:
        workspace = AttentionWorkspace(dev)
    code = _lib.lib().jf_tree_attention(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_table), block_table.shape[1] if block_table.dim() == 2 else 0,
        _ptr(prefix_lens), _ptr(tree_offsets), _ptr(parent), B, T, Hq, Hkv, D, page, num_pages, float(sm_scale),
        _ptr(out), _ptr(lse), _ptr(workspace.buf), workspace.nbytes, _ptr(dev_status), _stream(stream))
    _lib.check("jf_tree_attention", code)
    return out


def tree_attention_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: float,
                       v_scale: float, block_table: torch.Tensor, prefix_lens: torch.Tensor, tree_offsets: torch.Tensor,
                       parent: torch.Tensor, sm_scale: float, out: Optional[torch.Tensor] = None,
                       lse: Optional[torch.Tensor] = None, workspace: Optional[AttentionWorkspace] = None,
                       dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """jf_tree_attention_fp8: as :func:`tree_attention`, with k/v_cache uint8 E4M3 codes [pages, 16, Hkv, 128]
    standing for decode(code) * k_scale / v_scale.  Returns out (bf16)."""
    dev = q.device
    T, Hq, D = q.shape
    num_pages, page, Hkv, D2 = k_cache.shape
    _need(q, "q", torch.bfloat16, dev)
    _need(k_cache, "k_cache", torch.uint8, dev)
    _need(v_cache, "v_cache", torch.uint8, dev)
    for name, t in (("block_table", block_table), ("prefix_lens", prefix_lens), ("tree_offsets", tree_offsets),
                    ("parent", parent)):
        _need(t, name, torch.int32, dev)
    if v_cache.shape != k_cache.shape:
        raise ValueError("k_cache and v_cache shapes differ")
    B = prefix_lens.numel()
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, dev)
    if lse is not None:
        _need(lse, "lse", torch.float32, dev)
    if workspace is None:
        workspace = AttentionWorkspace(dev)
    code = _lib.lib().jf_tree_attention_fp8(
        _ptr(q), _ptr(k_cache), _ptr(v_cache), float(k_scale), float(v_scale), _ptr(block_table),
        block_table.shape[1] if block_table.dim() == 2 else 0, _ptr(prefix_lens), _ptr(tree_offsets), _ptr(parent), B,
        T, Hq, Hkv, D, page, num_pages, float(sm_scale), _ptr(out), _ptr(lse), _ptr(workspace.buf), workspace.nbytes,
        _ptr(dev_status), _stream(stream))
    _lib.check("jf_tree_attention_fp8", code)
    return out


def build_tree_workspace(batch: int, depths: int, vocab: int, topk: int, device) -> torch.Tensor:
    n = _lib.lib().jf_build_tree_workspace_size(batch, depths, vocab, topk)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def build_tree(draft_logits: torch.Tensor, root_tokens: torch.Tensor, topk: int, budget: int, max_depth: int,
               workspace: Optional[torch.Tensor] = None, out: Optional[dict] = None,
               dev_status: Optional[torch.Tensor] = None, stream=None) -> dict:
    """jf_build_tree: draft_logits fp32 [B, depths, V], root_tokens int32 [B] -> dict of parent, token,
    depth (int32 [B, budget]) and score (fp32 [B, budget])."""
    dev = draft_logits.device
    B, depths, V = draft_logits.shape
    _need(draft_logits, "draft_logits", torch.float32, dev)
    _need(root_tokens, "root_tokens", torch.int32, dev)
    if out is None:
        out = dict(parent=torch.empty(B, budget, dtype=torch.int32, device=dev),
                   token=torch.empty(B, budget, dtype=torch.int32, device=dev),
                   score=torch.empty(B, budget, dtype=torch.float32, device=dev),
                   depth=torch.empty(B, budget, dtype=torch.int32, device=dev))
    if workspace is None:
        workspace = build_tree_workspace(B, depths, V, topk, dev)
    code = _lib.lib().jf_build_tree(
        _ptr(draft_logits), _ptr(root_tokens), B, depths, V, topk, budget, max_depth, _ptr(out["parent"]),
        _ptr(out["token"]), _ptr(out["score"]), _ptr(out.get("depth")), _ptr(workspace), workspace.numel(),
        _ptr(dev_status), _stream(stream))
    _lib.check("jf_build_tree", code)
    return out


class FrontierTree:
    """A batch of trees grown round by round with :func:`expand_frontier`: the tree arrays (parent, token, depth
    int32 [B, budget], score fp32 [B, budget]), the node counts and frontier starts (int32 [B]) and the state the
    library carries between rounds.  ``reset()`` starts new trees (the next round creates the roots)."""

    def __init__(self, batch: int, budget: int, topk: int, device):
        self.batch, self.budget, self.topk = batch, budget, topk
        self.parent = torch.full((batch, budget), -1, dtype=torch.int32, device=device)
        self.token = torch.zeros(batch, budget, dtype=torch.int32, device=device)
        self.depth = torch.zeros(batch, budget, dtype=torch.int32, device=device)
        self.score = torch.zeros(batch, budget, dtype=torch.float32, device=device)
        self.num_nodes = torch.zeros(batch, dtype=torch.int32, device=device)
        self.frontier_begin = torch.zeros(batch, dtype=torch.int32, device=device)
        n = _lib.lib().jf_expand_frontier_state_size(batch, budget, topk)
        self.state = torch.empty(max(n, 256), dtype=torch.uint8, device=device)

    def reset(self) -> None:
        self.num_nodes.zero_()
        self.frontier_begin.zero_()


def expand_frontier_workspace(batch: int, frontier_rows: int, vocab: int, device) -> torch.Tensor:
    n = _lib.lib().jf_expand_frontier_workspace_size(batch, frontier_rows, vocab)
    return torch.empty(max(n, 16), dtype=torch.uint8, device=device)


def expand_frontier(node_logits: torch.Tensor, root_tokens: torch.Tensor, tree: FrontierTree, max_depth: int,
                    width: int, workspace: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None,
                    stream=None) -> FrontierTree:
    """jf_expand_frontier: one round.  node_logits fp32 [B, F, V] (row j of sequence b = the draft head's logits at
    node tree.frontier_begin[b] + j); root_tokens int32 [B].  Updates ``tree`` in place and returns it."""
    dev = node_logits.device
    B, F, V = node_logits.shape
    _need(node_logits, "node_logits", torch.float32, dev)
    _need(root_tokens, "root_tokens", torch.int32, dev)
    if B != tree.batch:
        raise ValueError("node_logits and tree have different batch sizes")
    if workspace is None:
        workspace = expand_frontier_workspace(B, F, V, dev)
    code = _lib.lib().jf_expand_frontier(
        _ptr(node_logits), _ptr(root_tokens), B, F, V, tree.topk, tree.budget, max_depth, width, _ptr(tree.parent),
        _ptr(tree.token), _ptr(tree.score), _ptr(tree.depth), _ptr(tree.num_nodes), _ptr(tree.frontier_begin),
        _ptr(tree.state), tree.state.numel(), _ptr(workspace), workspace.numel(), _ptr(dev_status), _stream(stream))
    _lib.check("jf_expand_frontier", code)
    return tree


def accept(token: torch.Tensor, parent: torch.Tensor, target_logits: torch.Tensor, max_depth: int,
           out: Optional[dict] = None, dev_status: Optional[torch.Tensor] = None, stream=None) -> dict:
    """jf_accept: token, parent int32 [B, N]; target_logits fp32 [B, N, V] -> dict of accepted_len int32 [B],
    path int32 [B, max_depth + 1], bonus int32 [B]."""
    dev = target_logits.device
    B, N, V = target_logits.shape
    _need(token, "token", torch.int32, dev)
    _need(parent, "parent", torch.int32, dev)
    _need(target_logits, "target_logits", torch.float32, dev)
    if out is None:
        out = dict(accepted_len=torch.empty(B, dtype=torch.int32, device=dev),
                   path=torch.empty(B, max_depth + 1, dtype=torch.int32, device=dev),
                   bonus=torch.empty(B, dtype=torch.int32, device=dev))
    code = _lib.lib().jf_accept(_ptr(token), _ptr(parent), _ptr(target_logits), B, N, V, max_depth,
                                _ptr(out["accepted_len"]), _ptr(out["path"]), _ptr(out["bonus"]), _ptr(dev_status),
                                _stream(stream))
    _lib.check("jf_accept", code)
    return out


def commit_kv(k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor, prefix_lens: torch.Tensor,
              tree_offsets: torch.Tensor, path: torch.Tensor, accepted_len: torch.Tensor,
              new_prefix_lens: Optional[torch.Tensor] = None, dev_status: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """jf_commit_kv: moves the accepted path's K/V (path, accepted_len as :func:`accept` returns them) to slots
    P + 1 .. P + L of each sequence, in place in k_cache / v_cache bf16 [pages, 16, Hkv, 128].  Returns
    new_prefix_lens int32 [B] (= P + L + 1; it may be prefix_lens itself)."""
    dev = k_cache.device
    _need(k_cache, "k_cache", torch.bfloat16, dev)
    _need(v_cache, "v_cache", torch.bfloat16, dev)
    for t, name in ((block_table, "block_table"), (prefix_lens, "prefix_lens"), (tree_offsets, "tree_offsets"),
                    (path, "path"), (accepted_len, "accepted_len")):
        _need(t, name, torch.int32, dev)
    if k_cache.shape != v_cache.shape or k_cache.dim() != 4:
        raise ValueError("k_cache and v_cache must both be [pages, 16, Hkv, 128]")
    num_pages, page, Hkv, D = k_cache.shape
    B = prefix_lens.shape[0]
    if path.dim() != 2 or path.shape[0] != B:
        raise ValueError("path must be [B, max_depth + 1]")
    if new_prefix_lens is None:
        new_prefix_lens = torch.empty(B, dtype=torch.int32, device=dev)
    _need(new_prefix_lens, "new_prefix_lens", torch.int32, dev)
    code = _lib.lib().jf_commit_kv(_ptr(k_cache), _ptr(v_cache), _ptr(block_table), block_table.shape[1],
                                   _ptr(prefix_lens), _ptr(tree_offsets), _ptr(path), _ptr(accepted_len), B,
                                   path.shape[1] - 1, Hkv, D, page, num_pages, _ptr(new_prefix_lens), _ptr(dev_status),
                                   _stream(stream))
    _lib.check("jf_commit_kv", code)
    return new_prefix_lens


def tree_kv_append(k_new: torch.Tensor, v_new: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   block_table: torch.Tensor, prefix_lens: torch.Tensor, tree_offsets: torch.Tensor,
                   depth: torch.Tensor, rope_theta: float, q: Optional[torch.Tensor] = None,
                   dev_status: Optional[torch.Tensor] = None, stream=None) -> None:
    """jf_tree_kv_append: k_new, v_new bf16 [T, Hkv, 128] of the tree tokens go to cache slots P + j of their
    sequences, K rotated at position P + depth; q bf16 [T, Hq, 128], when given, is rotated in place."""
    dev = k_cache.device
    for t, name in ((k_new, "k_new"), (v_new, "v_new"), (k_cache, "k_cache"), (v_cache, "v_cache")):
        _need(t, name, torch.bfloat16, dev)
    for t, name in ((block_table, "block_table"), (prefix_lens, "prefix_lens"), (tree_offsets, "tree_offsets"),
                    (depth, "depth")):
        _need(t, name, torch.int32, dev)
    if q is not None:
        _need(q, "q", torch.bfloat16, dev)
    if k_cache.shape != v_cache.shape or k_cache.dim() != 4 or k_new.shape != v_new.shape or k_new.dim() != 3:
        raise ValueError("caches must be [pages, 16, Hkv, 128] and k_new / v_new [T, Hkv, 128]")
    num_pages, page, Hkv, D = k_cache.shape
    T = k_new.shape[0]
    if depth.numel() != T or (q is not None and q.shape[0] != T):
        raise ValueError("depth must have one entry per tree node, q one row per node")
    B = prefix_lens.shape[0]
    code = _lib.lib().jf_tree_kv_append(_ptr(k_new), _ptr(v_new), _ptr(q), _ptr(k_cache), _ptr(v_cache),
                                        _ptr(block_table), block_table.shape[1], _ptr(prefix_lens), _ptr(tree_offsets),
                                        _ptr(depth), B, T, q.shape[1] if q is not None else 0, Hkv, D, page, num_pages,
                                        float(rope_theta), _ptr(dev_status), _stream(stream))
    _lib.check("jf_tree_kv_append", code)


# ----------------------------------------------------------------------------------------------
# Serving several sampled continuations of one prompt (include/jf_serving.h)
# ----------------------------------------------------------------------------------------------
_LOGITS_TYPE = {torch.float32: 0, torch.bfloat16: 1}


def _call(fn: str, dev: torch.device, stream, *args) -> None:
    """Calls a library function with ``dev`` current and, without a stream of the caller's, on that device's current
    stream (the stream is the call's last argument)."""
    if dev.type != "cuda":
        raise ValueError(f"the tensors must live on a CUDA device, got {dev}")
    s = torch.cuda.current_stream(dev).cuda_stream if stream is None else _stream(stream)
    call = getattr(_lib.lib(), fn)
    if dev.index is None or dev.index == torch.cuda.current_device():
        code = call(*args, s)
    else:
        with torch.cuda.device(dev):
            code = call(*args, s)
    _lib.check(fn, code)


def _allocating_on(stream, dev: torch.device):
    """Allocations for a call on a stream of the caller's come from that stream's memory: a block of another stream may
    still be in use by work queued there."""
    if stream is None or dev.type != "cuda":
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else
                             torch.cuda.ExternalStream(_stream(stream), device=dev))


def _need_status(dev_status: Optional[torch.Tensor], dev: torch.device) -> None:
    if dev_status is not None:
        _need(dev_status, "dev_status", torch.int32, dev)
        if dev_status.numel() < 1:
            raise ValueError("dev_status must hold one int32")


def _sampling_params(n: int, dev: torch.device, temperature, top_k, top_p, min_p) -> list:
    """Checks the per-row sampling parameters; top_k, top_p and min_p may be None (off)."""
    for t, name, dtype in ((temperature, "temperature", torch.float32), (top_k, "top_k", torch.int32),
                           (top_p, "top_p", torch.float32), (min_p, "min_p", torch.float32)):
        if t is None and name != "temperature":
            continue
        _need(t, name, dtype, dev)
        if t.shape != (n,):
            raise ValueError(f"{name} must be [{n}], got {list(t.shape)}")
    return [_ptr(temperature), _ptr(top_k), _ptr(top_p), _ptr(min_p)]


def _outputs(out: Optional[dict], dev: torch.device, stream, **want) -> dict:
    """``out`` after a check of the tensors it holds, or newly allocated ones; want: name=(shape, dtype).  The last
    of the names, the log-probabilities, may be left out of ``out``."""
    if out is None:
        with _allocating_on(stream, dev):
            return {k: torch.empty(shape, dtype=dtype, device=dev) for k, (shape, dtype) in want.items()}
    for k, (shape, dtype) in want.items():
        if k == "logprob" and out.get(k) is None:
            continue
        _need(out[k], k, dtype, dev)
        if tuple(out[k].shape) != shape:
            raise ValueError(f"{k} must be {list(shape)}, got {list(out[k].shape)}")
    return out


def sample(logits: torch.Tensor, u: torch.Tensor, temperature: torch.Tensor, top_k: Optional[torch.Tensor] = None,
           top_p: Optional[torch.Tensor] = None, min_p: Optional[torch.Tensor] = None, out: Optional[dict] = None,
           dev_status: Optional[torch.Tensor] = None, stream=None) -> dict:
    """jf_sample: logits fp32 or bf16 [R, V] (rows may be strided, entries not; they start on a 16-byte boundary), u and
    temperature fp32 [R] (u in [0, 1); temperature 0 = greedy), top_k int32 [R] (0 = off), top_p fp32 [R] (1 = off),
    min_p fp32 [R] (0 = off), each of the last three optional -> dict of token int32 [R] and logprob fp32 [R]."""
    dev = logits.device
    if logits.dtype not in _LOGITS_TYPE:
        raise TypeError(f"logits must be float32 or bfloat16, got {logits.dtype}")
    if logits.dim() != 2 or (logits.numel() and logits.stride(1) != 1):
        raise ValueError("logits must be [R, V] with consecutive entries")
    R, V = logits.shape
    stride = logits.stride(0) if R > 1 else V
    _need(u, "u", torch.float32, dev)
    if u.shape != (R,):
        raise ValueError(f"u must be [{R}], got {list(u.shape)}")
    params = _sampling_params(R, dev, temperature, top_k, top_p, min_p)
    _need_status(dev_status, dev)
    out = _outputs(out, dev, stream, token=((R,), torch.int32), logprob=((R,), torch.float32))
    _call("jf_sample", dev, stream, _ptr(logits), _LOGITS_TYPE[logits.dtype], stride, R, V, _ptr(u), *params,
          _ptr(out["token"]), _ptr(out.get("logprob")), _ptr(dev_status))
    return out


def accept_sampled(token: torch.Tensor, parent: torch.Tensor, target_logits: torch.Tensor, u: torch.Tensor,
                   temperature: torch.Tensor, max_depth: int, top_k: Optional[torch.Tensor] = None,
                   top_p: Optional[torch.Tensor] = None, min_p: Optional[torch.Tensor] = None,
                   out: Optional[dict] = None, dev_status: Optional[torch.Tensor] = None, stream=None) -> dict:
    """jf_accept_sampled: :func:`accept` with a token sampled per step in place of the argmax.  token, parent int32
    [B, N]; target_logits fp32 or bf16 [B, N, V]; u fp32 [B, max_depth + 1]; the parameters of :func:`sample` per
    sequence, [B] -> dict of accepted_len int32 [B], path int32 [B, max_depth + 1], bonus int32 [B] and logprob fp32
    [B, max_depth + 1] (of the token drawn at each step of the walk)."""
    dev = target_logits.device
    if target_logits.dtype not in _LOGITS_TYPE:
        raise TypeError(f"target_logits must be float32 or bfloat16, got {target_logits.dtype}")
    _need(target_logits, "target_logits", target_logits.dtype, dev)
    if target_logits.dim() != 3:
        raise ValueError("target_logits must be [B, N, V]")
    B, N, V = target_logits.shape
    for t, name in ((token, "token"), (parent, "parent")):
        _need(t, name, torch.int32, dev)
        if t.shape != (B, N):
            raise ValueError(f"{name} must be [{B}, {N}], got {list(t.shape)}")
    _need(u, "u", torch.float32, dev)
    if max_depth < 0 or u.shape != (B, max_depth + 1):
        raise ValueError(f"u must be [{B}, max_depth + 1] with max_depth >= 0, got {list(u.shape)}")
    params = _sampling_params(B, dev, temperature, top_k, top_p, min_p)
    _need_status(dev_status, dev)
    out = _outputs(out, dev, stream, accepted_len=((B,), torch.int32), path=((B, max_depth + 1), torch.int32),
                   bonus=((B,), torch.int32), logprob=((B, max_depth + 1), torch.float32))
    _call("jf_accept_sampled", dev, stream, _ptr(token), _ptr(parent), _ptr(target_logits),
          _LOGITS_TYPE[target_logits.dtype], _ptr(u), *params, B, N, V, max_depth, _ptr(out["accepted_len"]),
          _ptr(out["path"]), _ptr(out["bonus"]), _ptr(out.get("logprob")), _ptr(dev_status))
    return out


class SharedAttentionWorkspace:
    """Scratch for :func:`tree_attention_shared` calls of up to ``total_nodes`` tree nodes with ``num_q_heads`` heads.
    One per stream; needs no initialisation and is reusable across calls."""

    def __init__(self, total_nodes: int, num_q_heads: int, device):
        n = _lib.lib().jf_tree_attention_shared_workspace_size(total_nodes, num_q_heads)
        self.buf = torch.empty(n, dtype=torch.uint8, device=device)

    @property
    def nbytes(self) -> int:
        return self.buf.numel()


def _attention_shared(fn, cache_dtype, scales, q, k_cache, v_cache, block_table, prefix_lens, tree_offsets, parent,
                      group_offsets, shared_lens, sm_scale, out, lse, workspace, dev_status, stream):
    dev = q.device
    _need(q, "q", torch.bfloat16, dev)
    _need(k_cache, "k_cache", cache_dtype, dev)
    _need(v_cache, "v_cache", cache_dtype, dev)
    for name, t in (("block_table", block_table), ("prefix_lens", prefix_lens), ("tree_offsets", tree_offsets),
                    ("parent", parent), ("group_offsets", group_offsets), ("shared_lens", shared_lens)):
        _need(t, name, torch.int32, dev)
    if q.dim() != 3 or k_cache.dim() != 4 or v_cache.shape != k_cache.shape:
        raise ValueError("q must be [T, Hq, 128], k_cache and v_cache both [pages, 16, Hkv, 128]")
    T, Hq, D = q.shape
    num_pages, page, Hkv, cache_dim = k_cache.shape
    B, G = prefix_lens.numel(), shared_lens.numel()
    if cache_dim != D:
        raise ValueError("q and the caches have different head dimensions")
    if block_table.dim() != 2 or block_table.shape[0] != B or tree_offsets.numel() != B + 1:
        raise ValueError("block_table must be [B, max_pages] and tree_offsets [B + 1]")
    if group_offsets.numel() != G + 1 or parent.numel() != T:
        raise ValueError("group_offsets must be [G + 1] for G shared_lens, parent [T]")
    _need_status(dev_status, dev)
    if out is None:
        with _allocating_on(stream, dev):
            out = torch.empty_like(q)
    _need(out, "out", torch.bfloat16, dev)
    if out.shape != q.shape:
        raise ValueError("out must have q's shape")
    if lse is not None:
        _need(lse, "lse", torch.float32, dev)
        if lse.shape != (T, Hq):
            raise ValueError("lse must be [T, Hq]")
    if workspace is None:
        with _allocating_on(stream, dev):  # freed on return, and not reused but on the same stream
            workspace = SharedAttentionWorkspace(T, Hq, dev)
    elif workspace.buf.device != dev:
        raise ValueError(f"the workspace must be on {dev}, got {workspace.buf.device}")
    _call(fn, dev, stream, _ptr(q), _ptr(k_cache), _ptr(v_cache), *scales, _ptr(block_table), block_table.shape[1],
          _ptr(prefix_lens), _ptr(tree_offsets), _ptr(parent), _ptr(group_offsets), _ptr(shared_lens), G, B, T, Hq, Hkv,
          D, page, num_pages, float(sm_scale), _ptr(out), _ptr(lse), _ptr(workspace.buf), workspace.nbytes,
          _ptr(dev_status))
    return out


def tree_attention_shared(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                          prefix_lens: torch.Tensor, tree_offsets: torch.Tensor, parent: torch.Tensor,
                          group_offsets: torch.Tensor, shared_lens: torch.Tensor, sm_scale: float,
                          out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                          workspace: Optional[SharedAttentionWorkspace] = None,
                          dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """jf_tree_attention_shared: :func:`tree_attention` of a batch made of groups of consecutive sequences, group g =
    sequences [group_offsets[g], group_offsets[g + 1]) (int32 [G + 1]) with the first shared_lens[g] tokens (int32 [G])
    in common; the whole pages of that prefix are read through the group's first block-table row, once for all its
    nodes.  Returns out."""
    return _attention_shared("jf_tree_attention_shared", torch.bfloat16, (), q, k_cache, v_cache, block_table,
                             prefix_lens, tree_offsets, parent, group_offsets, shared_lens, sm_scale, out, lse,
                             workspace, dev_status, stream)


def tree_attention_shared_fp8(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scale: float,
                              v_scale: float, block_table: torch.Tensor, prefix_lens: torch.Tensor,
                              tree_offsets: torch.Tensor, parent: torch.Tensor, group_offsets: torch.Tensor,
                              shared_lens: torch.Tensor, sm_scale: float, out: Optional[torch.Tensor] = None,
                              lse: Optional[torch.Tensor] = None,
                              workspace: Optional[SharedAttentionWorkspace] = None,
                              dev_status: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """jf_tree_attention_shared_fp8: as :func:`tree_attention_shared`, with k/v_cache uint8 E4M3 codes [pages, 16, Hkv,
    128] standing for decode(code) * k_scale / v_scale.  Returns out (bf16)."""
    return _attention_shared("jf_tree_attention_shared_fp8", torch.uint8, (float(k_scale), float(v_scale)), q, k_cache,
                             v_cache, block_table, prefix_lens, tree_offsets, parent, group_offsets, shared_lens,
                             sm_scale, out, lse, workspace, dev_status, stream)
