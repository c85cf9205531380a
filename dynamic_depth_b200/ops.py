"""Serving operators over a caller-owned paged cache (include/tl.h, "serving operators").

Marshalling only: shapes, types and strides are checked here, everything else by the library.  Every call runs on
the current stream of its tensors' device and allocates only its outputs (and a workspace where none is given).

No operator has a backward form: outside torch.no_grad() a tensor that requires a gradient is refused.  What only the
device sees (a page id, a slot, a length, a wait that ran out) skips its access and sets a bit of `status`, an int32
tensor of one element that the caller clears and reads; without one it goes unreported.

The cache is one tensor of pages, [n_pages, 2 (keys, values), kv heads, page tokens, head width], fp16 or bf16.
"""
from __future__ import annotations

import ctypes as C
from typing import NamedTuple, Optional

import torch

from ._lib import TL_BF16, TL_F16, TL_F32, TlKvPool, check, lib

_DT = {torch.float32: TL_F32, torch.float16: TL_F16, torch.bfloat16: TL_BF16}


class TokenLogprobs(NamedTuple):
    """Outputs of token_logprobs, one row per row of logits (None where not asked for)."""
    logprob: Optional[torch.Tensor]
    rank: Optional[torch.Tensor]
    entropy: torch.Tensor
    lse: torch.Tensor
    top_ids: Optional[torch.Tensor]
    top_logprobs: Optional[torch.Tensor]


class BatchPlan(NamedTuple):
    """Outputs of plan_batch (the block table is extended in place)."""
    cu: torch.Tensor
    lens: torch.Tensor
    granted: torch.Tensor
    free_head: torch.Tensor
    slots: torch.Tensor
    positions: torch.Tensor
    masks: Optional[torch.Tensor]


def _need(ok, what):
    if not ok:
        raise ValueError(what)


def _forward_only():
    """A call was given a tensor that requires a gradient."""
    if torch.is_grad_enabled():
        raise ValueError("no backward form: detach the tensors or call under torch.no_grad()")


def _flat(t, dtype, n, name, dev):
    """A contiguous vector of n elements on CUDA device `dev` (None passes as a null pointer)."""
    if t is None:
        return None
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous() or t.get_device() != dev:
        raise ValueError(f"{name}: a contiguous {dtype} tensor of {n} elements on cuda:{dev} is wanted")
    return t.data_ptr()


def _at(t):
    return None if t is None else t.data_ptr()


# A call costs its wrapper before it costs the GPU anything: streams and outputs come from torch's raw entry points
# where it has them (0.1 against 3.3 us for the current stream, 0.6 against 2.3 us for an empty tensor), and devices
# are compared by index.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda i: torch.cuda.current_stream(i).cuda_stream)
_current = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
try:
    from torch._C._dynamo.guards import _empty_strided_cuda as _alloc  # (sizes, strides, dtype), on the current device
except ImportError:
    def _alloc(sizes, strides, dtype):
        return torch.empty(sizes, dtype=dtype, device="cuda")


def _elsewhere(dev):
    """Whether a call's device is not the current one (it then runs again with that made current)."""
    if dev < 0:
        raise ValueError("the tensors must be on a CUDA device")
    return dev != _current()


def _pool(pool) -> TlKvPool:
    _need(pool.dim() == 5 and pool.shape[1] == 2 and pool.is_contiguous() and pool.dtype in _DT,
          "pool: a contiguous [pages, 2, kv heads, page tokens, head width] tensor of fp16 or bf16 is wanted")
    n, _, h, p, d = pool.shape
    return TlKvPool(pool.data_ptr(), n, _DT[pool.dtype], h, d, p)


def token_logprobs(logits, targets=None, n_top: int = 0) -> TokenLogprobs:
    """Log probability and rank of each row's target, entropy, log-sum-exp and the n_top best tokens of logits
    [rows, vocab] (fp32, fp16 or bf16; rows may be strided).  targets int32 [rows], -1 for none."""
    if logits.requires_grad:
        _forward_only()
    _need(logits.dim() == 2 and logits.dtype in _DT and (logits.shape[1] <= 1 or logits.stride(1) == 1),
          "logits: [rows, vocab] of fp32, fp16 or bf16 with adjacent columns is wanted")
    rows, vocab = logits.shape
    dev = logits.get_device()
    f32, i32 = torch.float32, torch.int32
    tp = _flat(targets, i32, rows, "targets", dev)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return token_logprobs(logits, targets, n_top)
    lp = rank = ids = top = None
    one = (rows,), (1,)
    if targets is not None:
        lp, rank = _alloc(*one, f32), _alloc(*one, i32)
    ent, lse = _alloc(*one, f32), _alloc(*one, f32)
    if n_top:
        _need(n_top > 0, "n_top: 0 or more")
        ids, top = _alloc((rows, n_top), (n_top, 1), i32), _alloc((rows, n_top), (n_top, 1), f32)
    check(lib().tl_token_logprobs(
        logits.data_ptr(), _DT[logits.dtype], rows, vocab, logits.stride(0) if rows > 1 else vocab, tp, n_top,
        _at(lp), _at(rank), ent.data_ptr(), lse.data_ptr(), _at(ids), _at(top), _raw_stream(dev)),
        "tl_token_logprobs")
    return TokenLogprobs(lp, rank, ent, lse, ids, top)


def plan_batch(cached, fresh, block_table, free_pages, free_head, page_tokens: int, n_rows: int, parents=None,
               mask_words: int = 0, status=None) -> BatchPlan:
    """Row offsets, slots, positions and tree masks of a batch's new tokens from the request lengths; the block table
    [R, max_pages] (int32) gets the pages granted from free_pages[free_head[0]:].  n_rows: rows of the row outputs
    (at least the sum of fresh; rows past that sum are rows of no token: slot -1, position 0, no mask bits)."""
    R = cached.numel()
    dev = cached.get_device()
    _need(block_table.dim() == 2 and block_table.shape[0] == R and block_table.dtype == torch.int32
          and block_table.is_contiguous() and block_table.get_device() == dev,
          "block_table: a contiguous int32 [R, max_pages] tensor is wanted")
    _need(free_pages.dim() == 1, "free_pages: a vector is wanted")
    i32 = torch.int32
    args = (_flat(cached, i32, R, "cached", dev), _flat(fresh, i32, R, "fresh", dev), R, page_tokens,
            block_table.data_ptr(), block_table.shape[1],
            _flat(free_pages, i32, free_pages.numel(), "free_pages", dev), free_pages.numel(),
            _flat(free_head, i32, 1, "free_head", dev), _flat(parents, i32, n_rows, "parents", dev), n_rows,
            mask_words)
    st = _flat(status, i32, 1, "status", dev)
    _need(0 <= mask_words <= 8 and 0 <= n_rows < 1 << 31, "mask_words 0 .. 8 and n_rows of 0 or more are wanted")
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return plan_batch(cached, fresh, block_table, free_pages, free_head, page_tokens, n_rows, parents,
                              mask_words, status)
    per_request = (R,), (1,)
    cu, lens, granted = _alloc((R + 1,), (1,), i32), _alloc(*per_request, i32), _alloc(*per_request, i32)
    head = _alloc((1,), (1,), i32)
    slots, pos = _alloc((n_rows,), (1,), torch.int64), _alloc((n_rows,), (1,), i32)
    masks = _alloc((n_rows, mask_words), (mask_words, 1), i32) if mask_words else None
    check(lib().tl_plan_batch_padded(*args, cu.data_ptr(), lens.data_ptr(), granted.data_ptr(), head.data_ptr(),
                                     slots.data_ptr(), pos.data_ptr(), _at(masks), st, _raw_stream(dev)),
          "tl_plan_batch_padded")
    return BatchPlan(cu, lens, granted, head, slots, pos, masks)


def rope_table(length: int, head_dim: int, base: float = 1e4, device="cuda") -> torch.Tensor:
    """(cos, sin) of position * base^(-2i / head_dim): fp32 [length, head_dim / 2, 2], angles in fp64."""
    with torch.cuda.device(device):
        t = torch.empty((length, head_dim // 2, 2), dtype=torch.float32, device="cuda")
        check(lib().tl_rope_table(t.data_ptr(), length, head_dim, float(base), _raw_stream(t.device.index)),
              "tl_rope_table")
    return t


def norm_rope_append(qkv, n_heads: int, pool, slots, positions, rope, q_gain=None, k_gain=None, eps: float = 1e-6,
                     q_out=None, status=None) -> torch.Tensor:
    """Per-head RMSNorm (with gains) and rotation of the queries and keys of qkv [rows, (q | k | v) heads * width],
    keys and values stored at `slots` of the pool; returns the queries [rows, n_heads, width] in the pool's type."""
    if (qkv.requires_grad or pool.requires_grad or rope.requires_grad or q_gain is not None and q_gain.requires_grad
            or k_gain is not None and k_gain.requires_grad or q_out is not None and q_out.requires_grad):
        _forward_only()
    p = _pool(pool)
    dev, rows, hd = pool.get_device(), qkv.shape[0], p.head_dim
    _need(qkv.dim() == 2 and qkv.dtype in _DT and qkv.shape[1] == (n_heads + 2 * p.n_kv_heads) * hd
          and qkv.stride(1) == 1 and qkv.get_device() == dev, "qkv: [rows, (q + 2 kv heads) * width] of the pool's device")
    _need(rope.dim() == 3 and rope.shape[1:] == (hd // 2, 2), "rope: a rope_table of the pool's head width is wanted")
    i32, f32 = torch.int32, torch.float32
    sp = _flat(slots, torch.int64, rows, "slots", dev)
    pp = _flat(positions, i32, rows, "positions", dev)
    rp = _flat(rope, f32, rope.numel(), "rope", dev)
    gq, gk = _flat(q_gain, f32, hd, "q_gain", dev), _flat(k_gain, f32, hd, "k_gain", dev)
    st = _flat(status, i32, 1, "status", dev)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return norm_rope_append(qkv, n_heads, pool, slots, positions, rope, q_gain, k_gain, eps, q_out, status)
    if q_out is None:
        q_out = _alloc((rows, n_heads, hd), (n_heads * hd, hd, 1), pool.dtype)
    qp = _flat(q_out, pool.dtype, rows * n_heads * hd, "q_out", dev)
    check(lib().tl_norm_rope_append(qkv.data_ptr(), _DT[qkv.dtype], rows, qkv.stride(0) if rows > 1 else qkv.shape[1],
                                    n_heads, gq, gk, eps, rp, rope.shape[0], pp, sp, C.byref(p), qp, st,
                                    _raw_stream(dev)), "tl_norm_rope_append")
    return q_out


_workspace_sizes = {}


def _workspace_bytes(hd, H, Hk, max_nodes, device_index):
    key = (hd, H, Hk, max_nodes, device_index)
    n = _workspace_sizes.get(key)
    if n is None:
        c = C.c_size_t()
        check(lib().tl_tree_attention_workspace(hd, H, Hk, max_nodes, C.byref(c)), "tl_tree_attention_workspace")
        n = _workspace_sizes[key] = c.value
    return n


def tree_attention_workspace(head_dim: int, n_heads: int, n_kv_heads: int, max_nodes: int, device="cuda"):
    """A workspace for tree_attention calls of these sizes (one per call that may run at the same time)."""
    with torch.cuda.device(device):
        n = _workspace_bytes(head_dim, n_heads, n_kv_heads, max_nodes, _current())
        return torch.empty(n, dtype=torch.uint8, device="cuda")


def tree_attention(q, pool, block_table, ctx_lens, cu, max_nodes: int, masks=None, scale: float = 0.0, out=None,
                   return_lse: bool = False, workspace=None, status=None):
    """Attention of draft trees over the pool's pages: rows cu[r] .. cu[r+1] of q [rows, heads, width] see request r's
    first ctx_lens[r] positions and the nodes behind them that their mask words name (None: the earlier nodes and
    themselves).  out: a given tensor's type (the pool's or fp32), else the pool's; it may be q.  Rows of no request are
    left as they are, so in a new tensor undefined.  Returns out, or (out, lse)."""
    if q.requires_grad or pool.requires_grad or out is not None and out.requires_grad:
        _forward_only()
    p = _pool(pool)
    dev, hd = pool.get_device(), p.head_dim
    _need(q.dim() == 3 and q.dtype == pool.dtype and q.shape[2] == hd and q.stride(2) == 1
          and (q.stride(1) == hd or q.shape[1] == 1) and q.get_device() == dev, "q: [rows, heads, width] of the pool's type, heads adjacent")
    rows, H = q.shape[0], q.shape[1]
    R = ctx_lens.numel()
    i32 = torch.int32
    _need(block_table.dim() == 2 and block_table.shape[0] == R and block_table.dtype == i32
          and block_table.is_contiguous() and block_table.get_device() == dev,
          "block_table: a contiguous int32 [R, max_pages] tensor is wanted")
    cp, up = _flat(ctx_lens, i32, R, "ctx_lens", dev), _flat(cu, i32, R + 1, "cu", dev)
    words = 0
    if masks is not None:
        _need(masks.dim() == 2 and masks.shape[0] == rows and masks.shape[1] > 0, "masks: int32 [rows, words] is wanted")
        words = masks.shape[1]
    mp = _flat(masks, i32, rows * words, "masks", dev)
    st = _flat(status, i32, 1, "status", dev)
    if _elsewhere(dev):
        with torch.cuda.device(dev):
            return tree_attention(q, pool, block_table, ctx_lens, cu, max_nodes, masks, scale, out, return_lse,
                                  workspace, status)
    if out is None:
        out = _alloc((rows, H, hd), (H * hd, hd, 1), q.dtype)
    else:
        _need(out.shape == q.shape and out.dtype in _DT and out.stride(2) == 1
              and (out.stride(1) == hd or H == 1) and out.get_device() == dev, "out: the shape of q, heads adjacent")
    lse = _alloc((rows, H), (H, 1), torch.float32) if return_lse else None
    if workspace is None:
        n = _workspace_bytes(hd, H, p.n_kv_heads, max_nodes, dev)
        workspace = _alloc((n,), (1,), torch.uint8)
    else:
        n = workspace.numel() * workspace.element_size()
        _need(workspace.is_contiguous() and workspace.get_device() == dev, "workspace: a tree_attention_workspace is wanted")
    check(lib().tl_tree_attention(
        q.data_ptr(), q.stride(0) if rows > 1 else H * hd, C.byref(p), block_table.data_ptr(),
        block_table.shape[1], cp, up, R, rows, H, max_nodes, mp, words, scale, out.data_ptr(), _DT[out.dtype],
        out.stride(0) if rows > 1 else H * hd, _at(lse), workspace.data_ptr(), n, st, _raw_stream(dev)),
        "tl_tree_attention")
    return (out, lse) if return_lse else out
