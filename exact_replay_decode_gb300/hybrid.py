"""PyTorch-facing binding of the serving operators of gated-delta-rule and attention layers (include/ers.h): prompts and
single tokens of the gated delta rule, attention of a tree of drafts over a paged cache, and the rows it takes.

Marshalling only, as in ops.py and serve.py."""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Tuple

import torch

from . import _abi
from .ops import Status, _finish, _io_from, _IO, _need
from .serve import (LinAttnCache, PagePool, _linattn_dims, _longest, _on_stream, _out, _read_arg, _seqlens, _slot, _status,
                    _tensor, _where)


# ---- gated delta rule --------------------------------------------------------------------------
def _gdn_args(q, k, v, g, beta, io, T, H, G, dk, dv):
    """Checked, as pointers."""
    return (_tensor(q, io, "q", (T, G, dk)), _tensor(k, io, "k", (T, G, dk)), _tensor(v, io, "v", (T, H, dv)),
            _tensor(g, torch.float32, "g", (T, H)), _tensor(beta, torch.float32, "beta", (T, H)))


def _workspace(size: int, device):
    """(The tensor, which has to live until the launch, its pointer and its size.)"""
    if size == 0:
        return None, None, 0
    t = torch.empty(size, dtype=torch.uint8, device=device)
    return t, t.data_ptr(), size


@_on_stream
def gdn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, g: torch.Tensor, beta: torch.Tensor,
            cu_seqlens: Optional[torch.Tensor] = None, init_state: Optional[torch.Tensor] = None, scale: float = 1.0,
            max_seqlen: Optional[int] = None, status: Optional[Status] = None, check: bool = True, stream=None,
            out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The gated delta rule over packed prompts (ers_gdn_fwd).

    q, k [T,G,dk], v [T,H,dv] (bf16 or fp32; dk, dv 64 or 128), g (log-gates, <= 0), beta [T,H] fp32; cu_seqlens, init_state
    and max_seqlen as in linattn_fwd (a short bf16 sequence has the recurrence's bits whatever max_seqlen and its neighbours are;
    ers.h has the workspace that a call allocates).  Returns (o [T,H,dv], final_state [S,H,dv,dk] fp32); a final state may
    start a GdnCache: anchor.copy_(state), read_copy.copy_(state)."""
    io = _io_from(q)
    T, G, dk = q.shape
    H, dv = v.shape[1], v.shape[2]
    dev = q.device
    cu_seqlens, S = _seqlens(cu_seqlens, T, dev)
    qkv = _gdn_args(q, k, v, g, beta, io, T, H, G, dk, dv)
    state = (S, H, dv, dk)
    init = None if init_state is None else _tensor(init_state, torch.float32, "init_state", state)
    if out is None:
        o, final = torch.empty_like(v), torch.empty(state, dtype=torch.float32, device=dev)
    else:
        o, final = out
        _out(o, v)
        _tensor(final, torch.float32, "out[1]", state)
    st = _status(status, check, dev)
    dims, longest = _linattn_dims(H, G, dk, dv, io, float(scale)), _longest(cu_seqlens, T, S, H, max_seqlen)
    keep, *ws = _workspace(_abi.lib().ers_gdn_fwd_workspace_size(dims, S, T, longest), dev)
    code = _abi.lib().ers_gdn_fwd(dims, S, T, longest, cu_seqlens.data_ptr(), *qkv, init, o.data_ptr(), final.data_ptr(),
                                  *ws, *_where(dev, st))
    _finish(code, "ers_gdn_fwd", st, check)
    return o, final


@_on_stream
def gdn_prefill(cache: LinAttnCache, q, k, v, g, beta, cu_seqlens: Optional[torch.Tensor] = None,
                slot: Optional[torch.Tensor] = None, read_page: Optional[torch.Tensor] = None, scale: float = 1.0,
                max_seqlen: Optional[int] = None, status: Optional[Status] = None, check: bool = True, stream=None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Packed prompts that go on from the slots' cached states (ers_gdn_prefill), whose pages are read and written as by
    linattn_prefill.  Returns o [T,H,dv]."""
    T, dev = q.shape[0], q.device
    cu_seqlens, S = _seqlens(cu_seqlens, T, dev)
    qkv = _gdn_args(q, k, v, g, beta, cache.io, T, cache.H, cache.G, cache.dk, cache.dv)
    o = _out(out, v)
    st = _status(status, check, dev)
    dims = _linattn_dims(cache.H, cache.G, cache.dk, cache.dv, cache.io, float(scale))
    longest = _longest(cu_seqlens, T, S, cache.H, max_seqlen)
    keep, *ws = _workspace(_abi.lib().ers_gdn_fwd_workspace_size(dims, S, T, longest), dev)
    code = _abi.lib().ers_gdn_prefill(dims, cache._c, S, T, longest, cu_seqlens.data_ptr(), _slot(slot, S),
                                      _read_arg(read_page, S), *qkv, o.data_ptr(), *ws, *_where(dev, st))
    _finish(code, "ers_gdn_prefill", st, check)
    return o


@_on_stream
def gdn_decode(cache: LinAttnCache, q, k, v, g, beta, slot: Optional[torch.Tensor] = None,
               read_page: Optional[torch.Tensor] = None, scale: float = 1.0, status: Optional[Status] = None,
               check: bool = True, stream=None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token per sequence (ers_gdn_decode): q, k [S,G,dk], v [S,H,dv], g, beta [S,H]; states as in gdn_prefill."""
    S, dev = q.shape[0], q.device
    qkv = _gdn_args(q, k, v, g, beta, cache.io, S, cache.H, cache.G, cache.dk, cache.dv)
    o = _out(out, v)
    st = _status(status, check, dev)
    dims = _linattn_dims(cache.H, cache.G, cache.dk, cache.dv, cache.io, float(scale))
    code = _abi.lib().ers_gdn_decode(dims, cache._c, S, _slot(slot, S), _read_arg(read_page, S), *qkv, o.data_ptr(),
                                     *_where(dev, st))
    _finish(code, "ers_gdn_decode", st, check)
    return o


# ---- attention over a paged cache ---------------------------------------------------------------------
class AttnCache:
    """The keys and values of an attention layer: k, v [npages, page_tokens, kv_heads, head_dim] in the io dtype, under a table
    of slot_pages pages per slot (pages: a PagePool of both), and the tokens in use pos [nslots] int32.

    npages None: nslots * slot_pages, slot s starting out with its share of them.  Otherwise every page starts out free, and
    pages_own(cache.pages, slots) hands them out.  k, v: tensors to use as the pages (they stay the cache's).  The page calls
    do not touch pos: after pages_fork(src, dst) the caller sets pos[dst] = pos[src], after pages_free pos[slot] = 0."""

    k = property(lambda self: self._k)
    v = property(lambda self: self._v)
    pos = property(lambda self: self._pos)
    pages = property(lambda self: self._pages)

    def __init__(self, nslots: int, kv_heads: int, head_dim: int = 128, page_tokens: int = 64, slot_pages: int = 1,
                 npages: Optional[int] = None, io_dtype: torch.dtype = torch.bfloat16, device="cuda",
                 k: Optional[torch.Tensor] = None, v: Optional[torch.Tensor] = None):
        if io_dtype not in _IO:
            raise TypeError(f"io dtype {io_dtype} not supported (bf16 or fp32)")
        if slot_pages < 1 or page_tokens < 1:
            raise ValueError(f"slot_pages {slot_pages}, page_tokens {page_tokens}: expected at least 1")
        self.nslots, self.kv_heads, self.head_dim, self.io = nslots, kv_heads, head_dim, io_dtype
        self.page_tokens, self.slot_pages = page_tokens, slot_pages
        self.npages = nslots * slot_pages if npages is None else npages
        shape = (self.npages, page_tokens, kv_heads, head_dim)
        if (k is None) != (v is None):
            raise ValueError("k, v: expected both or neither")
        if k is None:
            k, v = (torch.zeros(shape, dtype=io_dtype, device=device) for _ in range(2))
        _need(k, io_dtype, "k", shape)
        _need(v, io_dtype, "v", shape)
        d = dict(dtype=torch.int32, device=k.device)
        if npages is None:
            table = torch.arange(self.npages, **d).view(nslots, slot_pages)
        else:
            table = torch.full((nslots, slot_pages), -1, **d)
        refs = torch.full((self.npages,), int(npages is None), **d)
        self._k, self._v, self._pos = k, v, torch.zeros(nslots, **d)
        self._pages = PagePool([k, v], table, refs)
        self._c = ctypes.byref(_abi.AttnCache(k.data_ptr(), v.data_ptr(), table.data_ptr(), refs.data_ptr(),
                                              self._pos.data_ptr(), nslots, slot_pages, self.npages, page_tokens))

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.k, self.v, self.pos, self.pages.table, self.pages.refs))


@functools.lru_cache(maxsize=64)
def _attn_dims(H: int, kv_heads: int, head_dim: int, io: torch.dtype, scale: float):
    return ctypes.byref(_abi.AttnDims(H, kv_heads, head_dim, _IO[io], scale))


@_on_stream
def attn_verify(cache: AttnCache, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, parent: Optional[torch.Tensor] = None,
                slot: Optional[torch.Tensor] = None, scale: Optional[float] = None, max_len: Optional[int] = None,
                status: Optional[Status] = None, check: bool = True, stream=None,
                out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of T drafts per sequence over the slot's tokens and their own path (ers_attn_verify), outputs only.

    q [S,T,H,D], k, v [S,T,kv_heads,D], T up to 64 (1: the next token); parent [S,T] int32: the place of the draft that each one
    follows, -1 for the slot's last token, -2 for an empty place (zeros); default: a chain.  scale: default D ** -0.5.
    max_len, the most tokens of a slot, only chooses how the work is split (default: what the table has room for).  Returns o
    [S,T,H,D]."""
    if q.dim() != 4:
        raise ValueError(f"q: shape {tuple(q.shape)}, expected (sequences, drafts, heads, {cache.head_dim})")
    S, T, H, D = q.shape
    shape = (S, T, cache.kv_heads, cache.head_dim)
    args = (_tensor(q, cache.io, "q", (S, T, H, cache.head_dim)), _tensor(k, cache.io, "k", shape),
            _tensor(v, cache.io, "v", shape), None if parent is None else _tensor(parent, torch.int32, "parent", (S, T)))
    o, dev = _out(out, q), q.device
    st = _status(status, check, dev)
    dims = _attn_dims(H, cache.kv_heads, cache.head_dim, cache.io, D ** -0.5 if scale is None else float(scale))
    longest = cache.slot_pages * cache.page_tokens if max_len is None else int(max_len)
    keep, *ws = _workspace(_abi.lib().ers_attn_verify_workspace_size(dims, S, T, longest), dev)
    code = _abi.lib().ers_attn_verify(dims, cache._c, S, _slot(slot, S), T, longest, *args, o.data_ptr(), *ws, *_where(dev, st))
    _finish(code, "ers_attn_verify", st, check)
    return o


def _rows_dims(cache: AttnCache):
    return _attn_dims(cache.kv_heads, cache.kv_heads, cache.head_dim, cache.io, 1.0)


@_on_stream
def attn_append(cache: AttnCache, k: torch.Tensor, v: torch.Tensor, cu_seqlens: Optional[torch.Tensor] = None,
                slot: Optional[torch.Tensor] = None, status: Optional[Status] = None, check: bool = True,
                stream=None) -> None:
    """Packed new rows k, v [T,kv_heads,D] go behind their slots' tokens (ers_attn_append) and pos moves on; cu_seqlens
    int32 [S+1] (default: one sequence)."""
    T, dev = k.shape[0], k.device
    cu_seqlens, S = _seqlens(cu_seqlens, T, dev)
    shape = (T, cache.kv_heads, cache.head_dim)
    rows = _tensor(k, cache.io, "k", shape), _tensor(v, cache.io, "v", shape)
    st = _status(status, check, dev)
    code = _abi.lib().ers_attn_append(_rows_dims(cache), cache._c, S, T, cu_seqlens.data_ptr(), _slot(slot, S), *rows,
                                      *_where(dev, st))
    _finish(code, "ers_attn_append", st, check)


@_on_stream
def attn_commit(cache: AttnCache, k: torch.Tensor, v: torch.Tensor, accepted: torch.Tensor,
                path: Optional[torch.Tensor] = None, slot: Optional[torch.Tensor] = None, status: Optional[Status] = None,
                check: bool = True, stream=None) -> None:
    """The accepted drafts' rows of k, v [S,T,kv_heads,D] go behind their slots' tokens (ers_attn_commit) and pos moves on:
    drafts path[s][0 .. accepted[s]) (default: the first ones).  accepted [S], path [S,T] int32."""
    if k.dim() != 4:
        raise ValueError(f"k: shape {tuple(k.shape)}, expected (sequences, drafts, {cache.kv_heads}, {cache.head_dim})")
    S, T, dev = k.shape[0], k.shape[1], k.device
    shape = (S, T, cache.kv_heads, cache.head_dim)
    rows = _tensor(k, cache.io, "k", shape), _tensor(v, cache.io, "v", shape)
    args = (None if path is None else _tensor(path, torch.int32, "path", (S, T)),
            _tensor(accepted, torch.int32, "accepted", (S,)))
    st = _status(status, check, dev)
    code = _abi.lib().ers_attn_commit(_rows_dims(cache), cache._c, S, _slot(slot, S), T, *args, *rows, *_where(dev, st))
    _finish(code, "ers_attn_commit", st, check)
