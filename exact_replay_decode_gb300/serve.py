"""PyTorch-facing binding of the serving operators around a linear-attention layer (include/ers.h): linear
attention with a decay per head, the pages of a cache, and log probabilities of given tokens.

Marshalling only, as in ops.py: shape, dtype and contiguity checks, outputs and workspaces from torch,
the caller's stream.  A decode step's call is a few microseconds of kernel, so the checks of a call that passes
them are kept to one comparison each."""
from __future__ import annotations

import ctypes
import functools
from typing import Optional, Sequence, Tuple

import torch

from . import _abi
from .ops import ReplayCache, Status, _finish, _io_from, _IO, _need, _ptr


_raw_stream = torch._C._cuda_getCurrentRawStream


def _on_stream(f):
    """stream=: the call's allocations, its status word and its launches all belong to that stream."""
    @functools.wraps(f)
    def g(*args, stream=None, **kw):
        if stream is None:
            return f(*args, **kw)
        with torch.cuda.stream(stream):
            return f(*args, **kw)
    return g


def _status(status: Optional[Status], check: bool, device) -> Optional[Status]:
    return status if status is not None else (Status(device) if check else None)


def _tensor(t: torch.Tensor, dtype, name: str, shape) -> int:
    """The data pointer of a dense CUDA tensor of that type and shape; otherwise _need's error."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.shape == shape and t.is_contiguous()):
        _need(t, dtype, name, shape)
    return t.data_ptr()


def _where(device: torch.device, st: Optional[Status]):
    """The launch's stream and status word."""
    return _raw_stream(device.index), None if st is None else st.t.data_ptr()


# ---- pages of a cache --------------------------------------------------------------------------
class PagePool:
    """Counted references to the pages of a pool under a table of pages per slot.

    arrays: contiguous tensors whose first dimension is the page (the same number in all of them); one page
    index addresses all of them.  table [nslots, slot_pages] int32: the pages of each slot, -1 where it has
    none.  refs [npages] int32: how many table entries name a page; counted from the table when not given.
    The pool keeps and changes these tensors (and cannot be given others: its calls go by where they are); from then on pages
    change hands through the pages_* calls."""

    arrays = property(lambda self: self._arrays)
    table = property(lambda self: self._table)
    refs = property(lambda self: self._refs)

    def __init__(self, arrays: Sequence[torch.Tensor], table: torch.Tensor, refs: Optional[torch.Tensor] = None):
        self._arrays: Tuple[torch.Tensor, ...] = tuple(arrays)
        if not 0 < len(self.arrays) <= _abi.PAGE_ARRAYS_MAX:
            raise ValueError(f"a pool has 1 to {_abi.PAGE_ARRAYS_MAX} arrays, got {len(self.arrays)}")
        if table.dim() != 2:
            raise ValueError(f"table: shape {tuple(table.shape)}, expected (nslots, slot_pages)")
        npages = self.arrays[0].shape[0]
        _need(table, torch.int32, "table")
        if refs is None:
            held = table.flatten()
            refs = torch.zeros(npages + 1, dtype=torch.int32, device=table.device)
            named = (held >= 0) & (held < npages)   # others name no page (the calls report what is out of range)
            refs.index_add_(0, torch.where(named, held, npages).long(), torch.ones_like(held))
            refs = refs[:-1].contiguous()
        _need(refs, torch.int32, "refs", (npages,))
        for k, x in enumerate(self.arrays):
            _need(x, x.dtype, f"arrays[{k}]")
            if x.shape[0] != npages:
                raise ValueError(f"arrays[{k}]: {x.shape[0]} pages, expected {npages}")
        self._table, self._refs = table, refs
        self.npages, (self.nslots, self.slot_pages) = npages, table.shape
        self._c = ctypes.byref(_pool_c(self.arrays, table, refs))
        # scratch of the calls on this pool, which have to follow one another anyway
        L = _abi.lib()
        self._work = torch.empty(max(L.ers_pages_own_workspace_size(self._c, self.nslots),
                                     L.ers_pages_compact_workspace_size(self._c), 16),
                                 dtype=torch.uint8, device=table.device)


def _pool_c(arrays: Sequence[torch.Tensor], table: Optional[torch.Tensor], refs: Optional[torch.Tensor]):
    c = _abi.PagePool()
    c.npages, c.narrays = arrays[0].shape[0], len(arrays)
    if table is not None:
        c.table, c.refs = table.data_ptr(), refs.data_ptr()
        c.nslots, c.slot_pages = table.shape
    for k, x in enumerate(arrays):
        c.array[k] = x.data_ptr()
        c.page_bytes[k] = x[0].numel() * x.element_size() if x.shape[0] else 2
    return c


def _list_arg(t: torch.Tensor, name: str, n: Optional[int] = None) -> int:
    if not isinstance(t, torch.Tensor) or t.dim() != 1:
        raise ValueError(f"{name}: expected a one-dimensional tensor")
    return _tensor(t, torch.int32, name, (t.numel() if n is None else n,))


@_on_stream
def pages_fork(pool: PagePool, src: torch.Tensor, dst: torch.Tensor, status: Optional[Status] = None,
               check: bool = True, stream=None) -> None:
    """Slots dst (without pages) share the pages of slots src (ers_pages_fork); nothing is copied."""
    n = dst.numel()
    s, d = _list_arg(src, "src", n), _list_arg(dst, "dst", n)
    st = _status(status, check, dst.device)
    code = _abi.lib().ers_pages_fork(pool._c, n, s, d, *_where(dst.device, st))
    _finish(code, "ers_pages_fork", st, check)


@_on_stream
def pages_own(pool: PagePool, slot: torch.Tensor, copy: bool = True, status: Optional[Status] = None,
              check: bool = True, stream=None) -> torch.Tensor:
    """Every missing or shared page of the listed slots becomes a page of their own (ers_pages_own), with the old
    page's contents (zeros where there was none) when copy.  Returns the entries as they were [n, slot_pages]:
    with copy=False, the pages that linattn_decode and linattn_prefill read from (read_page)."""
    n = slot.numel()
    sp = _list_arg(slot, "slot")
    read = torch.empty(n, pool.slot_pages, dtype=torch.int32, device=slot.device)
    st = _status(status, check, slot.device)
    code = _abi.lib().ers_pages_own(pool._c, n, sp, _abi.FLAG_COPY if copy else 0, read.data_ptr(),
                                    pool._work.data_ptr(), pool._work.numel(), *_where(slot.device, st))
    _finish(code, "ers_pages_own", st, check)
    return read


@_on_stream
def pages_free(pool: PagePool, slot: torch.Tensor, status: Optional[Status] = None, check: bool = True,
               stream=None) -> None:
    """The listed slots give up their pages (ers_pages_free)."""
    sp = _list_arg(slot, "slot")
    st = _status(status, check, slot.device)
    code = _abi.lib().ers_pages_free(pool._c, slot.numel(), sp, *_where(slot.device, st))
    _finish(code, "ers_pages_free", st, check)


@_on_stream
def pages_compact(pool: PagePool, status: Optional[Status] = None, check: bool = True,
                  stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Moves the pages in use to the lowest indices (ers_pages_compact).  Returns (remap [npages]: each page's new
    index, -1 where it was free; live [1]: how many are in use), both on the device."""
    dev = pool.table.device
    remap = torch.empty(pool.npages, dtype=torch.int32, device=dev)
    live = torch.empty(1, dtype=torch.int32, device=dev)
    st = _status(status, check, dev)
    code = _abi.lib().ers_pages_compact(pool._c, remap.data_ptr(), live.data_ptr(), pool._work.data_ptr(),
                                        pool._work.numel(), *_where(dev, st))
    _finish(code, "ers_pages_compact", st, check)
    return remap, live


@_on_stream
def pages_copy(arrays: Sequence[torch.Tensor], src: torch.Tensor, dst: torch.Tensor, status: Optional[Status] = None,
               check: bool = True, stream=None) -> None:
    """Page dst[i] of every array receives page src[i] (ers_pages_copy); the page is the first dimension."""
    arrays = list(arrays)
    if not 0 < len(arrays) <= _abi.PAGE_ARRAYS_MAX:
        raise ValueError(f"1 to {_abi.PAGE_ARRAYS_MAX} arrays, got {len(arrays)}")
    for k, x in enumerate(arrays):
        _need(x, x.dtype, f"arrays[{k}]")
        if x.shape[0] != arrays[0].shape[0]:
            raise ValueError(f"arrays[{k}]: {x.shape[0]} pages, expected {arrays[0].shape[0]}")
    n = dst.numel()
    s, d = _list_arg(src, "src", n), _list_arg(dst, "dst", n)
    st = _status(status, check, dst.device)
    code = _abi.lib().ers_pages_copy(ctypes.byref(_pool_c(arrays, None, None)), n, s, d, *_where(dst.device, st))
    _finish(code, "ers_pages_copy", st, check)


def _pages_clone(pool: PagePool, src: torch.Tensor, dst: torch.Tensor, status: Optional[Status], check: bool) -> torch.Tensor:
    """Slots dst give up their pages for copies of src's (ers_pages_clone).  Returns src's entries, -2 after an error."""
    n = dst.numel()
    s, d = _list_arg(src, "src", n), _list_arg(dst, "dst", n)
    read = torch.empty(n, pool.slot_pages, dtype=torch.int32, device=dst.device)
    st = _status(status, check, dst.device)
    code = _abi.lib().ers_pages_clone(pool._c, n, s, d, read.data_ptr(), pool._work.data_ptr(), pool._work.numel(),
                                      *_where(dst.device, st))
    _finish(code, "ers_pages_clone", st, check)
    return read


@_on_stream
def fork_slots(cache: ReplayCache, src: torch.Tensor, dst: torch.Tensor, status: Optional[Status] = None,
               check: bool = True, stream=None) -> None:
    """Slots dst of a ReplayCache become copies of slots src (distinct, none of them in src): the state, the read
    copy, the position and the buffered rows, so that both decode on from there.  Paged buffers: dst gives up its
    pages and gets pages of its own from cache.page_pool(), in one decision with everything else: where that finds an
    error (too few free pages, lists that overlap), no slot is changed."""
    arrays = [t for t in (cache.state, cache.read_copy, cache.read_scale, cache.read_block_scale, cache.pos)
              if t is not None]
    if cache.buf_pages is None:
        arrays += [cache.buf_x, cache.buf_dt, cache.buf_B, cache.buf_C]
    else:
        read = _pages_clone(cache.page_pool(), src, dst, status, check)
        if not check:   # after an error known on the device only: sources that pages_copy leaves out
            src = torch.where(read[:, 0] == -2, -1, src)
    pages_copy(arrays, src, dst, status=status, check=check)


# ---- linear attention ----------------------------------------------------------------------------
class LinAttnCache:
    """The states of a linear-attention layer: pages of state [npages, H, dv, dk] fp32 under a table of one page per
    slot (pages: a PagePool).  npages None: as many as slots, slot s starting out with page s (zeros).  Otherwise
    every page starts out free, and pages_own(cache.pages, slots) hands them out.  state: a tensor to use as the pages (it
    stays the cache's; another one is another cache)."""

    state = property(lambda self: self._state)
    pages = property(lambda self: self._pages)

    def __init__(self, nslots: int, nheads: int, ngroups: int, dk: int = 128, dv: int = 128,
                 npages: Optional[int] = None, io_dtype: torch.dtype = torch.bfloat16, device="cuda",
                 state: Optional[torch.Tensor] = None):
        self.nslots, self.H, self.G, self.dk, self.dv, self.io = nslots, nheads, ngroups, dk, dv, io_dtype
        self.npages = nslots if npages is None else npages
        shape = (self.npages, nheads, dv, dk)
        if state is None:
            state = torch.zeros(shape, dtype=torch.float32, device=device)
        _need(state, torch.float32, "state", shape)
        self._state = state
        if npages is None:
            table = torch.arange(nslots, dtype=torch.int32, device=state.device).view(nslots, 1)
        else:
            table = torch.full((nslots, 1), -1, dtype=torch.int32, device=state.device)
        refs = torch.full((self.npages,), int(npages is None), dtype=torch.int32, device=state.device)
        self._pages = PagePool([state], table, refs)
        self._c = ctypes.byref(_abi.LinAttnCache(state.data_ptr(), table.data_ptr(), nslots, self.npages))

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size() for t in (self.state, self.pages.table, self.pages.refs))


@functools.lru_cache(maxsize=64)
def _linattn_dims(H: int, G: int, dk: int, dv: int, io: torch.dtype, scale: float):
    if io not in _IO:
        raise TypeError(f"io dtype {io} not supported (bf16 or fp32)")
    return ctypes.byref(_abi.LinAttnDims(H, G, dk, dv, _IO[io], scale))


def _qkv(q, k, v, log_decay, io, T, H, G, dk, dv):
    """Checked; (log_decay, (q, k, v)) as pointers."""
    return _tensor(log_decay, torch.float32, "log_decay", (H,)), (
        _tensor(q, io, "q", (T, G, dk)), _tensor(k, io, "k", (T, G, dk)), _tensor(v, io, "v", (T, H, dv)))


def _seqlens(cu_seqlens: Optional[torch.Tensor], T: int, device):
    if cu_seqlens is None:
        # made on the device: a copy from the host would wait, and cannot be captured
        d = dict(dtype=torch.int32, device=device)
        cu_seqlens = torch.arange(0, T + 1, T, **d) if T > 0 else torch.zeros(2, **d)
    S = cu_seqlens.numel() - 1
    _tensor(cu_seqlens, torch.int32, "cu_seqlens", (S + 1,))
    return cu_seqlens, S


def _longest(cu_seqlens: torch.Tensor, T: int, S: int, H: int, max_seqlen: Optional[int]) -> int:
    """max_seqlen, or the longest length that cu_seqlens has, which waits for the device (25 us).  T, an upper bound for which
    the work of several sequences may be split too far, while a stream is captured, and of up to 256 tokens of few heads or of
    few tokens a sequence (12 x 20 tokens x 16 heads: 22 us by T and 18 by 20; 28 x 9 x 64: 127 and 77, so it is read)."""
    if max_seqlen is not None:
        return int(max_seqlen)
    if S <= 1 or T <= 256 and (S * H <= 304 or T <= 8 * S) or torch.cuda.is_current_stream_capturing():
        return T
    at = cu_seqlens.tolist()
    return min(max(max(b - a for a, b in zip(at, at[1:])), 0), T)   # (whatever cu_seqlens holds)


def _out(out: Optional[torch.Tensor], v: torch.Tensor) -> torch.Tensor:
    if out is None:
        return torch.empty_like(v)
    _tensor(out, v.dtype, "out", v.shape)
    return out


@_on_stream
def linattn_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, log_decay: torch.Tensor,
                cu_seqlens: Optional[torch.Tensor] = None, init_state: Optional[torch.Tensor] = None,
                scale: float = 1.0, max_seqlen: Optional[int] = None, status: Optional[Status] = None,
                check: bool = True, stream=None,
                out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """Linear attention with a decay per head over packed prompts (ers_linattn_fwd).

    q, k [T,G,dk], v [T,H,dv] (bf16 or fp32; dk, dv 64 or 128), log_decay [H] fp32 (<= 0); cu_seqlens int32 [S+1]
    (default: one sequence); init_state [S,H,dv,dk] fp32 (default zeros).  max_seqlen, the longest sequence's length,
    only chooses how the work is split (default: read from cu_seqlens, which waits for the device; T for few tokens and while a
    stream is captured).  Returns (o [T,H,dv], final_state [S,H,dv,dk] fp32)."""
    io = _io_from(q)
    T, G, dk = q.shape
    H, dv = v.shape[1], v.shape[2]
    dev = q.device
    cu_seqlens, S = _seqlens(cu_seqlens, T, dev)
    decay, qkv = _qkv(q, k, v, log_decay, io, T, H, G, dk, dv)
    state = (S, H, dv, dk)
    init = None if init_state is None else _tensor(init_state, torch.float32, "init_state", state)
    if out is None:
        o, final = torch.empty_like(v), torch.empty(state, dtype=torch.float32, device=dev)
    else:
        o, final = out
        _out(o, v)
        _tensor(final, torch.float32, "out[1]", state)
    st = _status(status, check, dev)
    code = _abi.lib().ers_linattn_fwd(_linattn_dims(H, G, dk, dv, io, float(scale)), decay, S, T,
                                      _longest(cu_seqlens, T, S, H, max_seqlen), cu_seqlens.data_ptr(), *qkv,
                                      init, o.data_ptr(), final.data_ptr(), *_where(dev, st))
    _finish(code, "ers_linattn_fwd", st, check)
    return o, final


def _read_arg(read_page: Optional[torch.Tensor], S: int):
    if read_page is None:
        return None
    if read_page.dim() == 2:   # as pages_own returns it
        read_page = read_page[:, 0]
    return _tensor(read_page, torch.int32, "read_page", (S,))


def _slot(slot: Optional[torch.Tensor], S: int):
    return None if slot is None else _tensor(slot, torch.int32, "slot", (S,))


@_on_stream
def linattn_prefill(cache: LinAttnCache, q, k, v, log_decay, cu_seqlens: Optional[torch.Tensor] = None,
                    slot: Optional[torch.Tensor] = None, read_page: Optional[torch.Tensor] = None,
                    scale: float = 1.0, max_seqlen: Optional[int] = None, status: Optional[Status] = None,
                    check: bool = True, stream=None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Packed prompts that go on from the slots' cached states (ers_linattn_prefill): each state is read from
    read_page (default: the slot's own page; -1: zeros) and written to the slot's own page.  max_seqlen: as in
    linattn_fwd.  Returns o [T,H,dv]."""
    T, dev = q.shape[0], q.device
    cu_seqlens, S = _seqlens(cu_seqlens, T, dev)
    decay, qkv = _qkv(q, k, v, log_decay, cache.io, T, cache.H, cache.G, cache.dk, cache.dv)
    o = _out(out, v)
    st = _status(status, check, dev)
    dims = _linattn_dims(cache.H, cache.G, cache.dk, cache.dv, cache.io, float(scale))
    code = _abi.lib().ers_linattn_prefill(dims, decay, cache._c, S, T,
                                          _longest(cu_seqlens, T, S, cache.H, max_seqlen), cu_seqlens.data_ptr(),
                                          _slot(slot, S), _read_arg(read_page, S), *qkv, o.data_ptr(), *_where(dev, st))
    _finish(code, "ers_linattn_prefill", st, check)
    return o


@_on_stream
def linattn_decode(cache: LinAttnCache, q, k, v, log_decay, slot: Optional[torch.Tensor] = None,
                   read_page: Optional[torch.Tensor] = None, scale: float = 1.0, status: Optional[Status] = None,
                   check: bool = True, stream=None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One token per sequence (ers_linattn_decode): q, k [S,G,dk], v [S,H,dv]; states as in linattn_prefill."""
    S, dev = q.shape[0], q.device
    decay, qkv = _qkv(q, k, v, log_decay, cache.io, S, cache.H, cache.G, cache.dk, cache.dv)
    o = _out(out, v)
    st = _status(status, check, dev)
    dims = _linattn_dims(cache.H, cache.G, cache.dk, cache.dv, cache.io, float(scale))
    code = _abi.lib().ers_linattn_decode(dims, decay, cache._c, S, _slot(slot, S),
                                         _read_arg(read_page, S), *qkv, o.data_ptr(), *_where(dev, st))
    _finish(code, "ers_linattn_decode", st, check)
    return o


# ---- log probabilities -----------------------------------------------------------------------------
@_on_stream
def token_logprobs(logits: torch.Tensor, target: Optional[torch.Tensor] = None, top_k: int = 0, scale: float = 1.0,
                   status: Optional[Status] = None, check: bool = True, stream=None):
    """Log probabilities of the target tokens, entropy and top alternatives of each row (ers_token_logprobs).

    logits [R, V] bf16 or fp32, its rows contiguous and any distance apart; target [R] int32, -1 for none; scale: an inverse
    temperature.  Returns (logprob [R] or None, entropy [R], top_id [R,top_k] int32, top_logprob [R,top_k])."""
    io = _io_from(logits)
    if logits.dim() != 2:
        raise ValueError(f"logits: shape {tuple(logits.shape)}, expected (rows, vocabulary)")
    if not logits.is_cuda:
        raise ValueError("logits: must be a CUDA tensor")
    R, V = logits.shape
    if V > 1 and logits.stride(1) != 1 or R > 1 and logits.stride(0) < V:
        raise ValueError(f"logits: strides {logits.stride()}, expected contiguous rows")
    if target is not None:
        _tensor(target, torch.int32, "target", (R,))
    dev, k = logits.device, int(top_k)
    if not 0 <= k <= _abi.TOP_MAX:
        raise ValueError(f"top_k: {k}, expected 0 to {_abi.TOP_MAX}")
    logprob = None if target is None else torch.empty(R, dtype=torch.float32, device=dev)
    entropy = torch.empty(R, dtype=torch.float32, device=dev)
    top_id = torch.empty(R, k, dtype=torch.int32, device=dev)
    top_logprob = torch.empty(R, k, dtype=torch.float32, device=dev)
    st = _status(status, check, dev)
    code = _abi.lib().ers_token_logprobs(_IO[io], R, V, logits.stride(0) if R > 1 else V, logits.data_ptr(),
                                         _ptr(target), float(scale), k, _ptr(logprob), entropy.data_ptr(),
                                         top_id.data_ptr() if k else None, top_logprob.data_ptr() if k else None,
                                         *_where(dev, st))
    _finish(code, "ers_token_logprobs", st, check)
    return logprob, entropy, top_id, top_logprob
