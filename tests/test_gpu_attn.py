"""Attention of a tree of drafts over a paged cache on the GPU, against softmax attention in 64 bits, and the rows that go into the
pages against plain indexing.

Bounds.  With A = sum_j p_j |v_j| and X the largest sum of |scale q_i k_i| of a row, a score in fp32 is off by at most (D + 2) 2^-24 X, a
weight by that and its exponential's 2 units, relative, twice (it is divided by their sum), and the sums over L tokens by
(L + 8) 2^-24: fp32 outputs are within (2 (D + 4) X + 2 L + 16) 2^-24 A.  bf16 ones also round the weights (2^-8 A, as each weight is off
by at most 2^-8 of itself, and their sum by no more) and the output (2^-8).  In the 2-norm the roundings do not conspire: 2e-6, and
2.4e-3 (the output's rounding is 1.7e-3, the weights' at most as much again in quadrature for rows of a single
dominant token).  A score is a sum of D products in fp32, whose partial sums grow to X at most, each rounded by half of 2^-24 of
itself: sqrt(D / 3) / 2 2^-24 X in quadrature, an absolute error that its weight inherits as a relative one.  Where X is large
(434 in the mean for queries of size 60, D 128: 8e-5) that takes the place of 2e-6."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _ers():
    import exact_replay_decode_gb300 as ers
    return ers


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _cache(seed, lens, KV, D, page, io, room=0):
    """A cache of scattered pages that hold lens tokens, NaN in everything that no token is in."""
    S, per = len(lens), max(1, -(-(max(lens) + room) // page))
    cache = _ers().AttnCache(S, KV, D, page_tokens=page, slot_pages=per, npages=S * per + 2, io_dtype=io)
    order = torch.randperm(S * per + 2, device="cuda", generator=_gen(seed)).to(torch.int32)
    cache.pages.table.copy_(order[:S * per].view(S, per))
    cache.pages.refs[order[:S * per].long()] = 1
    cache.pos.copy_(torch.tensor(lens, dtype=torch.int32))
    for x in (cache.k, cache.v):
        x.fill_(math.nan)
        for i, n in enumerate(lens):
            rows = torch.randn(n, KV, D, device="cuda", generator=_gen(seed + 7 * i + (x is cache.v))).to(io)
            _put(cache, x, i, 0, rows)
    return cache


def _at(cache, slot, n):
    t = torch.arange(n, device="cuda")
    return cache.pages.table[slot].long()[t // cache.page_tokens] * cache.page_tokens + t % cache.page_tokens


def _put(cache, x, slot, start, rows):
    flat = x.view(-1, *x.shape[2:])
    flat[_at(cache, slot, start + rows.shape[0])[start:]] = rows


def _drafts(seed, S, T, H, KV, D, io, sharp=2.0):
    r = dict(device="cuda", generator=_gen(seed))
    return ((torch.randn(S, T, H, D, **r) * sharp).to(io), torch.randn(S, T, KV, D, **r).to(io), torch.randn(S, T, KV, D, **r).to(io))


def _trees(S, T, seed, empties=False):
    import random
    r = random.Random(seed)
    rows = []
    for _ in range(S):
        row = []
        for t in range(T):
            used = [p for p in range(t) if row[p] != -2]
            row.append(-2 if empties and r.random() < 0.3 else r.choice([-1] + used + used[-2:]))
        rows.append(row)
    return torch.tensor(rows, dtype=torch.int32, device="cuda")


def _sees(parent, T):
    seen = torch.zeros(T, T, dtype=torch.bool)
    for t, p in enumerate(parent):
        if p != -2:
            if p >= 0:
                seen[t] |= seen[p]
            seen[t, t] = True
    return seen.cuda()


def _check(o, cache, q, k, v, parent=None, scale=None, slots=None):
    S, T, H, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    rep = H // cache.kv_heads
    want, bound = torch.zeros(q.shape, dtype=torch.float64, device="cuda"), torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    largest = 0.0
    for i in range(S):
        slot = i if slots is None else slots[i]
        n = int(cache.pos[slot])
        rows = _at(cache, slot, n)
        kk, vv = (torch.cat([x.view(-1, *x.shape[2:])[rows], y[i]]).double().repeat_interleave(rep, 1).transpose(0, 1)
                  for x, y in ((cache.k, k), (cache.v, v)))                                       # [H, n + T, D]
        seen = torch.ones(T, n + T, dtype=torch.bool, device="cuda")
        row = list(range(-1, T - 1)) if parent is None else parent[i].tolist()
        seen[:, n:] = _sees(row, T)
        seen[torch.tensor(row, device="cuda") == -2] = False
        qq = q[i].double().transpose(0, 1)
        x = (qq @ kk.transpose(1, 2) * scale).masked_fill(~seen, -math.inf)
        p = torch.softmax(x, -1).nan_to_num(0.0)
        want[i] = (p @ vv).transpose(0, 1)
        X = (qq.abs() @ kk.abs().transpose(1, 2) * abs(scale)).masked_fill(~seen, 0).amax(-1, keepdim=True)
        largest = max(largest, X.mean().item())
        A = p @ vv.abs()
        bound[i] = ((2 * (D + 4) * X + 2 * n + 16) * 2.0 ** -24 * A + (2.0 ** -8 * A if q.dtype == BF16 else 0)).transpose(0, 1)
    if q.dtype == BF16:
        bound = bound * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs()
    assert ((o.double() - want).abs() <= bound).all()
    if want.norm() > 0:
        off = ((o.double() - want).norm() / want.norm()).item()
        assert off <= (2.4e-3 if q.dtype == BF16 else max(2e-6, math.sqrt(D / 3) / 2 * 2.0 ** -24 * largest))


IO = pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])


@IO
@pytest.mark.parametrize("T", [1, 2, 7, 33, 64])
@pytest.mark.parametrize("D,H,KV,page", [(128, 8, 2, 64), (64, 6, 6, 24), (128, 5, 1, 1), (64, 16, 2, 500)])
def test_trees(io, T, D, H, KV, page):
    lens = [130, 0, 1, 63, 300]
    cache = _cache(T + D, lens, KV, D, page, io)
    q, k, v = _drafts(T, 5, T, H, KV, D, io)
    for parent in (None, _trees(5, T, T), _trees(5, T, T + 1, empties=True)):
        o = _ers().attn_verify(cache, q, k, v, parent=parent)
        _check(o, cache, q, k, v, parent)


@IO
@pytest.mark.parametrize("lens,T,max_len", [([5000], 1, None), ([5000], 4, 5000), ([2049, 17, 0], 16, 2049), ([700, 4000], 3, 100),
                                            ([1000, 1000], 5, 10 ** 6)])
def test_long_pasts_are_shared_out(io, lens, T, max_len):
    """Whatever max_len says."""
    cache = _cache(3, lens, 2, 128, 48, io)
    q, k, v = _drafts(4, len(lens), T, 8, 2, 128, io)
    o = _ers().attn_verify(cache, q, k, v, max_len=max_len)
    _check(o, cache, q, k, v)


@IO
def test_a_wide_group_and_many_rows(io):
    cache = _cache(5, [100, 200], 2, 64, 16, io)
    q, k, v = _drafts(6, 2, 64, 32, 2, 64, io)
    parent = _trees(2, 64, 1)
    _check(_ers().attn_verify(cache, q, k, v, parent=parent, scale=-0.2), cache, q, k, v, parent, -0.2)


@IO
@pytest.mark.parametrize("sharp", [0.0, 60.0, 3e4])
def test_flat_and_sharp_rows(io, sharp):
    """Even weights; one dominant token; scores that only their differences keep in range."""
    cache = _cache(7, [500, 63], 2, 128, 64, io)
    q, k, v = _drafts(8, 2, 3, 4, 2, 128, io, sharp)
    if sharp < 1e4:
        _check(_ers().attn_verify(cache, q, k, v), cache, q, k, v)
        return
    o = _ers().attn_verify(cache, q, k, v)      # scores of 1e5, off by 1: no more than that it is an average of values
    assert torch.isfinite(o).all() and o.abs().max() <= max(cache.v.nan_to_num().abs().max(), v.abs().max())


@IO
def test_rows_that_rise_and_fall(io):
    """The running maximum moves at every tile, by far, in both directions."""
    cache = _cache(9, [1024], 1, 64, 64, io)
    level = torch.linspace(-8, 8, 1024, device="cuda").view(-1, 1, 1)
    q, k, v = _drafts(10, 1, 2, 2, 1, 64, io)
    q[:, :, 0], q[:, :, 1] = 1.0, -1.0
    _put(cache, cache.k, 0, 0, (torch.randn(1024, 1, 64, device="cuda", generator=_gen(1)) * 0.1 + level).to(io))
    _check(_ers().attn_verify(cache, q, k, v), cache, q, k, v)


@IO
def test_what_is_not_attended_to_may_be_anything(io):
    cache = _cache(11, [70, 64], 2, 128, 64, io)
    q, k, v = _drafts(12, 2, 6, 4, 2, 128, io)
    parent = torch.tensor([[-1, 0, -2, 0, 1, -2], [-1, -1, -1, -2, 2, 4]], dtype=torch.int32, device="cuda")
    good = _ers().attn_verify(cache, q, k, v, parent=parent)
    _check(good, cache, q, k, v, parent)
    for fill in (math.nan, math.inf, -math.inf, torch.finfo(io).max):
        q2, k2, v2 = q.clone(), k.clone(), v.clone()
        for x in (q2, k2, v2):
            x[0, 2], x[0, 5], x[1, 3] = fill, fill, fill        # empty places
        for x in (k2, v2):
            x[0, 3], x[1, 1] = fill, fill                       # leaves of other paths
        o = _ers().attn_verify(cache, q2, k2, v2, parent=parent)
        rows = torch.ones(2, 6, dtype=torch.bool, device="cuda")
        rows[0, 3], rows[1, 1] = False, False
        assert torch.equal(o[rows], good[rows])
        assert (o[0, 2] == 0).all() and (o[1, 3] == 0).all()
        if not math.isfinite(fill):
            v3 = v.clone()
            v3[1, 2] = fill
            o = _ers().attn_verify(cache, q, k, v3, parent=parent)
            assert not torch.isfinite(o[1, [2, 4, 5]]).any() and torch.equal(o[1, :2], good[1, :2])


@IO
def test_no_tokens_at_all(io):
    cache = _cache(13, [0, 5], 1, 64, 8, io)
    q, k, v = _drafts(14, 2, 3, 2, 1, 64, io)
    parent = torch.tensor([[-2, -2, -2], [-1, -2, -2]], dtype=torch.int32, device="cuda")
    o = _ers().attn_verify(cache, q, k, v, parent=parent)
    assert (o[0] == 0).all() and (o[1, 1:] == 0).all()
    _check(o, cache, q, k, v, parent)
    _ers().attn_verify(cache, q[:0], k[:0], v[:0])


@IO
def test_prompts_drafts_and_commits(io):
    """Rows from packed prompts and from accepted paths are where plain indexing puts them, and nothing else changes."""
    ers = _ers()
    cache = _cache(15, [10, 0, 33, 5], 2, 64, 24, io, room=200)
    want_k, want_v = cache.k.clone(), cache.v.clone()
    slot = torch.tensor([2, 0, 3], dtype=torch.int32, device="cuda")
    lens = [100, 0, 17]
    k, v = (torch.randn(117, 2, 64, device="cuda", generator=_gen(s)).to(io) for s in (1, 2))
    cu = torch.tensor([0, 100, 100, 117], dtype=torch.int32, device="cuda")
    _put_all(cache, want_k, want_v, [(2, 33, k[:100], v[:100]), (3, 5, k[100:], v[100:])])
    ers.attn_append(cache, k, v, cu, slot=slot)
    assert cache.pos.tolist() == [10, 0, 133, 22] and sum(lens) == 117
    assert _same(cache.k, want_k) and _same(cache.v, want_v)
    q, k, v = _drafts(16, 3, 6, 4, 2, 64, io)
    parent = _trees(3, 6, 5)
    o = ers.attn_verify(cache, q, k, v, parent=parent, slot=slot)
    _check(o, cache, q, k, v, parent, slots=slot.tolist())
    accepted = torch.tensor([3, 0, 6], dtype=torch.int32, device="cuda")
    path = torch.tensor([[1, 4, 5, -9, -9, 99], [-1] * 6, [0, 1, 2, 3, 4, 5]], dtype=torch.int32, device="cuda")
    at = [1, 4, 5]
    _put_all(cache, want_k, want_v, [(2, 133, k[0, at], v[0, at]), (3, 22, k[2], v[2])])
    ers.attn_commit(cache, k, v, accepted, path=path, slot=slot)
    assert cache.pos.tolist() == [10, 0, 136, 28]
    assert _same(cache.k, want_k) and _same(cache.v, want_v)
    ers.attn_commit(cache, k, v, torch.tensor([1, 2, 0], dtype=torch.int32, device="cuda"), slot=slot)   # the first drafts
    _put_all(cache, want_k, want_v, [(2, 136, k[0, :1], v[0, :1]), (0, 10, k[1, :2], v[1, :2])])
    assert cache.pos.tolist() == [12, 0, 137, 28] and _same(cache.k, want_k) and _same(cache.v, want_v)


def _put_all(cache, want_k, want_v, parts):
    for slot, start, k, v in parts:
        _put(cache, want_k, slot, start, k)
        _put(cache, want_v, slot, start, v)


def _same(x, y):
    view = torch.int16 if x.dtype == BF16 else torch.int32
    return torch.equal(x.view(view), y.view(view))


@pytest.mark.parametrize("page", [1, 7, 64])
def test_many_ragged_prompts(page):
    """Blocks of rows find their sequences, empty ones among them."""
    ers = _ers()
    lens = [0, 1, 16, 17, 0, 0, 300, 15, 33, 0, 2, 128, 0]
    cache = _cache(17, [0] * len(lens), 1, 64, page, F32, room=310)
    T = sum(lens)
    k, v = (torch.randn(T, 1, 64, device="cuda", generator=_gen(s)) for s in (3, 4))
    want_k, want_v = cache.k.clone(), cache.v.clone()
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
    at = 0
    for i, n in enumerate(lens):
        _put_all(cache, want_k, want_v, [(i, 0, k[at:at + n], v[at:at + n])])
        at += n
    ers.attn_append(cache, k, v, cu)
    assert cache.pos.tolist() == lens and _same(cache.k, want_k) and _same(cache.v, want_v)


def test_rows_that_cannot_be_added():
    """Each error leaves its sequence as it was; the others get their rows."""
    ers = _ers()
    k, v = (torch.randn(4, 3, 1, 64, device="cuda", generator=_gen(s)) for s in (5, 6))
    three = torch.full((4,), 3, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")

    def fresh():
        return _cache(18, [6, 6, 6, 6], 1, 64, 4, F32, room=4)

    def no_page(c): c.pages.table[1, 2] = -1          # the third row's
    def far_page(c): c.pages.table[1, 2] = c.npages
    def shared(c): c.pages.refs[c.pages.table[1, 1].long()] = 2
    def full(c): c.pos[1] = 10
    def outside(c): c.pos[1] = 13
    def before(c): c.pos[1] = -1

    for spoil, code in ((no_page, "ESLOT"), (far_page, "ESLOT"), (shared, "EINVAL"), (full, "EOVERFLOW"), (outside, "EALIGN"),
                        (before, "EALIGN")):
        for call in ("commit", "append"):
            c = fresh()
            spoil(c)
            pos, kept = c.pos.clone(), c.k.clone()
            with pytest.raises(ers.ErsError, match="ERS_" + code):
                if call == "commit":
                    ers.attn_commit(c, k, v, three)
                else:
                    ers.attn_append(c, k.view(12, 1, 64), v.view(12, 1, 64), torch.arange(0, 13, 3, **i32))
            moved = torch.tensor([3, 0, 3, 3], **i32)
            assert torch.equal(c.pos, pos + moved)
            for i in (0, 2, 3):
                _put(c, kept, i, 6, k[i])
            assert _same(c.k, kept)
    for bad in (dict(accepted=torch.tensor([3, 4, 3, 3], **i32)), dict(accepted=torch.tensor([3, -1, 3, 3], **i32)),
                dict(accepted=three, path=torch.tensor([[0, 1, 2], [0, 3, 2], [0, 1, 2], [0, 1, 2]], **i32))):
        c = fresh()
        with pytest.raises(ers.ErsError, match="ERS_ECOMMIT"):
            ers.attn_commit(c, k, v, **bad)
        assert c.pos.tolist() == [9, 6, 9, 9]
    c = fresh()
    with pytest.raises(ers.ErsError, match="ERS_EINVAL"):
        ers.attn_commit(c, k, v, three, slot=torch.tensor([0, 1, 1, 2], **i32))
    assert c.pos.tolist() == [9, 6, 9, 6]
    with pytest.raises(ers.ErsError, match="ERS_ESLOT"):
        ers.attn_commit(c, k, v, three, slot=torch.tensor([0, 4, -1, 3], **i32))
    assert c.pos.tolist() == [12, 6, 9, 9]
    for cu in ([0, 6, 3, 12, 12], [0, 3, 6, 9, 13], [-1, 3, 6, 9, 12]):
        c = fresh()
        kept = c.k.clone()
        with pytest.raises(ers.ErsError, match="ERS_EINVAL"):
            ers.attn_append(c, k.view(12, 1, 64), v.view(12, 1, 64), torch.tensor(cu, **i32))
        assert c.pos.tolist() == [6] * 4 and _same(c.k, kept)


@IO
def test_verify_errors_leave_their_sequence(io):
    ers = _ers()
    for lens in ([6, 6, 6], [6, 6, 3000]):             # in one part and in several
        cache = _cache(19, lens, 1, 64, 4, io)
        q, k, v = _drafts(20, 3, 3, 2, 1, 64, io)
        good = ers.attn_verify(cache, q, k, v, max_len=max(lens))
        for parent, slot, code in (([[-1, 0, 1], [-1, 1, 0], [-1, 0, 1]], None, "EINVAL"),
                                   ([[-1, 0, 1], [-2, 0, 0], [-1, 0, 1]], None, "EINVAL"),
                                   ([[-1, 0, 1], [-3, 0, 0], [-1, 0, 1]], None, "EINVAL"),
                                   ([[-1, 0, 1], [-1, 5, 0], [-1, 0, 1]], None, "EINVAL"),
                                   (None, [0, 3, 2], "ESLOT"), (None, [0, -1, 2], "ESLOT")):
            o = torch.full_like(q, 7.0)
            i32 = dict(dtype=torch.int32, device="cuda")
            with pytest.raises(ers.ErsError, match="ERS_" + code):
                ers.attn_verify(cache, q, k, v, parent=None if parent is None else torch.tensor(parent, **i32),
                                slot=None if slot is None else torch.tensor(slot, **i32), max_len=max(lens), out=o)
            assert (o[1] == 7.0).all() and torch.equal(o[0], good[0]) and torch.equal(o[2], good[2])
        cache.pages.table[1, 0] = -1                   # a page of the past
        with pytest.raises(ers.ErsError, match="ERS_ESLOT"):
            ers.attn_verify(cache, q, k, v, max_len=max(lens))


def test_arguments():
    ers = _ers()
    cache = _cache(21, [6, 6], 2, 64, 4, BF16)
    q, k, v = _drafts(22, 2, 3, 4, 2, 64, BF16)
    for bad, err in (((q.float(), k, v), TypeError), ((q, k[:, :2], v), ValueError), ((q, k, v[:1]), ValueError),
                     ((q[0], k, v), ValueError), ((q.transpose(1, 2), k, v), ValueError), ((q.cpu(), k, v), ValueError)):
        with pytest.raises(err):
            ers.attn_verify(cache, *bad)
    with pytest.raises(ers.ErsError, match="ESHAPE"):
        ers.attn_verify(cache, q[:, :, :3].contiguous(), k, v)
    long = _drafts(23, 2, 65, 4, 2, 64, BF16)
    with pytest.raises(ers.ErsError, match="EINVAL"):
        ers.attn_verify(cache, *long)
    with pytest.raises(ValueError):
        ers.AttnCache(2, 2, 64, page_tokens=0)
    with pytest.raises(ValueError):
        ers.AttnCache(2, 2, 64, k=cache.k)
    with pytest.raises(TypeError):
        ers.AttnCache(2, 2, 64, io_dtype=torch.float16)
    with pytest.raises(AttributeError):
        cache.pos = cache.pos.clone()


@IO
def test_captured_steps(io):
    """Two captured verifies of unlike sizes and a commit, replayed as the cache grows."""
    ers = _ers()
    cache = _cache(24, [900, 40], 2, 128, 64, io, room=64)
    sets = [_drafts(25, 2, 4, 8, 2, 128, io), _drafts(26, 2, 9, 4, 2, 128, io)]
    accepted = torch.tensor([2, 4], dtype=torch.int32, device="cuda")
    outs = []
    graphs = []
    for q, k, v in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(ers.attn_verify(cache, q, k, v, max_len=1000, check=False))
        graphs.append(graph)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ers.attn_commit(cache, *sets[0][1:], accepted, check=False)
    for step in range(3):
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, (q, k, v) in zip(outs, sets):
            _check(o, cache, q, k, v)
        graph.replay()
        torch.cuda.synchronize()
        assert cache.pos.tolist() == [902 + 2 * step, 44 + 4 * step]


def test_pools_beyond_32_bits():
    """Pages whose rows start beyond 2^31 elements and 2^32 bytes of the pool: read, written and committed to."""
    ers = _ers()
    KV, D, page, npages = 4, 128, 64, 70000                # 2.3e9 elements each
    k, v = (torch.empty(npages, page, KV, D, dtype=BF16, device="cuda") for _ in range(2))
    cache = ers.AttnCache(2, KV, D, page_tokens=page, slot_pages=4, npages=npages, k=k, v=v)
    cache.pages.table.copy_(torch.tensor([[npages - 1, 3, 66000, npages - 2], [1, 69000, 2, 68000]], dtype=torch.int32))
    cache.pages.refs[cache.pages.table.flatten().long()] = 1
    rows = [torch.randn(300, KV, D, device="cuda", generator=_gen(s)).to(BF16) for s in (7, 8)]
    ers.attn_append(cache, *rows, torch.tensor([0, 180, 300], dtype=torch.int32, device="cuda"))
    assert torch.equal(cache.k[npages - 1], rows[0][:64]) and torch.equal(cache.v[69000][:56], rows[1][244:])
    q, dk, dv = _drafts(27, 2, 3, 8, KV, D, BF16)
    _check(ers.attn_verify(cache, q, dk, dv), cache, q, dk, dv)
    ers.attn_commit(cache, dk, dv, torch.tensor([3, 2], dtype=torch.int32, device="cuda"))
    assert torch.equal(cache.k[66000][52:55], dk[0]) and torch.equal(cache.v[69000][56:58], dv[1, :2])
    _check(ers.attn_verify(cache, q, dk, dv, max_len=183), cache, q, dk, dv)


@IO
def test_on_another_stream(io):
    """stream=: every allocation, launch and status of the calls belongs to that stream."""
    ers = _ers()
    cache = _cache(28, [700, 20], 2, 128, 64, io, room=8)
    q, k, v = _drafts(29, 2, 4, 8, 2, 128, io)
    accepted = torch.tensor([4, 1], dtype=torch.int32, device="cuda")
    good = ers.attn_verify(cache, q, k, v, max_len=700)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = ers.attn_verify(cache, q, k, v, max_len=700, stream=side)
    ers.attn_commit(cache, k, v, accepted, stream=side)
    after = ers.attn_verify(cache, q, k, v, max_len=700, stream=side, check=False)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, good) and cache.pos.tolist() == [704, 21]
    _check(after, cache, q, k, v)


@IO
def test_a_fork_reads_its_parents_pages(io):
    """Slots that share a prompt's pages attend to them; a row may only be added once the page is the slot's own."""
    ers = _ers()
    cache = ers.AttnCache(3, 2, 64, page_tokens=16, slot_pages=3, npages=7, io_dtype=io)
    i32 = dict(dtype=torch.int32, device="cuda")
    ers.pages_own(cache.pages, torch.tensor([0], **i32))
    rows = [torch.randn(20, 2, 64, device="cuda", generator=_gen(s)).to(io) for s in (9, 10)]
    ers.attn_append(cache, *rows, slot=torch.tensor([0], **i32))
    ers.pages_fork(cache.pages, torch.tensor([0], **i32), torch.tensor([2], **i32))
    cache.pos[2] = cache.pos[0]
    q, k, v = _drafts(30, 2, 2, 4, 2, 64, io)
    slot = torch.tensor([0, 2], **i32)
    _check(ers.attn_verify(cache, q, k, v, slot=slot), cache, q, k, v, slots=[0, 2])
    one = torch.ones(2, **i32)
    with pytest.raises(ers.ErsError, match="ERS_EINVAL"):
        ers.attn_commit(cache, k, v, one, slot=slot)
    assert cache.pos.tolist() == [20, 0, 20]
    ers.pages_own(cache.pages, torch.tensor([2], **i32))
    ers.attn_commit(cache, k, v, one, slot=slot)
    assert cache.pos.tolist() == [21, 0, 21]
    _check(ers.attn_verify(cache, q, k, v, slot=slot), cache, q, k, v, slots=[0, 2])
