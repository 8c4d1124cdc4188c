"""Pages of a cache on the GPU: every decision equals a sequential model's (whole numbers, bytes moved), a call that finds an
error changes nothing, and a forked ReplayCache slot decodes on with its parent's bits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _ers():
    import exact_replay_decode_gb300 as ers
    return ers


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Model:
    """The pool's rules, one entry after the other, on the host."""

    def __init__(self, table, refs, arrays):
        self.table, self.refs = table.copy(), refs.copy()
        self.arrays = [x.copy() for x in arrays]

    def fork(self, src, dst):
        for s, d in zip(src, dst):
            self.table[d] = self.table[s]
            for p in self.table[s]:
                if p >= 0:
                    self.refs[p] += 1

    def free(self, slots):
        for s in slots:
            for p in self.table[s]:
                if p >= 0:
                    self.refs[p] -= 1
            self.table[s] = -1

    def own(self, slots, copy):
        start, old = self.refs.copy(), self.table[slots].copy()
        free = [p for p in range(len(start)) if start[p] == 0]
        source = [x.copy() for x in self.arrays]
        for s in slots:
            for c, p in enumerate(self.table[s]):
                if p >= 0 and start[p] <= 1:
                    continue
                new = free.pop(0)
                if p >= 0:
                    self.refs[p] -= 1
                self.refs[new] = 1
                self.table[s, c] = new
                for x, y in zip(self.arrays, source):
                    if copy:
                        x[new] = y[p] if p >= 0 else 0
        return old

    def compact(self):
        live = int((self.refs > 0).sum())
        remap = np.where(self.refs > 0, np.arange(len(self.refs)), -1).astype(np.int32)
        holes = [p for p in range(live) if self.refs[p] == 0]
        for p in range(live, len(self.refs)):
            if self.refs[p] > 0:
                h = holes.pop(0)
                remap[p] = h
                self.refs[h], self.refs[p] = self.refs[p], 0
                for x in self.arrays:
                    x[h] = x[p]
        self.table = np.where(self.table >= 0, remap[np.maximum(self.table, 0)], -1).astype(np.int32)
        return remap, live


def _same(pool, model):
    assert np.array_equal(pool.table.cpu().numpy(), model.table)
    assert np.array_equal(pool.refs.cpu().numpy(), model.refs)
    for x, y in zip(pool.arrays, model.arrays):
        assert np.array_equal(x.cpu().numpy(), y)


def _pool(seed, nslots, slot_pages, npages, shapes):
    rng = np.random.Generator(np.random.PCG64(seed))
    table = np.full((nslots, slot_pages), -1, dtype=np.int32)
    refs = np.zeros(npages, dtype=np.int32)
    arrays = [rng.integers(-30000, 30000, (npages, *s)).astype(np.int16) for s in shapes]
    pool = _ers().PagePool([torch.from_numpy(x).cuda() for x in arrays], _ints(table), _ints(refs))
    return pool, Model(table, refs, arrays), rng


@pytest.mark.parametrize("nslots,slot_pages,npages,shapes", [
    (1, 1, 3, [(8,)]), (7, 1, 20, [(24,), (3, 5)]), (40, 3, 200, [(1,), (64, 33), (8,)]),
    (700, 2, 2500, [(16,)]), (33, 1, 60, [(40000,), (17001,)])])
def test_random_histories_equal_the_model(nslots, slot_pages, npages, shapes):
    ers = _ers()
    pool, model, rng = _pool(nslots, nslots, slot_pages, npages, shapes)
    for step in range(25):
        held = [s for s in range(nslots) if (model.table[s] >= 0).any()]
        bare = [s for s in range(nslots) if (model.table[s] < 0).all()]
        what = rng.integers(0, 5)
        if what == 0 and bare:
            new = rng.permutation(bare)[: rng.integers(1, len(bare) + 1)]
            if (model.refs == 0).sum() >= len(new) * slot_pages:
                copy = bool(rng.integers(0, 2))
                read = ers.pages_own(pool, _ints(new), copy=copy)
                assert np.array_equal(read.cpu().numpy(), model.own(new, copy))
        elif what == 1 and bare and held:
            dst = rng.permutation(bare)[: rng.integers(1, len(bare) + 1)]
            src = rng.choice(held, len(dst))
            ers.pages_fork(pool, _ints(src), _ints(dst))
            model.fork(src, dst)
        elif what == 2 and held:
            some = rng.permutation(held)[: rng.integers(1, len(held) + 1)]
            if (model.refs == 0).sum() >= len(some) * slot_pages:
                read = ers.pages_own(pool, _ints(some))
                assert np.array_equal(read.cpu().numpy(), model.own(some, True))
        elif what == 3 and held:
            some = rng.permutation(nslots)[: rng.integers(1, nslots // 2 + 2)]
            ers.pages_free(pool, _ints(some))
            model.free(some)
        elif what == 4:
            remap, live = ers.pages_compact(pool)
            eremap, elive = model.compact()
            assert np.array_equal(remap.cpu().numpy(), eremap) and int(live) == elive
        _same(pool, model)


@pytest.mark.parametrize("size", [1, 7, 8, 4096, 16384 + 8, 100001])
def test_copy_of_pages_of_any_size(size):
    pool, model, rng = _pool(size, 1, 1, 12, [(size,), (8,)])
    _ers().pages_copy(pool.arrays, _ints([3, 3, 0]), _ints([5, 11, 7]))
    for x in model.arrays:
        x[[5, 11, 7]] = x[[3, 3, 0]]
    _same(pool, model)


def test_large_pages_past_32_bits():
    x = torch.empty(5, 600_000_000, dtype=torch.int16, device="cuda")   # 1.2 GB a page, 6 GB in all
    x[1].fill_(7)
    x[4].fill_(9)
    _ers().pages_copy([x], _ints([4]), _ints([3]))
    assert (x[3] == 9).all() and (x[4] == 9).all() and (x[1] == 7).all()


def test_errors_change_nothing():
    ers = _ers()
    pool, model, _ = _pool(3, 6, 2, 9, [(32,)])
    ers.pages_own(pool, _ints([0, 1, 2]))
    model.own([0, 1, 2], True)
    st = ers.Status("cuda")

    def fails(code, f, *args, **kw):
        st.reset()
        out = f(*args, status=st, check=False, **kw)
        assert st.read() == code
        _same(pool, model)
        return out

    read = fails(6, ers.pages_own, pool, _ints([3, 4]))                # four pages, three free
    assert (read == -2).all()
    fails(1, ers.pages_own, pool, _ints([3, 3]))
    fails(8, ers.pages_own, pool, _ints([3, 6]))
    fails(8, ers.pages_own, pool, _ints([-1]))
    fails(1, ers.pages_free, pool, _ints([1, 0, 1]))
    fails(8, ers.pages_free, pool, _ints([1, 600]))
    fails(1, ers.pages_fork, pool, _ints([0, 1]), _ints([3, 3]))
    fails(1, ers.pages_fork, pool, _ints([0]), _ints([1]))            # it holds pages already
    fails(1, ers.pages_fork, pool, _ints([0, 3]), _ints([3, 4]))      # both source and destination
    fails(8, ers.pages_fork, pool, _ints([6]), _ints([3]))
    fails(8, ers.pages_copy, pool.arrays, _ints([0]), _ints([9]))
    fails(8, ers.pages_copy, pool.arrays, _ints([-1]), _ints([0]))
    pool.table[2, 1] = 9
    model.table[2, 1] = 9
    fails(8, ers.pages_compact, pool)
    fails(8, ers.pages_free, pool, _ints([2]))
    fails(8, ers.pages_fork, pool, _ints([2]), _ints([3]))
    with pytest.raises(ers.ErsError):
        ers.pages_own(pool, _ints([2]))


def test_refusals():
    ers = _ers()
    x, table = torch.zeros(4, 8, device="cuda"), torch.full((2, 1), -1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        ers.PagePool([], table)
    with pytest.raises(ValueError):
        ers.PagePool([x, torch.zeros(3, 8, device="cuda")], table)
    with pytest.raises(TypeError):
        ers.PagePool([x], table.long())
    with pytest.raises(ValueError):
        ers.PagePool([x.t()], table)
    pool = ers.PagePool([x], table)
    with pytest.raises(ers.ErsError):
        ers.pages_free(pool, _ints([0, 1, 0]))                          # more slots than there are
    with pytest.raises(TypeError):
        ers.pages_free(pool, torch.zeros(1, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        ers.pages_fork(pool, _ints([0, 1]), _ints([0]))
    with pytest.raises(ers.ErsError):
        ers.PagePool([torch.zeros(4, 3, dtype=torch.uint8, device="cuda")], table) and ers.pages_copy(
            [torch.zeros(4, 3, dtype=torch.uint8, device="cuda")], _ints([0]), _ints([1]))
    with pytest.raises(ValueError):
        ers.ReplayCache(1, 4, 1, 64, 128, 16).page_pool()


def test_entries_without_a_reference_change_nothing():
    """A table that names a page more often than refs counts it: reported by every call that meets it, nothing changes."""
    ers = _ers()
    pool, model, _ = _pool(11, 6, 2, 12, [(32,)])
    ers.pages_own(pool, _ints([0, 1, 2]))
    model.own([0, 1, 2], True)
    ers.pages_free(pool, _ints([0]))                                  # pages 0 and 1: holes below the others
    model.free([0])
    st = ers.Status("cuda")

    def fails(f, *args, **kw):
        st.reset()
        out = f(*args, status=st, check=False, **kw)
        assert st.read() == 1
        _same(pool, model)
        return out

    pool.refs[4] = model.refs[4] = 0                                  # slot 2's first
    fails(ers.pages_free, pool, _ints([1, 2]))
    fails(ers.pages_fork, pool, _ints([1, 2]), _ints([3, 4]))
    for copy in (True, False):
        assert (fails(ers.pages_own, pool, _ints([3, 2]), copy=copy) == -2).all()
    remap, live = fails(ers.pages_compact, pool)
    assert int(live) == 3 and remap.tolist() == [-1, -1, 2, 3, -1, 5] + [-1] * 6
    pool.refs[4] = model.refs[4] = 1
    ers.pages_fork(pool, _ints([2, 2]), _ints([3, 4]))
    model.fork([2, 2], [3, 4])
    pool.refs[5] = model.refs[5] = 2                                  # named by three slots
    fails(ers.pages_free, pool, _ints([3, 2, 4]))
    for copy in (True, False):
        assert (fails(ers.pages_own, pool, _ints([0, 4, 2, 3]), copy=copy) == -2).all()
    pool.refs[5] = model.refs[5] = 3
    read = ers.pages_own(pool, _ints([4, 2]))
    assert np.array_equal(read.cpu().numpy(), model.own([4, 2], True))
    _same(pool, model)


def test_counting_a_table_that_names_pages_out_of_range():
    """The pool counts what is in range; the calls report the rest."""
    ers = _ers()
    x, st = torch.zeros(4, 8, device="cuda"), ers.Status("cuda")
    pool = ers.PagePool([x], _ints([[2, 4], [-5, 2], [1, 2**31 - 1], [-1, -(2**31)]]))
    assert pool.refs.tolist() == [0, 1, 2, 0]
    for slot in range(4):
        st.reset()
        ers.pages_free(pool, _ints([slot]), status=st, check=False)
        assert st.read() == 8
    assert pool.refs.tolist() == [0, 1, 2, 0]


def test_many_slots():
    """A table larger than the default shared memory's bitmap."""
    n = 600_000
    pool, _, _ = _pool(1, n, 1, 40, [(8,)])
    some = _ints([0, 599_999, 31, 32, 500_000])
    _ers().pages_own(pool, some)
    assert pool.table[some.long(), 0].tolist() == [0, 1, 2, 3, 4]


@pytest.mark.parametrize("paged", [None, (4, 16)], ids=["dense", "paged"])
def test_forked_replay_slots_decode_with_the_parents_bits(paged):
    ers = _ers()
    import synth
    from synth import torch_io
    H, G, P, N, Q = 8, 2, 64, 128, 16
    w = synth.Workload("fork", synth.Dims(H, G, P, N, Q), True, seqlens=(40,))
    params, toks, _ = synth.prefill_inputs(w, seed=5)
    prm = ers.LayerParams(*torch_io.params_to(params, torch.device("cuda")))
    x, dt, B, C = torch_io.tokens_to(toks, torch.device("cuda"))
    cache = ers.ReplayCache(3, H, G, P, N, Q, torch.bfloat16, paged=paged)
    zero = _ints([0])
    ers.chunked_prefill(cache, prm, x[:37], dt[:37], B[:37], C[:37], slot=zero)
    ers.fork_slots(cache, _ints([0, 0]), _ints([2, 1]))
    for t in range(37, 40):
        tok = [u[t:t + 1].expand(3, *u.shape[1:]).contiguous() for u in (x, dt, B, C)]
        y = ers.replay_decode(cache, prm, *tok)
        assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])
    y_ref, _ = ers.ssd_scan_fwd(x, dt, prm, B, C, chunk=Q)
    assert torch.equal(y[0].view(torch.int16), y_ref[-1].view(torch.int16))
    if paged:
        assert (cache.page_pool().refs[cache.buf_pages.long()] == 1).all()


def _replay_arrays(cache):
    return [t for t in (cache.state, cache.read_copy, cache.read_scale, cache.read_block_scale, cache.pos, cache.buf_x,
                        cache.buf_dt, cache.buf_B, cache.buf_C, cache.buf_pages) if t is not None]


def _filled(paged, **kw):
    cache = _ers().ReplayCache(4, 4, 2, 64, 128, 16, BF16, paged=paged, **kw)
    g = torch.Generator(device="cuda").manual_seed(2)
    for t in _replay_arrays(cache):
        if t is not cache.buf_pages:
            t.view(torch.uint8).random_(0, 256, generator=g)
    return cache


@pytest.mark.parametrize("paged", [None, (4, 24)], ids=["dense", "paged"])
@pytest.mark.parametrize("kw", [dict(), dict(read_copy=True), dict(read_copy=True, read_dtype="fp8"),
                                dict(read_copy=True, read_dtype="nvfp4", anchor="fp16_sr"),
                                dict(read_copy=True, read_dtype="nvfp4", anchor="nvfp4_sr_shared")], ids=str)
def test_fork_slots_copies_every_array(paged, kw):
    """Also the read copies with their scales, byte by byte; other slots keep theirs."""
    cache = _filled(paged, **kw)
    before = [t.clone() for t in _replay_arrays(cache)]
    _ers().fork_slots(cache, _ints([2, 2]), _ints([3, 0]))
    for t, old in zip(_replay_arrays(cache), before):
        if t is cache.buf_pages:
            assert torch.equal(t[[1, 2]], old[[1, 2]]) and t.unique().numel() == t.numel()
            continue
        own, was = t, old
        if paged and t.shape[0] == 24:                       # a slot's rows, through the table now and before
            own, was = t[cache.buf_pages.long()], old[before[-1].long()]
        own, was = (y.reshape(4, -1).contiguous().view(torch.uint8) for y in (own, was))
        for slot, source in enumerate((2, 1, 2, 2)):
            assert torch.equal(own[slot], was[source])


@pytest.mark.parametrize("paged,src,dst,code", [
    ((4, 18), [0, 1], [2, 3], 0), ((4, 16), [0, 1, 0], [2, 3, 2], 1), ((4, 24), [0, 2], [2, 3], 1), ((4, 24), [0, 4], [2, 3], 8),
    ((4, 24), [0, 1], [2, -1], 8), ((4, 10), [0], [3], 6), ((4, 10), [0, 1], [2, 3], 6), ((4, 11), [1], [2], 6)], ids=str)
def test_fork_slots_whole_or_not_at_all(paged, src, dst, code):
    """Too few free pages (a cache whose later slots share page 0), lists that overlap, slots that are none."""
    ers = _ers()
    for check in (True, False):
        cache = _filled(paged)
        refs = cache.page_pool().refs
        before = [t.clone() for t in _replay_arrays(cache) + [refs]]
        if check and code:
            with pytest.raises(ers.ErsError):
                ers.fork_slots(cache, _ints(src), _ints(dst))
        else:
            st = ers.Status("cuda")
            ers.fork_slots(cache, _ints(src), _ints(dst), status=st, check=False)
            assert st.read() == code
            if code:                                           # and without a word
                ers.fork_slots(cache, _ints(src), _ints(dst), check=False)
        after = _replay_arrays(cache) + [refs]
        same = [torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(after, before)]
        assert all(same) if code else not any(same[:2])


def test_clone_equals_free_fork_and_own():
    """One decision, against the model's three; pages that dst gives up are handed out again."""
    ers = _ers()
    from exact_replay_decode_gb300 import serve
    for seed in range(12):
        pool, model, rng = _pool(seed, 9, 2, 22, [(24,), (3, 5)])
        ers.pages_own(pool, _ints([8, 1, 4, 0]))
        model.own([8, 1, 4, 0], True)
        ers.pages_fork(pool, _ints([1, 1]), _ints([3, 6]))
        model.fork([1, 1], [3, 6])
        dst = rng.permutation(9)[:4]
        src = rng.choice(np.setdiff1d(np.arange(9), dst), 4)
        read = serve._pages_clone(pool, _ints(src), _ints(dst), None, True)
        model.free(dst)
        assert np.array_equal(read.cpu().numpy(), model.table[src])
        model.fork(src, dst)
        model.own(dst, True)
        _same(pool, model)


def test_clone_with_entries_that_are_not_counted():
    ers = _ers()
    pool, model, _ = _pool(5, 5, 1, 9, [(16,)])
    ers.pages_own(pool, _ints([0, 1]))
    model.own([0, 1], True)
    ers.pages_fork(pool, _ints([0]), _ints([2]))
    model.fork([0], [2])
    for page, count in ((0, 1), (1, 0), (0, 0)):               # src and dst name page 0, counted once; dst's page 1 not at all
        pool.refs[page] = count
        model.refs[page] = count
        st = ers.Status("cuda")
        from exact_replay_decode_gb300 import serve
        read = serve._pages_clone(pool, _ints([0, 0]), _ints([2, 1]), st, False)
        assert st.read() == 1 and (read == -2).all()
        _same(pool, model)
        pool.refs[page] = model.refs[page] = 2 if page == 0 else 1


def test_page_pool_follows_replaced_tensors():
    """Every other call reads a cache's tensors when it is made; so does a fork."""
    ers = _ers()
    cache = _filled((4, 24))
    old = cache.page_pool()
    table = _ints([[4 * s + c for c in range(4)] for s in (5, 4, 3, 2)])
    kept = cache.buf_pages.clone()
    cache.buf_pages, cache.buf_x = table, cache.buf_x.clone()
    was = [cache.buf_x[table.long()].clone(), cache.buf_dt[table.long()].clone()]
    ers.fork_slots(cache, _ints([1]), _ints([0]))
    assert cache.page_pool() is not old and cache.page_pool() is cache.page_pool()
    assert cache.buf_pages[0].tolist() == [0, 1, 2, 3] and torch.equal(old.table, kept)
    for t, rows in zip((cache.buf_x, cache.buf_dt), was):
        now = t[cache.buf_pages.long()]
        for slot, source in enumerate((1, 1, 2, 3)):
            assert torch.equal(now[slot].view(torch.uint8), rows[source].view(torch.uint8))


def test_tensors_of_a_pool_or_a_state_cache_cannot_be_replaced():
    """Their calls go by where the tensors are, so another one would be passed over in silence."""
    ers = _ers()
    cache = ers.LinAttnCache(2, 2, 2)
    for name in ("state", "pages"):
        with pytest.raises(AttributeError):
            setattr(cache, name, getattr(cache, name))
    for name in ("table", "refs", "arrays"):
        with pytest.raises(AttributeError):
            setattr(cache.pages, name, getattr(cache.pages, name))
    with pytest.raises(TypeError):
        cache.pages.arrays[0] = cache.state.clone()
