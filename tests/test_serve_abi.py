"""Host validation of the serving operators' C ABI: bad calls are refused before any launch (no GPU needed), empty ones
are fine, and the workspace queries."""
import ctypes

import pytest

needs_no_gpu = pytest.mark.skipif(__import__("torch").cuda.is_available(), reason="host-only validation test")

FAKE = 1 << 20          # 16-byte aligned, never dereferenced
OFF = FAKE + 4


@pytest.fixture(scope="module")
def lib():
    from exact_replay_decode_gb300 import build, _abi
    build.build()
    return _abi.lib()


def _dims(**kw):
    from exact_replay_decode_gb300 import _abi
    d = dict(nheads=8, ngroups=2, dk=128, dv=128, io_dtype=_abi.DTYPE_BF16, scale=1.0)
    d.update(kw)
    return ctypes.byref(_abi.LinAttnDims(**d))


def _fwd(lib, dims=None, nseq=0, ntokens=32, max_len=32, decay=FAKE, cu=FAKE, q=FAKE, final=FAKE, init=None):
    return lib.ers_linattn_fwd(dims or _dims(), decay, nseq, ntokens, max_len, cu, q, FAKE, FAKE, init, FAKE, final, None, None)


@needs_no_gpu
def test_linattn_refusals(lib):
    assert _fwd(lib) == 0                                            # an empty batch
    for bad, code in ((dict(io_dtype=7), 3), (dict(ngroups=3), 2), (dict(dk=32), 2), (dict(dv=96), 2),
                      (dict(nheads=0), 2), (dict(nheads=70000, ngroups=1), 2), (dict(scale=float("nan")), 1),
                      (dict(scale=float("inf")), 1)):
        assert _fwd(lib, _dims(**bad)) == code, bad
    assert _fwd(lib, nseq=-1) == 1 and _fwd(lib, ntokens=-1) == 1 and _fwd(lib, max_len=-1) == 1
    assert _fwd(lib, ntokens=1 << 31) == 1
    for kw in (dict(q=None), dict(cu=None), dict(final=None), dict(decay=None)):
        assert _fwd(lib, nseq=1, **kw) == 1, kw
    for kw in (dict(q=OFF), dict(cu=OFF), dict(final=OFF), dict(init=OFF), dict(decay=OFF)):
        assert _fwd(lib, nseq=1, **kw) == 4, kw
    assert lib.ers_linattn_fwd(None, FAKE, 0, 0, 0, FAKE, FAKE, FAKE, FAKE, None, FAKE, FAKE, None, None) == 1


@needs_no_gpu
def test_linattn_cache_refusals(lib):
    from exact_replay_decode_gb300 import _abi

    def decode(cache, nseq, slot=None, q=FAKE):
        return lib.ers_linattn_decode(_dims(), FAKE, ctypes.byref(cache), nseq, slot, None, q, FAKE, FAKE, FAKE, None, None)

    good = _abi.LinAttnCache(FAKE, FAKE, 4, 8)
    assert decode(good, 0) == 0
    assert decode(good, 5) == 1 and decode(good, -1) == 1            # more sequences than slots
    assert decode(good, 2, q=None) == 1 and decode(good, 2, q=OFF) == 4 and decode(good, 2, slot=OFF) == 4
    assert decode(_abi.LinAttnCache(None, FAKE, 4, 8), 1) == 1
    assert decode(_abi.LinAttnCache(FAKE, OFF, 4, 8), 1) == 4
    assert decode(_abi.LinAttnCache(FAKE, FAKE, -1, 8), 0) == 1
    assert lib.ers_linattn_prefill(_dims(), FAKE, ctypes.byref(good), 1, 4, 4, None, None, None, FAKE, FAKE, FAKE, FAKE,
                                   None, None) == 1


def _pool(**kw):
    from exact_replay_decode_gb300 import _abi
    p = _abi.PagePool()
    p.table, p.refs, p.nslots, p.slot_pages, p.npages, p.narrays = FAKE, FAKE, 4, 2, 9, 1
    p.array[0], p.page_bytes[0] = FAKE, 64
    for k, v in kw.items():
        setattr(p, k, v)
    return p


@needs_no_gpu
def test_pages_refusals(lib):
    ref = ctypes.byref
    assert lib.ers_pages_free(ref(_pool()), 0, None, None, None) == 0
    for kw, code in ((dict(nslots=(1 << 20) + 1), 2), (dict(slot_pages=0), 2), (dict(narrays=13), 1), (dict(npages=-1), 1),
                     (dict(table=OFF), 4), (dict(refs=None), 1)):
        assert lib.ers_pages_free(ref(_pool(**kw)), 0, None, None, None) == code, kw
    assert lib.ers_pages_free(ref(_pool()), 5, FAKE, None, None) == 1          # more slots than there are
    assert lib.ers_pages_free(ref(_pool()), 1, None, None, None) == 1
    assert lib.ers_pages_fork(ref(_pool()), 1, FAKE, OFF, None, None) == 4
    odd = _pool()
    odd.page_bytes[0] = 3
    assert lib.ers_pages_copy(ref(odd), 1, FAKE, FAKE, None, None) == 2
    assert lib.ers_pages_own_workspace_size(ref(_pool()), 3) >= 3 * 2 * 8
    assert lib.ers_pages_own(ref(_pool()), 1, FAKE, 8, FAKE, None, 0, None, None) == 10
    assert lib.ers_pages_own(ref(_pool()), 1, FAKE, 1, FAKE, FAKE, 1 << 20, None, None) == 1     # an unknown flag
    assert lib.ers_pages_compact_workspace_size(ref(_pool())) >= 19 * 4
    assert lib.ers_pages_compact(ref(_pool()), FAKE, FAKE, FAKE, 16, None, None) == 10
    assert lib.ers_pages_compact(ref(_pool()), FAKE, None, FAKE, 1 << 20, None, None) == 1


@needs_no_gpu
def test_pages_past_32_bits_are_refused(lib):
    # counts that the deciding CTA's steps of 1024 would carry past 32 bits (699734 * 3069 = 2^31 - 2)
    for kw in (dict(npages=2**31 - 1), dict(npages=0x7ffffc01), dict(nslots=699734, slot_pages=3069)):
        assert lib.ers_pages_free(ctypes.byref(_pool(**kw)), 0, None, None, None) == 1, kw
    assert lib.ers_pages_free(ctypes.byref(_pool(npages=0x7ffffc00)), 0, None, None, None) == 0


@needs_no_gpu
def test_pages_clone_refusals(lib):
    def clone(n=1, src=FAKE, dst=FAKE, read=FAKE, ws=FAKE, size=1 << 20, **kw):
        return lib.ers_pages_clone(ctypes.byref(_pool(**kw)), n, src, dst, read, ws, size, None, None)

    assert clone(n=0, src=None, dst=None, read=None, ws=None, size=0) == 0
    assert clone(n=5) == 1 and clone(n=-1) == 1
    for kw in (dict(src=None), dict(dst=None), dict(read=None)):
        assert clone(**kw) == 1, kw
    for kw in (dict(src=OFF), dict(dst=OFF), dict(read=OFF), dict(ws=OFF)):
        assert clone(**kw) == 4, kw
    assert clone(ws=None) == 10 and clone(size=8) == 10
    assert clone(slot_pages=0) == 2


@needs_no_gpu
def test_logprobs_refusals(lib):
    from exact_replay_decode_gb300 import _abi

    def call(io=_abi.DTYPE_BF16, rows=0, vocab=100, stride=100, logits=FAKE, target=FAKE, scale=1.0, k=0, lp=FAKE, ent=FAKE,
             ids=None, tops=None):
        return lib.ers_token_logprobs(io, rows, vocab, stride, logits, target, scale, k, lp, ent, ids, tops, None, None)

    assert call() == 0
    assert call(io=5) == 3
    for kw in (dict(rows=-1), dict(vocab=0), dict(stride=99), dict(k=33), dict(k=-1), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf"))):
        assert call(**kw) == 1, kw
    for kw in (dict(logits=None), dict(target=None), dict(lp=None), dict(k=2), dict(k=2, ids=FAKE)):
        assert call(rows=1, **kw) == 1, kw
    for kw in (dict(logits=FAKE + 1), dict(target=OFF), dict(ent=OFF), dict(k=1, ids=OFF, tops=FAKE)):
        assert call(rows=1, **kw) == 4, kw
