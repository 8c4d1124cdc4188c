"""Host validation of the C ABI of the gated delta rule over states and of attention over a paged cache: bad calls are refused
before any launch (no GPU needed), empty ones are fine, and the workspace queries."""
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
    d = dict(nheads=8, ngroups=2, dk=128, dv=128, io_dtype=_abi.DTYPE_F32, scale=1.0)
    d.update(kw)
    return ctypes.byref(_abi.LinAttnDims(**d))


def _fwd(lib, dims=None, nseq=0, ntokens=32, max_len=32, cu=FAKE, q=FAKE, g=FAKE, final=FAKE, init=None, ws=FAKE, size=1 << 40,
         status=None):
    return lib.ers_gdn_fwd(dims or _dims(), nseq, ntokens, max_len, cu, q, FAKE, FAKE, g, FAKE, init, FAKE, final, ws, size, None,
                           status)


@needs_no_gpu
def test_gdn_refusals(lib):
    assert _fwd(lib) == 0                                            # an empty batch
    for bad, code in ((dict(io_dtype=7), 3), (dict(ngroups=3), 2), (dict(dk=32), 2), (dict(dv=96), 2), (dict(nheads=0), 2),
                      (dict(nheads=70000, ngroups=1), 2), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1)):
        assert _fwd(lib, _dims(**bad)) == code, bad
    assert _fwd(lib, nseq=-1) == 1 and _fwd(lib, ntokens=-1) == 1 and _fwd(lib, max_len=-1) == 1
    assert _fwd(lib, ntokens=1 << 31) == 1 and _fwd(lib, nseq=1 << 28) == 1
    assert _fwd(lib, _dims(nheads=128), ntokens=0x7fffffff) == 1
    for kw in (dict(q=None), dict(cu=None), dict(final=None), dict(g=None)):
        assert _fwd(lib, nseq=1, **kw) == 1, kw
    for kw in (dict(q=OFF), dict(cu=OFF), dict(final=OFF), dict(init=OFF), dict(g=OFF), dict(status=OFF), dict(ws=OFF)):
        assert _fwd(lib, nseq=1, **kw) == 4, kw


@needs_no_gpu
def test_gdn_workspace(lib):
    from exact_replay_decode_gb300 import _abi
    size = lib.ers_gdn_fwd_workspace_size
    assert size(_dims(), 0, 0, 0) == 0 and size(_dims(dk=32), 1, 64, 64) == 0 and size(_dims(), -1, 64, 64) == 0
    bf16 = _dims(io_dtype=_abi.DTYPE_BF16)
    need = size(bf16, 2, 4096, 4000)
    if need:
        assert _fwd(lib, bf16, nseq=2, ntokens=4096, max_len=4000, ws=FAKE, size=need - 1) == 10
        assert _fwd(lib, bf16, nseq=2, ntokens=4096, max_len=4000, ws=None) == 10


@needs_no_gpu
def test_gdn_cache_refusals(lib):
    from exact_replay_decode_gb300 import _abi

    def decode(cache, nseq, slot=None, read=None, q=FAKE):
        return lib.ers_gdn_decode(_dims(), ctypes.byref(cache), nseq, slot, read, q, FAKE, FAKE, FAKE, FAKE, FAKE, None, None)

    good = _abi.LinAttnCache(FAKE, FAKE, 4, 8)
    assert decode(good, 0) == 0
    assert decode(good, 5) == 1 and decode(good, -1) == 1            # more sequences than slots
    assert decode(good, 2, q=None) == 1 and decode(good, 2, q=OFF) == 4 and decode(good, 2, slot=OFF) == 4
    assert decode(good, 2, read=OFF) == 4
    assert decode(_abi.LinAttnCache(None, FAKE, 4, 8), 1) == 1 and decode(_abi.LinAttnCache(FAKE, OFF, 4, 8), 1) == 4
    assert decode(_abi.LinAttnCache(FAKE, FAKE, -1, 8), 0) == 1
    assert lib.ers_gdn_prefill(_dims(), ctypes.byref(good), 1, 4, 4, None, None, None, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, 0,
                               None, None) == 1


def _attn(lib, call, dims={}, cache={}, nseq=0, T=4, max_len=100, slot=None, q=FAKE, parent=None, ws=FAKE, size=1 << 40, ntokens=9,
          cu=FAKE, accepted=FAKE, path=None):
    from exact_replay_decode_gb300 import _abi
    d = dict(nheads=8, kv_heads=2, head_dim=128, io_dtype=_abi.DTYPE_F32, scale=1.0)
    c = dict(k=FAKE, v=FAKE, table=FAKE, refs=FAKE, pos=FAKE, nslots=4, slot_pages=3, npages=9, page_tokens=16)
    d.update(dims)
    c.update(cache)
    d, c = ctypes.byref(_abi.AttnDims(**d)), ctypes.byref(_abi.AttnCache(**c))
    if call == "verify":
        return lib.ers_attn_verify(d, c, nseq, slot, T, max_len, q, FAKE, FAKE, parent, FAKE, ws, size, None, None)
    if call == "append":
        return lib.ers_attn_append(d, c, nseq, ntokens, cu, slot, q, FAKE, None, None)
    return lib.ers_attn_commit(d, c, nseq, slot, T, path, accepted, q, FAKE, None, None)


@needs_no_gpu
@pytest.mark.parametrize("call", ["verify", "append", "commit"])
def test_attention_refusals(lib, call):
    assert _attn(lib, call) == 0
    for bad, code in ((dict(io_dtype=7), 3), (dict(kv_heads=3), 2), (dict(head_dim=96), 2), (dict(nheads=0), 2), (dict(kv_heads=0), 2),
                      (dict(nheads=8200, kv_heads=8200), 2), (dict(scale=float("nan")), 1)):
        assert _attn(lib, call, dims=bad) == code, bad
    for bad, code in ((dict(k=None), 1), (dict(v=OFF), 4), (dict(table=None), 1), (dict(refs=OFF), 4), (dict(pos=None), 1),
                      (dict(nslots=-1), 1), (dict(slot_pages=0), 1), (dict(npages=-1), 1), (dict(page_tokens=0), 1),
                      (dict(slot_pages=1 << 16, page_tokens=1 << 16), 1)):
        assert _attn(lib, call, cache=bad) == code, bad
    assert _attn(lib, call, nseq=-1) == 1 and _attn(lib, call, nseq=5) == 1
    assert _attn(lib, call, nseq=2, q=None) == 1 and _attn(lib, call, nseq=2, q=OFF) == 4 and _attn(lib, call, nseq=2, slot=OFF) == 4
    if call != "append":
        assert _attn(lib, call, T=0) == 1 and _attn(lib, call, T=65) == 1
    if call == "verify":
        assert _attn(lib, call, max_len=-1) == 1 and _attn(lib, call, nseq=2, parent=OFF) == 4
        assert _attn(lib, call, nseq=2, max_len=4000, ws=None) == 10 and _attn(lib, call, nseq=2, max_len=4000, size=100) == 10
        assert _attn(lib, call, nseq=2, max_len=4000, ws=OFF) == 4
    if call == "append":
        assert _attn(lib, call, ntokens=-1) == 1 and _attn(lib, call, nseq=1, cu=None) == 1 and _attn(lib, call, nseq=1, cu=OFF) == 4
    if call == "commit":
        assert _attn(lib, call, nseq=1, accepted=None) == 1 and _attn(lib, call, nseq=1, path=OFF) == 4


@needs_no_gpu
def test_attention_workspace(lib):
    from exact_replay_decode_gb300 import _abi
    dims = ctypes.byref(_abi.AttnDims(8, 2, 128, _abi.DTYPE_F32, 1.0))
    size = lib.ers_attn_verify_workspace_size
    assert size(dims, 0, 1, 100) == 0 and size(dims, 1, 65, 100) == 0 and size(dims, 1, 1, -1) == 0 and size(None, 1, 1, 1) == 0
    assert size(dims, 1, 1, 64) == 0 and size(dims, 1, 1, 100000) > size(dims, 1, 1, 5000) > 0
