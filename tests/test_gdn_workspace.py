"""The workspace that the gated delta rule asks for, on the host (no GPU needed): what the header says, and refused when it is less."""
import pytest

from test_hybrid_abi import FAKE, _dims, _fwd, lib, needs_no_gpu  # noqa: F401

KB = 1024


def _said(nseq, T, H, G, few):
    return (T // 64 + min(nseq, T // (few + 1))) * (81 * H + 32 * G) * KB


@pytest.mark.parametrize("nseq,T,longest,H,G", [(1, 131072, 131072, 64, 8), (2, 4096, 4000, 8, 2), (256, 256, 256, 64, 8),
                                                (64, 256, 256, 64, 8), (257, 2304, 2048, 64, 8), (4, 3339, 2048, 64, 8)])
def test_size(lib, nseq, T, longest, H, G):  # noqa: F811
    from exact_replay_decode_gb300 import _abi
    size = lib.ers_gdn_fwd_workspace_size
    dims = _dims(nheads=H, ngroups=G, io_dtype=_abi.DTYPE_BF16)
    few = 32 if nseq * H <= 64 else 24
    assert size(dims, nseq, T, longest) == _said(nseq, T, H, G, few) > 0
    assert size(dims, nseq, T, few) == 0                                  # all by the recurrence
    assert size(_dims(nheads=H, ngroups=G), nseq, T, longest) == 0        # fp32


@needs_no_gpu
def test_less_is_refused(lib):  # noqa: F811
    from exact_replay_decode_gb300 import _abi
    bf16 = _dims(io_dtype=_abi.DTYPE_BF16)
    need = lib.ers_gdn_fwd_workspace_size(bf16, 2, 4096, 4000)
    assert need > 0
    assert _fwd(lib, bf16, nseq=2, ntokens=4096, max_len=4000, ws=FAKE, size=need - 1) == 10
    assert _fwd(lib, bf16, nseq=2, ntokens=4096, max_len=4000, ws=None) == 10
