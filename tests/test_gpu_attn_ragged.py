"""Attention of drafts over pasts of unlike lengths: tiles that change hands between the warps of a CTA in every order, and batches
in which one past is far longer than the others.  Bounds as in test_gpu_attn.py."""
import pytest
import torch

from test_gpu_attn import BF16, IO, _cache, _check, _drafts, _ers, _trees

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [64, 8, 24, 500])
@pytest.mark.parametrize("D", [64, 128])
def test_tiles_change_hands(page, D):
    """One to seven tiles of 64 tokens in every mixture of whole ones (copied by one lane where a page has a multiple of 8
    tokens) and a last one that has some, none or all but one of its rows, by one part and by several."""
    lens = [64 * n + r for n in range(7) for r in (0, 1, 63)]
    cache = _cache(41, lens, 2, D, page, BF16)
    for T, max_len in ((1, 64), (5, 64), (5, 449), (33, 10 ** 6)):
        q, k, v = _drafts(42 + T, len(lens), T, 4, 2, D, BF16)
        parent = _trees(len(lens), T, T)
        _check(_ers().attn_verify(cache, q, k, v, parent=parent, max_len=max_len), cache, q, k, v, parent)


@IO
@pytest.mark.parametrize("max_len", [8192, None])
def test_one_long_past_among_many_short_ones(io, max_len):
    """Enough sequences to fill the GPU, one of them with most of the tokens; the same bits every time."""
    lens = [(37 * i) % 500 for i in range(38)]
    lens[11] = 8192
    cache = _cache(43, lens, 8, 64, 64, io)
    q, k, v = _drafts(44, 38, 2, 16, 8, 64, io)
    o = _ers().attn_verify(cache, q, k, v, max_len=max_len)
    _check(o, cache, q, k, v)
    assert torch.equal(o, _ers().attn_verify(cache, q, k, v, max_len=max_len))
