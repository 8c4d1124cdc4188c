"""Calls of the gated delta rule whose sequences have unlike lengths: each goes by the recurrence or by chunks by its own length, with
the bits that it has alone, whatever its neighbours are and whatever the caller knows of the longest.  Bounds as in
test_gpu_gdn_rule.py."""
import pytest
import torch

from test_gpu_gdn_rule import BF16, F32, _check, _cu, _ers, _gen, _inputs, _norm, _rule

pytestmark = pytest.mark.gpu


def _parts(lens):
    at = 0
    for n in lens:
        yield slice(at, at + n)
        at += n


@pytest.mark.parametrize("H,G,few", [(2, 1, 32), (16, 4, 24)])
@pytest.mark.parametrize("hint", ["longest", "none", "loose", "captured"])
def test_short_sequences_have_their_own_bits(H, G, few, hint):
    """Beside prompts, empty ones and one another, with the recurrence's precision."""
    lens = [300, 1, few, 0, few + 1, 5, 64, 0, 0, 17, 129, 3]
    args = _inputs(61, sum(lens), H, G, 128, 128, BF16)
    init = torch.randn(len(lens), H, 128, 128, device="cuda", generator=_gen(62)) * 0.3
    ers, cu = _ers(), _cu(lens)
    if hint == "captured":
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            o, fin = ers.gdn_fwd(*args, cu, init_state=init, check=False)
        graph.replay()
        torch.cuda.synchronize()
    else:
        o, fin = ers.gdn_fwd(*args, cu, init_state=init, max_seqlen={"longest": 300, "none": None, "loose": 10 ** 9}[hint])
    _check(o, fin, args, lens, init)
    for i, part in enumerate(_parts(lens)):
        if lens[i] > few:
            continue
        alone = [x[part].clone() for x in args]
        o1, fin1 = ers.gdn_fwd(*alone, init_state=init[i:i + 1])
        assert torch.equal(o[part], o1) and torch.equal(fin[i], fin1[0])
        _check(o1, fin1, alone, [lens[i]], init[i:i + 1], chunks=False)


@pytest.mark.parametrize("hint", [None, 1000, 10 ** 6])
def test_a_prompt_among_many_single_tokens(hint):
    """On the cache, as a server's mixed step is: the tokens' states are as near the rule as gdn_decode's."""
    ers, S, H = _ers(), 200, 8
    lens = [1] * 70 + [1000] + [1] * (S - 71)
    args = _inputs(63, sum(lens), H, 2, 128, 128, BF16)
    cache = ers.LinAttnCache(S, H, 2)
    cache.state.copy_(torch.randn(cache.state.shape, device="cuda", generator=_gen(64)) * 0.3)
    init = cache.state.clone()
    o = ers.gdn_prefill(cache, *args, _cu(lens), max_seqlen=hint)
    _check(o, cache.state, args, lens, init)
    _, want, _, _ = _rule(*args, lens, init)
    single = torch.tensor(lens, device="cuda") == 1
    assert _norm(cache.state[single], want[single]) <= 2e-6


@pytest.mark.parametrize("captured", [False, True])
def test_many_short_sequences_and_no_hint(captured):
    """Branches of a tree, and single tokens, without max_seqlen: bits and precision of the recurrence, a workspace of some chunks."""
    ers = _ers()
    for lens, H, G in (([4] * 64, 16, 2), ([1] * 256, 16, 2), ([3, 7, 0, 24] * 12, 16, 2)):
        args = _inputs(65, sum(lens), H, G, 128, 128, BF16)
        init = torch.randn(len(lens), H, 128, 128, device="cuda", generator=_gen(66)) * 0.3
        want = ers.gdn_fwd(*args, _cu(lens), init_state=init, max_seqlen=max(lens))
        cu = _cu(lens)
        torch.cuda.synchronize()
        torch.cuda.reset_peak_memory_stats()
        before = torch.cuda.memory_allocated()
        if captured:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                o, fin = ers.gdn_fwd(*args, cu, init_state=init, check=False)
            graph.replay()
        else:
            o, fin = ers.gdn_fwd(*args, cu, init_state=init)
        torch.cuda.synchronize()
        used = torch.cuda.max_memory_allocated() - before - (fin.numel() * 4 + o.numel() * 2)
        assert torch.equal(o, want[0]) and torch.equal(fin, want[1])
        _check(o, fin, args, lens, init, chunks=False)
        T = sum(lens)
        assert used <= (T // 64 + T // 25) * (81 * H + 32 * G) * 1024 + (4 << 20)


@pytest.mark.parametrize("seed", range(6))
def test_ragged_batches(seed):
    """Chunk numbers of sequences of any lengths, more of them than a CTA has threads, in any order, tokens left over at both ends."""
    import random
    r = random.Random(seed)
    S = r.choice([3, 40, 700])
    lens = [r.choice([0, 1, r.randint(0, 30), r.randint(20, 70), r.randint(0, 200)]) for _ in range(S)]
    lens[r.randrange(S)] = 65
    lead, rest = r.choice([0, 100]), r.choice([0, 50])
    args = _inputs(67 + seed, lead + sum(lens) + rest, 2, 1, 64, 64, BF16)
    cu = _cu(lens) + lead
    o, fin = torch.full_like(args[2], 7.0), torch.empty(S, 2, 64, 64, device="cuda")
    _ers().gdn_fwd(*args, cu, max_seqlen=r.choice([max(lens), 10 ** 6]), out=(o, fin))
    end = lead + sum(lens)
    assert (o[:lead] == 7.0).all() and (o[end:] == 7.0).all()
    _check(o[lead:end], fin, [x[lead:end] for x in args], lens)


@pytest.mark.parametrize("io,lens", [(F32, [300, 280, 0, 310, 17]), (BF16, [24, 20, 23, 1, 24])], ids=["f32", "bf16"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128), (128, 64), (64, 64)])
def test_heads_enough_for_four_rows_a_lane(io, lens, dk, dv):
    """More CTAs of 16 state rows than fit four a SM (608), by the lengths and by the sum of tokens: the recurrence's widest form."""
    H = 64 if dv == 128 else 160
    assert 3 * H * dv // 16 > 608
    args = _inputs(73, sum(lens), H, 16, dk, dv, io)
    init = torch.randn(len(lens), H, dv, dk, device="cuda", generator=_gen(74)) * 0.3
    o, fin = _ers().gdn_fwd(*args, _cu(lens), init_state=init, scale=dk ** -0.5, max_seqlen=max(lens))
    _check(o, fin, args, lens, init, dk ** -0.5, chunks=False)
