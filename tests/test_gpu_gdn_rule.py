"""Prompts and single tokens of the gated delta rule on the GPU, against the rule token by token in 64 bits.

Bounds.  For keys of norm at most 1, gates and beta in [0, 1], a token maps a state row S_d by a (I - beta k k^T), whose norm is at
most 1, so errors add up and are forgotten as the state is: with c the relative error that one token (or, of a chunk, each
of its tokens) adds, |dS_d| <= E with E_t = a_t E_(t-1) + c (|S_d| + |v_d|), and an output is within |scale| |q| (E + c |S_d|) of
the formula's before its one rounding to bf16 (2^-8 of its value).  The recurrence sums dk products in fp32 and rounds
some ten times: c = (dk + 16) 2^-24.  Chunks make products of operands that carry at least 16 bits: three such
roundings (2^-17 each) and the sums of 64 tokens: c = 2^-15.  Rounding errors do not conspire: in the 2-norm fp32 results
stay within 2e-6, states from chunks within 1e-5 (a rounding of 2^-17 at most is 2^-18 in the mean, 3.8e-6, and three of them in
quadrature 6.6e-6), bf16 outputs within 2.2e-3 (their own rounding is 1.7e-3)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _ers():
    import exact_replay_decode_gb300 as ers
    return ers


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _inputs(seed, T, H, G, dk, dv, io, strong=1.0):
    g = _gen(seed)
    r = dict(device="cuda", generator=g)
    q, k = (torch.randn(T, G, dk, **r) for _ in range(2))
    q, k = ((x / (x.norm(dim=-1, keepdim=True) * 1.01)).to(io) for x in (q, k))     # (rounded ones have norms below 1 too)
    v = torch.randn(T, H, dv, **r).to(io)
    gate = -strong * torch.rand(T, H, **r) * torch.exp2(-8.0 * torch.arange(H, dtype=F32, device="cuda") / H)
    beta = torch.rand(T, H, **r)
    return q, k, v, gate, beta


def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _rule(q, k, v, g, beta, lens, init=None, scale=1.0, c=0.0):
    """Outputs, final states, and how far each may be off for a relative error c a token."""
    H, G = v.shape[1], q.shape[1]
    group = torch.arange(H, device="cuda") // (H // G)
    q, k, v, g, beta = q.double()[:, group], k.double()[:, group], v.double(), g.double(), beta.double()
    o, o_off = torch.zeros_like(v), torch.zeros_like(v)
    finals, offs, t = [], [], 0
    for i, n in enumerate(lens):
        S = init[i].double() if init is not None else torch.zeros(H, v.shape[2], q.shape[2], dtype=torch.float64, device="cuda")
        E = torch.zeros(H, v.shape[2], dtype=torch.float64, device="cuda")
        for t in range(t, t + n):
            a = torch.exp(g[t])
            S = S * a[:, None, None]
            u = beta[t][:, None] * (v[t] - (S @ k[t][..., None])[..., 0])
            S = S + u[..., None] * k[t][:, None]
            o[t] = scale * (S @ q[t][..., None])[..., 0]
            size = S.norm(dim=-1)
            E = a[:, None] * E + c * (size + v[t].abs())
            o_off[t] = abs(scale) * q[t].norm(dim=-1)[:, None] * (E + c * size)
        t = t + 1 if n else t
        finals.append(S)
        offs.append(E)
    return o, torch.stack(finals), o_off, torch.stack(offs)


def _norm(x, y):
    d, n = (x.double() - y).norm().item(), y.norm().item()
    return d / n if n else d


def _check(o, state, args, lens, init=None, scale=1.0, chunks=None):
    q = args[0]
    chunks = q.dtype == BF16 if chunks is None else chunks
    c = 2.0 ** -15 if chunks else (q.shape[2] + 16) * 2.0 ** -24
    oe, se, oo, so = _rule(*args, lens, init, scale, c)
    if o.numel():
        bound = oo + (2.0 ** -8 * oe.abs() if o.dtype == BF16 else 0)
        assert ((o.double() - oe).abs() <= bound + 1e-30).all()
        assert _norm(o, oe) <= (2.2e-3 if o.dtype == BF16 else 2e-6)
    assert ((state.double() - se).norm(dim=-1) <= so + 1e-30).all()
    assert _norm(state, se) <= (1e-5 if chunks else 2e-6)


LENS = [[1], [63, 64, 65], [5, 0, 300, 1, 64], [700], [0, 0], [129, 2, 2, 191]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
def test_prompts_match_the_rule(lens, io):
    args = _inputs(len(lens), sum(lens), 8, 4, 128, 128, io)
    init = torch.randn(len(lens), 8, 128, 128, device="cuda", generator=_gen(1)) * 0.3
    for start in (None, init):
        o, fin = _ers().gdn_fwd(*args, _cu(lens), init_state=start, max_seqlen=max(lens))
        _check(o, fin, args, lens, start)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("H,G", [(1, 1), (6, 3), (8, 1)])
@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
def test_shapes(dk, dv, H, G, io):
    lens = [150, 33]
    args = _inputs(dk + dv + H, 183, H, G, dk, dv, io)
    init = torch.randn(2, H, dv, dk, device="cuda", generator=_gen(2)) * 0.3
    o, fin = _ers().gdn_fwd(*args, _cu(lens), init_state=init, scale=dk ** -0.5)
    _check(o, fin, args, lens, init, dk ** -0.5)


@pytest.mark.parametrize("strong", [0.0, 30.0, 3000.0])
@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
def test_gates_from_none_to_all(strong, io):
    """Nothing forgotten; nearly everything; and gates whose running sum would leave fp32 little of a difference."""
    args = list(_inputs(5, 333, 4, 2, 128, 128, io, strong))
    args[3][100] = -1e5                              # one token forgets everything
    args[3][200:210] = -float("inf")
    o, fin = _ers().gdn_fwd(*args, scale=0.3)
    _check(o, fin, args, [333], None, 0.3)


@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
def test_keys_that_repeat(io):
    """The same key over and over at beta 1: every token replaces what the last one wrote (an inverse of full size)."""
    args = list(_inputs(6, 200, 4, 2, 128, 128, io))
    args[1][:] = args[1][:1]
    args[4][:] = 1.0
    o, fin = _ers().gdn_fwd(*args)
    _check(o, fin, args, [200])


def test_long_memory():
    args = list(_inputs(7, 5000, 2, 1, 128, 128, BF16, 0.001))
    o, fin = _ers().gdn_fwd(*args)
    _check(o, fin, args, [5000])


@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
def test_a_state_in_place_and_parts_of_a_prompt(io):
    ers = _ers()
    args = _inputs(8, 200, 4, 4, 128, 128, io)
    state = torch.randn(1, 4, 128, 128, device="cuda", generator=_gen(3)) * 0.3
    init = state.clone()
    outs = []
    for a, b in ((0, 70), (70, 71), (71, 200)):
        part = [x[a:b].contiguous() for x in args]
        o = torch.empty_like(part[2])
        ers.gdn_fwd(*part, init_state=state, out=(o, state))
        outs.append(o)
    _check(torch.cat(outs), state, args, [200], init)


@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("dk,dv,S,H", [(128, 128, 3, 8), (64, 128, 1, 2), (128, 64, 90, 8), (128, 128, 80, 8), (64, 64, 77, 8)])
def test_decode_matches_the_rule(io, dk, dv, S, H):
    """Single tokens, of few heads and of enough to fill the GPU, states read from other pages than they go to."""
    ers = _ers()
    cache = ers.LinAttnCache(S, H, H // 2, dk, dv, npages=2 * S + 1, io_dtype=io)
    cache.state.copy_(torch.randn(cache.state.shape, device="cuda", generator=_gen(4)) * 0.3)
    order = torch.randperm(2 * S + 1, device="cuda", generator=_gen(5)).to(torch.int32)
    cache.pages.table.copy_(order[:S].view(S, 1))
    read = order[S:2 * S].clone()
    read[0] = -1                                     # zeros
    before = cache.state.clone()
    init = before[read.long()]
    init[0] = 0
    args = _inputs(9, S, H, H // 2, dk, dv, io)
    o = ers.gdn_decode(cache, *args, read_page=read, scale=0.5)
    _check(o, cache.state[order[:S].long()], args, [1] * S, init, 0.5, chunks=False)
    rest = order[S:].long()
    assert torch.equal(cache.state[rest], before[rest])


@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
def test_prompts_on_the_cache_and_tokens_after_them(io):
    ers = _ers()
    lens = [130, 7, 0]
    cache = ers.LinAttnCache(5, 4, 2, npages=7, io_dtype=io)
    slot = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    ers.pages_own(cache.pages, slot)
    args = _inputs(10, 140, 4, 2, 128, 128, io)
    prompt = [x[:137].contiguous() for x in args]
    o = ers.gdn_prefill(cache, *prompt, _cu(lens), slot=slot)
    alone, fin = ers.gdn_fwd(*prompt, _cu(lens))
    assert torch.equal(o, alone) and torch.equal(cache.state[cache.pages.table[slot.long(), 0].long()], fin)
    token = [x[137:140].contiguous() for x in args]
    o2 = ers.gdn_decode(cache, *token, slot=slot)
    seq = [torch.cat([x[:130], x[137:138], x[130:137], x[138:]]) for x in args]   # each prompt and its token
    _check(torch.cat([o[:130], o2[:1], o[130:], o2[1:]]), cache.state[cache.pages.table[slot.long(), 0].long()], seq, [131, 8, 1],
           chunks=io == BF16)


def test_it_starts_a_speculative_cache():
    """A prompt's final state as the anchor of a GdnCache: the drafts' outputs are the rule's from there (bf16 read copy)."""
    ers = _ers()
    args = _inputs(11, 104, 4, 2, 128, 128, BF16)
    prompt, drafts = [x[:100].contiguous() for x in args], [x[100:].contiguous() for x in args]
    _, fin = ers.gdn_fwd(*prompt)
    gc = ers.GdnCache(1, 4, 2)
    gc.anchor.copy_(fin)
    gc.read_copy.copy_(fin)
    o = ers.gdn_verify(gc, *[x.view(1, 4, *x.shape[1:]) for x in drafts])
    want, state, _, _ = _rule(*args, [104])
    # a read copy rounded by 2^-8 an element, at most, and two roundings of outputs (residuals read the copy too)
    assert _norm(o[0], want[100:]) <= 8e-3
    ers.gdn_commit(gc, torch.full((1,), 4, dtype=torch.int32, device="cuda"), 4)
    ers.gdn_refresh(gc, 16)
    assert _norm(gc.anchor, state) <= 1e-5


@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
def test_what_is_not_finite_stays_behind(io):
    """Nothing before a bad token changes, no other sequence and no other head does."""
    ers = _ers()
    lens = [150, 60]
    args = list(_inputs(12, 210, 4, 2, 128, 128, io))
    good, state = ers.gdn_fwd(*args, _cu(lens))
    for which, place in ((2, (70, 1, 3)), (1, (70, 0, 5)), (0, (70, 0, 5)), (4, (70, 1)), (3, (70, 1))):
        bad = [x.clone() for x in args]
        bad[which][place] = float("nan")
        if which == 2:
            bad[2][170, 3, 1] = float("inf")
        o, fin = ers.gdn_fwd(*bad, _cu(lens))
        assert torch.equal(o[:70], good[:70]) and not torch.isfinite(o[70, 1]).all()
        assert torch.equal(o[:150, 2:], good[:150, 2:]) and torch.equal(fin[0, 2:], state[0, 2:])
        if which == 2:
            assert torch.equal(o[150:170], good[150:170]) and torch.equal(fin[1, :3], state[1, :3])
            assert not torch.isfinite(o[170, 3, 1]) and not torch.isfinite(fin[1, 3, 1]).all()
        else:
            assert torch.equal(o[150:], good[150:]) and torch.equal(fin[1], state[1])


@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
def test_errors_are_reported_and_touch_nothing(io):
    ers = _ers()
    args = _inputs(13, 100, 2, 1, 128, 128, io)
    cu = torch.tensor([0, 40, 30, 100], dtype=torch.int32, device="cuda")
    o, fin = torch.full_like(args[2], 7.0), torch.full((3, 2, 128, 128), 7.0, device="cuda")
    with pytest.raises(ers.ErsError, match="ERS_EINVAL"):
        ers.gdn_fwd(*args, cu, out=(o, fin), max_seqlen=100)
    assert (fin[1] == 7.0).all()
    cache = ers.LinAttnCache(3, 2, 1, io_dtype=io)
    for slot in ([0, 5], [0, -1]):
        cache.state.fill_(1.0)
        token = [x[:2].contiguous() for x in args]
        o = torch.full_like(token[2], 7.0)
        with pytest.raises(ers.ErsError, match="ERS_ESLOT"):
            ers.gdn_decode(cache, *token, slot=torch.tensor(slot, dtype=torch.int32, device="cuda"), out=o)
        assert (o[1] == 7.0).all() and (cache.state[1:] == 1.0).all() and not (cache.state[0] == 1.0).all()
        with pytest.raises(ers.ErsError, match="ERS_ESLOT"):
            ers.gdn_prefill(cache, *token, _cu([1, 1]), slot=torch.tensor(slot, dtype=torch.int32, device="cuda"), out=o)
        assert (o[1] == 7.0).all() and (cache.state[1:] == 1.0).all()


def test_arguments():
    ers = _ers()
    args = list(_inputs(14, 10, 2, 1, 128, 128, BF16))
    for n, bad, err in ((0, args[0].float(), TypeError), (1, args[1][:9], ValueError), (2, args[2][:, :1], ValueError),
                        (3, args[3].double(), TypeError), (4, args[4][:, :1], ValueError), (4, args[4].cpu(), ValueError)):
        with pytest.raises((err, ers.ErsError)):
            ers.gdn_fwd(*[bad if m == n else x for m, x in enumerate(args)])


@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
def test_captured_and_on_other_streams(io):
    """Two captured prompts and a decode step, replayed, with calls on another stream in between."""
    ers = _ers()
    sets = [_inputs(s, 300, 4, 2, 128, 128, io) for s in (15, 16)]
    want = [ers.gdn_fwd(*x) for x in sets]
    cache = ers.LinAttnCache(300, 4, 2, io_dtype=io)
    graphs, outs = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for x in sets:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs.append((ers.gdn_fwd(*x, check=False), ers.gdn_decode(cache, *x, check=False)))
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
        with torch.cuda.stream(side):
            other = ers.gdn_fwd(*sets[1], check=False, stream=side)
    torch.cuda.synchronize()
    for (prompt, _), w in zip(outs, want):
        assert torch.equal(prompt[0], w[0]) and torch.equal(prompt[1], w[1])
    assert torch.equal(other[0], want[1][0]) and torch.equal(other[1], want[1][1])
    six = [torch.cat([y for _ in range(3) for y in (a, b)]).view(6, 300, *a.shape[1:]).transpose(0, 1).reshape(1800, *a.shape[1:])
           for a, b in zip(*sets)]
    _, states, _, off = _rule(*six, [6] * 300, c=(128 + 16) * 2.0 ** -24)
    assert ((cache.state.double() - states).norm(dim=-1) <= off).all()


@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
def test_states_beyond_32_bits(io):
    """A pool of 2.2e9 floats: its last pages are read and written, by prompts and by tokens."""
    ers = _ers()
    H, npages = 32, 4200
    cache = ers.LinAttnCache(2, H, 16, npages=npages, io_dtype=io, state=torch.empty(npages, H, 128, 128, device="cuda"))
    cache.pages.table.copy_(torch.tensor([[npages - 1], [5]], dtype=torch.int32))
    read = torch.tensor([-1, npages - 2], dtype=torch.int32, device="cuda")
    cache.state[npages - 2] = torch.randn(H, 128, 128, device="cuda", generator=_gen(17)) * 0.3
    init = torch.stack([torch.zeros_like(cache.state[0]), cache.state[npages - 2]])
    args = _inputs(18, 72, H, 16, 128, 128, io)
    prompt, token = [x[:70].contiguous() for x in args], [x[70:].contiguous() for x in args]
    lens = [40, 30]
    o = ers.gdn_prefill(cache, *prompt, _cu(lens), read_page=read)
    o2 = ers.gdn_decode(cache, *token)
    seq = [torch.cat([x[:40], x[70:71], x[40:70], x[71:]]) for x in args]
    _check(torch.cat([o[:40], o2[:1], o[40:], o2[1:]]), cache.state[[npages - 1, 5]], seq, [41, 31], init, chunks=io == BF16)


def test_more_sequences_than_tokens():
    """Empty sequences around a few tokens, by chunks and by the recurrence."""
    for n in (3, 40):
        lens = [0] * 50 + [n] + [0] * 50 + [1, 0]
        args = _inputs(19, n + 1, 4, 2, 64, 64, BF16)
        init = torch.randn(len(lens), 4, 64, 64, device="cuda", generator=_gen(20))
        o, fin = _ers().gdn_fwd(*args, _cu(lens), init_state=init, max_seqlen=n)
        _check(o, fin, args, lens, init)
        still = [i for i, m in enumerate(lens) if m == 0]
        assert torch.equal(fin[still], init[still])


@pytest.mark.parametrize("hint", [1, 10 ** 9])
def test_max_seqlen_never_changes_what_is_computed(hint):
    lens = [100, 3, 64]
    args = _inputs(21, 167, 4, 2, 128, 128, BF16)
    o, fin = _ers().gdn_fwd(*args, _cu(lens), max_seqlen=hint)
    _check(o, fin, args, lens)
