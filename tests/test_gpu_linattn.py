"""Linear attention with a decay per head on the GPU, against the token-by-token recurrence in 64 bits.

Bounds.  With A the same recurrence over absolute values (A_o = |scale| |S| |q|, A_S = the state's), every
kernel computes sums of at most T + dk + dv terms in fp32 from operands that are exact or carry at least 16
significant bits (the scores and the state inside a chunk), so an output is within (2^-15 + (T + 256) 2^-23) A_o and a
state, whose operands carry 24 bits, within (T + 256) 2^-22 A_S, before the output's one rounding to bf16
(2^-8 of its value).  Rounding errors that do not conspire are far smaller: in the 2-norm fp32 results stay within 2e-6,
bf16 outputs within 2.2e-3 (their own rounding is 1.7e-3)."""
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


def _inputs(seed, T, H, G, dk, dv, io):
    g = _gen(seed)
    r = dict(device="cuda", generator=g)
    q = (torch.randn(T, G, dk, **r) * dk ** -0.5).to(io)
    k = (torch.randn(T, G, dk, **r) * dk ** -0.5).to(io)
    v = torch.randn(T, H, dv, **r).to(io)
    decay = -torch.exp2(-8.0 * torch.arange(1, H + 1, dtype=F32, device="cuda") / H)
    return q, k, v, decay


def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def _recurrence(q, k, v, decay, lens, init=None, scale=1.0, absolute=False):
    """o and final states in 64 bits, token by token."""
    H, G = v.shape[1], q.shape[1]
    group = torch.arange(H, device="cuda") // (H // G)
    f = (lambda x: x.double().abs()) if absolute else (lambda x: x.double())
    q, k, v = f(q)[:, group], f(k)[:, group], f(v)
    lam = torch.exp(decay.double())[:, None, None]
    o = torch.zeros(v.shape, dtype=torch.float64, device="cuda")
    out, t = [], 0
    for i, n in enumerate(lens):
        S = f(init[i]) if init is not None else torch.zeros(H, v.shape[2], q.shape[2], dtype=torch.float64, device="cuda")
        for t in range(t, t + n):
            S = lam * S + v[t][:, :, None] * k[t][:, None, :]
            o[t] = abs(scale) * (S @ q[t][..., None])[..., 0] if absolute else scale * (S @ q[t][..., None])[..., 0]
        t = t + 1 if n else t
        out.append(S)
    return o, torch.stack(out)


def _norm(x, y):
    d, n = (x.double() - y).norm().item(), y.norm().item()
    return d / n if n else d


def _check(o, state, q, k, v, decay, lens, init=None, scale=1.0):
    oe, se = _recurrence(q, k, v, decay, lens, init, scale)
    oa, sa = _recurrence(q, k, v, decay, lens, init, scale, absolute=True)
    T = max(list(lens) + [1])
    if o.numel():
        bound = (2.0 ** -15 + (T + 256) * 2.0 ** -23) * oa
        if o.dtype == BF16:
            bound = bound + 2.0 ** -8 * oe.abs()
        assert ((o.double() - oe).abs() <= bound + 1e-30).all()
        assert _norm(o, oe) <= (2.2e-3 if o.dtype == BF16 else 2e-6)
    assert ((state.double() - se).abs() <= (T + 256) * 2.0 ** -22 * sa + 1e-30).all()
    assert _norm(state, se) <= 2e-6


LENS = [[1], [127, 128, 129], [5, 0, 300, 1, 64], [700], [0, 0]]


@pytest.mark.parametrize("lens", LENS, ids=str)
@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
def test_prompts_match_the_recurrence(lens, io):
    q, k, v, decay = _inputs(len(lens), sum(lens), 8, 4, 128, 128, io)
    init = torch.randn(len(lens), 8, 128, 128, device="cuda", generator=_gen(1)) * 0.3
    for start in (None, init):
        o, fin = _ers().linattn_fwd(q, k, v, decay, _cu(lens), init_state=start, max_seqlen=max(lens))
        _check(o, fin, q, k, v, decay, lens, start)


@pytest.mark.parametrize("H,G", [(1, 1), (4, 4), (6, 2), (3, 1)])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
def test_prompts_head_layouts(H, G, dk, dv, io):
    lens = [130, 1, 77]
    q, k, v, decay = _inputs(H + dk, sum(lens), H, G, dk, dv, io)
    init = torch.randn(3, H, dv, dk, device="cuda", generator=_gen(2)) * 0.3
    o, fin = _ers().linattn_fwd(q, k, v, decay, _cu(lens), init_state=init, scale=0.7)
    _check(o, fin, q, k, v, decay, lens, init, scale=0.7)


@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
def test_extreme_decays(io):
    """No decay at all, hardly any, one that underflows within a chunk, and one that forgets everything."""
    lens = [300, 140]
    q, k, v, _ = _inputs(3, sum(lens), 6, 6, 128, 128, io)
    decay = torch.tensor([0.0, -1e-6, -0.5, -30.0, -200.0, -float("inf")], device="cuda")
    init = torch.randn(2, 6, 128, 128, device="cuda", generator=_gen(3))
    o, fin = _ers().linattn_fwd(q, k, v, decay, _cu(lens), init_state=init)
    _check(o, fin, q, k, v, decay, lens, init)


@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("power", [-105, -66, -40, 40, 66, 105])
def test_extreme_scales(io, power):
    """Outputs that are in range are right although scale times a factor of the sums' level is not."""
    scale = 2.0 ** power
    lens = [40, 200, 300]
    for n in lens:                                      # a tile, a chunk and two, by the recurrence and by chunks
        q, k, v, _ = _inputs(3, n, 5, 5, 128, 128, io)
        decay = torch.tensor([-1.0, -0.98, -0.6, -0.1, -5.0], device="cuda")
        init = torch.randn(1, 5, 128, 128, device="cuda", generator=_gen(3))
        o, fin = _ers().linattn_fwd(q, k, v, decay, init_state=init, scale=scale)
        _check(o * 2.0 ** -power, fin, q, k, v, decay, [n], init)


@pytest.mark.parametrize("sign", ["any", "positive"])
def test_states_that_forget_little(sign):
    """A prompt's state is added up by 24 truncated sums in 128 tokens, each off by at most 2^-23 of the sum so far."""
    T = 8192
    q, k, v, _ = _inputs(21, T, 4, 1, 128, 128, BF16)
    if sign == "positive":
        k, v = k.abs(), v.abs()
    decay = torch.tensor([0.0, -1e-5, -1e-4, -1e-3], device="cuda")
    o, fin = _ers().linattn_fwd(q, k, v, decay)
    oe, se = _recurrence(q, k, v, decay, [T])
    for h in range(4):
        assert _norm(fin[0, h], se[0, h]) <= T * 24 / 128 * 2.0 ** -23 + 2e-6
    assert _norm(o, oe) <= 2.2e-3


@pytest.mark.parametrize("power", [-20, -30, -40])
def test_small_values(power):
    """States of 1e-6 to 1e-12.  With E = exp(64 |a|), operands (scores, states) of bf16 prompts are off by 2^-134 E besides their
    16 bits, and sums of up to 512 products by 2^-149 E each: an output by that times the sums of |q| and, over its chunk, of |v|."""
    T = 300
    q, k, v, _ = _inputs(3, T, 5, 5, 128, 128, BF16)
    v = v * 2.0 ** power
    decay = torch.tensor([-1.0, -0.9, -0.5, -0.1, -5.0], device="cuda")
    init = torch.randn(1, 5, 128, 128, device="cuda", generator=_gen(3)) * 2.0 ** power
    o, fin = _ers().linattn_fwd(q, k, v, decay, init_state=init)
    oe, se = _recurrence(q, k, v, decay, [T], init)
    oa, sa = _recurrence(q, k, v, decay, [T], init, absolute=True)
    E = torch.exp(torch.where(decay.abs() <= 1, 64 * decay.abs(), torch.zeros_like(decay)).double())[None, :, None]
    values = torch.stack([v.double().abs()[c:c + 128].sum(0) for c in range(0, T, 128)]).repeat_interleave(128, 0)[:T]
    small = E * (2.0 ** -134 * (q.double().abs().sum(-1, keepdim=True) + values) + 512 * 2.0 ** -149)
    assert ((o.double() - oe).abs() <= (2.0 ** -15 + (T + 256) * 2.0 ** -23) * oa + 2.0 ** -8 * oe.abs() + small).all()
    assert ((fin.double() - se).abs() <= (T + 256) * 2.0 ** -22 * sa + 1e-30).all()


@pytest.mark.parametrize("lens,H", [([2500], 1), ([1500, 1], 8), ([900, 1100, 700], 40), ([130] * 30, 8)],
                         ids=["split8", "split", "few", "none"])
def test_long_prompts_whatever_the_split(lens, H):
    """Work split over a sequence or not, the sum is the same."""
    q, k, v, decay = _inputs(5, sum(lens), H, 1, 128, 128, BF16)
    init = torch.randn(len(lens), H, 128, 128, device="cuda", generator=_gen(4)) * 0.3
    o, fin = _ers().linattn_fwd(q, k, v, decay, _cu(lens), init_state=init, max_seqlen=max(lens))
    _check(o, fin, q, k, v, decay, lens, init)
    again, fin2 = _ers().linattn_fwd(q, k, v, decay, _cu(lens), init_state=init, max_seqlen=max(lens))
    assert torch.equal(o, again) and torch.equal(fin, fin2)
    # a caller's wrong guess of the longest sequence changes the order of sums only
    o, fin = _ers().linattn_fwd(q, k, v, decay, _cu(lens), init_state=init, max_seqlen=1)
    _check(o, fin, q, k, v, decay, lens, init)


@pytest.mark.parametrize("lens,H", [([2048] * 4, 32), ([700, 300, 900], 8), ([1] * 30 + [400, 200], 16)], ids=["even", "few", "short"])
def test_the_default_call_is_planned_by_its_lengths(lens, H):
    """Without max_seqlen a call of several sequences gives the bits, and so takes the split, of one with the right length."""
    ers = _ers()
    q, k, v, decay = _inputs(H, sum(lens), H, 4, 128, 128, BF16)
    cu = _cu(lens)
    o, fin = ers.linattn_fwd(q, k, v, decay, cu, max_seqlen=max(lens))
    p, fin2 = ers.linattn_fwd(q, k, v, decay, cu)
    assert torch.equal(o, p) and torch.equal(fin, fin2)
    cache = ers.LinAttnCache(len(lens), H, 4)
    p = ers.linattn_prefill(cache, q, k, v, decay, cu)
    assert torch.equal(o, p) and torch.equal(fin, cache.state)


@pytest.mark.parametrize("lens,H", [([129, 1, 0], 2), ([256], 3), ([385, 640], 20), ([512], 8), ([1025, 3, 0, 128], 16),
                                    ([1100] + [1] * 12, 8), ([897], 36)], ids=str)
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_runs_of_few_chunks(lens, H, dk, dv):
    """Sequences cut into runs of one chunk or two, some CTAs of a sequence without any."""
    q, k, v, decay = _inputs(H, sum(lens), H, 1, dk, dv, BF16)
    init = torch.randn(len(lens), H, dv, dk, device="cuda", generator=_gen(2)) * 0.3
    for most in (max(lens), max(lens) + 700):
        o, fin = _ers().linattn_fwd(q, k, v, decay, _cu(lens), init_state=init, max_seqlen=most)
        _check(o, fin, q, k, v, decay, lens, init)


@pytest.mark.parametrize("lens,H,most", [([2048], 160, 2048), ([1000, 2200], 24, 3200), ([1500] * 12, 16, 1500)], ids=str)
def test_many_chunks_through_one_staging_buffer(lens, H, most):
    """dk 64, dv 128: outputs do not fit a K tile, so every chunk of a CTA is staged in the same buffer and must wait for the
    last one's store.  Whole sequences and runs of many chunks, next to traffic that holds stores up; bits stay over repeats."""
    q, k, v, decay = _inputs(H, sum(lens), H, 1, 64, 128, BF16)
    init = torch.randn(len(lens), H, 128, 64, device="cuda", generator=_gen(6)) * 0.3
    cu = _cu(lens)
    o, fin = _ers().linattn_fwd(q, k, v, decay, cu, init_state=init, max_seqlen=most)
    _check(o, fin, q, k, v, decay, lens, init)
    busy, side = torch.empty(1 << 29, dtype=torch.uint8, device="cuda"), torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(side):
            busy.add_(1)
        again, fin2 = _ers().linattn_fwd(q, k, v, decay, cu, init_state=init, max_seqlen=most, check=False)
        assert torch.equal(o, again) and torch.equal(fin, fin2)
    torch.cuda.synchronize()


@pytest.mark.parametrize("lens,H", [([56], 8), ([31, 57], 4), ([57], 8), ([32, 0, 25], 20), ([33, 1], 20)], ids=str)
@pytest.mark.parametrize("decays", ["graded", "strong"])
def test_few_tokens_by_either_form(lens, H, decays):
    q, k, v, decay = _inputs(H, sum(lens), H, 2, 128, 128, BF16)
    if decays == "strong":   # either side of -1, where the state is no longer held at a common level
        decay = torch.linspace(-0.9, -3.0, H, device="cuda")
    init = torch.randn(len(lens), H, 128, 128, device="cuda", generator=_gen(4)) * 0.3
    o, fin = _ers().linattn_fwd(q, k, v, decay, _cu(lens), init_state=init, max_seqlen=max(lens))
    _check(o, fin, q, k, v, decay, lens, init)


@pytest.mark.parametrize("lens,H", [([95], 3), ([64, 1, 33], 16), ([200], 40), ([45, 0] + [40] * 40, 16)], ids=["few", "odd", "heads", "many"])
def test_fp32_tiles_at_every_decay(lens, H):
    q, k, v, decay = _inputs(H, sum(lens), H, 1, 64, 128, F32)
    decay = -torch.logspace(-4, 0.5, H, device="cuda")
    init = torch.randn(len(lens), H, 128, 64, device="cuda", generator=_gen(5)) * 0.3
    o, fin = _ers().linattn_fwd(q, k, v, decay, _cu(lens), init_state=init, max_seqlen=max(lens))
    _check(o, fin, q, k, v, decay, lens, init)


@pytest.mark.parametrize("lens,H", [([1] * 20 + [200] + [0, 3, 8, 9, 1], 16), ([300] + [1] * 70, 5), ([0] * 40 + [25], 8)],
                         ids=["among", "first", "last"])
@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 128)])
def test_a_prompt_among_single_tokens(lens, H, dk, dv):
    q, k, v, decay = _inputs(H, sum(lens), H, 1, dk, dv, BF16)
    init = torch.randn(len(lens), H, dv, dk, device="cuda", generator=_gen(3)) * 0.3
    for most in (max(lens), max(lens) + 700):
        o, fin = _ers().linattn_fwd(q, k, v, decay, _cu(lens), init_state=init, max_seqlen=most)
        _check(o, fin, q, k, v, decay, lens, init)


@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
def test_neighbours_do_not_leak(io):
    """A sequence of NaN and infinities between two others touches neither, nor their final states."""
    lens = [100, 40, 90]
    q, k, v, decay = _inputs(6, sum(lens), 4, 2, 128, 128, io)
    for x, bad in ((q, float("nan")), (k, float("inf")), (v, float("nan"))):
        x[100:140] = bad
    o, fin = _ers().linattn_fwd(q, k, v, decay, _cu(lens))
    keep = list(range(100)) + list(range(140, 230))
    o2, fin2 = o[keep].contiguous(), fin[[0, 2]].contiguous()
    _check(o2, fin2, q[keep], k[keep], v[keep], decay, [100, 90])


@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
def test_future_tokens_do_not_leak(io):
    """Causality holds for values that are not finite: tokens before a NaN or infinite value keep their outputs."""
    lens = [200]
    q, k, v, decay = _inputs(16, 200, 4, 4, 128, 128, io)
    o, _ = _ers().linattn_fwd(q, k, v, decay, _cu(lens))
    w = v.clone()
    w[150, 1] = float("nan")
    w[60, 2, 5] = float("inf")
    w[61, 2, 5] = -float("inf")
    p, _ = _ers().linattn_fwd(q, k, w, decay, _cu(lens))
    assert torch.equal(p[:, [0, 3]], o[:, [0, 3]])
    assert torch.isfinite(p[:150, 1]).all() and torch.isnan(p[150:, 1]).all()
    others = [d for d in range(128) if d != 5]
    assert torch.isfinite(p[:60, 2]).all() and torch.isfinite(p[:, 2][:, others]).all()
    assert not torch.isfinite(p[60:, 2, 5]).any() and torch.isnan(p[61:, 2, 5]).all()
    assert _norm(p[:150, 1], o[:150, 1].double()) <= 1e-2 and _norm(p[:, 2][:, others], o[:, 2][:, others].double()) <= 1e-2


def test_prefill_and_decode_through_the_cache():
    """Prompts written into scattered pages, resumed, decoded token by token; other pages keep their bytes."""
    ers = _ers()
    H, G, n = 8, 4, 3
    lens, more = [150, 1, 40], [30, 200, 0]
    cache = ers.LinAttnCache(5, H, G, npages=9)
    slots = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    cache.state.copy_(torch.randn(cache.state.shape, device="cuda", generator=_gen(7)))
    cache.pages.table.copy_(torch.tensor([[7], [1], [0], [5], [3]], dtype=torch.int32))
    before = cache.state.clone()
    q, k, v, decay = _inputs(8, sum(lens), H, G, 128, 128, BF16)
    q2, k2, v2, _ = _inputs(9, sum(more), H, G, 128, 128, BF16)
    fresh = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    o = ers.linattn_prefill(cache, q, k, v, decay, _cu(lens), slots, read_page=fresh)
    pages = [3, 7, 0]
    _check(o, cache.state[pages], q, k, v, decay, lens)
    mid = cache.state[pages].clone()
    o = ers.linattn_prefill(cache, q2, k2, v2, decay, _cu(more), slots)
    _check(o, cache.state[pages], q2, k2, v2, decay, more, mid)
    for step in range(3):
        mid = cache.state[pages].clone()
        qd, kd, vd, _ = _inputs(20 + step, n, H, G, 128, 128, BF16)
        o = ers.linattn_decode(cache, qd, kd, vd, decay, slots, scale=0.5)
        _check(o, cache.state[pages], qd, kd, vd, decay, [1] * n, mid, scale=0.5)
    rest = [1, 2, 4, 5, 6, 8]
    assert torch.equal(cache.state[rest], before[rest])


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
def test_prompts_on_the_cache_have_the_bits_of_prompts_alone(dk, dv, io):
    """Every shape and type, from other slots' pages, zeros or the slot's own, into scattered pages."""
    ers = _ers()
    H, G, lens = 6, 2, [150, 0, 40, 1]
    cache = ers.LinAttnCache(6, H, G, dk, dv, npages=9, io_dtype=io)
    cache.state.copy_(torch.randn(cache.state.shape, device="cuda", generator=_gen(7)))
    cache.pages.table.copy_(torch.tensor([[7], [1], [0], [5], [3], [8]], dtype=torch.int32))
    slots = torch.tensor([4, 0, 2, 5], dtype=torch.int32, device="cuda")       # pages 3, 7, 0 and 8
    q, k, v, decay = _inputs(dk + dv, sum(lens), H, G, dk, dv, io)
    for read in ([5, 6, -1, 8], None):
        before = cache.state.clone()
        init = torch.stack([before[p] if p >= 0 else torch.zeros_like(before[0]) for p in (read or [3, 7, 0, 8])])
        o = ers.linattn_prefill(cache, q, k, v, decay, _cu(lens), slots, max_seqlen=150,
                                read_page=None if read is None else torch.tensor(read, dtype=torch.int32, device="cuda"))
        want, fin = ers.linattn_fwd(q, k, v, decay, _cu(lens), init_state=init, max_seqlen=150)
        assert torch.equal(o, want) and torch.equal(cache.state[[3, 7, 0, 8]], fin)
        assert torch.equal(cache.state[[1, 2, 4, 5, 6]], before[[1, 2, 4, 5, 6]])
        _check(o, fin, q, k, v, decay, lens, init)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("B,H", [(1, 2), (7, 6), (200, 4)])
def test_decode_matches_the_recurrence(B, H, dk, dv, io):
    ers = _ers()
    cache = ers.LinAttnCache(B, H, 2, dk, dv, io_dtype=io)
    cache.state.copy_(torch.randn(cache.state.shape, device="cuda", generator=_gen(11)))
    init = cache.state.clone()
    q, k, v, decay = _inputs(12, B, H, 2, dk, dv, io)
    o = ers.linattn_decode(cache, q, k, v, decay)
    _check(o, cache.state, q, k, v, decay, [1] * B, init)


def test_fork_then_decode_reads_the_parents_page():
    """After a fork, one decode step takes the children from the shared page into their own; the parent's stays."""
    ers = _ers()
    H = 4
    cache = ers.LinAttnCache(4, H, H, npages=6)
    one = torch.tensor([1], dtype=torch.int32, device="cuda")
    kids = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    ers.pages_own(cache.pages, one)
    q, k, v, decay = _inputs(13, 50, H, H, 128, 128, BF16)
    ers.linattn_prefill(cache, q, k, v, decay, slot=one)
    parent = cache.state[cache.pages.table[1, 0]].clone()
    ers.pages_fork(cache.pages, one.repeat(2), kids)
    read = ers.pages_own(cache.pages, kids, copy=False)
    qd, kd, vd, _ = _inputs(14, 2, H, H, 128, 128, BF16)
    o = ers.linattn_decode(cache, qd, kd, vd, decay, kids, read_page=read)
    got = cache.state[cache.pages.table[kids.long(), 0].long()]
    _check(o, got, qd, kd, vd, decay, [1, 1], torch.stack([parent, parent]))
    assert torch.equal(cache.state[cache.pages.table[1, 0]], parent)


def test_offsets_past_32_bits():
    ers = _ers()
    npages = 140000                                   # 9.2 GB of states of one head
    state = torch.empty(npages, 1, 128, 128, device="cuda")
    cache = ers.LinAttnCache(2, 1, 1, npages=npages, state=state)
    cache.pages.table.copy_(torch.tensor([[npages - 1], [131072]], dtype=torch.int32))
    state[npages - 1].normal_(generator=_gen(1))
    state[131072].normal_(generator=_gen(2))
    init = state[[npages - 1, 131072]].clone()
    q, k, v, decay = _inputs(15, 2, 1, 1, 128, 128, BF16)
    o = ers.linattn_decode(cache, q, k, v, decay)
    _check(o, state[[npages - 1, 131072]], q, k, v, decay, [1, 1], init)


def test_another_stream():
    ers = _ers()
    lens = [300]
    q, k, v, decay = _inputs(17, 300, 4, 4, 128, 128, BF16)
    ref, fin = ers.linattn_fwd(q, k, v, decay, _cu(lens))
    cu = _cu(lens)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    o, f = ers.linattn_fwd(q, k, v, decay, cu, stream=side)
    side.synchronize()
    assert torch.equal(o, ref) and torch.equal(f, fin)


def test_one_prompt_without_cu_seqlens():
    ers = _ers()
    q, k, v, decay = _inputs(23, 300, 4, 4, 128, 128, BF16)
    for T in (300, 1, 0):
        one = ers.linattn_fwd(q[:T], k[:T], v[:T], decay)
        two = ers.linattn_fwd(q[:T], k[:T], v[:T], decay, _cu([T]))
        assert all(torch.equal(a, b) for a, b in zip(one, two))


def test_a_serving_step_is_captured_with_default_arguments():
    """A prompt, a fork, a token of each branch, their scores, the losers' pages and a compaction as one graph: with
    check=False no call copies from or waits for the device, and the replay has the eager calls' bits."""
    ers = _ers()
    H, V = 4, 5003
    q, k, v, decay = _inputs(24, 500, H, 2, 128, 128, BF16)
    qd, kd, vd, _ = _inputs(25, 3, H, 2, 128, 128, BF16)
    logits = (torch.randn(3, V, device="cuda", generator=_gen(26)) * 3).to(BF16)
    target = torch.tensor([5, 7, 9], dtype=torch.int32, device="cuda")
    root = torch.zeros(1, dtype=torch.int32, device="cuda")
    kids, losers = torch.arange(1, 4, dtype=torch.int32, device="cuda"), torch.tensor([1, 3], dtype=torch.int32, device="cuda")
    parents = root.repeat(3)

    def step(cache):
        ers.pages_own(cache.pages, root, check=False)
        out = [ers.linattn_prefill(cache, q, k, v, decay, slot=root, check=False),
               *ers.linattn_fwd(q, k, v, decay, check=False)]
        ers.pages_fork(cache.pages, parents, kids, check=False)
        read = ers.pages_own(cache.pages, kids, copy=False, check=False)
        out.append(ers.linattn_decode(cache, qd, kd, vd, decay, kids, read_page=read, check=False))
        out += ers.token_logprobs(logits, target, top_k=4, check=False)
        ers.pages_free(cache.pages, losers, check=False)
        return out + list(ers.pages_compact(cache.pages, check=False)) + [cache.state, cache.pages.table, cache.pages.refs]

    want = step(ers.LinAttnCache(4, H, 2, npages=6))
    cache = ers.LinAttnCache(4, H, 2, npages=6)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(cache)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_errors_leave_outputs_unwritten():
    ers = _ers()
    cache = ers.LinAttnCache(3, 2, 2)
    cache.state.fill_(2.0)
    q, k, v, decay = _inputs(18, 2, 2, 2, 128, 128, BF16)
    for table, slot, read, code in (([0, 1, 2], [0, 3], None, 8), ([0, 1, 2], [0, -1], None, 8),
                                    ([0, 3, 2], [0, 1], None, 8), ([0, -1, 2], [0, 1], None, 8),
                                    ([0, 1, 2], [0, 1], [0, 3], 8), ([0, 1, 2], [0, 1], [0, -2], 8)):
        cache.pages.table.copy_(torch.tensor(table, dtype=torch.int32).view(3, 1))
        cache.state.fill_(2.0)
        for decode in (True, False):
            st, out = ers.Status("cuda"), torch.full_like(v, 9.0)
            dev = dict(slot=torch.tensor(slot, dtype=torch.int32, device="cuda"), status=st, check=False, out=out,
                       read_page=None if read is None else torch.tensor(read, dtype=torch.int32, device="cuda"))
            if decode:
                ers.linattn_decode(cache, q, k, v, decay, **dev)
            else:
                ers.linattn_prefill(cache, q, k, v, decay, _cu([1, 1]), **dev)
            assert st.read() == code
            assert (out[1] == 9.0).all() and not (out[0] == 9.0).all()
            assert (cache.state[1:] == 2.0).all()
    for cu in ([0, 3, 2], [-1, 1, 2], [0, 1, 5], [2, 1, 2]):
        st, out = ers.Status("cuda"), (torch.full_like(v, 9.0), torch.full((2, 2, 128, 128), 9.0, device="cuda"))
        ers.linattn_fwd(q, k, v, decay, torch.tensor(cu, dtype=torch.int32, device="cuda"), status=st, check=False,
                        out=out, max_seqlen=2)
        assert st.read() == 1
        bad = [i for i in range(2) if cu[i] < 0 or cu[i + 1] < cu[i] or cu[i + 1] > 2]
        assert (out[1][bad] == 9.0).all()


def test_refusals():
    ers = _ers()
    q, k, v, decay = _inputs(19, 4, 2, 2, 128, 128, BF16)
    with pytest.raises(ers.ErsError):
        ers.linattn_fwd(q[..., :32].contiguous(), k[..., :32].contiguous(), v, decay)
    with pytest.raises(ers.ErsError):
        ers.linattn_fwd(q, k, v, decay, scale=float("inf"))
    with pytest.raises(TypeError):
        ers.linattn_fwd(q.half(), k.half(), v.half(), decay)
    with pytest.raises(TypeError):
        ers.linattn_fwd(q, k.float(), v, decay)
    with pytest.raises(ValueError):
        ers.linattn_fwd(q, k, v.transpose(1, 2), decay)
    with pytest.raises(ValueError):
        ers.linattn_fwd(q, k[:3].contiguous(), v, decay)
    with pytest.raises(ValueError):
        ers.linattn_fwd(q, k, v, decay, init_state=torch.zeros(1, 2, 128, 64, device="cuda"))
    cache = ers.LinAttnCache(3, 2, 2)
    with pytest.raises(ers.ErsError):
        ers.linattn_decode(cache, q, k, v, decay)            # four sequences, three slots
    with pytest.raises(ValueError):
        ers.linattn_decode(cache, q, k, v, decay, slot=torch.zeros(3, dtype=torch.int32, device="cuda"))
