"""Log probabilities of given tokens, entropy and top alternatives on the GPU, against 64 bits and a sort.

Bounds.  d = scale (x - m) carries two roundings (2^-23 of |d|), exp and log a few units, and z is a sum of V
non-negative terms added in pairs and strides (at most V / 256 + 16 terms in a row): log z is within (V / 256 + 32) 2^-23,
and a log probability within that and 2^-22 of its value; the entropy, whose terms weigh d by e^d <= 1, within
(V / 256 + 32) 2^-22 (1 + entropy).  Ids are equal."""
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


def _expected(logits, target, k, scale):
    x = logits.double()
    odd = (torch.isnan(x) | (x == math.inf)).any(1)
    x = torch.where(odd[:, None], torch.zeros_like(x), x)
    top = x.max(1, keepdim=True).values
    empty = (top == -math.inf)[:, 0]
    d = (x - torch.where(top == -math.inf, torch.zeros_like(top), top)) * scale
    z = torch.where(empty, torch.ones_like(top[:, 0]), d.exp().sum(1))
    lp = d - z.log()[:, None]
    lp = torch.where(lp < -torch.finfo(F32).max, torch.full_like(lp, -math.inf), lp)
    entropy = torch.where(empty, torch.zeros_like(z), -torch.where(lp == -math.inf, torch.zeros_like(lp),
                                                                   lp.exp() * lp).sum(1))
    nan = torch.full_like(z, math.nan)
    entropy = torch.where(odd, nan, entropy)
    V = x.shape[1]
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    value = x.gather(1, order)
    gone = (value == -math.inf) | odd[:, None]
    top_id = torch.where(gone, -1, order)
    top_lp = torch.where(gone, torch.full_like(value, -math.inf), lp.gather(1, order))
    top_lp = torch.where(odd[:, None], nan[:, None], top_lp)
    if V < k:
        top_id = torch.cat([top_id, torch.full((x.shape[0], k - V), -1, device="cuda")], 1)
        fill = torch.where(odd, nan, torch.full_like(z, -math.inf))[:, None].expand(-1, k - V)
        top_lp = torch.cat([top_lp, fill], 1)
    out = None
    if target is not None:
        t = target.long()
        out = torch.where(odd, nan, lp.gather(1, t.clamp(min=0)[:, None])[:, 0])
        out = torch.where(t < 0, torch.zeros_like(out), out)
    return out, entropy, top_id, top_lp


def _close(got, want, bound):
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    ok = torch.isfinite(want)
    rest = ~ok & ~torch.isnan(want)
    assert torch.equal(got[rest], want[rest])
    assert ((got - want).abs()[ok] <= bound[ok]).all()


def _check(logits, target, k, scale=1.0):
    lp, entropy, top_id, top_lp = _ers().token_logprobs(logits, target, top_k=k, scale=scale)
    elp, eent, eid, etop = _expected(logits, target, k, scale)
    eps = (logits.shape[1] / 256 + 32) * 2.0 ** -23
    if target is None:
        assert lp is None
    else:
        _close(lp, elp, eps + 2.0 ** -22 * elp.abs())
    _close(entropy, eent, 2 * eps * (1 + eent.abs()))
    assert torch.equal(top_id.long(), eid)
    _close(top_lp, etop, eps + 2.0 ** -22 * etop.abs())


def _target(R, V, seed=0):
    t = torch.randint(0, V, (R,), device="cuda", generator=_gen(seed)).to(torch.int32)
    t[R // 2:: 3] = -1
    return t


@pytest.mark.parametrize("V", [1, 2, 7, 255, 256, 257, 1000, 4099, 50001, 131072, 300007])
@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R,k", [(1, 5), (3, 32), (5, 0), (160, 1)])
def test_matches_64_bits(V, io, R, k):
    x = (torch.randn(R, V, device="cuda", generator=_gen(V + R)) * 3).to(io)
    _check(x, _target(R, V), k, scale=1.0)
    _check(x, None, k, scale=0.6)


@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("offset,pad", [(0, 1), (1, 0), (3, 5), (8, 64), (5, 3)])
def test_rows_anywhere(io, offset, pad):
    """Rows at odd distances and odd starts: views into a padded buffer, poisoned around the rows."""
    R, V = 6, 5003
    buf = torch.full((offset + R * (V + pad),), float("nan"), device="cuda", dtype=io)
    x = buf[offset:].view(R, V + pad)[:, :V]
    x.copy_((torch.randn(R, V, device="cuda", generator=_gen(3)) * 2).to(io))
    _check(x, _target(R, V), 20)


@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [100, 40000])
def test_masks_and_rows_that_are_left_nothing(io, V):
    low = torch.finfo(io).min
    x = (torch.randn(12, V, device="cuda", generator=_gen(5)) * 3).to(io)
    x[0] = -math.inf                                   # nothing
    x[1] = low                                         # the type's lowest value: an even distribution
    x[2, 3:] = -math.inf                               # three alternatives left
    x[3, 1:] = low                                     # one, and the rest at the lowest
    x[4, :-1] = -math.inf                              # one, at the end
    x[5, ::2] = low
    x[5, 1::2] = -math.inf                             # half at the lowest, half masked
    x[6] = 0.0
    x[6, 1::2] = -0.0                                  # all equal: the lowest indices
    x[7] = torch.finfo(io).max                         # even again, at the other end
    x[8, V // 2] = math.nan
    x[9, V - 1] = math.inf
    x[10, V // 3:] = -math.inf
    t = torch.zeros(12, dtype=torch.int32, device="cuda")
    t[4], t[2], t[10] = V - 1, 50, V - 1               # the last two masked
    for scale in (1.0, 1.3):
        _check(x, t, 8, scale)
        _check(x, t, 32, scale)


@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [100, 5003, 131072])
def test_finite_values_of_any_size(io, V):
    """Rows under an additive mask of any usual size, at the front (whole turns of threads see nothing else), at the end and
    scattered; even rows, and rows around a large value, of either sign and any size."""
    g = _gen(V)
    noise = (torch.randn(V, device="cuda", generator=g) * 3).to(io)
    scattered = torch.rand(V, device="cuda", generator=g) < 0.99
    scattered[V // 2] = False
    rows = []
    for size in (1e5, 1e6, 1e9, 2.1e9, 1e10, 1e12, 1e15, 1e20, 1e25, 1e29, 1e30, 1e35):
        for mask in (slice(None, V - 3), slice(3, None), scattered):
            rows.append(noise.clone())
            rows[-1][mask] = -size
            rows.append(noise.clone())
            rows[-1][mask] -= size
        for value in (-size, size):
            rows.append(torch.full_like(noise, value))
            rows.append(torch.full_like(noise, value))
            rows[-1][V // 2] *= 1 + 2.0 ** -7            # one step of a bf16 away
            rows.append((torch.full_like(noise, value).float() * (1 + noise.float() * 1e-7)).to(io))
            rows[-1][1] = -math.inf
    x = torch.stack(rows)
    for R in (len(rows), 5, 1):                          # whole rows, and rows split over a cluster
        for r in range(0, len(rows), R):
            _check(x[r:r + R].contiguous(), _target(len(rows), V)[r:r + R].clone(), 20)


@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("V", [7, 5003, 131072])
@pytest.mark.parametrize("power", [-149, -130, -120, -96, -40, -10, 10, 21, 27, 28, 60, 100, 127])
def test_any_scale(io, V, power):
    """Inverse temperatures (powers of two, exact in fp32) from the least float to the largest."""
    low, high = torch.finfo(io).min, torch.finfo(io).max
    x = (torch.randn(12, V, device="cuda", generator=_gen(power + 200)) * 3).to(io)
    x[1, : V // 2] = -math.inf
    x[2, 1:] = -math.inf
    x[3] = -math.inf
    x[4, ::2] = low
    x[5, ::3] = high
    x[5, 1] = low
    x[6] = 0.0
    x[7] *= 2.0 ** 100
    x[8] *= 2.0 ** -100
    x[8, 0] = -math.inf
    x[9, V // 2] = math.nan
    x[10] = x[10] * 2.0 ** -120
    x[10, 3:] = low
    x[11, ::2] = -1e9
    t = _target(12, V)
    _check(x, t, 7, 2.0 ** power)
    _check(x[:4].contiguous(), t[:4].clone(), 7, 2.0 ** power)


@pytest.mark.parametrize("V", [5000, 131072])
def test_ties_and_orders(V):
    """Few distinct values, ascending and descending rows, and the best alternatives side by side."""
    x = torch.randint(-4, 5, (4, V), device="cuda", generator=_gen(7)).to(BF16)
    up = torch.arange(V, device="cuda", dtype=F32)
    y = torch.stack([up, -up, torch.zeros_like(up), (up % 97)])
    y[2, 1000:1032] = 1.0
    for k in (1, 20, 32):
        _check(x, _target(4, V), k)
        _check(y / V, _target(4, V), k)
        _check((y * 0.01).to(BF16), _target(4, V), k)


def test_offsets_past_32_bits():
    R, V = 20000, 131072
    x = torch.empty(R, V, dtype=BF16, device="cuda")
    rows = [0, 16384, 16385, R - 1]
    for r in range(0, R, 500):
        x[r:r + 500].normal_(generator=_gen(r))
    t = _target(R, V)
    lp, ent, ids, top = _ers().token_logprobs(x, t, top_k=4)
    sub = x[rows].contiguous()
    elp, eent, eid, etop = _expected(sub, t[rows], 4, 1.0)
    eps = (V / 256 + 32) * 2.0 ** -23
    _close(lp[rows], elp, eps + 2.0 ** -22 * elp.abs())
    _close(ent[rows], eent, 2 * eps * (1 + eent))
    assert torch.equal(ids[rows].long(), eid)


def test_repeats_and_other_streams_give_the_same_bits():
    x = (torch.randn(3, 70001, device="cuda", generator=_gen(9)) * 3).to(BF16)
    t = _target(3, 70001)
    one = _ers().token_logprobs(x, t, top_k=7)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    two = _ers().token_logprobs(x, t, top_k=7, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(one, two))


@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("R", [1, 2, 17, 30])
def test_rows_split_over_a_cluster(R, io):
    """Slices of 8 KB, so short that a CTA may be done with its own before another of its row has started: what it hands over
    waits for that.  Beside a kernel that holds part of the SMs, and over and over, the bits stay."""
    V = 8 * 8192 // io.itemsize
    x = (torch.randn(R, V, device="cuda", generator=_gen(R)) * 3).to(io)
    t = _target(R, V)
    _check(x, t, 20)
    one = _ers().token_logprobs(x, t, top_k=20)
    load = torch.randn(2048, 2048, device="cuda", generator=_gen(1)).to(BF16)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(20):
        with torch.cuda.stream(side):
            load @ load
        again = _ers().token_logprobs(x, t, top_k=20, check=False)
        assert all(torch.equal(a, b) for a, b in zip(one, again))


def test_refusals_and_errors():
    ers = _ers()
    x = torch.zeros(4, 64, dtype=BF16, device="cuda")
    t = torch.tensor([0, 64, -2, 5], dtype=torch.int32, device="cuda")
    st = ers.Status("cuda")
    lp, *_ = ers.token_logprobs(x, t, status=st, check=False)
    assert st.read() == 1
    assert torch.isnan(lp[1:3]).all() and torch.isfinite(lp[[0, 3]]).all()
    with pytest.raises(ers.ErsError):
        ers.token_logprobs(x, t)
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(ers.ErsError):
            ers.token_logprobs(x, scale=scale)
    for bad in (dict(top_k=33), dict(top_k=-1)):
        with pytest.raises(ValueError):
            ers.token_logprobs(x, **bad)
    with pytest.raises(ValueError):
        ers.token_logprobs(x.t())
    with pytest.raises(ValueError):
        ers.token_logprobs(x, t[:3])
    with pytest.raises(TypeError):
        ers.token_logprobs(x.half())
    with pytest.raises(TypeError):
        ers.token_logprobs(x, t.long())
    lp, ent, ids, top = ers.token_logprobs(x[:0], t[:0], top_k=3)
    assert lp.shape == (0,) and ids.shape == (0, 3)
