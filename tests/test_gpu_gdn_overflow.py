"""Finite tokens of the gated delta rule whose sums leave fp32: by the recurrence they reach their own outputs and later ones, by
chunks those from the start of their chunk of 64 tokens, of their state row (or, where products of keys overflow, of their head), and
nothing else.  Bounds as in test_gpu_gdn_rule.py."""
import pytest
import torch

from test_gpu_gdn_rule import BF16, F32, _cu, _ers, _gen, _inputs, _rule

pytestmark = pytest.mark.gpu

IO = pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])


def _reached(at, io):
    """The first token that one whose sums overflow may reach."""
    return at // 64 * 64 if io == BF16 else at


def _same_as_the_rule(o, args, init, rows=...):
    n = o.shape[0]
    c = 2.0 ** -15 if o.dtype == BF16 else (args[0].shape[2] + 16) * 2.0 ** -24
    oe, _, oo, _ = _rule(*[x[:n] for x in args], [n], init, 1.0, c)
    bound = oo + (2.0 ** -8 * oe.abs() if o.dtype == BF16 else 0) + 1e-30
    assert ((o.double() - oe).abs() <= bound)[:, rows].all()


@IO
@pytest.mark.parametrize("dv,H", [(128, 2), (64, 2), (128, 80)])
@pytest.mark.parametrize("at", [70, 127, 128])
def test_a_residual_that_overflows(io, dv, H, at):
    """One state row so large that a strong key's product with it overflows: that row's outputs from there on, no others."""
    args = list(_inputs(51, 200, H, 1, 128, dv, io))
    args[1][at] = 8.0
    init = torch.randn(1, H, dv, 128, device="cuda", generator=_gen(52)) * 0.3
    init[0, 1, 3] = 1e37
    args[3][:] = 0.0                                  # nothing is forgotten
    args[4][:at] = 0.01
    o, fin = _ers().gdn_fwd(*args, init_state=init)
    _same_as_the_rule(o[:_reached(at, io)], args, init)
    assert not torch.isfinite(o[at:, 1, 3]).any() and not torch.isfinite(fin[0, 1, 3]).any()
    rows = torch.ones(H, dv, dtype=torch.bool, device="cuda")
    rows[1, 3] = False
    init[0, 1, 3] = 0.0                               # rows depend on no other
    _same_as_the_rule(o[:at], args, init, rows)
    assert torch.isfinite(o[:, rows]).all() and torch.isfinite(fin[0][rows]).all()


@IO
@pytest.mark.parametrize("at", [7, 60, 100, 191])
def test_a_key_whose_products_overflow(io, at):
    """Its row of the triangular system is infinite in places; the head of the other key group has none of that."""
    args = list(_inputs(53, 260, 2, 2, 128, 128, io))
    init = torch.randn(1, 2, 128, 128, device="cuda", generator=_gen(54)) * 0.3
    args[1][at // 2, 1] = 1 / 12.0                    # (a product of 3e39 for certain)
    good, state = _ers().gdn_fwd(*args, init_state=init)
    args[1][at, 1] = 3e38
    o, fin = _ers().gdn_fwd(*args, init_state=init)
    _same_as_the_rule(o[:_reached(at, io)], args, init)
    assert not torch.isfinite(o[at:, 1]).any() and not torch.isfinite(fin[0, 1]).any()
    assert torch.equal(o[:, 0], good[:, 0]) and torch.equal(fin[0, 0], state[0, 0])


@IO
def test_a_state_that_grows_out_of_range(io):
    """The same strong key at beta 1 over and over multiplies the state by -999 a token, until it overflows; the next sequence
    is none the worse."""
    T, at = 150, 100
    args = list(_inputs(55, T + 20, 2, 1, 128, 128, io))
    key = args[1][at].float()
    args[1][at:T] = (key / key.norm() * 1000.0 ** 0.5).to(io)
    args[4][at:T] = 1.0
    args[3][at:T] = 0.0
    o, fin = _ers().gdn_fwd(*args, _cu([T, 20]), max_seqlen=T)
    _same_as_the_rule(o[:_reached(at, io)], args, None)
    assert not torch.isfinite(o[T - 1]).any() and not torch.isfinite(fin[0]).all()
    _same_as_the_rule(o[T:], [x[T:] for x in args], None)
    assert torch.isfinite(fin[1]).all()
