"""What the gated delta rule remembers over long prompts, on the GPU.

A state element that the keys do not reach (they are zero there) has one formula, S_T = S_0 exp(sum of the gates), whatever the
other elements do, and each time the kernels move the state by a chunk of 64 tokens (fp32 prompts: a batch of eight) they round it
once, to nearest: by 2^-24 of itself at most.  Roundings of unlike values do not conspire: over n of them the 2-norm is within
sqrt(n) 2^-24.  A factor that were rounded the same way each time would add up to n times its error, a chunk's single float to as
much as n 2^-25.  The gates' own sums and exponentials are within 2^-22 of the whole decay's exponent: three roundings of the
sum, its product with a constant and the exponential, 2^-24 each and counted twice."""
import math

import pytest
import torch

from test_gpu_gdn_rule import BF16, F32, _check, _ers, _gen, _inputs, _norm, _rule

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("io,T", [(BF16, 8192), (BF16, 32768), (F32, 8192)], ids=str)
@pytest.mark.parametrize("total", [0.5, 2.0])
def test_what_the_keys_do_not_reach_is_only_forgotten(io, T, total):
    """A constant gate a head, with 16 of them around total / T, and keys and queries in the first half of dk."""
    H = 16
    q, k, v, _, beta = _inputs(31, T, H, 1, 128, 128, io)
    k[..., 64:] = 0
    rate = total / T * (1 + torch.arange(H, device="cuda") / (2 * H))
    g = (-rate).expand(T, H).contiguous().float()
    init = torch.randn(1, H, 128, 128, device="cuda", generator=_gen(32))
    _, fin = _ers().gdn_fwd(q, k, v, g, beta, init_state=init)
    exponent = g[:1].double().view(1, H, 1, 1) * T
    want = init[..., 64:].double() * torch.exp(exponent)
    off = (fin[..., 64:].double() - want).flatten(2).norm(dim=-1) / want.flatten(2).norm(dim=-1)
    rounds = T // (64 if io == BF16 else 8)
    assert (off <= math.sqrt(rounds) * 2.0 ** -24 - exponent.flatten() * 2.0 ** -22).all()


@pytest.mark.parametrize("io,T", [(BF16, 8192), (F32, 4096)], ids=str)
def test_weak_writes_over_a_long_memory(io, T):
    """beta near 0 and a weak gate: a state that holds thousands of tokens, and a resumed one, against the rule."""
    args = list(_inputs(33, T, 2, 1, 128, 128, io, 1.0 / T))
    args[4] *= 4.0 / T
    init = torch.randn(1, 2, 128, 128, device="cuda", generator=_gen(34)) * 0.3
    o, fin = _ers().gdn_fwd(*args, init_state=init)
    _check(o, fin, args, [T], init)


@pytest.mark.parametrize("weak", ["none", "gates", "gates and writes"])
@pytest.mark.parametrize("dk", [64, 128])
@pytest.mark.parametrize("io,T", [(BF16, 1), (BF16, 24), (BF16, 97), (BF16, 1025), (BF16, 4096), (F32, 24), (F32, 300), (F32, 4096)], ids=str)
def test_final_states_are_as_near_as_the_header_says(io, T, dk, weak):
    """Chunks: three operands of 16 bits whose roundings, 2^-17 at most and 2^-18 in the mean, add up in quadrature (6.6e-6), and the
    state's own rounding every 64 tokens.  The recurrence: for each token a rounded product and sum into the state, an eighth of
    its factor's rounding, and the residual's own error, whose sum of dk products is as far off as sqrt(dk) 2^-24 / 2 of |S k|, which is
    |S| / sqrt(dk) for keys that point anywhere: half a rounding of S.  Together less than two a token, in quadrature, for no
    longer than the state remembers."""
    args = list(_inputs(35, T, 4, 2, dk, 128, io, 1.0 if weak == "none" else 1.0 / T))
    if weak == "gates and writes":
        args[4] *= 4.0 / T
    init = torch.randn(1, 4, 128, dk, device="cuda", generator=_gen(36)) * 0.3
    _, fin = _ers().gdn_fwd(*args, init_state=init)
    _, want, _, _ = _rule(*args, [T], init)
    chunks = io == BF16 and T > 32
    assert _norm(fin, want) <= ((6.6e-6 + math.sqrt(T / 64) * 2.0 ** -24) if chunks else (math.sqrt(2 * T) + 2) * 2.0 ** -24)
