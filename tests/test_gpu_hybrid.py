"""A hybrid of a gated-delta-rule and an attention layer served speculatively with a tree of drafts: prompts into both caches, the
tree's branches on forked states and its drafts against the pages, the accepted path into both, and the next token.  What comes
out is what the same tokens give when they are read as one prompt, and what the layers' formulas give in 64 bits."""
import math

import pytest
import torch

from test_gpu_gdn_rule import BF16, F32, _cu, _gen, _inputs, _norm, _rule

pytestmark = pytest.mark.gpu

PARENT = [-1, 0, 0, 1, -1, 4, 3]                         # two drafts after the past; leaves 2, 5 and 6
LEAVES = {2: [0, 2], 5: [4, 5], 6: [0, 1, 3, 6]}


@pytest.mark.parametrize("io", [BF16, F32], ids=["bf16", "f32"])
def test_a_tree_through_both_layers(io):
    import exact_replay_decode_gb300 as ers
    H, G, KV, D, T = 4, 2, 2, 64, len(PARENT)
    lens, S = [70, 131], 2
    i32 = dict(dtype=torch.int32, device="cuda")
    gdn = [_inputs(30 + i, lens[i] + T + 1, H, G, 128, 128, io) for i in range(S)]          # prompt, drafts, one more token
    r = dict(device="cuda", generator=_gen(40))
    att = [[(torch.randn(lens[i] + T + 1, n, D, **r)).to(io) for n in (H, KV, KV)] for i in range(S)]

    # prompts
    states = ers.LinAttnCache(S * (1 + len(LEAVES)), H, G, npages=S * (1 + len(LEAVES)) + 1, io_dtype=io)
    rows = ers.AttnCache(S, KV, D, page_tokens=16, slot_pages=12, io_dtype=io)
    roots = torch.arange(S, **i32)
    ers.pages_own(states.pages, roots)
    prompt = [torch.cat([gdn[i][x][:lens[i]] for i in range(S)]) for x in range(5)]
    o_prompt = ers.gdn_prefill(states, *prompt, _cu(lens), slot=roots)
    ers.attn_append(rows, *(torch.cat([att[i][x][:lens[i]] for i in range(S)]) for x in (1, 2)), cu_seqlens=_cu(lens))

    # the tree: a branch of states for each leaf, and all drafts against the pages at once
    src, dst = roots.repeat_interleave(len(LEAVES)), torch.arange(S, S * (1 + len(LEAVES)), **i32)
    ers.pages_fork(states.pages, src, dst)
    read = ers.pages_own(states.pages, dst, copy=False)
    paths = [(i, path) for i in range(S) for path in LEAVES.values()]
    branch = [torch.cat([gdn[i][x][lens[i]:][path] for i, path in paths]) for x in range(5)]
    o_tree = ers.gdn_prefill(states, *branch, _cu([len(p) for _, p in paths]), slot=dst, read_page=read)
    parent = torch.tensor([PARENT] * S, **i32)
    drafts = [torch.stack([att[i][x][lens[i]:lens[i] + T] for i in range(S)]) for x in range(3)]
    a_tree = ers.attn_verify(rows, *drafts, parent=parent)

    # accepted: all of the longest branch by the first sequence, one draft of the second leaf's by the other
    taken = [LEAVES[6], LEAVES[5]]
    path = torch.tensor([p + [0] * (T - len(p)) for p in taken], **i32)
    ers.attn_commit(rows, drafts[1], drafts[2], torch.tensor([len(p) for p in taken], **i32), path=path)
    winners = torch.tensor([S + 2, S + len(LEAVES) + 1], **i32)
    ers.pages_free(states.pages, torch.tensor([s for s in range(S * (1 + len(LEAVES))) if s not in winners.tolist()], **i32))
    assert int((states.pages.refs > 0).sum()) == S and rows.pos.tolist() == [lens[i] + len(taken[i]) for i in range(S)]

    # the next token
    token = [torch.stack([gdn[i][x][-1] for i in range(S)]) for x in range(5)]
    o_next = ers.gdn_decode(states, *token, slot=winners)
    a_next = ers.attn_verify(rows, *[torch.stack([att[i][x][-1:] for i in range(S)]) for x in range(3)])

    at = 0
    for n, (i, p) in enumerate(paths):
        whole = [torch.cat([x[:lens[i]], x[lens[i]:][p], x[-1:]]) for x in gdn[i]]
        want, state, off, state_off = _rule(*whole, [whole[0].shape[0]], c=2.0 ** -15 if io is BF16 else 144 * 2.0 ** -24)
        mine = o_tree[at:at + len(p)]
        at += len(p)
        assert _norm(mine, want[lens[i]:-1]) <= (2.2e-3 if io is BF16 else 2e-6)
        if p == taken[i]:
            assert _norm(o_next[i], want[-1]) <= (2.4e-3 if io is BF16 else 2e-6)      # (few values: the mean is not quite one)
            page = states.pages.table[winners[i].long(), 0].long()
            assert ((states.state[page].double() - state[0]).norm(dim=-1) <= state_off[0]).all()
        # the attention layer: each draft of the branch, and the next token where it was taken
        q, k, v = ([torch.cat([x[:lens[i]], x[lens[i]:][p], x[-1:]]).double() for x in att[i]])
        k, v = (x.repeat_interleave(H // KV, 1).transpose(0, 1) for x in (k, v))
        x = q.transpose(0, 1) @ k.transpose(1, 2) * D ** -0.5
        past = torch.ones(x.shape[1:], dtype=torch.bool, device="cuda").tril()
        w = (torch.softmax(x.masked_fill(~past, -math.inf), -1) @ v).transpose(0, 1)
        bound = 2.4e-3 if io is BF16 else 2e-6
        assert _norm(a_tree[i][p], w[lens[i]:-1]) <= bound
        if p == taken[i]:
            assert _norm(a_next[i, 0], w[-1]) <= bound * 1.2
    whole, _ = ers.gdn_fwd(*prompt, _cu(lens))
    assert torch.equal(o_prompt, whole)
