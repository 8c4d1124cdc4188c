"""Warp-wide instructions of the aligned kind are for converged warps.  Lanes may come to them from a section that one lane had
to itself (a loop that issues copies, a bounded wait), and nothing but a __syncwarp promises that they have met again; a warp whose
lanes leave a loop one by one must not vote in it.  The sources are read: what goes wrong otherwise is a hang."""
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "exact_replay_decode_gb300", "csrc")


def _source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _body(text, opening):
    """From the first brace after `opening` to the one that closes it."""
    start = text.index("{", text.index(opening))
    depth = 0
    for at in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[at], 0)
        if depth == 0:
            return text[start:at + 1]
    raise AssertionError(opening)


@pytest.mark.parametrize("name", ["void named_sync(", "bool named_sync_and(", "void tmem_alloc(", "void tmem_dealloc("])
def test_lanes_meet_before_barriers_and_tensor_memory_changes_hands(name):
    body = _body(_source("tc_common.cuh"), name)
    assert 0 <= body.find("__syncwarp();") < body.index("asm volatile")


def test_attentions_issuing_warp_goes_on_or_leaves_as_one():
    """Its lanes vote on whether the next tile is there, so none may have left on its own: a wait's end is voted on as well."""
    text = _source("ers_attn_tc.cu")
    start = text.index("if (tid >= kIssueThread)")
    body = text[start:text.index("else if (tid >= kLoadThread)", start)]
    assert "__all_sync(kFull, mbar_test(" in body and "break;" in body
    for m in re.finditer(r"\bwait\(", body):
        assert body[:m.start()].endswith("__all_sync(kFull, ")


def test_attention_outputs_meet_before_every_load():
    text = _source("ers_attn_tc.cu")
    loop = text[text.rindex("for (int x = 0; x < D; x += 32)"):]
    assert "continue;" in loop and loop.index("__syncwarp();") < loop.index("tmem_ld32_begin")
