"""Prefill through BeamStack over paged caches in calls where something is out of range, where
the page table is large, or between replays of a captured step."""
import pytest
import torch

from synth import TINY
from hybrid_attention_moe_gb300 import beam as B
from hybrid_attention_moe_gb300.stack import BeamStack
from test_gpu_paged import status
from test_gpu_paged_stack import PAGE, PAGES, SEQS, paged_caches, prefill, tokens, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [PAGE * PAGES + 1, PAGE * PAGES + 60, 300])
def test_a_token_past_the_page_table_leaves_the_others_as_they_are(bad):
    """max_pos may lie past the table's reach: a token between the two is flagged, its sequence's
    other tokens give the bits that they give beside a good token of another sequence."""
    W = weights()
    runs = []
    for last in ((2, 18), (0, bad)):
        st = BeamStack(TINY, W, paged_caches("fp8"))
        prefill(st)
        seq, pos = [1] * 30 + [0] * 30 + [last[0]], list(range(34, 64)) + list(range(50, 80)) + [last[1]]
        e, s, p = tokens(seq, pos, 7)
        runs.append(st.forward(e, s, p, 300, max_q_per_seq=31)[:60].clone())
        assert status() == (B.DEV_BAD_POSITION if last[0] == 0 else 0)
    assert torch.equal(*runs)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_tokens_whose_keys_are_not_read_attend_to_nothing(fmt):
    """One entry of sequence 0's table names no page: the tokens whose keys lie there attend to
    nothing (the first layer's attention output is zero), never to what the copy held before;
    those before it and the other sequence's give the bits that they give without the fault."""
    W = weights()
    seq, pos = [0] * 60 + [1] * 9, list(range(3, 63)) + list(range(34, 43))
    e, s, p = tokens(seq, pos, 7)
    runs = []
    for entry in (None, -1, 10 ** 6):
        caches = paged_caches(fmt)
        st = BeamStack(TINY, W, caches)
        prefill(st)
        if entry is not None:
            for c in caches:
                c.page_table[0, 1] = entry      # positions 33 .. 64
        trace = []
        st.forward(e, s, p, max(pos), trace=trace, max_q_per_seq=60)
        assert status() & B.DEV_BAD_PAGE == (0 if entry is None else B.DEV_BAD_PAGE)
        runs.append(trace)
    good = runs[0]
    for trace in runs[1:]:
        for layer, t in enumerate(trace):
            assert not t["attn"][30:60].any(), layer
            assert torch.equal(t["attn"][:30], good[layer]["attn"][:30])
            assert torch.equal(t["attn"][60:], good[layer]["attn"][60:])


def test_tokens_of_a_sequence_too_far_apart_attend_to_nothing():
    """A sliding window's copy holds the window of consecutive tokens; tokens of one sequence further
    apart are flagged and attend to nothing there, the other sequence's are as they were."""
    W = weights()
    runs = []
    for far in (53, 170):
        caches = paged_caches("fp8")
        st = BeamStack(TINY, W, caches)
        prefill(st)
        seq, pos = [0] * 5 + [1] * 7, [50, 51, 52, far, far + 1] + list(range(34, 41))
        e, s, p = tokens(seq, pos, 8)
        trace = []
        st.forward(e, s, p, 171, trace=trace, max_q_per_seq=7)
        assert status() & B.DEV_BAD_POSITION == (0 if far == 53 else B.DEV_BAD_POSITION)
        runs.append(trace)
    layer = next(i for i, c in enumerate(caches) if c.window)
    assert not runs[1][layer]["attn"][:5].any()
    assert torch.equal(runs[0][layer]["attn"][5:], runs[1][layer]["attn"][5:])
