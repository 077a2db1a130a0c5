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
