"""Prefill through BeamStack over paged caches in calls where something is out of range, where
the page table is large, or between replays of a captured step."""
import pytest
import torch

from synth import TINY
from hybrid_attention_moe_gb300 import beam as B
from hybrid_attention_moe_gb300.stack import BeamStack
from test_gpu_paged import status
from test_gpu_paged_stack import CHUNKS, PAGE, PAGES, SEQS, paged_caches, prefill, tokens, weights

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


ROWS = {0: 35, 1: 2, 2: 17}      # where the small table's sequences lie in the large one


def large(caches, rows=40):
    """The same caches under a table of many sequences, the others' entries naming no page."""
    table = torch.full((rows, PAGES), -1, dtype=torch.int32, device="cuda")
    for small, s in ROWS.items():
        table[s] = caches[0].page_table[small]
    return [B.PagedKVCache(c.k, c.v, table, c.row_scale, c.block_scale, c.window) for c in caches]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("n_seqs", [None, 2, 7])
def test_prefill_out_of_a_large_table(fmt, n_seqs):
    """Chunks of two sequences out of a table of 40 give the bits of a table of three, then a decode
    step over what they wrote does; the copies have rows for the call's sequences only."""
    W = weights()
    a, b = BeamStack(TINY, W, paged_caches(fmt)), BeamStack(TINY, W, large(paged_caches(fmt)))
    for n, (seq, pos, most) in enumerate(CHUNKS + [([0, 1, 2], [50, 34, 18], 1)]):
        e, s, p = tokens(seq, pos, n)
        x = a.forward(e, s, p, max(pos), max_q_per_seq=most)
        y = b.forward(e, torch.tensor([ROWS[i] for i in seq], dtype=torch.int32, device="cuda"), p, max(pos),
                      max_q_per_seq=most, n_seqs=n_seqs)
        assert torch.equal(x, y)
    assert status() == 0
    assert {k[0] for k in b._copies} == {40 if n_seqs is None else n_seqs}


def test_more_sequences_than_were_said_are_flagged():
    """n_seqs = 1 with two sequences: the first is served, the other's tokens attend to nothing."""
    W = weights()
    seq, pos, most = CHUNKS[0]
    e, s, p = tokens(seq, pos, 0)
    runs = []
    for n_seqs in (2, 1):
        trace = []
        BeamStack(TINY, W, paged_caches("fp8")).forward(e, s, p, max(pos), trace=trace, max_q_per_seq=most, n_seqs=n_seqs)
        assert status() == (0 if n_seqs == 2 else B.DEV_BAD_SEQ)
        runs.append(trace[0]["attn"])
    assert torch.equal(runs[0][:40], runs[1][:40]) and not runs[1][40:].any()


def test_prefill_of_one_sequence_takes_the_memory_of_one():
    """One sequence out of a table of 512 that reaches 102,400 positions, and a bound as high."""
    W = weights()
    table = torch.full((512, 3200), -1, dtype=torch.int32, device="cuda")
    table[300, :PAGES] = torch.arange(PAGES)
    st = BeamStack(TINY, W, [B.PagedKVCache.empty(PAGES, PAGE, TINY.n_kv, TINY.head_dim, table, B.BEAM_PAGED_FP8, c.window)
                             for c in paged_caches("fp8")])
    e, s, p = tokens([300] * 100, list(range(1, 101)), 3)
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    got = st.forward(e, s, p, 102400)
    assert status() == 0
    # one row of keys and values of both kinds of layer, and less than 256 MiB for all else
    assert torch.cuda.max_memory_allocated() - before < 102400 * TINY.n_kv * TINY.head_dim * 4 + (256 << 20)
    ref = BeamStack(TINY, W, paged_caches("fp8"))
    assert torch.equal(got, ref.forward(e, torch.zeros_like(s), p, 100))
