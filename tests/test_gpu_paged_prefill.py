"""Prefill through BeamStack over paged caches in calls where something is out of range, where
the page table is large, or between replays of a captured step."""
import pytest
import torch

from synth import TINY
from hybrid_attention_moe_gb300 import beam as B
from hybrid_attention_moe_gb300.stack import BeamStack
from test_gpu_paged import status
from test_gpu_paged_stack import CHUNKS, PAGE, PAGES, SEQS, contiguous_caches, paged_caches, prefill, tokens, weights

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


def test_replays_after_prefills_of_other_sizes():
    """A server's order: a decode step captured, a longer prefill chunk (other buffers, a larger
    workspace, a larger copy) between its replays, memory handed out again in between. The replays
    give the eager steps' bits and write no one else's memory."""
    W = weights()
    outs = []
    for captured in (False, True):
        st = BeamStack(TINY, W, paged_caches("nvfp4"))
        prefill(st)
        e, s, p = tokens([0, 1, 2], [50, 34, 18], 10)
        args = dict(max_q_per_seq=1)
        if captured:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                h = st.forward(e, s, p, 64, **args)
        out, junk = [], []
        for n in range(3):
            ce, cs, cp = tokens([0] * (40 + 7 * n), [60 + 35 * n + i for i in range(40 + 7 * n)], 30 + n)
            st.forward(ce, cs, cp, PAGE * PAGES, max_q_per_seq=40 + 7 * n, n_seqs=1)
            junk += [torch.full((2 ** i,), 77, dtype=torch.uint8, device="cuda") for i in range(9, 23)]
            e2, s2, p2 = tokens([0, 1, 2], [51 + n, 34 + n, 18 + n], 20 + n)
            for x, y in ((e, e2), (s, s2), (p, p2)):
                x.copy_(y)
            if captured:
                graph.replay()
            else:
                h = st.forward(e, s, p, 64, **args)
            out.append(h.clone())
        torch.cuda.synchronize()
        assert all(bool((x == 77).all()) for x in junk)
        outs.append(out)
    assert status() == 0
    for x, y in zip(*outs):
        assert torch.equal(x, y)


def test_captured_prefill_chunk_equals_the_eager_one():
    """A chunk captured once (n_seqs said) and replayed for other sequences and positions, with eager
    calls of other sizes between the replays."""
    W = weights()
    caches = [paged_caches("fp8"), paged_caches("fp8")]
    a, b = (BeamStack(TINY, W, large(c)) for c in caches)
    T = 12

    def chunk(n):
        seq = [ROWS[n % 3]] * 7 + [ROWS[(n + 1) % 3]] * 5
        return tokens(seq, list(range(1, 8)) + list(range(1, 6)), 50 + n)

    e, s, p = chunk(0)
    for st in (a, b):
        st.forward(e, s, p, 96, max_q_per_seq=7, n_seqs=2)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h = b.forward(e, s, p, 96, max_q_per_seq=7, n_seqs=2)
    assert h.shape[0] == T
    for n in range(1, 5):
        for x, y in zip((e, s, p), chunk(n)):
            x.copy_(y)
        ref = a.forward(e, s, p, 96, max_q_per_seq=7, n_seqs=2).clone()
        graph.replay()
        assert torch.equal(h, ref)
        ce, cs, cp = tokens([ROWS[n % 3]] * 30, list(range(20, 50)), 70 + n)
        for st in (a, b):
            st.forward(ce, cs, cp, 150, max_q_per_seq=30, n_seqs=n % 3 + 1)
    assert status() == 0


def test_a_padded_decode_batch_sets_no_bit():
    """A captured decode batch of four rows, some of them padding (position 0, any sequence): no
    device status, nothing written for them, zeros from their attention, and the other rows' bits
    are those beside real tokens. A negative position is flagged still."""
    W = weights()
    caches = paged_caches("fp8")
    st = BeamStack(TINY, W, caches)
    prefill(st)
    e, s, p = tokens([0, 1, 2, 0], [50, 34, 18, 0], 10)
    st.forward(e, s, p, 64, max_q_per_seq=1)
    torch.cuda.synchronize()
    graph, trace = torch.cuda.CUDAGraph(), []
    with torch.cuda.graph(graph):
        h = st.forward(e, s, p, 64, trace=trace, max_q_per_seq=1)
    rows = []
    for seq, pos in (([0, 1, 2, 0], [50, 34, 18, 0]), ([0, 99, 2, -4], [50, 0, 18, 0]), ([0, 1, 2, 0], [50, 34, 18, 51])):
        s.copy_(torch.tensor(seq)), p.copy_(torch.tensor(pos))
        before = [c.k.clone() for c in caches]
        graph.replay()
        assert status() == 0
        for t in trace:
            for i, x in enumerate(pos):
                assert bool(t["attn"][i].any()) == (x > 0)
        if pos[3] == 0 and rows:       # the same rows again, and nothing else
            assert all(torch.equal(a, c.k) for a, c in zip(before, caches))
        rows.append(h[[0, 2]].clone())
    assert torch.equal(rows[0], rows[1]) and torch.equal(rows[0], rows[2])
    p.copy_(torch.tensor([50, -1, 18, 0]))
    graph.replay()
    assert status() == B.DEV_BAD_POSITION


@pytest.mark.parametrize("paged", [False, True])
def test_a_call_on_another_stream_waits_for_no_other(paged):
    """forward(stream=...) while the current stream is busy: the input's copy, the buffers and the
    trace belong to the call's stream, so its results are those of a call by itself."""
    W = weights()
    runs = []
    busy = torch.randn(4096, 4096, device="cuda")
    for side in (None, torch.cuda.Stream()):
        st = BeamStack(TINY, W, paged_caches("bf16") if paged else contiguous_caches(40))
        got = []
        for n, (seq, pos, most) in enumerate(CHUNKS + [([0, 1, 2], [50, 34, 18], 1)]):
            e, s, p = tokens(seq, pos, n)
            torch.cuda.synchronize()
            trace = []
            if side is not None:
                x = busy
                for _ in range(40):      # tens of milliseconds
                    x = x @ busy
            h = st.forward(e, s, p, max(pos), stream=side, trace=trace, max_q_per_seq=most)
            (side or torch.cuda.current_stream()).synchronize()
            with torch.cuda.stream(side):
                got += [h.clone()] + [t[k].clone() for t in trace for k in ("u_attn", "attn", "h")]
            torch.cuda.synchronize()
        runs.append(got)
    assert status() == 0
    for x, y in zip(*runs):
        assert torch.equal(x, y)
