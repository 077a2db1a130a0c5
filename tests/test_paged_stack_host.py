"""What BeamStack works out on the host and in torch for a prefill over paged caches, on the CPU."""
import weakref

import pytest
import torch

from synth import TINY
from hybrid_attention_moe_gb300 import beam as B
from hybrid_attention_moe_gb300 import stack as S


def paged(rows=4, pages=5, page_size=16, window=0):
    c = object.__new__(B.PagedKVCache)
    c.page_table, c.window, c.page_size = torch.zeros((rows, pages), dtype=torch.int32), window, page_size
    return c


def stack(caches=()):
    """A stack without weights: enough for the context of a prefill."""
    return S.BeamStack(TINY, [], list(caches), device="cpu")


def ints(x):
    return torch.tensor(x, dtype=torch.int32)


@pytest.mark.parametrize("window", [0, TINY.window])
@pytest.mark.parametrize("bad", [81, 200])
def test_context_leaves_tokens_past_the_page_table_out(window, bad):
    """max_pos is an upper bound that may lie past the page table (here 80 positions): a token
    between the two is no one's last position, and the copy is no longer than the table."""
    st, kc = stack(), paged(window=window)
    seq, pos = [2] * 9 + [0] * 6, list(range(30, 39)) + list(range(1, 7))

    def ranges(seq, pos):
        copy, every, first, last, longest = st.context(kc, ints(seq), ints(pos), 300, 9)
        assert longest <= 80
        return every.tolist(), first.tolist(), last.tolist(), longest

    assert ranges(seq + [2], pos + [bad]) == ranges(seq, pos)


@pytest.mark.parametrize("window", [0, 20])
def test_tokens_with_keys_that_are_not_read_attend_to_nothing(window):
    """readable() against the definition: every key of the token in a page of the pool, and the
    sequence's range within the copy."""
    st, kc = stack(), paged(rows=3, pages=6, page_size=16, window=window)
    kc.num_pages = 9
    kc.page_table.copy_(ints([[0, 1, 2, 3, 4, 5], [6, -1, 7, 8, 0, 1], [2, 3, 9, 4, 5, 6]]))
    seq = [s for s in range(3) for _ in range(97)]
    pos = [p for _ in range(3) for p in range(97)]
    first, last = ints([1, 1, 1]), ints([96, 96, 96])
    got = st.readable(kc, ints(seq + [-1, 3]), ints(pos + [0, 0]), first, last, 96).tolist()
    for s, p, g in zip(seq, pos, got):
        keys = range(max(1, p - window + 1) if window else 1, p + 1)
        ok = all(0 <= int(kc.page_table[s, (k - 1) // 16]) < 9 for k in keys)
        assert g == (p if ok else 0), (s, p)
    assert got[-2:] == [0, 0]
    # a range longer than the copy is not read at all: sequence 0's tokens attend to nothing
    got = st.readable(kc, ints([0, 0, 1]), ints([1, 96, 9]), ints([1, 1, 1]), ints([96, 9, 0]), 90).tolist()
    assert got == [0, 0, 9]


@pytest.mark.parametrize("window", [0, TINY.window])
@pytest.mark.parametrize("n_seqs", [None, 2, 3, 50])
def test_context_has_rows_for_the_call_only(window, n_seqs):
    """A table of 50 sequences, two of which have tokens in the call: the copy holds n_seqs rows, whose
    ranges are those of the full table's, and every token finds its sequence's row."""
    kc = paged(rows=50, pages=8, window=window)
    seq, pos = [47] * 9 + [-1, 50, 3] + [11] * 6, list(range(30, 39)) + [5, 6, 0] + list(range(1, 7))
    full = stack().context(kc, ints(seq), ints(pos), 60, 9)
    copy, every, first, last, longest = got = stack().context(kc, ints(seq), ints(pos), 60, 9, n_seqs)
    assert copy.k.shape[0] == copy.v.shape[0] == every.numel() == (n_seqs or 50) and longest == full[4]
    assert copy.k.shape[2:] == full[0].k.shape[2:]
    row = stack().rows(kc, ints(seq), ints(pos), every, first, last)
    for t, s in enumerate(seq):
        r = int(row[t])
        if s in (47, 11):
            assert int(every[r]) == s and int(first[r]) == int(full[2][s]) and int(last[r]) == int(full[3][s])
        elif 0 <= s < 50:
            assert 0 <= r < every.numel()            # position 0: any row, flagged for the position
        else:
            assert not 0 <= r < every.numel()        # flagged for the sequence
    reads = [int(every[r]) for r in range(every.numel()) if int(last[r]) >= int(first[r])]
    assert sorted(reads) == [11, 47]
    p = stack().readable(kc, row, ints(pos), first, last, longest, every)
    assert p.tolist() == pos
    assert got[0].k.dtype == torch.bfloat16


def test_context_of_more_sequences_than_were_said():
    """The first n_seqs sequences are served, the others' tokens name no row."""
    kc = paged(rows=9, pages=8)
    seq, pos = ints([7, 7, 2, 4, 4]), ints([1, 2, 9, 5, 6])
    copy, every, first, last, _ = stack().context(kc, seq, pos, 60, 5, 2)
    row = stack().rows(kc, seq, pos, every, first, last)
    assert every.tolist() == [2, 4] and last.tolist() == [9, 6] and row.tolist() == [-1, -1, 0, 1, 1]


def test_the_copy_grows_and_is_kept():
    """One copy for a window: kept for calls that fit in it, a quarter larger than asked where a
    context has outgrown it, never longer than the page table."""
    st, kc = stack(), paged(rows=50, pages=100)
    seq, pos = ints([3] * 6), ints(list(range(1, 7)))

    def cap(max_pos, n=1):
        c = st.context(kc, seq, pos, max_pos, 6, n)[0]
        assert len(st._copies) == 1 and next(iter(st._copies.values())) is c
        return tuple(c.k.shape[::2])
    assert cap(200) == (1, 200) and cap(100) == (1, 200)
    assert cap(400) == (1, 500) and cap(500) == (1, 500)
    assert cap(1590) == (1, 1600) and cap(5000) == (1, 1600)
    assert cap(100, 2) == (2, 100) and cap(100, 1) == (2, 100)
    st.context(paged(rows=50, pages=100, window=16), seq, pos, 300, 6, 1)
    assert len(st._copies) == 2


def test_the_sequences_of_a_large_call_are_counted():
    """A call that does not say how many sequences it has: counted where T rows would take more
    than COPY_BYTES, else not."""
    seq = ints([3, 3, 90, 3] * 30)
    st = stack([paged(rows=128, pages=6400), paged(rows=128, pages=6400, window=16)])
    assert st.count(seq, 102400, None) == 2
    assert st.count(seq, 1024, None) is None
    assert stack([paged(rows=128, pages=6400, window=16)]).count(seq, 102400, None) is None
    copy = st.context(st.caches[0], seq, ints([1] * 120), 102400, 5, 2)[0]
    assert copy.k.nbytes + copy.v.nbytes == 2 * 102400 * TINY.n_kv * TINY.head_dim * 4


def test_captured_calls_keep_their_buffers(monkeypatch):
    """Buffers that a captured call got outlive calls of other sizes (a replay writes them), are
    used again by calls of their size, and what no capture used is dropped."""
    st, kc = stack(), paged(rows=8, pages=100)
    seq, pos = ints([3] * 6), ints(list(range(1, 7)))

    def use(T, max_pos, nbytes):
        st.ws.device = "cpu"
        got = [st.buffers(T)["h"], st.stage(T)[0].k, st.stage(T)[1],
               st.context(kc, seq, pos, max_pos, 6, 1)[0].k, st.ws.get(nbytes)]
        return [weakref.ref(x) for x in got]

    early = use(3, 100, 1000)
    monkeypatch.setattr(B, "capturing", lambda: True, raising=False)
    first = use(4, 200, 2000)
    monkeypatch.setattr(B, "capturing", lambda: False, raising=False)
    between = use(70, 900, 50000)
    again = use(4, 100, 100)
    assert all(x() is not None for x in first)
    assert [a() is b() for a, b in zip(first[:3], again[:3])] == [True] * 3
    assert early[0]() is None and early[1]() is None and early[4]() is None
    assert between[3]() is again[3]() and between[4]() is again[4]()
    use(5, 100, 100)
    assert between[0]() is None and between[1]() is None and all(x() is not None for x in first)


def test_padding_rows_are_projected_at_a_position_that_there_is(monkeypatch):
    """Position 0 reaches the write and the attention, which take it for padding, and not the
    projection, which flags it; one tensor serves all layers."""
    import synth
    caches = [paged(window=TINY.window), paged(window=TINY.window)]
    st = S.BeamStack(TINY, [synth.layer_weights(TINY, layer, 0) for layer in range(2)], caches, device="cpu")
    seen = {}
    for name in ("beam_qkv_gate", "beam_attn", "beam_boundary_norm", "beam_dense_mlp", "beam_route", "beam_moe",
                 "beam_paged_kv_write", "beam_paged_kv_read", "beam_paged_attn"):
        monkeypatch.setattr(B, name, lambda *a, _n=name, **k: seen.setdefault(_n, []).append(a))
    monkeypatch.setattr(B, "workspace_bytes", lambda *a: 100)
    monkeypatch.setattr(B, "paged_workspace_bytes", lambda *a: 100)
    e = torch.zeros((4, TINY.hidden), dtype=torch.bfloat16)
    st.forward(e, ints([0, 1, 2, 0]), ints([7, 0, -3, 1]), 7, max_q_per_seq=1)
    assert [a[6].tolist() for a in seen["beam_qkv_gate"]] == [[7, 1, 1, 1]] * 2
    assert seen["beam_qkv_gate"][0][6] is seen["beam_qkv_gate"][1][6]
    assert [a[3].tolist() for a in seen["beam_paged_kv_write"]] == [[7, 0, -3, 1]] * 2
    assert [a[6].tolist() for a in seen["beam_paged_attn"]] == [[7, 0, -3, 1]] * 2


def test_layers_share_what_they_read_over_one_table_only(monkeypatch):
    """Layers over one table and window use the ranges that the first of them found; another table
    or window has its own, and so has the next call."""
    import synth
    one, other = ints([[0, 1, 2, 3, 4]] * 4), ints([[0, 1, -1, 3, 4]] * 4)
    caches = [paged(window=w) for w in (TINY.window, 0, TINY.window, TINY.window, 0)]
    for c, t in zip(caches, (one, one, one, other, other)):
        c.page_table, c.num_pages = t, 9
    st = S.BeamStack(TINY, [synth.layer_weights(TINY, 0, 0) for _ in caches], caches, device="cpu")
    st.dense = [True] * 5
    seen = {}
    for name in ("beam_qkv_gate", "beam_attn", "beam_boundary_norm", "beam_dense_mlp", "beam_paged_kv_write",
                 "beam_paged_kv_read"):
        monkeypatch.setattr(B, name, lambda *a, _n=name, **k: seen.setdefault(_n, []).append(a))
    monkeypatch.setattr(B, "workspace_bytes", lambda *a: 100)
    monkeypatch.setattr(B, "paged_workspace_bytes", lambda *a: 100)
    for start in (30, 33):
        seen.clear()
        e, pos = torch.zeros((9, TINY.hidden), dtype=torch.bfloat16), list(range(start, start + 9))
        st.forward(e, ints([2] * 9), ints(pos), max(pos), max_q_per_seq=9)
        reads, attns = seen["beam_paged_kv_read"], seen["beam_attn"]
        assert reads[0][2] is reads[2][2] and reads[0][1] is reads[2][1] and attns[0][6] is attns[2][6]
        for read, attn, c in zip(reads, attns, caches):
            lo = max(1, start - c.window + 1) if c.window else 1
            assert read[2].tolist() == [1, 1, lo, 1] and read[3].tolist() == [0, 0, start + 8, 0]
            assert attn[4] is read[5] and attn[5].tolist() == [2] * 9
            # page 2, positions 33 .. 48, is none in the other table
            sees = [c.page_table is other and p >= 33 and (c.window == 0 or p - c.window + 1 <= 48) for p in pos]
            assert attn[6].tolist() == [0 if bad else p for p, bad in zip(pos, sees)]


@pytest.mark.parametrize("window", [0, 512, 2 ** 31 - 1])
def test_any_position_stays_inside_the_page_table(window):
    """Positions that the library flags, as far out as there are, index nothing outside the table."""
    st, kc = stack(), paged(rows=3, pages=6, page_size=16, window=window)
    far = [-2 ** 31, -2 ** 31 + 5, -600, -1, 0, 2 ** 31 - 1, 97]
    first, last = ints([1] * 3), ints([96] * 3)
    got = st.readable(kc, ints([0, 1, 2, -2 ** 31, 2 ** 31 - 1, 1, 0]), ints(far), first, last, 96)
    assert got.tolist() == far       # left to the library to flag
    seq, pos = ints([0, -2 ** 31, 2 ** 31 - 1, 1, 2, 2]), ints([-2 ** 31, 5, 5, 2 ** 31 - 1, 3, 4])
    for n_seqs in (None, 1):
        copy, every, first, last, longest = st.context(kc, seq, pos, 90, 6, n_seqs)
        row = st.rows(kc, seq, pos, every, first, last)
        st.readable(kc, row, pos, first, last, longest, every)
        assert [int(x) for x in every[last >= first]] == [2] and int(last.max()) == 4


def test_the_sequences_of_a_windowed_call_are_counted_too():
    """A window's rings for 2048 rows of window + chunk slots pass COPY_BYTES as a context does."""
    seq = ints([5] * 2048)
    st = stack([paged(rows=4096, pages=200, window=16)])
    assert st.count(seq, 3000, None, 2048) == 1            # 2048 rings of 2176 slots, 512 bytes each
    assert st.count(seq, 3000, None, 100) is None          # of 128
