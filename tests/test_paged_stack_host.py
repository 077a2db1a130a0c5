"""What BeamStack works out on the host and in torch for a prefill over paged caches, on the CPU."""
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
