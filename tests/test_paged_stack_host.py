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
