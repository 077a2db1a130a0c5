"""A drafted tree's bookkeeping where a sample failed, node 0 is no root, a context's length is none, or sequences share
pages."""
import numpy as np
import pytest
import torch

from oracle import tree as OT
from hybrid_attention_moe_gb300 import beam as B
from test_gpu_paged import host, ints, make_cache, status

pytestmark = pytest.mark.gpu
DEV = "cuda"


def accept(parent, token, sampled, start=None):
    start = [0, len(parent)] if start is None else start
    N = len(start) - 1
    count, path, nxt = ints([77] * N), torch.full((N, 8), 77, dtype=torch.int32, device=DEV), ints([77] * N)
    B.beam_tree_accept(ints(parent), ints(token), ints(sampled), ints(start), count, path, nxt)
    return count.tolist(), path.tolist(), nxt.tolist()


def same_as_the_oracle(trees):
    start = np.cumsum([0] + [len(t[0]) for t in trees]).tolist()
    got = accept(*(sum((t[i] for t in trees), []) for i in range(3)), start)
    assert status() == 0
    for i, t in enumerate(trees):
        path, after = OT.accept(*t)
        assert (got[0][i], got[1][i], got[2][i]) == (len(path), path + [-1] * (8 - len(path)), after), i


def test_a_failed_sample_names_no_child():
    """-1, which sampling gives where a row has no distribution, ends the path, whatever a drafter filled its tokens with."""
    same_as_the_oracle([([-1, 0, 1], [5, -1, 6], [-1, 6, 7]), ([-1, 0, 1], [5, 4, -1], [4, -1, 7]), ([-1], [-1], [-1]),
                        ([-1, 0, 0, 2], [5, -1, 4, 9], [4, 3, 9, 1]), ([-1, 0], [5, -7], [-7, 1])])
    assert OT.accept([-1, 0, 1], [5, -1, 6], [-1, 6, 7]) == ([0], -1)


def test_a_node_0_that_is_no_root():
    """What the plan leaves out is not accepted."""
    for up in (0, 3, -2, 7):
        same_as_the_oracle([([-1, 0], [1, 2], [2, 3]), ([up, 0, 1, 1], [1, 2, 3, 4], [2, 3, 4, 5]), ([-1, 0], [1, 2], [2, 3])])
        assert OT.accept([up, 0, 1, 1], [1, 2, 3, 4], [2, 3, 4, 5]) == ([], -1)


@pytest.mark.parametrize("base", [-1, -5, -64, -2 ** 31, 2 ** 31 - 1, 2 ** 31 - 64])
def test_a_plan_behind_a_length_that_is_none(base):
    """A negative length (or one whose slots pass 32 bits) would put the tree's later nodes into the slots of real tokens."""
    parent, start = [-1, 0, 1, 2, 3, 4, 5] + [-1, 0] + [-1], [0, 7, 9, 10]
    out = [torch.full((10,), 77, dtype=torch.int64 if x == 0 else torch.int32, device=DEV) for x in range(4)]
    B.beam_tree_plan(ints(parent), ints(start), ints([0, 1, 2]), ints([base, 10, 0]), *out)
    assert status() == B.DEV_BAD_POSITION
    assert out[0].tolist() == [0] * 7 + [1, 3, 1]
    assert out[1].tolist() == [0] * 7 + [11, 12, 1] and out[2].tolist() == [0] * 7 + [11, 12, 1]


def test_a_plan_at_the_last_length():
    out = [torch.full((64,), 77, dtype=torch.int64 if x == 0 else torch.int32, device=DEV) for x in range(4)]
    base = 2 ** 31 - 1 - 64
    B.beam_tree_plan(ints(list(range(-1, 63))), ints([0, 64]), ints([0]), ints([base]), *out)
    assert status() == 0 and out[1].tolist() == out[2].tolist() == list(range(base + 1, 2 ** 31))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_keep_of_sequences_that_share_their_prefix(fmt):
    """Two sequences whose tables name the same pages for their common context: each moves rows of its own pages."""
    c, *_ = make_cache(fmt, 2, 64, 32, [96, 96], 4400)
    c.page_table[1, :2] = c.page_table[0, :2]
    ref, before = host(c), host(c)
    paths = [[0, 3, 4, 9], [1, 2, 7, 20]]
    for s, p in enumerate(paths):
        for i, x in enumerate(p):
            (pa, oa), (pb, ob) = before.place(s, 64 + 1 + x), before.place(s, 64 + 1 + i)
            for name in ("k", "v"):
                getattr(ref, name)[pb, :, ob] = getattr(before, name)[pa, :, oa]
            for name in ("row", "block"):
                if getattr(ref, name) is not None:
                    getattr(ref, name)[pb, :, :, ob] = getattr(before, name)[pa, :, :, oa]
    B.beam_paged_kv_keep(c, ints([0, 1]), ints([64, 64]), ints([4, 4]), ints(paths))
    assert status() == 0
    after = host(c)
    for name in ("k", "v", "row", "block"):
        a, b = getattr(ref, name), getattr(after, name)
        assert a is None or np.array_equal(a, b, equal_nan=a.dtype.kind == "f"), name
