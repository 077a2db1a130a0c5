"""Tree attention over pages: NaN and infinities that reach a row from one of the two streams, which take an item's blocks of 64
keys in turn, alone; and rows that see nothing beside gates that hold no numbers."""
import numpy as np
import pytest
import torch

from oracle import tree as OT
from hybrid_attention_moe_gb300 import beam as B
from parity import np64
from test_gpu_paged import FMT, cfg_for, host, ints, randn, status
from test_gpu_tree import attend, case, check, run, words

pytestmark = pytest.mark.gpu
DEV = "cuda"
D = 64
NAN, INF = float("nan"), float("inf")


def filled(fmt, k, v, window=0):
    """A cache of one sequence and one head with keys k and values v, from slot 1 on."""
    n = k.shape[0]
    pages = -(-n // 32) + 1
    c = B.PagedKVCache.empty(pages, 32, 1, D, ints([list(range(pages))]), FMT[fmt], window)
    i = torch.arange(1, n + 1, dtype=torch.int32, device=DEV)
    B.beam_paged_kv_write(k.view(n, 1, D).to(torch.bfloat16), v.view(n, 1, D).to(torch.bfloat16), torch.zeros_like(i), i, c)
    return c


def finite_as_the_oracle(fmt, k, v, q, base, window=0):
    """The rows of a chain of len(q) nodes behind `base` keys, and which elements the oracle says are numbers."""
    c = filled(fmt, k, v, window)
    n = q.shape[0]
    nodes = [set(range(j + 1)) for j in range(n)]
    out = attend(cfg_for(1, 1, D), c, q.to(torch.bfloat16), ints([0]), ints([0, n]), ints([base]), words(nodes), base + n)
    assert status() == 0
    with np.errstate(invalid="ignore"):
        ref = OT.tree_attention(1, np64(q.to(torch.bfloat16)), host(c), 0, base, nodes)[0]
    assert np.array_equal(np.isfinite(np64(out)), np.isfinite(ref))
    return np64(out), ref


def rows(n, seed):
    return randn(seed, n, D).float(), randn(seed + 1, n, D).float()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("base", [64, 128, 192, 2560])
def test_a_stream_of_nothing_but_nan_logits(fmt, base):
    """The last block's only key is the node's own, and its key row is NaN: the other stream's finite logits do not hide it. (At
    2,560 keys the item is cut into ranges.) The same with a NaN in q."""
    k, v = rows(base + 1, 10)
    q = randn(12, 1, 1, D).float()
    k[base, 5] = NAN
    out, _ = finite_as_the_oracle(fmt, k, v, q, base)
    assert np.isnan(out).all()
    k[base, 5] = 0
    q[0, 0, 7] = NAN
    out, _ = finite_as_the_oracle(fmt, k, v, q, base)
    assert np.isnan(out).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_a_row_that_sees_one_stream_only(fmt):
    """A window of one key: the second node sees itself alone, in the second block, the first one itself, in the first."""
    k, v = rows(65, 20)
    q = randn(22, 2, 1, D).float()
    _, ref = finite_as_the_oracle(fmt, k, v, q, 63, window=1)
    assert np.isfinite(ref).all()
    k[64, 0] = NAN
    out, _ = finite_as_the_oracle(fmt, k, v, q, 63, window=1)
    assert np.isfinite(out[0]).all() and np.isnan(out[1]).all()
    k[64, 0] = 1
    q[1, 0, 3] = NAN
    out, _ = finite_as_the_oracle(fmt, k, v, q, 63, window=1)
    assert np.isfinite(out[0]).all() and np.isnan(out[1]).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("base,spot,lead", [(64, 5, 64), (129, 70, 3), (129, 5, 70)])
def test_values_of_a_stream_that_the_other_outweighs(fmt, bad, base, spot, lead):
    """A value that is no number, in a block whose keys weigh e^-512 of one in the other stream's."""
    k, v = torch.zeros(base + 1, D, device=DEV), randn(30, base + 1, D).float()
    k[lead] = 8.0
    q = torch.full((1, 1, D), 8.0, device=DEV)
    v[spot, 3] = bad
    out, ref = finite_as_the_oracle(fmt, k, v, q, base)
    assert not np.isfinite(out[0, 3]) and np.isfinite(out).any() == (fmt == "bf16")
    v[spot, 3] = 0
    out, ref = finite_as_the_oracle(fmt, k, v, q, base)
    # where the leading value is 0 the others' are due, e^-512 of values below 2^3: FP32 loses weights below 2^-126, so that up to
    # 130 keys come to less than 2^-115 in all
    assert np.all(np.abs(out - ref) <= (2.0 ** -8 + 2.0 ** -11) * np.abs(ref) + 2.0 ** -115)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("base", [100, 20000])
def test_gates_of_rows_that_see_nothing(fmt, base):
    """Rows of a tree with mask 0, rows outside all trees and rows without a page give zero, whatever their gates hold; at 20,000
    keys the item is cut into ranges, whose parts are joined."""
    k = case(fmt, 6, 2, 128, 32, [base, 40], [9, 5], 3700, pad=(1, 2), spread=0)
    nodes = [set() if i in (3, 6) else x for i, x in enumerate(k["nodes"])]
    clean = run(k, nodes)
    check(k["cfg"], k["c"], k["q"], k["seq"], k["start"], k["base"], nodes, clean, k["g"], k["bias"], only=[0, 1] if base == 100 else [1])
    idle = [0, 3, 6, 15, 16]
    for x in (NAN, INF, -INF):
        g = k["g"].clone()
        g[idle] = x
        out = run(k, nodes, g=g)
        assert status() == 0 and torch.equal(out, clean) and not out[idle].any()
    bias = k["bias"].clone()
    bias[1] = NAN
    out = run(k, nodes, bias=bias).view(-1, 6, 128)
    assert status() == 0 and not out[idle].any() and torch.isnan(out[[1, 2, 10], 1]).all()
    k["c"].page_table[1] = -1          # the second sequence has no page at all
    g = k["g"].clone()
    g[10:15] = NAN
    out = run(k, nodes, g=g)
    assert status() == B.DEV_BAD_PAGE and not out[10:15].any() and torch.equal(out[:10], clean[:10])


@pytest.mark.parametrize("base", [64, 65, 127, 128, 2560, 2561])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_a_value_beside_a_logit_of_minus_infinity(base, bad):
    """It is the row's like any other that it reads, wherever the item is cut: the key of -inf is the last block's only one at 64, 128
    and 2,560 keys. The other columns are as if the key were not there."""
    k, v = rows(base + 1, 40)
    q = randn(42, 1, 1, D).float()
    q[0, 0, 0] = -1.0
    k[base, 0] = INF
    clean, _ = finite_as_the_oracle("bf16", k, v, q, base)
    v[base, 3] = bad
    out, ref = finite_as_the_oracle("bf16", k, v, q, base)
    assert not np.isfinite(out[0, 3]) and np.array_equal(np.delete(out, 3, 1), np.delete(clean, 3, 1))


def test_a_row_of_logits_of_minus_infinity_alone():
    """Zero, but for a value that is no number."""
    k, v = rows(65, 50)
    q = randn(52, 2, 1, D).to(torch.bfloat16)
    q[1, 0, 0] = -1.0
    k[64, 0] = INF
    v[64, 7] = NAN
    out = attend(cfg_for(1, 1, D), filled("bf16", k, v, 1), q, ints([0]), ints([0, 2]), ints([63]), words([{0}, {0, 1}]), 65)
    out = np64(out)
    assert status() == 0 and np.isfinite(out[0]).all() and np.isnan(out[1, 7]) and not np.delete(out[1], 7).any()


@pytest.mark.parametrize("base,first,last,spot", [(128, 64, 128, 70), (128, 0, 64, 5), (2560, 0, 1280, 100), (2560, 1280, 2560, 1300)])
@pytest.mark.parametrize("bad", [NAN, INF])
def test_whole_blocks_of_logits_of_minus_infinity(base, first, last, spot, bad):
    """All keys of a stream's blocks, or of a range's, weigh nothing, and one's value is no number."""
    k, v = rows(base + 1, 60)
    q = randn(62, 1, 1, D).float()
    q[0, 0, 0] = -1.0
    k[first:last, 0] = INF
    clean, _ = finite_as_the_oracle("bf16", k, v, q, base)
    assert np.isfinite(clean).all()
    v[spot, 3] = bad
    out, ref = finite_as_the_oracle("bf16", k, v, q, base)
    assert not np.isfinite(out[0, 3]) and np.array_equal(np.delete(out, 3, 1), np.delete(clean, 3, 1))
