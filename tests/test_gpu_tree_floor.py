"""Tree attention over quantised pages: what the rounding of a weight times its value row's power of two to f16 may cost.

Each such product is off by at most 2^-11 of it, or 2^-32 of the row's largest where that is more. One key of interest has a small
product; another, in the second 32 keys of the same block or in a later one, a far larger one, with a value row that is zero in
the upper half of its columns. There the result is w v of the first key alone, so with the key's code c (v is c times its row's power of
two) and the largest product M it is off by at most 2^-11 w |v| + 2^-32 M |c|, by the weight's own error (2^-15, as for
every row), and by half a bf16 step."""
import numpy as np
import pytest
import torch

from hybrid_attention_moe_gb300 import beam as B
from parity import np64
from test_gpu_paged import cfg_for, host, ints, status
from test_gpu_tree import attend, words
from test_gpu_tree_no_numbers import D, filled

pytestmark = pytest.mark.gpu
DEV = "cuda"


def upper_half(fmt, n, at, v_at, lead, k_lead, v_lead):
    """Columns D/2.. of the only row over n keys, their exact value and the bound. Key `at` has the logit 0 and values v_at, key
    `lead` the logit k_lead and values v_lead in the lower columns; other keys the logit 0 and values of zero."""
    k, v = torch.zeros(n, D, device=DEV), torch.zeros(n, D, device=DEV)
    k[lead, 0] = k_lead
    v[at] = v_at
    v[lead, :D // 2] = v_lead
    c = filled(fmt, k, v)
    q = torch.zeros((1, 1, D), device=DEV, dtype=torch.bfloat16)
    q[0, 0, 0] = D ** 0.5
    out = attend(cfg_for(1, 1, D), c, q, ints([0]), ints([0, 1]), ints([n - 1]), words([{0}]), n)
    assert status() == 0
    hc = host(c)
    K, V = (x[0] for x in hc.load(0, np.arange(1, n + 1)))
    x = K[:, 0]
    w = np.exp(x - x.max())
    unit = np.array([2.0 ** (int(hc.row[int(hc.table[0, i // 32]), 0, 1, i % 32]) - 127) for i in range(n)])
    most = float(np.max(w * unit)) / w.sum()
    w /= w.sum()
    ref = w @ V
    assert not V[lead, D // 2:].any() and ref[-1] == w[at] * V[at, -1] != 0
    tol = (2.0 ** -11 + 2.0 ** -15 + 2.0 ** -8) * np.abs(ref) + 2.0 ** -32 * most * np.abs(V[at] / unit[at])
    o = np64(out)[0]
    low = np.abs(o - ref)[:D // 2] <= (2.0 ** -8 + 2.0 ** -10) * np.abs(ref)[:D // 2]
    assert low.all()
    return o[D // 2:], ref[D // 2:], tol[D // 2:]


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("n,at,lead", [(63, 3, 40), (64, 31, 32), (63, 40, 3), (300, 10, 290), (300, 70, 170)])
@pytest.mark.parametrize("e", [5, 12, 20, 24, 25, 26, 27, 28, 29, 30])
def test_small_value_rows_beside_large_ones(fmt, n, at, lead, e):
    for sign in (1.0, -1.5):
        o, ref, tol = upper_half(fmt, n, at, sign, lead, 0.0, 2.0 ** e)
        assert np.all(np.abs(o - ref) <= tol), (float(np.max(np.abs(o - ref) / np.abs(ref))), float(np.max(tol / np.abs(ref))))
        assert e > 29 or np.all(o * ref > 0)


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("n,at,lead", [(63, 3, 40), (64, 31, 32), (63, 40, 3), (300, 10, 290), (300, 70, 170)])
@pytest.mark.parametrize("x", [6.0, 12.0, 16.0, 18.0, 20.0])
def test_small_weights_beside_large_ones(fmt, n, at, lead, x):
    o, ref, tol = upper_half(fmt, n, at, 3.0, lead, x, 1.0)
    assert np.all(np.abs(o - ref) <= tol), (float(np.max(np.abs(o - ref) / np.abs(ref))), float(np.max(tol / np.abs(ref))))
    assert np.all(o > 0)


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
@pytest.mark.parametrize("n,lead", [(63, 40), (63, 20), (300, 40), (300, 130), (300, 200)])
@pytest.mark.parametrize("e", range(4, 20))
def test_products_that_rise_beside_a_row_that_sees_nothing(fmt, n, lead, e):
    """Rows without keys have the references looked at in every block, and a row beside them moves its own only where its products
    have risen enough: up to there P has to be a number of f16. Keys of equal logits, one value row 2^e times the others."""
    k, v = torch.zeros(n + 2, D, device=DEV), torch.ones(n + 2, D, device=DEV)
    v[lead, :D // 2] = 2.0 ** e
    v[lead, D // 2:] = -(2.0 ** e)
    c = filled(fmt, k, v)
    q = torch.zeros((3, 1, D), device=DEV, dtype=torch.bfloat16)
    out = attend(cfg_for(1, 1, D), c, q, ints([0]), ints([0, 3]), ints([n - 1]), words([{0}, set(), {0, 2}]), n + 2)
    assert status() == 0
    V = host(c).load(0, np.arange(1, n + 1))[1][0]
    o, ref = np64(out), V.mean(0)
    assert np.all(np.abs(o[0] - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -15) * np.abs(V).mean(0))
    V = np.concatenate([V, host(c).load(0, np.array([n + 2]))[1][0]])
    ref = V.mean(0)
    assert not o[1].any() and np.all(np.abs(o[2] - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -15) * np.abs(V).mean(0))
