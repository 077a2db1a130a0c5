"""Decode attention over pages where value rows of very different magnitudes have very different
weights, against float64 (oracle/paged.py).

Bound per element, as in test_gpu_paged.py but for the f16 floor:
    2^-8 |ref| + W (2 d + r) + n 2^-31 F,   F = max over the row's keys of p max|v|
A quantised cache's P = p 2^e (e: the exponent of the value row's scale) is held in f16 at a
reference that lies at most at the largest p 2^e of the row's keys, which stands at 2^7 there. A P
below f16's smallest step 2^-24 is off by half of it: 2^-32 of that largest p 2^e. It multiplies a
code of at most C = 448 (2688), and C 2^e < 2 max|v| of the row that has the largest p 2^e, since e is the
least that fits: 2^-31 F a key. Values of negligible weight therefore count with their weight.
"""
import numpy as np
import pytest
import torch

from oracle import paged as OP
from hybrid_attention_moe_gb300 import beam as B
from parity import np64
from test_gpu_paged import DEV, FMT, attend, cfg_for, host, ints, randn, status

pytestmark = pytest.mark.gpu


def check(cfg, hc, q, pos, out):
    """One row of sequence 0 at position pos."""
    D, grp = cfg.head_dim, cfg.n_q // cfg.n_kv
    ref, mag = OP.paged_attention(cfg.n_q, q, hc, [0], [pos])
    lo = max(1, pos - hc.window + 1) if hc.window else 1
    K, V = hc.load(0, np.arange(lo, pos + 1))
    worst = 0.0
    for h in range(cfg.n_q):
        k, v, sl = K[h // grp], V[h // grp], slice(h * D, (h + 1) * D)
        x = k @ q[0, h] / np.sqrt(D)
        p = np.exp(x - x.max())
        p /= p.sum()
        d = D * 2.0 ** -23 * np.max(np.abs(k) @ np.abs(q[0, h])) / np.sqrt(D)
        r, floor = 2.0 ** -15, 0.0
        if hc.fmt != "bf16":
            r, floor = r + 2.0 ** -11, len(p) * 2.0 ** -31 * np.max(p * np.abs(v).max(1))
        tol = 2.0 ** -8 * np.abs(ref[0, sl]) + mag[0, sl] * (2 * d + r) + floor
        worst = max(worst, float(np.max(np.abs(out[0, sl] - ref[0, sl]) / tol)))
    print(f"largest error / bound {worst:.3f}")
    assert np.all(np.isfinite(out)) and worst <= 1.0, worst


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("D,G,n,window", [(128, 5, 16384, 0), (64, 12, 5000, 0), (64, 6, 200, 0), (128, 16, 900, 600)])
@pytest.mark.parametrize("big,at", [(20, 0.01), (20, 0.9), (60, 0.5), (100, 0.3)])
def test_value_rows_of_large_magnitude_and_small_weight(fmt, D, G, n, window, big, at):
    """A sink of weight 1, a long tail of 2^-13 each, and one value row 2^big times larger whose
    weight differs by head: nothing, as much as evens its size out, and all of it."""
    cfg = cfg_for(G, 1, D)
    page = 32
    per = -(-n // page)
    order = torch.randperm(per, generator=torch.Generator().manual_seed(1)).tolist()
    c = B.PagedKVCache.empty(per, page, 1, D, ints([order]), FMT[fmt], window)
    first = n - window if window else 0
    row, sink = first + int((n - first) * at), first + 40
    # head h reads its logits off element h of the keys, at a scale that makes the row's all -1 (4-bit
    # keys keep their differences)
    fits = -float(np.log(2.0)) * big
    want = [(-1.4 * big - 41.0, fits, 0.0, -300.0, fits - 6, -69.0)[h % 6] for h in range(G)]
    s = torch.tensor([max(14.0, -x) for x in want])
    logit = torch.full((n, G), -13 * float(np.log(2.0)))
    logit[sink] = 0.0
    logit[row] = torch.tensor(want)
    k = torch.zeros((n, 1, D))
    k[:, 0, :G] = logit / s
    v = randn(301, n, 1, D).float().cpu() * 2.0 ** (-big // 2)
    v[row] *= 2.0 ** big
    k, v = k.to(torch.bfloat16).to(DEV), v.to(torch.bfloat16).to(DEV)
    B.beam_paged_kv_write(k, v, ints([0] * n), ints(list(range(1, n + 1))), c)
    q = torch.zeros((1, G, D), dtype=torch.bfloat16, device=DEV)
    q[0, torch.arange(G), torch.arange(G)] = (s * np.sqrt(D)).to(torch.bfloat16).to(DEV)
    out = attend(cfg, c, q, ints([0]), ints([n]), n)
    assert status() == 0
    check(cfg, host(c), np64(q), n, np64(out))


@pytest.mark.parametrize("D,G,n", [(128, 5, 700), (64, 12, 3000), (128, 16, 90)])
def test_infinities_over_bf16_pages(D, G, n):
    """Keys with an infinity: logits of -inf weigh nothing, +inf makes NaN, all of -inf give zero. A
    value with one makes its element of what reads it infinite or NaN, and no other output."""
    cfg = cfg_for(2 * G, 2, D)
    page, inf = 32, float("inf")
    per = -(-n // page)
    lens = [n, n, n, 3]
    c = B.PagedKVCache.empty(4 * per, page, 2, D, torch.arange(4 * per, dtype=torch.int32, device=DEV).view(4, per))
    seq = [s for s, m in enumerate(lens) for _ in range(m)]
    pos = [p for m in lens for p in range(1, m + 1)]
    k, v = randn(311, len(seq), 2, D), randn(312, len(seq), 2, D)
    q = randn(313, 4, 2 * G, D).abs()
    k[[n // 2, n - 1], 0, 5] = -inf         # sequence 0, KV head 0: two keys of -inf for every query
    k[n + n // 3, 1, 7] = inf               # sequence 1, KV head 1: +inf
    v[2 * n + n // 4, 0, 9] = inf           # sequence 2, KV head 0: an infinite value
    k[3 * n:, 1, 0] = -inf                  # sequence 3, KV head 1: nothing but -inf
    B.beam_paged_kv_write(k, v, ints(seq), ints(pos), c)
    out = np64(attend(cfg, c, q, ints([0, 1, 2, 3]), ints(lens), n)).reshape(4, 2, G, D)
    assert status() == 0
    # the same without those keys and values
    k2, v2 = k.clone(), v.clone()
    k2[torch.isinf(k2)] = 0
    v2[torch.isinf(v2)] = 0
    B.beam_paged_kv_write(k2, v2, ints(seq), ints(pos), c)
    ref = np64(attend(cfg, c, q, ints([0, 1, 2, 3]), ints(lens), n)).reshape(4, 2, G, D)
    assert np.array_equal(out[0, 1], ref[0, 1]) and np.array_equal(out[1, 0], ref[1, 0])
    assert np.all(np.isnan(out[1, 1]))
    hit = ~np.isfinite(out[2, 0])
    assert np.all(hit[:, 9]) and not np.any(np.delete(hit, 9, axis=1))
    assert np.array_equal(np.delete(out[2, 0], 9, axis=1), np.delete(ref[2, 0], 9, axis=1))
    assert np.array_equal(out[2, 1], ref[2, 1]) and np.array_equal(out[3, 0], ref[3, 0])
    assert not np.any(out[3, 1])
    # sequence 0, KV head 0: the other keys' softmax
    keep = np.array([i for i in range(n) if i not in (n // 2, n - 1)])
    K, V = np64(k[:n, 0])[keep], np64(v[:n, 0])[keep]
    for g in range(G):
        qh = np64(q[0, g])
        x = K @ qh / np.sqrt(D)
        p = np.exp(x - x.max())
        p /= p.sum()
        want, mag = p @ V, p @ np.abs(V)
        d = D * 2.0 ** -23 * np.max(np.abs(K) @ np.abs(qh)) / np.sqrt(D)
        assert np.all(np.abs(out[0, 0, g] - want) <= 2.0 ** -8 * np.abs(want) + mag * (2 * d + 2.0 ** -15))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("D,G,big", [(128, 5, 30), (64, 12, 30), (128, 5, 33), (64, 12, 34)])
def test_query_elements_of_very_different_magnitude(fmt, D, G, big):
    """One element of q 2^big times the others, where the keys hold nothing or little: over quantised
    caches the others are f16 relative to it, off by at most 2^-39 of it each (2^14 of f16's 2^-25):
    a logit by 2^-39 max|q| sum|k| / sqrt(D), which joins the bound's d. Up to 2^31 nothing is lost."""
    n = 1500
    cfg = cfg_for(G, 1, D)
    per = -(-n // 64)
    c = B.PagedKVCache.empty(per, 64, 1, D, torch.arange(per, dtype=torch.int32, device=DEV)[None], FMT[fmt])
    k, v = randn(321, n, 1, D), randn(322, n, 1, D)
    k[:, 0, 3] = 0
    if big > 31:
        k[::2, 0, 3] = 2.0 ** -40      # of the BF16 cache only: 0 in a code
    B.beam_paged_kv_write(k, v, ints([0] * n), ints(list(range(1, n + 1))), c)
    q = randn(323, 1, G, D)
    q[0, :, 3] = 2.0 ** big
    out = np64(attend(cfg, c, q, ints([0]), ints([n]), n))
    assert status() == 0
    hc, qn = host(c), np64(q)
    ref, mag = OP.paged_attention(G, qn, hc, [0], [n])
    K, V = (x[0] for x in hc.load(0, np.arange(1, n + 1)))
    for h in range(G):
        sl = slice(h * D, (h + 1) * D)
        d = D * 2.0 ** -23 * np.max(np.abs(K) @ np.abs(qn[0, h])) / np.sqrt(D)
        r, floor = 2.0 ** -15, 0.0
        if fmt != "bf16":
            x = K @ qn[0, h] / np.sqrt(D)
            p = np.exp(x - x.max())
            p /= p.sum()
            r, floor = r + 2.0 ** -11, n * 2.0 ** -31 * np.max(p * np.abs(V).max(1))
            if big > 31:
                d += 2.0 ** -39 * 2.0 ** big * np.max(np.abs(K).sum(1)) / np.sqrt(D)
        # weights e^x: a logit's error d moves a normalised weight by a factor of e^(2d) at most
        tol = 2.0 ** -8 * np.abs(ref[0, sl]) + mag[0, sl] * (np.expm1(2 * d) * (1 + r) + r) + floor
        assert np.all(np.abs(out[0, sl] - ref[0, sl]) <= tol), h


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("qe,ke", [(120, 100), (60, 115), (-120, -100), (-130, 120), (120, -130)])
def test_logits_of_zero_from_large_and_small_factors(fmt, qe, ke):
    """Queries and keys of 2^qe and 2^ke in different elements: every product is 0 whatever their powers
    of two come to together, and the weights are equal."""
    D, G, n = 128, 5, 300
    cfg = cfg_for(G, 1, D)
    c = B.PagedKVCache.empty(10, 32, 1, D, torch.arange(10, dtype=torch.int32, device=DEV)[None], FMT[fmt])
    k, v = torch.zeros((n, 1, D), dtype=torch.bfloat16, device=DEV), randn(332, n, 1, D)
    k[:, 0, 5::2] = 2.0 ** ke
    B.beam_paged_kv_write(k, v, ints([0] * n), ints(list(range(1, n + 1))), c)
    q = torch.zeros((1, G, D), dtype=torch.bfloat16, device=DEV)
    q[0, :, 4::2] = 2.0 ** qe
    out = np64(attend(cfg, c, q, ints([0]), ints([n]), n))
    assert status() == 0
    check(cfg, host(c), np64(q), n, out)
