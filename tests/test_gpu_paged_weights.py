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
