"""Decode attention over pages in the forms that a CTA takes: pairs of up to eight blocks whole,
several to a CTA and shared by its groups, with and without a finisher; split pairs; every head
layout; with the gate. Against float64 with the bounds of test_gpu_paged.py."""
import pytest
import torch

from test_gpu_paged import attend, cfg_for, check_attn, ints, make_cache, randn, status

pytestmark = pytest.mark.gpu


def run(fmt, n_q, n_kv, D, page, lens, window=0, bound=None, seed=501):
    cfg = cfg_for(n_q, n_kv, D)
    c, *_ = make_cache(fmt, n_kv, D, page, lens, seed, window=window)
    T = len(lens)
    q, g, bias = randn(seed + 1, T, n_q, D), randn(seed + 2, T, n_q * D), randn(seed + 3, n_q)
    seq, pos = ints(list(range(T))), ints(lens)
    out = attend(cfg, c, q, seq, pos, max(lens) if bound is None else bound, g, bias)
    assert status() == 0
    check_attn(cfg, c, q, seq, pos, out, g, bias)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("D,G", [(128, 6), (128, 16), (64, 3), (64, 12)])
def test_short_pairs_several_to_a_cta(fmt, D, G):
    """More pairs than CTAs, of 1 to 4 blocks and a few keys each."""
    lens = [1 + (37 * i) % 250 for i in range(70)]
    run(fmt, 8 * G, 8, D, 32, lens)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("D,G", [(128, 6), (128, 16), (64, 3), (64, 12)])
@pytest.mark.parametrize("n", [500, 1000])
def test_pairs_of_five_to_eight_blocks(fmt, D, G, n):
    """A batch with pairs enough for every SM (whole pairs where blocks hold 128 or 64 keys, split ones
    else), full attention and as a window in longer sequences, with rows that see nothing."""
    run(fmt, 4 * G, 4, D, 64, [n - (53 * i) % (n // 2) for i in range(60)])
    lens = [n + 300 + (91 * i) % 400 for i in range(56)] + [5, n]
    run(fmt, 4 * G, 4, D, 16 if (fmt, D) != ("nvfp4", 64) else 32, lens, window=n - 11)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("n_q,n_kv,D", [(9, 1, 64), (32, 2, 64), (11, 1, 128), (24, 2, 64)])
def test_nine_to_sixteen_heads_gated(fmt, n_q, n_kv, D):
    """Two tiles of heads: one short pair, and long pairs split over the ranges."""
    run(fmt, n_q, n_kv, D, 128, [40])
    run(fmt, n_q, n_kv, D, 128, [9000, 1, 4100, 130], bound=9001)
