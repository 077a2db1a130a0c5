"""The stack over paged caches: prefill, a second chunk and decode steps through BeamStack, as a
server runs them, with sequences of unequal lengths whose pages lie anywhere in the pools.

With BF16 pages the keys and values are those of the contiguous caches, so the prefill, which
reads them back for the same attention, has to give the same bits. Every step's attention and
o_proj is recomputed by the oracle from exactly what the GPU's step had (its q, g and pages).

Bounds. The gated output og is within tol of the 64-bit one (test_gpu_paged.py derives tol; the
prefill attention of beam_attn rounds o once more before the gate: half a bf16 step, 2^-8 |og|,
and carries P in bf16 halves like the decode over bf16 pages). o_proj is linear, so
    |out - ref| <= tol |W_o|^T + n 2^-23 |og| |W_o|^T + 2^-8 |ref|
with n = n_q D exact products summed in FP32 and one rounding of the result."""
import numpy as np
import pytest
import torch

import synth
from oracle import paged as OP
from oracle.codecs import bf16_round
from synth import TINY
from hybrid_attention_moe_gb300 import beam as B
from hybrid_attention_moe_gb300.stack import BeamStack, is_nope_layer
from parity import np64
from test_gpu_paged import FMT, cfg_for, host, ints, status, tolerance

pytestmark = pytest.mark.gpu
DEV = "cuda"
SEQS, PAGE, PAGES = 3, 32, 6     # pages of a sequence


def weights(seed=0):
    return [{k: v.to(DEV) for k, v in synth.layer_weights(TINY, l, seed).items()}
            for l in range(TINY.n_layers)]


def windows():
    L = TINY.n_layers
    return [0 if is_nope_layer(l, L) else TINY.window for l in range(L)]


def paged_caches(fmt):
    order = torch.randperm(SEQS * PAGES, generator=torch.Generator().manual_seed(3))
    table = order.view(SEQS, PAGES).to(torch.int32).to(DEV)
    return [B.PagedKVCache.empty(SEQS * PAGES, PAGE, TINY.n_kv, TINY.head_dim, table, FMT[fmt], w)
            for w in windows()]


def contiguous_caches(tokens):
    out = []
    for w in windows():
        cap = PAGE * PAGES if w == 0 else (w - 1 + tokens + 127) // 128 * 128
        dims = (SEQS, TINY.n_kv, cap, TINY.head_dim)
        out.append(B.KVCache(*(torch.zeros(dims, dtype=torch.bfloat16, device=DEV) for _ in "kv"), window=w))
    return out


def check_attention(W, cache, t, seq, pos, what, twice=False):
    """One layer's attention output t["attn"] against the oracle on its own inputs."""
    hc, q, w = host(cache), np64(t["q"]), np64(W["w_o"])
    og, mag = OP.paged_attention(TINY.n_q, q, hc, seq, pos, np64(t["g"]), np64(W["gate_bias"]))
    tol = tolerance(cfg_for(TINY.n_q, TINY.n_kv, TINY.head_dim), hc, q, seq, pos, og, mag)
    if twice:
        tol += 2.0 ** -8 * np.abs(og)
    ref = og @ w.T
    bound = tol @ np.abs(w).T + og.shape[1] * 2.0 ** -23 * (np.abs(og) @ np.abs(w).T) + 2.0 ** -8 * np.abs(ref)
    worst = float(np.max(np.abs(np64(t["attn"]) - ref) / bound))
    print(f"{what}: largest error / bound {worst:.3f}")
    assert worst <= 1.0, what


CHUNKS = [([0] * 40 + [2] * 17, list(range(1, 41)) + list(range(1, 18)), 40),   # two sequences' prompts
          ([1] * 33 + [0] * 9, list(range(1, 34)) + list(range(41, 50)), 33)]   # a third's, and more of one
STEPS = [([0, 1, 2], [50, 34, 18]), ([2, 0, 1], [19, 51, 35]), ([1], [36]),
         ([0, 0, 0, 1], [52, 53, 54, 37])]                                       # the last: drafted tokens


def tokens(seq, pos, call):
    e = synth.activations(len(seq), TINY.hidden, 40 + call, "embed").to(DEV)
    return e, ints(seq), ints(pos)


def prefill(st):
    out = []
    for n, (seq, pos, most) in enumerate(CHUNKS):
        e, s, p = tokens(seq, pos, n)
        out.append(st.forward(e, s, p, max(pos), max_q_per_seq=most).clone())
    return out


def test_prefill_over_bf16_pages_is_the_contiguous_one():
    W = weights()
    a = prefill(BeamStack(TINY, W, paged_caches("bf16")))
    b = prefill(BeamStack(TINY, W, contiguous_caches(40)))
    assert status() == 0
    for x, y in zip(a, b):
        assert torch.equal(x, y)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_prefill_then_decode_steps(fmt):
    W = weights()
    st = BeamStack(TINY, W, paged_caches(fmt))
    h = prefill(st)
    assert status() == 0 and all(torch.isfinite(x.float()).all() for x in h)
    for n, (seq, pos) in enumerate(STEPS):
        e, s, p = tokens(seq, pos, 10 + n)
        trace = []
        most = max(seq.count(x) for x in seq)
        st.forward(e, s, p, max(pos), trace=trace, max_q_per_seq=most)
        assert status() == 0
        for l, t in enumerate(trace):
            check_attention(W[l], st.caches[l], t, seq, pos, f"step {n} L{l}.attn {fmt}")


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_prefill_reads_what_the_pages_hold(fmt):
    """The copy that the prefill's attention read holds the pages' values, and its attention is
    the oracle's over them."""
    W = weights()
    st = BeamStack(TINY, W, paged_caches(fmt))
    prefill(st)
    seq, pos, most = CHUNKS[1]
    e, s, p = tokens(seq, pos, 1)
    trace = []
    st.forward(e, s, p, max(pos), trace=trace, max_q_per_seq=most)
    assert status() == 0
    for l, t in enumerate(trace):
        hc = host(st.caches[l])
        check_attention(W[l], st.caches[l], t, seq, pos, f"prefill L{l}.attn {fmt}", twice=True)
        copy = st._copies[(SEQS, hc.window)]
        # the copy is shared by the layers of a window: the last of them is in it
        if l == max(i for i in range(TINY.n_layers) if windows()[i] == hc.window):
            lo = 1 if hc.window == 0 else max(1, 41 - hc.window + 1)
            K, V = hc.load(0, np.arange(lo, 50))
            slots = (np.arange(lo, 50) - 1) % copy.k.shape[2]
            assert np.array_equal(np64(copy.k)[0][:, slots], bf16_round(K))
            assert np.array_equal(np64(copy.v)[0][:, slots], bf16_round(V))


def test_captured_decode_step_equals_the_eager_one():
    W = weights()
    runs = []
    for captured in (False, True):
        st = BeamStack(TINY, W, paged_caches("fp8"))
        prefill(st)
        e, s, p = tokens(*STEPS[0], 10)
        st.forward(e, s, p, 64, max_q_per_seq=1)      # buffers exist before a capture
        out = []
        if captured:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                h = st.forward(e, s, p, 64, max_q_per_seq=1)
        for n in range(3):
            e2, s2, p2 = tokens([0, 1, 2], [50 + n, 34 + n, 18 + n], 20 + n)
            for x, y in ((e, e2), (s, s2), (p, p2)):
                x.copy_(y)
            if captured:
                graph.replay()
            else:
                h = st.forward(e, s, p, 64, max_q_per_seq=1)
            out.append(h.clone())
        runs.append(out)
    assert status() == 0
    for x, y in zip(*runs):
        assert torch.equal(x, y)


@pytest.mark.parametrize("bad", [(0, 0), (1, -3), (-1, 5), (SEQS, 5)])
def test_a_bad_token_of_a_chunk_leaves_the_others_as_they_are(bad):
    """(sequence, position) of a token that the library flags, last of a chunk: the other tokens'
    results are those beside a good one of a third sequence."""
    W = weights()
    runs = []
    for last in ((2, 18), bad):
        st = BeamStack(TINY, W, paged_caches("fp8"))
        prefill(st)
        seq, pos = [1] * 30 + [0] * 30 + [last[0]], list(range(34, 64)) + list(range(50, 80)) + [last[1]]
        e, s, p = tokens(seq, pos, 7)
        runs.append(st.forward(e, s, p, max(pos), max_q_per_seq=30)[:60].clone())
        assert bool(status()) == (last is bad)
    assert torch.equal(*runs)


def test_paged_buffers_belong_to_the_stream_of_the_call():
    st = BeamStack(TINY, weights(), paged_caches("fp8"))
    side, seen = torch.cuda.Stream(), []
    for name in ("stage", "context"):
        def wrapped(*a, _f=getattr(st, name)):
            seen.append(torch.cuda.current_stream())
            return _f(*a)
        setattr(st, name, wrapped)
    e, s, p = tokens([0] * 9, list(range(1, 10)), 3)
    torch.cuda.synchronize()
    st.forward(e, s, p, 9, stream=side, max_q_per_seq=9)
    torch.cuda.synchronize()
    assert len(seen) == 2 * TINY.n_layers and all(x == side for x in seen)
