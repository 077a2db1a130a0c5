"""GPU parity of a step of speculative decoding over the paged cache against float64 NumPy
(oracle/tree.py), at the sizes, masks and values where it can go wrong.

Tree attention: |out - ref| <= 2^-8 |ref| (half a bf16 step, the one rounding of the result) plus
W (2 d + r), W = sum p|v| (64 bits, gated). d bounds the logit error: D products summed in FP32,
each sum off by at most 2^-23 of the sum of magnitudes: d = D 2^-23 max_i sum|q k_i| / sqrt(D). r
bounds the relative error of a weight and of the sum of O: 2^-15 for P in two bf16 halves (2^-17), exp2
(2^-21), the joins and the row sums, and 2^-24 of the running sum for each accumulating MMA, two per 16 keys,
at most 1024 of them before a flush; flushed parts add up in FP32. Over quantised pages the codes are exact in f16 and P,
the weight times its value row's power of two, is rounded to f16 once: half a step, 2^-11, more to r, and the f16 floor: a
P below f16's smallest step 2^-24 is off by half of it where the largest of the row is 2^7 or more, so by 2^-32 of the
largest weighted value max|v| for each of the row's keys. q's f16 values are exact down to 2^-31 of the row's largest
magnitude, and below off by 2^-39 of it: far below d. A weight below FP32's smallest normal 2^-126 (relative to the running max, which is the largest logit's or
less) is lost, and so is a low half below it: 2^-125 max|v| for each of the row's keys; a result below bf16's normal
range is off by half its step there, 2^-134. The gate's sigmoid is within 2^-20 and scales what it gates.

Append: q' and k' are FP32 results rounded to bf16 once: 2^-8 |x| and the error before it, which is bounded
per pair (x, y) of the rotation: norm 2^-20, sine and cosine 2^-22 (the angle is reduced in double; sincosf is within
two units), products and their sum 2^-23 each: 2^-19 (|x| + |y|). Codes are exact functions of the bf16 rows that
the test takes back from the pages of a BF16 cache. Bookkeeping and moves are exact."""
import numpy as np
import pytest
import torch

import synth
from oracle import paged as OP
from oracle import tree as OT
from synth import TINY
from hybrid_attention_moe_gb300 import beam as B
from hybrid_attention_moe_gb300.stack import BeamStack
from parity import np64
from test_gpu_paged import FMT, cfg_for, gen, host, ints, make_cache, randn, status
from test_gpu_paged_stack import PAGE, PAGES, SEQS, paged_caches, weights

pytestmark = pytest.mark.gpu
DEV = "cuda"


def random_tree(seed, n):
    r = np.random.default_rng(seed)
    return [-1] + [int(r.integers(max(0, j - 9), j)) for j in range(1, n)] if n else []


def words(nodes):
    return torch.tensor([OT.bits(x) for x in nodes], dtype=torch.int64, device=DEV)


def attend(cfg, c, q, seq, start, base, mask, most, g=None, bias=None, w_o=None, stream=None, ws=None, out=None):
    T = q.shape[0]
    width = cfg.hidden if w_o is not None else cfg.n_q * cfg.head_dim
    if out is None:
        out = torch.full((T, width), 7.0, dtype=torch.bfloat16, device=DEV)
    if ws is None:
        ws = torch.full((B.paged_tree_workspace_bytes(cfg, T),), 255, dtype=torch.uint8, device=DEV)
    B.beam_paged_tree_attn(cfg, q, g, bias, c, seq, start, base, mask, most, w_o, out, ws, stream)
    return out


def bound(cfg, fmt, ref, mag, counts, logit, most):
    D = cfg.head_dim
    r = 2.0 ** -15 + (0.0 if fmt == "bf16" else 2.0 ** -11) + np.minimum(counts / 8 + 2, 1024) * 2.0 ** -24
    d = D * 2.0 ** -23 * logit
    floor = counts[:, None] * (2.0 ** -125 if fmt == "bf16" else 2.0 ** -32) * most + 2.0 ** -133
    return 2.0 ** -8 * np.abs(ref) + mag * np.repeat(2 * d + r[:, None], D, axis=1) + np.repeat(floor, D, axis=1)


def check(cfg, c, q, seq, start, base, nodes, out, g=None, bias=None, only=None):
    """Rows of `out` against the oracle; nodes: a set per row. Rows of no tree are zero."""
    hc, o, qq = host(c), np64(out), np64(q)
    gg, bb = (None, None) if g is None else (np64(g), np64(bias))
    seen = np.zeros(q.shape[0], bool)
    worst = 0.0
    for i in range(len(seq)):
        a, b = start[i], start[i + 1]
        seen[a:b] = True
        if only is not None and i not in only:
            continue
        ref, *sizes = OT.tree_attention(cfg.n_q, qq[a:b], hc, seq[i], base[i], nodes[a:b],
                                                    None if gg is None else gg[a:b], bb)
        err, tol = np.abs(o[a:b] - ref), bound(cfg, hc.fmt, ref, *sizes)
        assert np.array_equal(np.isfinite(o[a:b]), np.isfinite(ref))
        fin = np.isfinite(ref)
        if fin.any():
            worst = max(worst, float(np.max(err[fin] / np.maximum(tol[fin], 1e-300))))
        assert np.all(err[fin] <= tol[fin]), (i, worst)
    assert not o[~seen].any()
    print(f"tree attention: largest error / bound {worst:.3f}")


def case(fmt, n_q, n_kv, D, page, bases, sizes, seed, window=0, gate=True, spread=2, pad=(0, 0), order=None):
    """A cache of the sequences' contexts and trees, and a call over it."""
    order = list(range(len(bases))) if order is None else order
    lens = [0] * len(bases)
    for i, s in enumerate(order):
        lens[s] = bases[i] + sizes[i]
    c, *_ = make_cache(fmt, n_kv, D, page, lens, seed, window, spread)
    start = [pad[0]]
    for n in sizes:
        start.append(start[-1] + n)
    T = start[-1] + pad[1]
    parents = [random_tree(seed + i, n) for i, n in enumerate(sizes)]
    nodes = [set()] * pad[0] + [x for p in parents for x in OT.masks(p)] + [set()] * pad[1]
    cfg = cfg_for(n_q, n_kv, D)
    q = randn(seed + 90, T, n_q, D)
    g = randn(seed + 91, T, n_q * D) if gate else None
    bias = randn(seed + 92, n_q) if gate else None
    return dict(cfg=cfg, c=c, q=q, seq=order, start=start, base=list(bases), nodes=nodes, g=g, bias=bias, most=max(lens),
                parents=parents)


def run(k, nodes=None, **kw):
    n = k["nodes"] if nodes is None else nodes
    return attend(k["cfg"], k["c"], k["q"], ints(k["seq"]), ints(k["start"]), ints(k["base"]), words(n), k["most"],
                  kw.pop("g", k["g"]), kw.pop("bias", k["bias"]), **kw)


def verify(k, nodes=None, only=None):
    n = k["nodes"] if nodes is None else nodes
    out = run(k, n)
    assert status() == 0
    check(k["cfg"], k["c"], k["q"], k["seq"], k["start"], k["base"], n, out, k["g"], k["bias"], only)
    return out


# -------------------------------------------------------------------- tree attention ----

@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("n_q,n_kv,D,page", [(12, 2, 128, 16), (6, 1, 128, 64), (8, 2, 64, 32), (16, 1, 64, 256),
                                             (3, 3, 128, 128), (32, 2, 128, 32)])
def test_attention_matches_the_oracle(fmt, n_q, n_kv, D, page):
    """Trees of one to 64 nodes (rows at and around whole tiles of 128), contexts that end at, before and
    behind a block's end, one of nothing, sequences in another order, an empty tree, padding rows on both sides."""
    verify(case(fmt, n_q, n_kv, D, page, [0, 1, 63, 64, 130, 700, 5], [1, 5, 21, 22, 0, 64, 43], 1000 + n_q + D,
                pad=(3, 2), order=[4, 2, 6, 0, 1, 5, 3]))


@pytest.mark.parametrize("n", [1, 8, 9, 16, 17, 24, 25, 63, 64])
def test_attention_at_tile_edges(n):
    """16 heads a KV head: 8 nodes fill a tile."""
    verify(case("bf16", 16, 1, 64, 16, [77], [n], 1100 + n))
    verify(case("fp8", 16, 1, 128, 16, [300], [n], 1200 + n, gate=False))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("window", [1, 3, 17, 64, 65, 512])
def test_attention_window(fmt, window):
    """A window takes context keys and far ancestors from each row by its own depth; pages before the window
    are gone."""
    k = case(fmt, 6, 2, 128, 32, [0, 2, 40, 900], [9, 64, 30, 50], 1300 + window, window=window)
    table = k["c"].page_table
    for s, b in enumerate(k["base"]):
        gone = max(0, b + 2 - window - 1) // 32
        table[s, :gone] = -3
    verify(k)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_attention_masks_of_any_kind(fmt):
    """Masks that no tree has: nothing, the last node alone, every node, later nodes; bits past the tree's
    size are ignored."""
    k = case(fmt, 4, 2, 64, 32, [50, 0, 129], [40, 64, 6], 1400)
    r = np.random.default_rng(7)
    nodes = []
    for n in (40, 64, 6):
        for j in range(n):
            nodes.append([set(), {n - 1}, set(range(n)), set(np.nonzero(r.random(n) < 0.3)[0].tolist())][j % 4])
    out = verify(k, nodes)
    assert not out[0].any()
    more = [x | ({45, 63} if i < 40 else set()) for i, x in enumerate(nodes)]
    more = [x if nodes[i] else set() for i, x in enumerate(more)]
    assert torch.equal(run(k, more), out)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_attention_leaves_bad_pages_out(fmt):
    k = case(fmt, 6, 2, 128, 16, [300, 70], [20, 12], 1500)
    k["c"].page_table[0, 3], k["c"].page_table[0, 18], k["c"].page_table[1, 0] = 10 ** 6, -1, -5
    out = run(k)
    assert status() == B.DEV_BAD_PAGE
    check(k["cfg"], k["c"], k["q"], k["seq"], k["start"], k["base"], k["nodes"], out, k["g"], k["bias"])
    k["c"].page_table[1] = -1          # no page at all: nothing to see
    out = run(k)
    assert status() == B.DEV_BAD_PAGE and not out[20:].any()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_bad_sequences_are_zero(fmt):
    k = case(fmt, 4, 2, 64, 32, [40, 40, 40, 40], [3, 5, 4, 6], 1600)
    good = run(k)
    assert status() == 0
    reach = k["c"].positions
    for name, i, x, bit in (("seq", 1, 4, 2), ("seq", 1, -1, 2), ("base", 2, -1, 1), ("base", 0, reach - 2, 1),
                            ("base", 3, 2 ** 31 - 1, 1)):
        bad = {**k, name: k[name][:i] + [x] + k[name][i + 1:], "most": 2 ** 31 - 1}
        out = run(bad)
        assert status() == bit, (name, x)
        a, b = k["start"][i], k["start"][i + 1]
        assert not out[a:b].any() and torch.equal(out[:a], good[:a]) and torch.equal(out[b:], good[b:])
    out = run({**k, "most": 44})                       # a bound that the last three pass
    assert status() == 1 and torch.equal(out[:3], good[:3]) and not out[3:8].any() and torch.equal(out[8:12], good[8:12])
    # a tree of more than 64 rows, rows past the call's, a row_start that decreases
    big = case("bf16", 2, 1, 64, 16, [10], [64], 1601, pad=(0, 1))
    big["start"] = [0, 65]
    assert not run(big).any() and status() == 2
    # (in the second the first tree's nine rows pass the bound of 46 as well)
    for start, bits in (([0, 3, 8, 12, 19], 2), ([0, 9, 8, 12, 18], 3), ([-2, 3, 8, 12, 18], 2)):
        run({**k, "start": start})
        assert status() == bits


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("qe,ke,ve", [(0, 0, 100), (40, -40, -100), (-60, 60, 0), (6, 0, 0)])
def test_attention_magnitudes(fmt, qe, ke, ve):
    """Large, small and peaked logits and values whose magnitudes leave f16's range."""
    n_q, n_kv, D, n = 6, 2, 64, 400
    k = case(fmt, n_q, n_kv, D, 32, [n - 20], [20], 1700, gate=False)
    kk, vv = (randn(1701 + i, n, n_kv, D, spread=3).float() * 2.0 ** e for i, e in enumerate((ke, ve)))
    B.beam_paged_kv_write(kk.to(torch.bfloat16), vv.to(torch.bfloat16), ints([0] * n), ints(list(range(1, n + 1))), k["c"])
    k["q"] = (k["q"].float() * 2.0 ** qe).to(torch.bfloat16)
    verify(k)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_no_numbers_reach_their_readers_only(fmt):
    """NaN and infinities in keys and values of single nodes, of context keys that a window takes from some rows, and
    of a key that all rows see."""
    n_q, n_kv, D = 4, 2, 64
    for window, most in ((0, 6), (0, 4), (20, 6)):      # 4: the nodes' only
        k = case(fmt, n_q, n_kv, D, 32, [100, 50], [30, 30], 1800, window=window, gate=False)
        table = k["c"].page_table.cpu()
        clean = run(k)
        assert status() == 0
        spots = [(0, 100 + 7, "v", float("nan")), (0, 100 + 12, "v", float("inf")), (0, 100 + 20, "k", float("nan")),
                 (1, 50 + 3, "v", -float("inf")), (0, 84, "v", float("nan")), (1, 33, "v", float("inf"))]
        for s, p, which, x in spots[:most]:
            pg, off = int(table[s, p // 32]), p % 32
            t = getattr(k["c"], which)
            if fmt == "bf16":
                t[pg, 1, off, 5] = x
            else:
                k["c"].row_scale[pg, 1, int(which == "v"), off] = 255
        out = run(k)
        assert status() == 0
        # the oracle decides who reads what; outputs are no numbers where it says so, and right elsewhere
        with np.errstate(invalid="ignore"):
            hc = host(k["c"])
            for i in range(2):
                a, b = k["start"][i], k["start"][i + 1]
                ref = OT.tree_attention(n_q, np64(k["q"])[a:b], hc, i, k["base"][i], k["nodes"][a:b])[0]
                o = np64(out)[a:b]
                assert np.array_equal(np.isfinite(o), np.isfinite(ref)), (fmt, window, i)
                ok = np.isfinite(ref).all(1)
                assert not ok.all() and (ok.any() or (window, most) == (0, 6))   # there every row reads one
                assert torch.equal(out[a:b][torch.from_numpy(ok).to(DEV)][:, :2 * D], clean[a:b][torch.from_numpy(ok).to(DEV)][:, :2 * D])
        assert torch.equal(out[:, :2 * D], clean[:, :2 * D])      # the other KV head's


def test_attention_over_shared_pages_and_padding_between():
    """Two trees behind one context: the second sequence's table names the first one's pages."""
    k = case("bf16", 6, 2, 64, 16, [64, 64], [10, 12], 1900)
    k["c"].page_table[1, :4] = k["c"].page_table[0, :4]
    verify(k)


@pytest.mark.parametrize("fmt,D", [("bf16", 128), ("nvfp4", 64), ("fp8", 128)])
def test_long_contexts_are_flushed(fmt, D):
    """Ranges of more than 128 blocks to a stream, of one tile (streams in turn) and of two."""
    for n, base in ((3, 30000), (40, 30000)):
        seqs = 16 if n == 3 else 12
        k = case(fmt, 8, 2, D, 256, [base] * seqs, [n] * seqs, 2000 + n, spread=0)
        k["c"].k.view(torch.uint8)
        # 188 blocks of 64 keys... per (sequence, head): 16 x 2 x 469 / 152 = 98 blocks to a range of one tile
        verify(k, only=[0, seqs - 1])


def test_many_sequences_and_a_long_row_list():
    """More sequences than one launch takes."""
    sizes = [i % 3 for i in range(1030)]
    k = case("fp8", 2, 1, 64, 16, [(i * 7) % 20 for i in range(1030)], sizes, 2100, gate=False)
    verify(k, only=list(range(0, 1030, 37)) + [1023, 1024, 1025, 1029])


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("window", [0, 70])
def test_attention_of_many_short_items(fmt, window):
    """Several items of one, two and three tiles of rows and of one to six blocks to each range, whole and cut."""
    sizes, bases = [(i * 29) % 65 for i in range(300)], [(i * 53) % 310 for i in range(300)]
    k = case(fmt, 12, 2, 64, 32, bases, sizes, 2150, window=window)
    verify(k, only=list(range(0, 300, 7)) + [298, 299])


def test_offsets_past_32_bits():
    """Pages past 4 GiB of keys give the bits of a small cache."""
    n_kv, D, page = 8, 128, 256
    pages = (1 << 32) // (n_kv * page * D * 2) + 5
    dims = (pages, n_kv, page, D)
    far = B.PagedKVCache(*(torch.empty(dims, dtype=torch.bfloat16, device=DEV) for _ in "kv"), ints([[pages - 1, 0, pages - 2]]))
    near = B.PagedKVCache.empty(3, page, n_kv, D, ints([[0, 1, 2]]))
    n, cfg = 600, cfg_for(16, n_kv, D)
    kk, vv = randn(2201, n, n_kv, D), randn(2202, n, n_kv, D)
    q, nodes = randn(2203, 20, 16, D), OT.masks(random_tree(5, 20))
    outs = []
    for c in (far, near):
        B.beam_paged_kv_write(kk, vv, ints([0] * n), ints(list(range(1, n + 1))), c)
        outs.append(attend(cfg, c, q, ints([0]), ints([0, 20]), ints([580]), words(nodes), n))
    assert status() == 0 and torch.equal(*outs)


def test_attention_with_o_proj():
    k = case("bf16", 4, 2, 64, 32, [100, 7], [9, 5], 2300, pad=(0, 2))
    k["cfg"].hidden = 256
    w = randn(2301, 256, 256)
    og = run(k)
    out = run(k, w_o=w)
    assert status() == 0 and out.shape == (16, 256)
    ref = np64(og) @ np64(w).T
    tol = 256 * 2.0 ** -23 * np.abs(np64(og)) @ np.abs(np64(w)).T + 2.0 ** -8 * np.abs(ref)
    assert np.all(np.abs(np64(out) - ref) <= tol) and not out[14:].any()


def test_attention_agrees_with_single_rows():
    """A chain's rows are those of beam_paged_attn over the same pages, within both bounds."""
    k = case("fp8", 12, 2, 128, 32, [500], [7], 2400)
    nodes = [set(range(j + 1)) for j in range(7)]
    out = run(k, nodes)
    ws = torch.empty(B.paged_workspace_bytes(k["cfg"], 7, 507), dtype=torch.uint8, device=DEV)
    one = torch.empty_like(out)
    B.beam_paged_attn(k["cfg"], k["q"], k["g"], k["bias"], k["c"], ints([0] * 7), ints(list(range(501, 508))), 507, None, one, ws)
    assert status() == 0
    assert float((out.float() - one.float()).abs().max()) <= 2.0 ** -6 * float(one.float().abs().max())


def test_attention_repeats_streams_and_replays():
    """Repeated calls give the same bits; two streams with their own workspaces; a captured call replayed with
    new lengths, masks, rows and queries."""
    k = case("fp8", 12, 2, 128, 32, [1500, 90, 0], [16, 5, 11], 2500, pad=(0, 4))
    other = case("bf16", 12, 2, 128, 32, [700, 333, 1], [9, 64, 2], 2510)
    a, b = run(k), run(other)
    for _ in range(3):
        assert torch.equal(run(k), a)
    st, st2 = torch.cuda.Stream(), torch.cuda.Stream()
    held = [[ints(x["seq"]), ints(x["start"]), ints(x["base"]), words(x["nodes"])] for x in (k, other)]   # alive throughout
    for _ in range(3):
        outs = [torch.zeros_like(a), torch.zeros_like(b)]
        ws = [torch.empty(B.paged_tree_workspace_bytes(k["cfg"], 80), dtype=torch.uint8, device=DEV) for _ in range(2)]
        torch.cuda.synchronize()
        for i, (x, s) in enumerate(((k, st), (other, st2))):
            attend(x["cfg"], x["c"], x["q"], *held[i], x["most"], x["g"], x["bias"], stream=s, ws=ws[i], out=outs[i])
        torch.cuda.synchronize()
        assert torch.equal(outs[0], a) and torch.equal(outs[1], b)
    q, seq, start, base, mask = k["q"].clone(), ints(k["seq"]), ints(k["start"]), ints(k["base"]), words(k["nodes"])
    out, ws = torch.empty_like(a), torch.empty(B.paged_tree_workspace_bytes(k["cfg"], 36), dtype=torch.uint8, device=DEV)
    call = lambda: attend(k["cfg"], k["c"], q, seq, start, base, mask, 4000, k["g"], k["bias"], ws=ws, out=out)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, a)
    for step, (starts, bases) in enumerate((([0, 3, 3, 20], [1200, 0, 40]), ([1, 30, 32, 36], [3, 95, 9]))):
        nodes = [set()] * 36
        for i in range(3):
            t = OT.masks(random_tree(step * 5 + i, starts[i + 1] - starts[i]))
            nodes[starts[i]:starts[i + 1]] = t
        q.copy_(randn(2520 + step, *q.shape))
        start.copy_(ints(starts))
        base.copy_(ints(bases))
        mask.copy_(words(nodes))
        lens = [b + starts[i + 1] - starts[i] for i, b in enumerate(bases)]
        T = sum(lens)
        B.beam_paged_kv_write(randn(2530, T, 2, 128), randn(2531, T, 2, 128), torch.cat([ints([i] * n) for i, n in enumerate(lens)]),
                              torch.cat([torch.arange(1, n + 1, dtype=torch.int32, device=DEV) for n in lens]), k["c"])
        graph.replay()
        check(k["cfg"], k["c"], q, [0, 1, 2], starts, bases, nodes, out, k["g"], k["bias"])
        again = attend(k["cfg"], k["c"], q, seq, start, base, mask, 4000, k["g"], k["bias"])
        assert torch.equal(out, again)
    assert status() == B.DEV_BAD_PAGE      # the last step's second sequence ends past its pages


def test_captured_calls_share_a_workspace():
    """Two graphs over one workspace, replayed in turn, of calls that split their items (partials, flushed parts and the
    list of what to join lie there) and of one that does not; garbage in it between the replays."""
    ks = [case("bf16", 12, 2, 128, 64, [20000], [33], 2600), case("nvfp4", 12, 2, 128, 64, [3000, 50], [64, 3], 2610),
          case("fp8", 2, 1, 128, 64, [40], [4], 2620)]
    refs = [run(k) for k in ks]
    ws = torch.empty(max(B.paged_tree_workspace_bytes(k["cfg"], k["q"].shape[0]) for k in ks), dtype=torch.uint8, device=DEV)
    held = [[ints(k["seq"]), ints(k["start"]), ints(k["base"]), words(k["nodes"]), torch.zeros_like(r)] for k, r in zip(ks, refs)]
    torch.cuda.synchronize()
    graphs = []
    for k, h in zip(ks, held):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            attend(k["cfg"], k["c"], k["q"], *h[:4], k["most"], k["g"], k["bias"], ws=ws, out=h[4])
        graphs.append(g)
    for i in (0, 1, 2, 1, 0, 2, 2, 0):
        ws.fill_(255 if i else 1)
        held[i][4].zero_()
        graphs[i].replay()
        assert torch.equal(held[i][4], refs[i])
    for i in (0, 1, 2):          # and without a change between them
        graphs[i].replay()
    assert all(torch.equal(h[4], r) for h, r in zip(held, refs)) and status() == 0


def test_bindings_refuse_wrong_tensors():
    k = case("bf16", 4, 2, 64, 16, [20], [4], 2600)
    m = words(k["nodes"])

    def call(**kw):
        d = dict(cfg=k["cfg"], c=k["c"], q=k["q"], seq=ints([0]), start=ints([0, 4]), base=ints([20]), mask=m, most=24,
                 g=None, bias=None)
        d.update(kw)
        return attend(**d)

    ref = call()
    assert torch.equal(call(q=k["q"].view(4, 256)), ref)
    for kw in (dict(q=k["q"].float()), dict(q=k["q"][:, :2]), dict(q=k["q"].transpose(1, 2)), dict(seq=ints([0]).long()),
               dict(start=ints([0])), dict(base=ints([20, 1])), dict(mask=m.int()), dict(mask=m[:3]), dict(mask=m.cpu()),
               dict(g=randn(1, 4, 256)), dict(bias=randn(1, 4)), dict(g=randn(1, 4, 128), bias=randn(1, 4)),
               dict(out=torch.empty(4, 128, dtype=torch.bfloat16, device=DEV)), dict(w_o=randn(1, 256, 128)),
               dict(ws=torch.empty(4096, dtype=torch.uint8, device=DEV)), dict(most=-1)):
        with pytest.raises(B.BeamError):
            call(**kw)
    i4 = ints([0, 0, 1, 1])
    for f in (lambda: B.beam_tree_plan(i4.long(), ints([0, 4]), ints([0]), ints([1]), m, i4, i4, i4),
              lambda: B.beam_tree_plan(i4, ints([0, 4]), ints([0]), ints([1]), i4, i4, i4, i4),
              lambda: B.beam_tree_accept(i4, i4, i4, ints([0]), ints([0]), ints([[0]]), ints([0])),
              lambda: B.beam_tree_accept(i4, i4, i4, ints([0, 4]), ints([0]), ints([0]), ints([0])),
              lambda: B.beam_paged_kv_keep(k["c"], ints([0]), ints([1]), ints([1, 2]), ints([[0]])),
              lambda: B.beam_paged_kv_keep(k["c"], ints([0]), ints([1]), ints([1]), ints([0]))):
        with pytest.raises(B.BeamError):
            f()
    assert status() == 0 and torch.equal(call(), ref)


# ------------------------------------------------------------------------------ append ----

def append(cfg, c, z, gains, seq, pos, slot=None, gate=True, stream=None):
    T = z.shape[0]
    q = torch.full((T, cfg.n_q, cfg.head_dim), 5.0, dtype=torch.bfloat16, device=DEV)
    g = torch.full((T, cfg.n_q * cfg.head_dim), 5.0, dtype=torch.bfloat16, device=DEV) if gate else None
    B.beam_paged_append(cfg, z, *(gains or (None, None)), seq, pos, slot, q, g, c, stream)
    return q, g


def append_cfg(n_q, n_kv, D, kind):
    cfg = cfg_for(n_q, n_kv, D)
    cfg.kind = B.BEAM_ATTN_SWA_ROPE if kind == "rope" else B.BEAM_ATTN_NOPE_SSMAX
    return cfg


def same(a, b):
    """Bit for bit: the pools hold NaN."""
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def near(got, ref, pair, what):
    err, tol = np.abs(got - ref), 2.0 ** -8 * np.abs(ref) + 2.0 ** -19 * pair
    assert np.all(err <= tol), (what, float(np.max(err / np.maximum(tol, 1e-300))))


@pytest.mark.parametrize("kind", ["rope", "ssmax"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("n_q,n_kv,D,page", [(12, 2, 128, 16), (6, 3, 64, 32), (5, 5, 128, 256), (16, 1, 64, 64), (48, 8, 128, 64)])
def test_append_matches_the_oracle(kind, norm, n_q, n_kv, D, page):
    """Queries, gate rows and bf16 pages against 64 bits; quantised pages hold the codes of the bf16 rows, and all else
    in the pools is left as it was. Slots apart from positions, padding rows, far positions."""
    cfg, T = append_cfg(n_q, n_kv, D, kind), 21
    pos = [1, 2, 3, 100001, 2048, 0, 77] + list(range(500, 512)) + [5, 1048576]
    seq, slot = [0, 1, 2] * 7, [1, 5, 9, 2, 6, 0, 3, 7, 33, 34, 35, 36, 40, 41, 42, 17, 18, 19, 48, 50, 47]
    z = randn(3000 + n_q, T, (2 * n_q + 2 * n_kv) * D)
    gains = tuple((1 + 0.1 * torch.randn(D, generator=gen(3001 + i), device=DEV)).to(torch.bfloat16) for i in range(2)) if norm else None
    got = {}
    for fmt in ("bf16", "fp8", "nvfp4"):
        if fmt == "nvfp4" and D == 64 and page == 16:
            continue
        c, *_ = make_cache(fmt, n_kv, D, page, [50, 50, 50], 3002)
        before = host(c)
        q, g = append(cfg, c, z, gains, ints(seq), ints(pos), ints(slot))
        assert status() == 0
        after = host(c)
        got[fmt] = (q, g)
        zz = np64(z).reshape(T, -1, D)
        rows = [zz[:, :n_q], zz[:, n_q:n_q + n_kv]]
        out = [OT.append_rows(x, None if not norm else np64(gains[i]), pos, kind, cfg.rope_theta, cfg.ssmax_base,
                              cfg.ssmax_exp, cfg.eps, i == 0) for i, x in enumerate(rows)]
        flip = lambda x: np.abs(x) + np.abs(np.roll(x, D // 2, -1))  # noqa: E731
        if fmt == "bf16":
            near(np64(q), out[0], flip(out[0]), "q")
            assert np.array_equal(np64(g), zz[:, n_q + 2 * n_kv:].reshape(T, -1))
            stored = np.zeros((T, n_kv, D))
            for t in range(T):
                if slot[t]:
                    pg, off = before.place(seq[t], slot[t])
                    stored[t] = after.k[pg, :, off]
                    near(stored[t], out[1][t], flip(out[1])[t], "k")
            kept_rows = stored
        else:
            assert all(torch.equal(a, b) for a, b in zip(got["bf16"], got[fmt]))
        for t in range(T):
            before.store(seq[t], slot[t], kept_rows[t], zz[t, n_q + n_kv:n_q + 2 * n_kv])
        for name in ("k", "v", "row", "block"):
            a, b = getattr(before, name), getattr(after, name)
            assert a is None or np.array_equal(a, b, equal_nan=a.dtype.kind == "f"), (fmt, name)


def test_append_equals_projection_epilogue_and_write():
    """The same rows as beam_paged_kv_write of what the append stored, and the slot argument left out."""
    cfg = append_cfg(12, 2, 128, "rope")
    z, pos, seq = randn(3100, 9, 28 * 128), ints([3, 4, 5, 6, 7, 8, 9, 10, 11]), ints([1] * 9)
    a, *_ = make_cache("nvfp4", 2, 128, 16, [30, 30], 3101)
    b, *_ = make_cache("nvfp4", 2, 128, 16, [30, 30], 3101)
    w, *_ = make_cache("bf16", 2, 128, 16, [30, 30], 3101)
    gains = (randn(3102, 128), randn(3103, 128))
    append(cfg, a, z, gains, seq, pos)
    append(cfg, w, z, gains, seq, pos, pos.clone())
    to = B.KVCache(*(torch.zeros((1, 2, 30, 128), dtype=torch.bfloat16, device=DEV) for _ in "kv"))
    B.beam_paged_kv_read(w, ints([1]), ints([3]), ints([11]), 9, to)
    B.beam_paged_kv_write(to.k[0, :, 2:11].transpose(0, 1).contiguous(), to.v[0, :, 2:11].transpose(0, 1).contiguous(), seq, pos, b)
    assert status() == 0
    for name in ("k", "v", "row_scale", "block_scale"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name


def test_append_refuses_and_skips():
    """Bad tokens are left out one by one; wrong tensors are refused; rows of a wider buffer are taken as they lie."""
    cfg = append_cfg(4, 2, 64, "rope")
    wide = randn(3200, 6, 12 * 64 + 72)
    z = wide[:, 8:8 + 12 * 64]
    seq, slot = [0, 2, 0, -1, 1, 0], [1, 1, 10 ** 6, 3, 5, -4]
    c, *_ = make_cache("bf16", 2, 64, 16, [20, 20], 3201)
    ref, *_ = make_cache("bf16", 2, 64, 16, [20, 20], 3201)
    ref.page_table[1, 0] = c.page_table[1, 0] = -9        # token 4's page
    q, g = append(cfg, c, z, None, ints(seq), ints([1] * 6), ints(slot))
    assert status() == B.DEV_BAD_POSITION | B.DEV_BAD_SEQ | B.DEV_BAD_PAGE
    q1, g1 = append(cfg, ref, z[:1].contiguous(), None, ints([0]), ints([1]), ints([1]))
    assert status() == 0 and same(c.k, ref.k) and same(c.v, ref.v)
    assert torch.equal(q[:1], q1) and torch.equal(g[:1], g1) and torch.isfinite(q.float()).all()
    assert torch.equal(g, z[:, 8 * 64:])
    append(cfg, c, z, None, ints([0] * 6), ints([-1] * 6), ints([9] * 6))
    assert status() == B.DEV_BAD_POSITION and same(c.k, ref.k)
    i6 = ints([1, 2, 3, 4, 5, 6])
    for kw in (dict(z=z.float()), dict(z=z[:, :-8]), dict(z=wide.t()[:6, :]), dict(seq=i6.long()), dict(pos=i6[:5]),
               dict(slot=i6.float()), dict(gains=(randn(1, 64), None)), dict(gains=(randn(1, 32), randn(2, 64))),
               dict(z=wide[:, 4:4 + 12 * 64])):
        d = dict(cfg=cfg, c=c, z=z, gains=None, seq=i6, pos=i6, slot=i6)
        d.update(kw)
        with pytest.raises(B.BeamError):
            append(**d)
    empty = append(cfg, c, z[:0], None, ints([]), ints([]))
    assert empty[0].shape[0] == 0 and status() == 0


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_append_no_numbers_and_extremes(fmt):
    """Rows of NaN, infinities, zeros and bf16's ends give the codes of beam_paged_kv_write."""
    cfg = append_cfg(2, 2, 128, "ssmax")          # no norm, keys are not scaled: rows pass through
    z = randn(3300, 8, 6 * 128, spread=100)
    z[0, 2 * 128 + 5], z[1, 4 * 128 + 3], z[2, 3 * 128:4 * 128] = float("nan"), float("inf"), 0
    z[3, 2 * 128:] = 2.0 ** -133
    z[4, 2 * 128:] = 3.3e38
    a, *_ = make_cache(fmt, 2, 128, 16, [16], 3301)
    b, *_ = make_cache(fmt, 2, 128, 16, [16], 3301)
    i8 = ints(list(range(1, 9)))
    append(cfg, a, z, None, ints([0] * 8), i8, gate=False)
    B.beam_paged_kv_write(z[:, 256:512].reshape(8, 2, 128), z[:, 512:].reshape(8, 2, 128), ints([0] * 8), i8, b)
    assert status() == 0
    for name in ("k", "v", "row_scale") + (("block_scale",) if fmt == "nvfp4" else ()):
        assert torch.equal(getattr(a, name), getattr(b, name)), name


# ------------------------------------------------------------------------- bookkeeping ----

@pytest.mark.parametrize("sizes", [[1], [64], [0, 3, 64, 1, 0, 17, 2, 40], [5] * 300])
def test_plan_matches_the_oracle(sizes):
    start = [2]
    for n in sizes:
        start.append(start[-1] + n)
    N, T = len(sizes), start[-1] + 3
    trees = [random_tree(4000 + i, n) for i, n in enumerate(sizes)]
    parent = [9, 9] + sum(trees, []) + [9] * 3
    base, seq = [3 * i for i in range(N)], [N - 1 - i for i in range(N)]
    out = [torch.full((T,), 77, dtype=torch.int64 if x == 0 else torch.int32, device=DEV) for x in range(4)]
    B.beam_tree_plan(ints(parent), ints(start), ints(seq), ints(base), *out)
    assert status() == 0
    want = [[0] * T for _ in range(4)]
    for i, t in enumerate(trees):
        for j, m in enumerate(OT.masks(t)):
            r = start[i] + j
            want[0][r], want[1][r], want[2][r], want[3][r] = OT.bits(m), base[i] + len(m), base[i] + 1 + j, seq[i]
    for got, ref in zip(out, want):
        assert got.tolist() == ref


def test_plan_leaves_lost_nodes_and_bad_sequences_out():
    parent = [-1, 0, 5, 2, -2, 1, 6] + [-1] * 70
    out = [torch.full((77,), 77, dtype=torch.int64 if x == 0 else torch.int32, device=DEV) for x in range(4)]
    B.beam_tree_plan(ints(parent), ints([0, 7, 77]), ints([3, 4]), ints([10, 20]), *out)
    assert status() == B.DEV_BAD_POSITION | B.DEV_BAD_SEQ
    assert out[0].tolist() == [1, 3, 0, 0, 0, 0b100011, 0] + [0] * 70
    assert out[1].tolist() == [11, 12, 0, 0, 0, 13, 0] + [0] * 70
    assert out[2].tolist() == [11, 12, 0, 0, 0, 16, 0] + [0] * 70


@pytest.mark.parametrize("tokens", [1, 2, 5, 1000])
def test_accept_matches_the_oracle(tokens):
    """Few tokens: long paths and equal siblings; many: short ones."""
    sizes = [0, 1, 64, 30, 7, 0, 64, 12, 3]
    start = [0]
    for n in sizes:
        start.append(start[-1] + n)
    r = np.random.default_rng(tokens)
    trees = [random_tree(4100 + i, n) for i, n in enumerate(sizes)]
    tok, sam = (r.integers(0, tokens, start[-1]).tolist() for _ in "ts")
    for stride in (64, 3):
        count, nxt = ints([77] * 9), ints([77] * 9)
        path = torch.full((9, stride), 77, dtype=torch.int32, device=DEV)
        B.beam_tree_accept(ints(sum(trees, [])), ints(tok), ints(sam), ints(start), count, path, nxt)
        assert status() == 0
        for i, t in enumerate(trees):
            a, b = start[i], start[i + 1]
            want, after = OT.accept(t, tok[a:b], sam[a:b])
            assert (int(count[i]), int(nxt[i])) == (len(want), after)
            assert path[i].tolist() == (want + [-1] * 64)[:stride]
    count = ints([7])
    B.beam_tree_accept(ints([-1] * 65), ints([1] * 65), ints([1] * 65), ints([0, 65]), count, ints([[7, 7]]), nxt[:1])
    assert status() == B.DEV_BAD_SEQ and int(count[0]) == 0 and int(nxt[0]) == -1


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("D,page,n_kv", [(128, 16, 3), (64, 32, 2), (128, 256, 1)])
def test_keep_moves_rows_as_if_at_once(fmt, D, page, n_kv):
    """Paths whose rows take the places of others of the path, rows that stay, no rows; pages that are crossed; all else
    in the pools is left."""
    bases = [0, 15, 16, 100, 3, 40]
    paths = [[0, 1, 2], [0, 2, 3, 4, 5, 9, 63], list(range(1, 64)), [5], [], [3, 2, 1, 0]]
    c, *_ = make_cache(fmt, n_kv, D, page, [b + 64 for b in bases], 4200)
    hc = host(c)
    before = host(c)
    for s, (b, p) in enumerate(zip(bases, paths)):
        for k, x in enumerate(p):
            (pa, oa), (pb, ob) = hc.place(s, b + 1 + x), hc.place(s, b + 1 + k)
            for name in ("k", "v"):
                getattr(hc, name)[pb, :, ob] = getattr(before, name)[pa, :, oa]
            for name in ("row", "block"):
                if getattr(hc, name) is not None:
                    getattr(hc, name)[pb, :, :, ob] = getattr(before, name)[pa, :, :, oa]
    order = [4, 0, 2, 5, 1, 3]
    path = torch.full((6, 64), -1, dtype=torch.int32)
    for i, s in enumerate(order):
        path[i, :len(paths[s])] = torch.tensor(paths[s], dtype=torch.int32)
    B.beam_paged_kv_keep(c, ints(order), ints([bases[s] for s in order]), ints([len(paths[s]) for s in order]), path.to(DEV))
    assert status() == 0
    after = host(c)
    for name in ("k", "v", "row", "block"):
        a, b = getattr(hc, name), getattr(after, name)
        assert a is None or np.array_equal(a, b, equal_nan=a.dtype.kind == "f"), name


def test_keep_leaves_bad_rows_out():
    c, *_ = make_cache("bf16", 2, 64, 16, [80, 80], 4300)
    ref = host(c)
    for seq, base, count, path, bit in ((0, 5, 3, [0, 64, -1], 1), (0, 5, -1, [0, 2, 3], 1), (0, 5, 4, [1, 2, 3], 1),
                                        (2, 5, 2, [1, 2, 3], 2), (0, -7, 2, [1, 2, 3], 1), (0, 2 ** 31 - 2, 2, [1, 2, 3], 1),
                                        (1, 92, 3, [4, 5, 6], 17)):    # past the table, and to a page that is none
        B.beam_paged_kv_keep(c, ints([seq]), ints([base]), ints([count]), ints([path]))
        assert status() == bit, (seq, base, count)
        assert np.array_equal(host(c).k, ref.k, equal_nan=True)
    c.page_table[0, 0] = -1
    B.beam_paged_kv_keep(c, ints([0]), ints([14]), ints([3]), ints([[1, 2, 3]]))
    assert status() == B.DEV_BAD_PAGE
    after = host(c)
    # of slots 16 to 18, which move to 15 to 17, the last alone goes from a page to a page
    (pa, oa), (pb, ob) = ref.place(0, 18), ref.place(0, 17)
    ref.k[pb, :, ob] = ref.k[pa, :, oa]
    assert np.array_equal(after.k, ref.k, equal_nan=True)


# --------------------------------------------------------------------------- together ----

def check_layer(W, cache, t, start, held, nodes, what):
    """One layer's attention output t["attn"] against the oracle on its own inputs: o_proj is linear, so the bound of og
    goes through |W_o|, with n_q D exact products summed in FP32 and one rounding of the result."""
    hc, q, g, w = host(cache), np64(t["q"]), np64(t["g"]), np64(W["w_o"])
    for s in range(3):
        a, b = start[s], start[s + 1]
        og, *sizes = OT.tree_attention(TINY.n_q, q[a:b], hc, s, held[s], nodes[a:b], g[a:b], np64(W["gate_bias"]))
        tol = bound(cfg_for(TINY.n_q, TINY.n_kv, TINY.head_dim), hc.fmt, og, *sizes)
        ref = og @ w.T
        lim = tol @ np.abs(w).T + og.shape[1] * 2.0 ** -23 * (np.abs(og) @ np.abs(w).T) + 2.0 ** -8 * np.abs(ref)
        worst = float(np.max(np.abs(np64(t["attn"])[a:b] - ref) / lim))
        assert worst <= 1.0, (what, s, worst)
    assert not t["attn"][start[-1]:].any()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_steps_through_the_stack(fmt):
    """Prompts, then steps of verify, LM head, sampling, acceptance and keep, as a server runs them. The sequences that
    the accepted tokens make up, decoded one token at a time by another stack, give the same hidden states up to
    what a bf16 flip in one layer does to the next, through the layers in front of the first router (where a flip
    may choose another expert); every layer's attention is recomputed by the oracle from the step's own q, g and
    pages; a captured step replays to the same bits."""
    W = weights()
    L, H, V = TINY.n_layers, TINY.hidden, 300
    st, one = BeamStack(TINY, W, paged_caches(fmt)), BeamStack(TINY, W, paged_caches(fmt))
    emb = synth.activations(V, H, 50, "embed").to(DEV)
    head = {k: v.to(DEV) for k, v in synth.lm_head_weights(TINY, V, 0).items()}
    front = st.dense.index(False)
    held = [20, 3, 41]
    hist = [[(7 * i + 3 * s) % V for i in range(n)] for s, n in enumerate(held)]
    for x in (st, one):
        seq = sum(([s] * n for s, n in enumerate(held)), [])
        x.forward(emb[torch.tensor(sum(hist, []), device=DEV)], ints(seq), ints(sum((list(range(1, n + 1)) for n in held), [])),
                  max(held), max_q_per_seq=max(held))
    r = np.random.default_rng(3)
    nxt = [1, 2, 3]
    for step in range(3):
        sizes = [[5, 9, 1], [12, 1, 30], [3, 3, 3]][step]
        start = [0]
        for n in sizes:
            start.append(start[-1] + n)
        trees = [random_tree(60 + 10 * step + s, n) for s, n in enumerate(sizes)]
        T = start[-1] + 2                                            # and two rows of padding
        tok = torch.zeros(T, dtype=torch.int32)
        for s in range(3):
            tok[start[s]:start[s + 1]] = torch.from_numpy(r.permutation(V)[:sizes[s]].astype(np.int32))
            tok[start[s]] = nxt[s]
        parent, rows, ids, base = ints(sum(trees, []) + [-1, -1]), ints(start), ints([0, 1, 2]), ints(held)
        e = emb[tok.long().to(DEV)]
        trace = []
        h = st.verify(e, parent, rows, ids, base, max(held) + 64, trace=trace).clone()
        assert status() == 0 and torch.isfinite(h.float()).all()
        nodes = [x for t in trees for x in OT.masks(t)]
        for l, (w, c, tr) in enumerate(zip(W, st.caches, trace)):
            check_layer(w, c, tr, start, held, nodes, f"step {step} layer {l}")
        u, logits = torch.empty_like(h), torch.empty((T, V), device=DEV)
        B.beam_boundary_norm(None, h, u, None, head["final_norm"], 1, TINY.eps)
        B.beam_lm_head(u, head["w_lm"], logits, 30.0)
        got, uni = torch.empty(T, dtype=torch.int32, device=DEV), torch.rand(T, generator=gen(step), device=DEV)
        B.beam_sample(logits, uni, got, temperature=torch.full((T,), 0.8, device=DEV), top_k=ints([20] * T))
        # a drafter that is right along one path
        lead = got.cpu()
        for s in range(3):
            t, at = trees[s], 0
            for j in range(1, sizes[s]):
                if t[j] == at and r.random() < 0.7:
                    tok[start[s] + j] = lead[start[s] + at]
                    at = j
        count, path, after = ints([0] * 3), torch.zeros((3, 64), dtype=torch.int32, device=DEV), ints([0] * 3)
        B.beam_tree_accept(parent, tok.to(DEV), got, rows, count, path, after)
        st.keep(ids, base, count, path)
        assert status() == 0
        # the same tokens one at a time: their embeddings are those that the tree was run with
        for s in range(3):
            p = path[s, :int(count[s])].tolist()
            want, _ = OT.accept(trees[s], tok[start[s]:start[s + 1]].tolist(), lead[start[s]:start[s + 1]].tolist())
            assert p == want
            for k, j in enumerate(p):
                single = []
                one.forward(e[start[s] + j:start[s] + j + 1], ints([s]), ints([held[s] + 1 + k]), held[s] + 1 + k, trace=single)
                for l in range(front):
                    a, b = trace[l]["h"][start[s] + j].float(), single[l]["h"][0].float()
                    rel = float((a - b).norm() / b.norm())
                    assert rel <= 0.05, (step, s, j, l, rel)
            held[s] += len(p)
        nxt = after.tolist()
    assert status() == 0
    if fmt == "bf16":     # the pages hold the same sequences, up to the same flips
        for a, b in zip(st.caches[:front], one.caches[:front]):
            for s in range(3):
                to = [B.KVCache(*(torch.zeros((1, TINY.n_kv, held[s], TINY.head_dim), dtype=torch.bfloat16, device=DEV) for _ in "kv"))
                      for _ in range(2)]
                for x, d in zip((a, b), to):
                    B.beam_paged_kv_read(x, ints([s]), ints([1]), ints([held[s]]), held[s], d)
                for name in ("k", "v"):
                    x, y = (getattr(d, name).float() for d in to)
                    rel = float((x - y).norm() / y.norm())
                    assert rel <= 0.05, rel
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    b0 = ints(held)
    h = st.verify(e, parent, rows, ids, b0, max(held) + 64).clone()
    with torch.cuda.graph(graph):
        out = st.verify(e, parent, rows, ids, b0, max(held) + 64)
    st.verify(torch.cat([e, e]), torch.cat([parent, parent]), rows, ids, b0, max(held) + 64)   # another size between
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, h) and status() == 0


@pytest.mark.parametrize("T", [5, 70])
def test_paged_projection_equals_its_parts(T):
    """beam_paged_qkv_gate against beam_qkv_gate into a staging row and beam_paged_kv_write: the same arithmetic in
    another order of summation, so bf16 results differ by a step where the norm's last bit tips one."""
    shape = TINY
    W = {k: v.to(DEV) for k, v in synth.layer_weights(shape, 0, 1).items()}
    cfg = B.LayerCfg.from_shape(shape, B.BEAM_ATTN_SWA_ROPE)
    u = synth.activations(T, shape.hidden, 9, "u").to(DEV)
    c, *_ = make_cache("bf16", shape.n_kv, shape.head_dim, 16, [80], 5000)
    q, g = (torch.empty((T, shape.n_q * shape.head_dim), dtype=torch.bfloat16, device=DEV) for _ in "qg")
    ws = torch.empty(B.workspace_bytes(cfg, T, 80), dtype=torch.uint8, device=DEV)
    seq, pos = ints([0] * T), ints(list(range(1, T + 1)))
    B.beam_paged_qkv_gate(cfg, u, W["w_qkvg"], W["q_norm"], W["k_norm"], seq, pos, None, q, g, c, ws)
    kc = B.KVCache(*(torch.zeros((1, shape.n_kv, 80, shape.head_dim), dtype=torch.bfloat16, device=DEV) for _ in "kv"))
    q2, g2 = torch.empty_like(q), torch.empty_like(g)
    B.beam_qkv_gate(cfg, u, W["w_qkvg"], W["q_norm"], W["k_norm"], seq, pos, q2, g2, kc, ws)
    to = B.KVCache(torch.zeros_like(kc.k), torch.zeros_like(kc.v))
    B.beam_paged_kv_read(c, ints([0]), ints([1]), ints([T]), T, to)
    assert status() == 0
    for a, b in ((q, q2), (g, g2), (to.k, kc.k), (to.v, kc.v)):
        a, b = np64(a), np64(b)
        assert np.all(np.abs(a - b) <= 2.0 ** -7 * np.abs(b) + 2.0 ** -12) and np.mean(a != b) < 0.02
