"""GPU parity of the paged cache's entry points against float64 NumPy (oracle/paged.py), at the
sizes, layouts and values where they can go wrong.

Writing and reading are exact by definition: codes, scales and values must be equal.

Attention: |out - ref| <= 2^-8 |ref| (half a bf16 step, the one rounding of the result) plus an
absolute term from the work before it, per element
    W (2 d + r) + n 2^-32 V
with W = sum p|v| (64 bits). d bounds the logit error: D products summed in FP32, each sum off by
at most 2^-23 of the sum of magnitudes: d = D 2^-23 max_i sum|q k_i| / sqrt(D). r bounds the
relative error of a weight p itself, which enters the sum as (p + dp) v with |dp| <= r p, so the
sum moves by at most r W: 2^-15 over a BF16 cache (P in two bf16 halves, 2^-17, exp2, 2^-21, and
the FP32 sums); over a quantised cache P is rounded to f16 once, half a step, 2^-11, and the rest
is 2^-15 as before. The last term is the f16 floor there: a P value below f16's smallest step
2^-24 at the bias 2^7 is off by half of it, 2^-32, times the largest stored magnitude V of the
row's n keys. The gate's sigmoid is within 2^-20 and scales what it gates.
"""
import numpy as np
import pytest
import torch

from oracle import paged as OP
from oracle.codecs import bf16_round
from hybrid_attention_moe_gb300 import beam as B
from parity import np64

pytestmark = pytest.mark.gpu
DEV = "cuda"
FMT = {"bf16": B.BEAM_PAGED_BF16, "fp8": B.BEAM_PAGED_FP8, "nvfp4": B.BEAM_PAGED_NVFP4}


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(seed, *shape, spread=0):
    g = gen(seed)
    x = torch.randn(shape, generator=g, device=DEV)
    if spread:   # each row its own magnitude
        x = x * torch.exp2(torch.randint(-spread, spread + 1, shape[:-1] + (1,), generator=g, device=DEV).float())
    return x.to(torch.bfloat16)


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def cfg_for(n_q, n_kv, D, hidden=None):
    return B.LayerCfg(hidden=hidden or n_q * D, n_q=n_q, n_kv=n_kv, head_dim=D,
                      kind=B.BEAM_ATTN_NOPE_SSMAX, n_experts=8, n_groups=1, topk_groups=1, topk=1,
                      d_ff_expert=128, d_ff_dense=128)


def make_cache(fmt, n_kv, D, page, lens, seed, window=0, spread=2, junk=True, spare=2):
    """Sequences of the given lengths in pages scattered over the pool, written by the library;
    everything that holds no key is junk: pages of 0xFF bytes (NaN in every format), table
    entries past the end that name no page."""
    per = max(1, -(-max(lens) // page)) + 1
    need = [-(-n // page) for n in lens]
    pool = sum(need) + spare
    order = torch.randperm(pool, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((len(lens), per), -7, dtype=torch.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    c = B.PagedKVCache.empty(pool, page, n_kv, D, table.to(DEV), FMT[fmt], window)
    if junk:
        for t in (c.k, c.v, c.row_scale, c.block_scale):
            if t is not None:
                t.view(torch.uint8).fill_(255)
    seq = torch.cat([torch.full((n,), i) for i, n in enumerate(lens)]).to(torch.int32).to(DEV)
    pos = torch.cat([torch.arange(1, n + 1) for n in lens]).to(torch.int32).to(DEV)
    T = seq.numel()
    k, v = randn(seed, T, n_kv, D), randn(seed + 1, T, n_kv, D, spread=spread)
    if T:
        B.beam_paged_kv_write(k, v, seq, pos, c)
    return c, k, v, seq, pos


def host(c):
    """Oracle copy of a cache."""
    fmt = {v: k for k, v in FMT.items()}[c.dtype]
    f = (lambda t: np64(t)) if fmt == "bf16" else (lambda t: t.cpu().numpy())
    return OP.PagedKV(fmt, f(c.k), f(c.v), c.page_table.cpu().numpy(),
                      None if c.row_scale is None else c.row_scale.cpu().numpy(),
                      None if c.block_scale is None else c.block_scale.cpu().numpy(), c.window)


def status():
    torch.cuda.synchronize()
    return B.beam_get_device_status()


def scratch(cfg, T, max_pos):
    return torch.empty(B.paged_workspace_bytes(cfg, T, max_pos), dtype=torch.uint8, device=DEV)


def attend(cfg, c, q, seq, pos, max_pos, g=None, bias=None, w_o=None):
    T = q.shape[0]
    out = torch.full((T, cfg.hidden if w_o is not None else cfg.n_q * cfg.head_dim), 7.0,
                     dtype=torch.bfloat16, device=DEV)
    B.beam_paged_attn(cfg, q, g, bias, c, seq, pos, max_pos, w_o, out, scratch(cfg, T, max_pos))
    return out


def tolerance(cfg, hc, q, seq, pos, ref, mag):
    """The bound of the module's docstring, per output element."""
    D, T = cfg.head_dim, len(pos)
    grp = cfg.n_q // cfg.n_kv
    tol = 2.0 ** -8 * np.abs(ref)
    for t in range(T):
        p = int(pos[t])
        if p == 0:
            continue
        lo = max(1, p - hc.window + 1) if hc.window else 1
        K, V = hc.load(int(seq[t]), np.arange(lo, p + 1))
        for h in range(cfg.n_q):
            d = D * 2.0 ** -23 * np.max(np.abs(K[h // grp]) @ np.abs(q[t, h])) / np.sqrt(D)
            sl = slice(h * D, (h + 1) * D)
            floor = 0.0 if hc.fmt == "bf16" else V.shape[1] * 2.0 ** -32 * np.max(np.abs(V[h // grp]))
            r = 2.0 ** -15 + (0.0 if hc.fmt == "bf16" else 2.0 ** -11)
            tol[t, sl] += mag[t, sl] * (2 * d + r) + floor
    return tol


def check_attn(cfg, c, q, seq, pos, out, g=None, bias=None):
    hc = host(c)
    s, p = seq.cpu().numpy(), pos.cpu().numpy()
    ref, mag = OP.paged_attention(cfg.n_q, np64(q), hc, s, p, None if g is None else np64(g),
                                  None if bias is None else np64(bias))
    err = np.abs(np64(out) - ref)
    tol = tolerance(cfg, hc, np64(q), s, p, ref, mag)
    worst = float(np.max(err / np.maximum(tol, 1e-300))) if err.size else 0.0
    print(f"attention: largest error / bound {worst:.3f}")
    assert np.all(np.isfinite(np64(out))) and np.all(err <= tol), worst


# ------------------------------------------------------------------ write and read ----

@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("D,n_kv,page,T", [(128, 8, 64, 1), (128, 3, 16, 37), (64, 2, 32, 130), (64, 1, 256, 5)])
def test_write_codes_match_the_oracle(fmt, D, n_kv, page, T):
    """Scattered positions of several sequences, rows of very different magnitudes; what is not
    written keeps its bytes."""
    n = 4
    c, *_ = make_cache(fmt, n_kv, D, page, [90] * n, 3)
    hc = host(c)
    perm = torch.randperm(4 * 90, generator=torch.Generator().manual_seed(9))[:T]
    seq, pos = ints((perm // 90).tolist()), ints((perm % 90 + 1).tolist())
    k, v = randn(11, T, n_kv, D, spread=40), randn(12, T, n_kv, D, spread=100)
    B.beam_paged_kv_write(k, v, seq, pos, c)
    assert status() == 0
    for t in range(T):
        hc.store(int(seq[t]), int(pos[t]), np64(k[t]), np64(v[t]))
    got = host(c)
    assert np.array_equal(got.k, hc.k, equal_nan=fmt == "bf16")
    assert np.array_equal(got.v, hc.v, equal_nan=fmt == "bf16")
    if fmt != "bf16":
        assert np.array_equal(got.row, hc.row)
    if fmt == "nvfp4":
        assert np.array_equal(got.block, hc.block)


@pytest.mark.parametrize("fmt", ["fp8", "nvfp4"])
def test_write_ties_and_extremes(fmt):
    """Rows made of the codes' midpoints, of bf16's largest and smallest magnitudes, of zeros
    and negative zeros, and rows with one infinity or NaN."""
    D, n_kv = 64, 1
    m = np.array([0, .25, .5, .75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, -.25] * 4)
    rows = [m, -m, m * 2.0 ** -100, m * 448 / 6, np.arange(64) * 6.5 + 1, np.arange(64) * 14.0,
            (np.arange(64) * 2 + 1) * 2.0 ** -10, np.full(64, 3.3895313892515355e38),
            np.full(64, 2.0 ** -133), np.zeros(64), -np.zeros(64), np.r_[np.full(63, 1e-30), 1e30],
            np.r_[np.inf, np.ones(63)], np.r_[np.ones(63), np.nan], np.r_[np.ones(20), -np.inf, np.ones(43)],
            # a block's largest value halfway between two block scales (6 * (17 / 16) and others)
            np.r_[448 * 6.0, np.full(15, 1.0), np.arange(48) * 6 * 17 / 16]]
    x = torch.tensor(np.array(rows), dtype=torch.float32).to(torch.bfloat16).to(DEV)[:, None]
    T = x.shape[0]
    c = B.PagedKVCache.empty(2, 32, n_kv, D, ints([[1, 0]]), FMT[fmt])
    hc = host(c)
    B.beam_paged_kv_write(x, x.flip(0).contiguous(), ints([0] * T), ints(list(range(1, T + 1))), c)
    assert status() == 0
    xs = np64(x)
    for t in range(T):
        hc.store(0, t + 1, xs[t], xs[T - 1 - t])
    got = host(c)
    assert np.array_equal(got.row, hc.row) and np.array_equal(got.k, hc.k) and np.array_equal(got.v, hc.v)
    if fmt == "nvfp4":
        assert np.array_equal(got.block, hc.block)
    # and back: the stored values, NaN rows as NaN
    dst = B.KVCache(torch.zeros((1, 1, T, D), dtype=torch.bfloat16, device=DEV),
                    torch.zeros((1, 1, T, D), dtype=torch.bfloat16, device=DEV))
    B.beam_paged_kv_read(c, ints([0]), ints([1]), ints([T]), T, dst)
    K, V = hc.load(0, np.arange(1, T + 1))
    fin = np.isfinite(K)
    assert np.array_equal(np64(dst.k)[0][fin], bf16_round(K)[fin]) and np.array_equal(np.isnan(np64(dst.k)[0]), ~fin)
    assert np.array_equal(np.isnan(np64(dst.v)[0]), np.isnan(V))


def test_write_strided_rows_padding_and_bad_tokens():
    """K and V as they lie in a packed projection; a padding row and tokens out of range write
    nothing, the others are flagged; the rest of the call goes through."""
    n_kv, D, page = 2, 64, 16
    T = 7
    packed = randn(5, T, 3 * n_kv * D)
    k = packed[:, n_kv * D:2 * n_kv * D].view(T, n_kv, D)
    v = packed[:, 2 * n_kv * D:].view(T, n_kv, D)
    assert k.stride(0) == 3 * n_kv * D
    table = ints([[2, 0, 9], [1, -1, 3]])
    seq, pos = ints([0, 1, 0, 2, 1, 1, -1]), ints([17, 3, 0, 4, 49, 18, 1])
    want = {(0, 17): 0, (1, 3): 1}
    for i, bits in ((3, B.DEV_BAD_SEQ), (4, B.DEV_BAD_POSITION), (5, B.DEV_BAD_PAGE), (6, B.DEV_BAD_SEQ)):
        c = B.PagedKVCache.empty(4, page, n_kv, D, table)
        keep = [0, 1, 2, i]
        B.beam_paged_kv_write(k[:3], v[:3], seq[:3], pos[:3], c)
        assert status() == 0
        B.beam_paged_kv_write(k[i:i + 1], v[i:i + 1], seq[i:i + 1], pos[i:i + 1], c)
        assert status() == bits, (i, keep)
        ref = torch.zeros_like(c.k)
        for (s, p), t in want.items():
            ref[int(table[s, (p - 1) // page]), :, (p - 1) % page] = k[t]
        assert torch.equal(c.k, ref)
    c = B.PagedKVCache.empty(4, page, n_kv, D, table)
    B.beam_paged_kv_write(k, v, seq, ints([-1] * T), c)
    assert status() == B.DEV_BAD_POSITION and not c.k.any()
    with pytest.raises(B.BeamError):
        B.beam_paged_kv_write(k[:, :, :32], v[:, :, :32], seq, pos, c)
    with pytest.raises(B.BeamError):
        B.beam_paged_kv_write(packed.view(T, 3 * n_kv, D)[:, ::3], v, seq, pos, c)
    with pytest.raises(B.BeamError):
        B.beam_paged_kv_write(k, v.contiguous(), seq, pos, c)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("D,n_kv,page", [(128, 2, 64), (64, 3, 32), (128, 1, 256)])
def test_read_back(fmt, D, n_kv, page):
    """Ranges of every kind: whole, empty, one key, a window that wraps in the destination's
    ring, the same sequence twice; slots that are not read into keep their contents."""
    lens = [1, 200, 333, 64]
    c, *_ = make_cache(fmt, n_kv, D, page, lens, 21)
    hc = host(c)
    ranges = [(0, 1, 1), (1, 1, 200), (2, 150, 333), (2, 330, 333), (3, 5, 4), (1, 100, 163), (1, 65, 65)]
    cap = 203
    mark = torch.full((len(ranges) + 1, n_kv, cap, D), 5.0, dtype=torch.bfloat16, device=DEV)
    dst = B.KVCache(mark.clone(), mark.clone())
    B.beam_paged_kv_read(c, ints([r[0] for r in ranges]), ints([r[1] for r in ranges]),
                         ints([r[2] for r in ranges]), 200, dst)
    assert status() == 0
    ref_k, ref_v = np64(mark), np64(mark)
    for i, (s, a, b) in enumerate(ranges):
        if b >= a:
            pos = np.arange(a, b + 1)
            K, V = hc.load(s, pos)
            ref_k[i][:, (pos - 1) % cap], ref_v[i][:, (pos - 1) % cap] = bf16_round(K), bf16_round(V)
    assert np.array_equal(np64(dst.k), ref_k) and np.array_equal(np64(dst.v), ref_v)


def test_read_refuses_bad_ranges():
    c, *_ = make_cache("fp8", 2, 64, 16, [40, 40], 5)
    mark = torch.full((1, 2, 30, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    for s, a, b, most, bits in ((0, 0, 9, 30, B.DEV_BAD_POSITION), (0, -5, -1, 30, B.DEV_BAD_POSITION),
                                (0, 1, 31, 40, B.DEV_BAD_POSITION),    # longer than the destination
                                (0, 1, 20, 19, B.DEV_BAD_POSITION),    # longer than max_len
                                (0, 60, 65, 30, B.DEV_BAD_POSITION),   # past the page table (4 x 16)
                                (0, 2147483600, 2147483647, 30, B.DEV_BAD_POSITION),
                                (2, 1, 9, 30, B.DEV_BAD_SEQ), (-1, 1, 9, 30, B.DEV_BAD_SEQ)):
        dst = B.KVCache(mark.clone(), mark.clone())
        B.beam_paged_kv_read(c, ints([s]), ints([a]), ints([b]), most, dst)
        assert status() == bits, (s, a, b)
        assert torch.equal(dst.k, mark) and torch.equal(dst.v, mark)
    # a page that is none: its positions are left out
    c.page_table[0, 1] = 99
    dst = B.KVCache(mark.clone(), mark.clone())
    B.beam_paged_kv_read(c, ints([0]), ints([10]), ints([34]), 25, dst)
    assert status() == B.DEV_BAD_PAGE
    assert torch.equal(dst.k[:, :, 16:30], mark[:, :, 16:30])
    assert not bool((dst.k[:, :, 9:16] == 5).all()) and not bool((dst.k[:, :, 2:4] == 5).all())


# ---------------------------------------------------------------------- attention ----

LENS = [1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513, 700]


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("n_q,n_kv,D,page", [(12, 2, 128, 16), (8, 8, 128, 64), (16, 1, 128, 32), (5, 1, 64, 32),
                                             (36, 4, 64, 128), (7, 1, 128, 256)])
def test_attention_matches_the_oracle(fmt, n_q, n_kv, D, page):
    """Lengths around every tile's edge, in one ragged batch, with the gate; the longest rows
    are split between CTAs."""
    cfg = cfg_for(n_q, n_kv, D)
    lens = LENS + [2500 if fmt == "bf16" else 3100]
    c, *_ = make_cache(fmt, n_kv, D, page, lens, 31)
    T = len(lens)
    q, g, bias = randn(32, T, n_q, D), randn(33, T, n_q * D), randn(34, n_q)
    seq, pos = ints(list(range(T))), ints(lens)
    out = attend(cfg, c, q, seq, pos, max(lens), g, bias)
    assert status() == 0
    check_attn(cfg, c, q, seq, pos, out, g, bias)
    # no gate, and an upper bound of the positions well above them
    out = attend(cfg, c, q, seq, pos, 1 << 20)
    assert status() == 0
    check_attn(cfg, c, q, seq, pos, out)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("lens", [[1], [40], [257], [1030]])
def test_attention_short_whole_pairs(fmt, lens):
    """Few keys and a tight bound: no pair is split."""
    cfg = cfg_for(12, 2, 128)
    c, *_ = make_cache(fmt, 2, 128, 32, lens, 41)
    q = randn(42, 1, 12, 128)
    out = attend(cfg, c, q, ints([0]), ints(lens), lens[0])
    assert status() == 0
    check_attn(cfg, c, q, ints([0]), ints(lens), out)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("window", [1, 16, 100, 513])
def test_attention_window_drops_pages(fmt, window):
    """A sliding window: the pages before it are given back (their entries name no page)."""
    cfg = cfg_for(6, 2, 64)
    lens = [5, 99, 100, 101, 640, 1500]
    c, *_ = make_cache(fmt, 2, 64, 32, lens, 51, window=window)
    for i, n in enumerate(lens):
        gone = max(0, n - window) // 32
        c.page_table[i, :gone] = -1
    q = randn(52, len(lens), 6, 64)
    seq, pos = ints(list(range(len(lens)))), ints(lens)
    out = attend(cfg, c, q, seq, pos, 1500)
    assert status() == 0
    check_attn(cfg, c, q, seq, pos, out)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_attention_rows_that_see_nothing(fmt):
    """Padding rows (position 0, any sequence id) and rows out of range give zeros, the latter
    set a bit; rows of one sequence at several positions each see their own keys."""
    cfg = cfg_for(12, 2, 128)
    c, *_ = make_cache(fmt, 2, 128, 16, [300, 77], 61)
    q = randn(62, 6, 12, 128)
    seq, pos = ints([0, 99, 0, 1, 0, -5]), ints([300, 0, 123, 77, 1, 0])
    out = attend(cfg, c, q, seq, pos, 300)
    assert status() == 0
    assert not out[1].any() and not out[5].any()
    hs = ints([0, 0, 0, 1, 0, 0])
    check_attn(cfg, c, q, hs, pos, out)
    for s, p, bits in ((2, 5, B.DEV_BAD_SEQ), (-1, 5, B.DEV_BAD_SEQ), (0, -1, B.DEV_BAD_POSITION),
                       (0, 301, B.DEV_BAD_POSITION), (1, 1 << 30, B.DEV_BAD_POSITION)):
        o = attend(cfg, c, q[:2], ints([s, 1]), ints([p, 77]), 300)
        assert status() == bits
        assert not o[0].any()
        check_attn(cfg, c, q[1:2], ints([1]), ints([77]), o[1:])
    o = attend(cfg, c, q[:3], ints([0] * 3), ints([0] * 3), 300)     # nothing at all
    assert status() == 0 and not o.any()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_attention_leaves_bad_pages_out(fmt):
    """Keys of an entry that names no page are left out and flagged: the result is that of the
    other keys."""
    cfg = cfg_for(6, 1, 128)
    c, k, v, *_ = make_cache(fmt, 1, 128, 16, [400], 71)
    q = randn(72, 1, 6, 128)
    good = c.page_table.clone()
    for entry in (-1, c.k.shape[0], 1 << 30):
        c.page_table[0, 3] = entry
        c.page_table[0, 24] = entry
        out = attend(cfg, c, q, ints([0]), ints([400]), 400)
        assert status() == B.DEV_BAD_PAGE
        c.page_table.copy_(good)
        # the same keys, as a sequence of the other pages
        hc = host(c)
        keep = [i for i in range(25) if i not in (3, 24)]
        hc.table = hc.table[:, keep]
        ref, mag = OP.paged_attention(6, np64(q), hc, [0], [16 * 23])
        tol = tolerance(cfg, hc, np64(q), [0], [16 * 23], ref, mag)
        assert np.all(np.abs(np64(out) - ref) <= tol)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("qe,ke,ve", [(0, 0, 60), (0, 0, -90), (60, -60, 0), (-40, 40, 3), (-100, 0, 0),
                                       (119, -122, 0)])
def test_attention_magnitudes(fmt, qe, ke, ve):
    """Queries, keys and values far from 1: the powers of two carry them."""
    cfg = cfg_for(4, 2, 128)
    n, page = 333, 64
    c = B.PagedKVCache.empty(7, page, 2, 128, ints([[6, 0, 5, 1, 2, 3]]), FMT[fmt])
    k = (randn(81, n, 2, 128).float() * 2.0 ** ke).to(torch.bfloat16)
    v = (randn(82, n, 2, 128, spread=2).float() * 2.0 ** ve).to(torch.bfloat16)
    B.beam_paged_kv_write(k, v, ints([0] * n), ints(list(range(1, n + 1))), c)
    q = (randn(83, 1, 4, 128).float() * 2.0 ** qe).to(torch.bfloat16)
    out = attend(cfg, c, q, ints([0]), ints([n]), n)
    assert status() == 0
    check_attn(cfg, c, q, ints([0]), ints([n]), out)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_attention_values_that_grow_along_the_sequence(fmt):
    """Value rows of steadily larger and then smaller magnitude (the accumulators' unit moves),
    and a sharp softmax."""
    cfg = cfg_for(6, 1, 64)
    n = 1100
    c = B.PagedKVCache.empty(40, 32, 1, 64, ints([list(range(39, 3, -1))]), FMT[fmt])
    ramp = torch.cat([torch.linspace(-12, 12, 700), torch.linspace(12, -12, 400)]).to(DEV)
    v = (randn(91, n, 1, 64).float() * torch.exp2(ramp.round())[:, None, None]).to(torch.bfloat16)
    k = randn(92, n, 1, 64)
    B.beam_paged_kv_write(k, v, ints([0] * n), ints(list(range(1, n + 1))), c)
    for scale in (1.0, 12.0):
        q = (randn(93, 1, 6, 64).float() * scale).to(torch.bfloat16)
        out = attend(cfg, c, q, ints([0]), ints([n]), n)
        assert status() == 0
        check_attn(cfg, c, q, ints([0]), ints([n]), out)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_attention_nan_rows_reach_their_readers_only(fmt):
    """A key or value row with a NaN makes the outputs that read it NaN, and no other."""
    cfg = cfg_for(4, 2, 128)
    c, k, v, seq, pos = make_cache(fmt, 2, 128, 16, [90, 90, 90], 101)
    k2, v2 = k.clone(), v.clone()
    k2[10, 0, 3] = float("nan")        # sequence 0, position 11, KV head 0
    v2[90 + 50, 1, 7] = float("nan")   # sequence 1, position 51, KV head 1
    B.beam_paged_kv_write(k2, v2, seq, pos, c)
    q = randn(102, 5, 4, 128)
    o = np64(attend(cfg, c, q, ints([0, 1, 2, 0, 1]), ints([90, 90, 90, 10, 50]), 90)).reshape(5, 4, 128)
    assert status() == 0
    assert np.all(np.isnan(o[0, :2])) and np.all(np.isfinite(o[0, 2:]))
    bad = np.isnan(o[1, 2:])
    assert np.all(np.isfinite(o[1, :2])) and np.all(bad if fmt != "bf16" else bad[:, 7])
    assert np.all(np.isfinite(o[2:]))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_attention_over_shared_pages(fmt):
    """Two sequences with a common prefix share its pages, a third repeats one page; a call with
    one row of each, and one whose every row is padding under a bound of 0."""
    cfg = cfg_for(6, 2, 64)
    c, *_ = make_cache(fmt, 2, 64, 32, [200, 150, 96], 231)
    c.page_table[1, :3] = c.page_table[0, :3]
    c.page_table[2, :3] = c.page_table[0, 1]
    q = randn(232, 3, 6, 64)
    seq, pos = ints([0, 1, 2]), ints([200, 150, 96])
    out = attend(cfg, c, q, seq, pos, 200)
    assert status() == 0
    check_attn(cfg, c, q, seq, pos, out)
    out = attend(cfg, c, q, seq, ints([0, 0, 0]), 0)
    assert status() == 0 and not out.any()
    out = attend(cfg, c, q, seq, pos, 0)
    assert status() == B.DEV_BAD_POSITION and not out.any()


def test_attention_many_rows():
    """More rows than one launch takes (1024): the slices share the workspace in order."""
    cfg = cfg_for(2, 1, 64)
    lens = [40, 7, 133]
    c, *_ = make_cache("fp8", 1, 64, 16, lens, 111)
    T = 1024 + 77
    r = np.random.default_rng(3)
    seq = r.integers(0, 3, T)
    pos = np.array([r.integers(0, lens[s] + 1) for s in seq])
    q = randn(112, T, 2, 64)
    out = attend(cfg, c, q, ints(seq.tolist()), ints(pos.tolist()), 133)
    assert status() == 0
    check_attn(cfg, c, q, ints(seq.tolist()), ints(pos.tolist()), out)


def test_attention_with_o_proj():
    """w_o given: the o_proj of the gated output, as beam_attn's, for one row (GEMV), a few, and
    from 64 rows (tensor-core GEMM)."""
    n_q, n_kv, D, H = 4, 2, 64, 264
    cfg = cfg_for(n_q, n_kv, D, hidden=H)
    w_o = (randn(121, H, n_q * D).float() * 0.05).to(torch.bfloat16)
    for T in (1, 5, 70):
        lens = [20 + 3 * i for i in range(T)]
        c, *_ = make_cache("bf16", n_kv, D, 16, lens, 122)
        q, g, bias = randn(123, T, n_q, D), randn(124, T, n_q * D), randn(125, n_q)
        seq, pos = ints(list(range(T))), ints(lens)
        og = attend(cfg, c, q, seq, pos, max(lens), g, bias)
        out = attend(cfg, c, q, seq, pos, max(lens), g, bias, w_o)
        assert status() == 0
        a, w = np64(og), np64(w_o)
        ref = a @ w.T
        # FP32 sums of n_q D exact products, then half a bf16 step
        tol = 2.0 ** -8 * np.abs(ref) + n_q * D * 2.0 ** -23 * (np.abs(a) @ np.abs(w).T)
        assert np.all(np.abs(np64(out) - ref) <= tol)


def test_attention_agrees_with_the_contiguous_cache():
    """beam_attn over a contiguous BF16 cache of the same keys: its output rounds once more."""
    n_q, n_kv, D, n = 12, 2, 128, 2300
    cfg = cfg_for(n_q, n_kv, D, hidden=256)
    c, k, v, *_ = make_cache("bf16", n_kv, D, 64, [n], 131, spread=0)
    kc = B.KVCache(k.permute(1, 0, 2)[None].contiguous(), v.permute(1, 0, 2)[None].contiguous())
    q, g, bias = randn(132, 1, n_q, D), randn(133, 1, n_q * D), randn(134, n_q)
    w_o = (randn(135, 256, n_q * D).float() * 0.05).to(torch.bfloat16)
    a = attend(cfg, c, q, ints([0]), ints([n]), n, g, bias, w_o)
    b = torch.empty_like(a)
    ws = torch.empty(B.workspace_bytes(cfg, 1, n), dtype=torch.uint8, device=DEV)
    B.beam_attn(cfg, q, g, bias, kc, ints([0]), ints([n]), n, w_o, b, ws, max_q_per_seq=1)
    assert status() == 0
    d = (a.float() - b.float()).abs().max() / b.float().abs().max()
    assert float(d) <= 2e-2


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_offsets_past_32_bits(fmt):
    """Pages past 4 GiB of codes (and of block scales): written, attended to and read back."""
    n_kv, D, page = 8, 128, 256
    per_page = n_kv * page * {"bf16": 256, "fp8": 128, "nvfp4": 64}[fmt]
    pages = (1 << 32) // per_page + 5
    if fmt == "nvfp4":
        pages = (1 << 32) // (n_kv * page * 2 * 8) + 5   # 4 GiB of block scales
    table = ints([[pages - 1, 0, pages - 2]])
    dims = (pages, n_kv, page, {"bf16": 128, "fp8": 128, "nvfp4": 64}[fmt])
    kind = torch.bfloat16 if fmt == "bf16" else torch.uint8
    row = None if fmt == "bf16" else torch.zeros((pages, n_kv, 2, page), dtype=torch.uint8, device=DEV)
    blk = torch.zeros((pages, n_kv, 2, page, 8), dtype=torch.uint8, device=DEV) if fmt == "nvfp4" else None
    c = B.PagedKVCache(torch.empty(dims, dtype=kind, device=DEV), torch.empty(dims, dtype=kind, device=DEV),
                       table, row, blk)
    n = 600
    k, v = randn(141, n, n_kv, D), randn(142, n, n_kv, D)
    seq, pos = ints([0] * n), ints(list(range(1, n + 1)))
    B.beam_paged_kv_write(k, v, seq, pos, c)
    # the same rows in a small cache give the same bits
    s, *_ = make_cache(fmt, n_kv, D, 16, [1], 143)
    s = B.PagedKVCache.empty(3, page, n_kv, D, ints([[0, 1, 2]]), FMT[fmt])
    B.beam_paged_kv_write(k, v, seq, pos, s)
    cfg = cfg_for(16, n_kv, D)
    q = randn(144, 1, 16, D)
    a, b = (attend(cfg, x, q, ints([0]), ints([n]), n) for x in (c, s))
    assert status() == 0 and torch.equal(a, b)
    got = []
    for x in (c, s):
        d = B.KVCache(*(torch.zeros((1, n_kv, n, D), dtype=torch.bfloat16, device=DEV) for _ in range(2)))
        B.beam_paged_kv_read(x, ints([0]), ints([1]), ints([n]), n, d)
        got.append(d)
    assert status() == 0 and torch.equal(got[0].k, got[1].k) and torch.equal(got[0].v, got[1].v)


# -------------------------------------------------------------- together, and replayed ----

@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_decode_steps_in_a_replayed_graph(fmt):
    """A decode loop as a server runs it: each step writes its rows and attends, captured once
    and replayed with positions, rows and page table updated in place, one row being padding.
    Every step is checked, and an eager run of the same steps gives the same bits."""
    n_q, n_kv, D, page = 12, 2, 128, 16
    cfg = cfg_for(n_q, n_kv, D)
    lens = [30, 500, 1]
    T = 4
    table = torch.full((4, 40), -1, dtype=torch.int32)
    nxt = 0
    for i, n in enumerate(lens):
        need = -(-(n + 6) // page)
        table[i, :need] = torch.arange(nxt, nxt + need)
        nxt += need

    def fresh():
        c = B.PagedKVCache.empty(nxt, page, n_kv, D, table.to(DEV), FMT[fmt])
        for i, n in enumerate(lens):
            B.beam_paged_kv_write(randn(150 + i, n, n_kv, D), randn(160 + i, n, n_kv, D, spread=1),
                                  ints([i] * n), ints(list(range(1, n + 1))), c)
        return c

    def step_inputs(s):
        return (randn(170 + s, T, n_kv, D), randn(180 + s, T, n_kv, D, spread=1), randn(190 + s, T, n_q, D),
                ints([n + 1 + s for n in lens] + [0]))

    seq = ints([0, 1, 2, 3])
    caches = [fresh(), fresh()]
    k, v, q, pos = step_inputs(0)
    ws = scratch(cfg, T, 512)
    out = torch.empty((T, n_q * D), dtype=torch.bfloat16, device=DEV)

    def step(c, st=None):
        B.beam_paged_kv_write(k, v, seq, pos, c, st)
        B.beam_paged_attn(cfg, q, None, None, c, seq, pos, 512, None, out, ws, st)

    step(caches[0])
    torch.cuda.synchronize()
    caches[0] = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(caches[0])
    for s in range(5):
        for dst, src in zip((k, v, q, pos), step_inputs(s)):
            dst.copy_(src)
        graph.replay()
        a = out.clone()
        check_attn(cfg, caches[0], q, ints([0, 1, 2, 0]), pos, a)
        step(caches[1])
        assert torch.equal(a, out) and not a[3].any()
    assert status() == 0
    assert torch.equal(caches[0].k, caches[1].k) and torch.equal(caches[0].v, caches[1].v)


def test_runs_are_repeatable_and_streams_are_used():
    """Calls on a side stream are ordered there (write, then attention, behind a slow producer),
    two streams with their own workspaces do not disturb one another, and repeated runs give the
    same bits."""
    cfg = cfg_for(12, 2, 128)
    lens = [3000, 900]
    c, k, v, seq, pos = make_cache("fp8", 2, 128, 32, lens, 201)
    q = randn(202, 2, 12, 128)
    s2, p2 = ints([0, 1]), ints(lens)
    ref = attend(cfg, c, q, s2, p2, 3000)
    torch.cuda.synchronize()
    for _ in range(3):
        assert torch.equal(attend(cfg, c, q, s2, p2, 3000), ref)
    other, *_ = make_cache("nvfp4", 2, 128, 32, lens, 203)
    ref2 = attend(cfg, other, q, s2, p2, 3000)
    torch.cuda.synchronize()
    st, st2 = torch.cuda.Stream(), torch.cuda.Stream()
    ws1, ws2 = scratch(cfg, 2, 3000), scratch(cfg, 2, 3000)
    o1, o2 = torch.zeros_like(ref), torch.zeros_like(ref)
    kk = torch.zeros_like(k)
    torch.cuda.synchronize()
    big = torch.randn(4096, 4096, device=DEV)
    for _ in range(4):
        with torch.cuda.stream(st):
            x = big
            for _ in range(3):
                x = x @ big
            kk.copy_(k)
        B.beam_paged_kv_write(kk, v, seq, pos, c, st)
        B.beam_paged_attn(cfg, q, None, None, c, s2, p2, 3000, None, o1, ws1, st)
        B.beam_paged_attn(cfg, q, None, None, other, s2, p2, 3000, None, o2, ws2, st2)
        torch.cuda.synchronize()
        assert torch.equal(o1, ref) and torch.equal(o2, ref2)
        kk.zero_()
        torch.cuda.synchronize()
    assert status() == 0


def test_bindings_refuse_wrong_tensors():
    cfg = cfg_for(4, 2, 64)
    c, *_ = make_cache("bf16", 2, 64, 16, [20], 211)
    q, seq, pos = randn(212, 1, 4, 64), ints([0]), ints([20])
    out, ws = torch.empty((1, 256), dtype=torch.bfloat16, device=DEV), scratch(cfg, 1, 20)

    def run(q=q, g=None, bias=None, c=c, seq=seq, pos=pos, out=out, ws=ws, w_o=None, max_pos=20):
        B.beam_paged_attn(cfg, q, g, bias, c, seq, pos, max_pos, w_o, out, ws)
    run()
    for kw in (dict(q=q.float()), dict(q=q[:, :2]), dict(seq=seq.long()), dict(pos=ints([1, 2])),
               dict(out=out.float()), dict(out=out[:, :128]), dict(g=randn(1, 1, 256)), dict(bias=randn(1, 4)),
               dict(w_o=randn(1, 256, 128)), dict(ws=ws[:1024]), dict(ws=ws[16:]), dict(max_pos=-1),
               dict(q=q.cpu()), dict(c=make_cache("bf16", 1, 64, 16, [20], 1)[0])):
        with pytest.raises(B.BeamError):
            run(**kw)
    dst = B.KVCache(torch.zeros((1, 2, 20, 64), dtype=torch.bfloat16, device=DEV),
                    torch.zeros((1, 2, 20, 64), dtype=torch.bfloat16, device=DEV))
    B.beam_paged_kv_read(c, seq, ints([1]), pos, 20, dst)
    with pytest.raises(B.BeamError):
        B.beam_paged_kv_read(c, seq, ints([1, 1]), pos, 20, dst)
    with pytest.raises(B.BeamError):
        B.beam_paged_kv_read(c, seq, ints([1]), pos, 20, B.KVCache(dst.k[:, :1].contiguous(), dst.v[:, :1].contiguous()))
    with pytest.raises(B.BeamError):
        B.beam_paged_kv_read(c, seq, ints([1]), pos, 20, B.KVCache(dst.k.view(torch.uint8), dst.v.view(torch.uint8)))
    assert status() == 0


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
@pytest.mark.parametrize("G", [5, 16])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_over_every_range(fmt, G, D):
    """More blocks than there are ranges on any GB300, so that every range writes partials: within
    a workspace of exactly the size asked for."""
    cfg, lens = cfg_for(8 * G, 8, D), [4000, 2500, 1900]
    c, *_ = make_cache(fmt, 8, D, 32, lens, 31)
    q, seq, pos = randn(33, 3, 8 * G, D), ints([2, 0, 1]), ints([1900, 4000, 2500])
    need = B.paged_workspace_bytes(cfg, 3, 4000)
    buf = torch.full((need + 65536,), 0x5A, dtype=torch.uint8, device=DEV)
    out = torch.full((3, 8 * G * D), 7.0, dtype=torch.bfloat16, device=DEV)
    B.beam_paged_attn(cfg, q, None, None, c, seq, pos, 4000, None, out, buf[:need])
    assert status() == 0
    check_attn(cfg, c, q, seq, pos, out)
    assert bool((buf[need:] == 0x5A).all())
