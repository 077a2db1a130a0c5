"""The paged cache without a GPU: the oracle's row formats against torch and closed forms, and
the host-side argument checks of its entry points, which answer before any launch (the
16-byte-aligned placeholder addresses are never dereferenced)."""
import ctypes

import numpy as np
import pytest
import torch

import synth
from oracle import paged as OP
from oracle.codecs import e4m3_decode
from test_abi import lib  # noqa: F401  (the built library)

P = ctypes.c_void_p
A, B_, C_ = 0x100000, 0x200000, 0x300000


def rows(seed, n, D, spread=True):
    r = np.random.default_rng(seed)
    x = r.standard_normal((n, D))
    if spread:
        x *= np.exp2(r.integers(-60, 60, (n, 1)))
    return torch.from_numpy(x).to(torch.bfloat16).double().numpy()


def test_e2m1_encode_matches_nearest_code_and_ties():
    grid = np.array([0, .5, 1, 1.5, 2, 3, 4, 6])
    x = np.linspace(-7, 7, 5601)
    v = np.where(OP.e2m1_encode(x) >= 8, -1, 1) * grid[OP.e2m1_encode(x) & 7]
    # the distance to the code's value is the least there is
    assert np.allclose(np.abs(v - x), np.min(np.abs(np.concatenate([grid, -grid])[None] - x[:, None]), 1))
    # midpoints: 0.25 -> 0, 0.75 -> 1, 1.25 -> 1, 1.75 -> 2, 2.5 -> 2, 3.5 -> 4, 5 -> 4
    ties = OP.e2m1_encode(np.array([.25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, 9.0]))
    assert list(ties) == [0, 2, 2, 4, 4, 6, 6, 7]


@pytest.mark.parametrize("fmt,most", [("fp8", 448.0), ("nvfp4", 2688.0)])
def test_row_byte_is_the_least_that_fits(fmt, most):
    x = rows(1, 400, 64)
    b = OP.row_byte(x, fmt).astype(int)
    amax = np.abs(x).max(1)
    assert np.all(amax <= most * 2.0 ** (b - 127)) and np.all(amax > most * 2.0 ** (b - 128))
    edge = np.zeros((4, 64))
    edge[0, 3], edge[1, 3], edge[3, 0] = most, most * (1 + 2.0 ** -7), np.inf
    assert list(OP.row_byte(edge, fmt)) == [127, 128, 0, 255]
    tiny = np.full((1, 64), 2.0 ** -133)          # bf16's smallest magnitude
    assert OP.row_byte(tiny, fmt)[0] == 0


def test_fp8_rows_match_torch():
    x = rows(2, 300, 128)
    codes, b, _ = OP.quantise(x, "fp8")
    y = torch.from_numpy(x * 2.0 ** (127.0 - b.astype(float))[:, None]).float()
    assert np.array_equal(codes, y.to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    # half a step: 2^-4 relative, or half of 2^-9 in the subnormal range
    v = OP.dequantise(codes, b, None, "fp8")
    assert np.all(np.abs(v - x) <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** (b.astype(float) - 137)[:, None]))


def test_nvfp4_rows_stay_within_half_a_step():
    x = rows(3, 300, 128)
    codes, b, s = OP.quantise(x, "nvfp4")
    v = OP.dequantise(codes, b, s, "nvfp4")
    step = (e4m3_decode(s).repeat(16, axis=1) * 2.0 ** (b.astype(float) - 127)[:, None])
    # steps of the grid: 0.5 below 2, 1 to 4, 2 to 6; saturation adds at most 6/16 of the scale
    # (the scale is e4m3(max / 6): at most half a step, 2^-4, or 2^-10 absolute, too small)
    y = np.abs(x) / np.where(step > 0, step, 1)
    half = np.where(y <= 2, 0.25, np.where(y <= 4, 0.5, 1.0))
    assert np.all((np.abs(v - x) <= half * step * (1 + 1e-12)) | (step == 0))
    assert np.all(v[step == 0] == 0)


def test_non_finite_and_zero_rows():
    # the third row's element is stored exactly: 1 = 1 * 2^0, 1.3125 = 6 * 448 * 2^-11
    for fmt, one in (("fp8", 1.0), ("nvfp4", 1.3125)):
        x = np.zeros((4, 64))
        x[0, 5], x[1, 6], x[2, 7] = np.nan, -np.inf, one
        codes, b, s = OP.quantise(x, fmt)
        v = OP.dequantise(codes, b, s, fmt)
        assert np.all(np.isnan(v[:2])) and np.all(codes[:2] == 0) and v[2, 7] == one
        assert b[3] == 0 and np.all(v[3] == 0)


def handle(**kw):
    from hybrid_attention_moe_gb300 import beam as B
    d = dict(k=A, v=B_, row_scale=0, block_scale=0, page_table=C_, dtype=0, num_pages=10,
             page_size=16, n_kv=8, head_dim=128, num_seqs=2, table_stride=4, window=0)
    d.update(kw)
    return B.PagedKVC(*[d[n] for n, _ in B.PagedKVC._fields_])


BAD_HANDLES = [
    (dict(k=0), 1), (dict(page_table=0), 1), (dict(k=A + 8), 1), (dict(v=B_ + 4), 1),
    (dict(page_table=C_ + 2), 1), (dict(dtype=3), 1), (dict(dtype=-1), 1), (dict(num_pages=0), 1),
    (dict(num_seqs=0), 1), (dict(table_stride=0), 1), (dict(window=-1), 1), (dict(n_kv=0), 1),
    (dict(row_scale=A), 1),                                  # scales on a BF16 cache
    (dict(dtype=1), 1), (dict(dtype=1, row_scale=A + 1), 1),  # FP8 without, or misaligned
    (dict(dtype=1, row_scale=A, block_scale=A), 1),
    (dict(dtype=2, row_scale=A), 1),
    (dict(head_dim=96), 2), (dict(head_dim=256), 2),
    (dict(page_size=8), 2), (dict(page_size=48), 2), (dict(page_size=512), 2),
    (dict(dtype=2, row_scale=A, block_scale=A, head_dim=64, page_size=16), 2),
    (dict(table_stride=1 << 28), 2), (dict(num_pages=1 << 29), 2),
]


@pytest.mark.parametrize("i", range(len(BAD_HANDLES)))
def test_bad_handles_are_refused_by_every_call(lib, i):  # noqa: F811
    from hybrid_attention_moe_gb300 import beam as B
    kw, want = BAD_HANDLES[i]
    h = handle(**kw)
    hr = ctypes.byref(h)
    kc = B.KVCacheC(A, B_, 0, 1.0, 1.0, 4, 64, 0)
    cfg = B.LayerCfg.from_shape(synth.BEAM, B.BEAM_ATTN_NOPE_SSMAX).c()
    assert lib.beam_paged_kv_write(P(A), P(B_), 1024, P(C_), P(C_), 1, hr, None) == want
    assert lib.beam_paged_kv_read(hr, P(A), P(A), P(A), 1, 10, ctypes.byref(kc), None) == want
    got = lib.beam_paged_attn(ctypes.byref(cfg), P(A), None, None, hr, P(C_), P(C_), 1, 10, None,
                              P(B_), P(A), 1 << 23, None)
    assert got == want


def test_write_argument_checks(lib):  # noqa: F811
    h = ctypes.byref(handle())
    a, b, c = P(A), P(B_), P(C_)
    w = lib.beam_paged_kv_write
    assert w(a, b, 1024, c, c, 0, h, None) == 0                 # no tokens: nothing
    assert w(None, None, 1024, None, None, 0, h, None) == 0
    assert w(a, b, 1024, c, c, -1, h, None) == 1
    assert w(None, b, 1024, c, c, 1, h, None) == 1
    assert w(a, P(B_ + 2), 1024, c, c, 1, h, None) == 1
    assert w(a, b, 1016, c, c, 1, h, None) == 1                 # shorter than a token's rows
    assert w(a, b, 1028, c, c, 1, h, None) == 1                 # not a multiple of 8
    assert w(a, b, 1024, None, c, 1, h, None) == 1
    assert w(a, b, 1024, c, c, 1 << 28, h, None) == 2
    assert w(a, b, 1024, c, c, 1, None, None) == 1


def test_read_argument_checks(lib):  # noqa: F811
    from hybrid_attention_moe_gb300 import beam as B
    h = ctypes.byref(handle())
    a = P(A)

    def read(N=1, max_len=10, dst=B.KVCacheC(A, B_, 0, 1.0, 1.0, 4, 64, 0), seq=a, first=a, last=a):
        return lib.beam_paged_kv_read(h, seq, first, last, N, max_len,
                                      None if dst is None else ctypes.byref(dst), None)
    assert read(N=0) == 0 and read(max_len=0) == 0
    assert read(N=-1) == 1 and read(max_len=-1) == 1 and read(N=5) == 1   # 4 rows in dst
    assert read(seq=None) == 1 and read(first=None) == 1 and read(last=None) == 1
    assert read(dst=None) == 1
    assert read(dst=B.KVCacheC(A + 2, B_, 0, 1.0, 1.0, 4, 64, 0)) == 1
    assert read(dst=B.KVCacheC(A, B_, 0, 1.0, 1.0, 4, 0, 0)) == 1
    assert read(dst=B.KVCacheC(A, B_, 1, 1.0, 1.0, 4, 64, 0)) == 2        # an FP8 destination
    assert read(N=70000, dst=B.KVCacheC(A, B_, 0, 1.0, 1.0, 70000, 64, 0)) == 2


def test_attn_argument_checks(lib):  # noqa: F811
    from hybrid_attention_moe_gb300 import beam as B
    import dataclasses
    a, b, c = P(A), P(B_), P(C_)
    beam = synth.BEAM

    def attn(shape=beam, h=handle(), q=a, g=None, gb=None, seq=c, pos=c, T=1, max_pos=10, wo=None,
             out=b, ws=a, n=1 << 23):
        cfg = B.LayerCfg.from_shape(shape, B.BEAM_ATTN_NOPE_SSMAX).c()
        return lib.beam_paged_attn(ctypes.byref(cfg), q, g, gb, ctypes.byref(h), seq, pos, T,
                                   max_pos, wo, out, ws, n, None)
    assert attn(T=0) == 0
    assert attn(T=-1) == 1 and attn(max_pos=-1) == 1
    assert attn(q=None) == 1 and attn(out=None) == 1 and attn(ws=None) == 1
    assert attn(seq=None) == 1 and attn(pos=None) == 1
    assert attn(g=a) == 1 and attn(gb=a) == 1                       # the gate's halves go together
    assert attn(q=P(A + 8)) == 1 and attn(out=P(A + 8)) == 1 and attn(ws=P(A + 16)) == 1
    assert attn(h=handle(n_kv=4)) == 1 and attn(h=handle(head_dim=64)) == 1
    assert attn(shape=dataclasses.replace(beam, n_q=8 * 17)) == 2   # 17 query heads per KV head
    cfg = B.LayerCfg.from_shape(beam, B.BEAM_ATTN_NOPE_SSMAX)
    assert attn(n=1 << 16) in (1, 2)      # workspace too small (2: no driver here to encode maps)
    # 1024 rows over 8 heads of 2^30 keys: flat block numbers would pass 32 bits
    big = handle(table_stride=1 << 26, page_size=16)
    assert attn(h=big, T=1024, max_pos=1 << 30) == 2
    assert B.paged_workspace_bytes(cfg, 1, 100) <= (8 << 20) + 48 * 128 * 2
    assert B.paged_workspace_bytes(cfg, 300, 100) <= (8 << 20) + 300 * 48 * 128 * 2


def test_paged_bytes(lib):  # noqa: F811
    from hybrid_attention_moe_gb300 import beam as B
    # per key and KV head, K and V: 512 B, 2 x 129 B, 2 x (64 + 8 + 1) B at head_dim 128
    assert B.paged_kv_bytes(1, 1, 16, 128) == 16 * 512
    assert B.paged_kv_bytes(10, 8, 64, 128, B.BEAM_PAGED_FP8) == 10 * 8 * 64 * 258
    assert B.paged_kv_bytes(10, 8, 64, 128, B.BEAM_PAGED_NVFP4) == 10 * 8 * 64 * 146
    assert B.paged_kv_bytes(1 << 22, 8, 64, 128) == (1 << 22) * 8 * 64 * 512
    assert B.paged_kv_bytes(1, 1, 16, 128, 7) == 0


def test_binding_refuses_wrong_tensors():
    from hybrid_attention_moe_gb300 import beam as B
    k = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16)
    table = torch.zeros((1, 3), dtype=torch.int32)
    for bad in (lambda: B.PagedKVCache(k, k, table.long()),
                lambda: B.PagedKVCache(k.float(), k.float(), table),
                lambda: B.PagedKVCache(k, k[:2], table),
                lambda: B.PagedKVCache(k.transpose(1, 2), k.transpose(1, 2), table),
                lambda: B.PagedKVCache(k[0], k[0], table),
                lambda: B.PagedKVCache(k, k, table, row_scale=torch.zeros((3, 2, 2, 16), dtype=torch.uint8)),
                lambda: B.PagedKVCache(k, k, table, block_scale=torch.zeros((3, 2, 2, 16, 4), dtype=torch.uint8))):
        with pytest.raises((B.BeamError, RuntimeError)):
            bad()


def test_stack_takes_paged_layers(monkeypatch):
    """BeamStack over paged caches (recorded calls, no kernel): up to PAGED_MAX_Q tokens per
    sequence write and attend in the pages; more read the context back for beam_attn, with the
    range of each sequence that has tokens in the call."""
    from hybrid_attention_moe_gb300 import beam as B
    from hybrid_attention_moe_gb300 import stack as S
    shape = synth.TINY
    W = [synth.layer_weights(shape, layer, 0) for layer in range(2)]

    def paged(window):
        c = object.__new__(B.PagedKVCache)
        c.page_table, c.window = torch.zeros((4, 5), dtype=torch.int32), window
        return c

    caches = [paged(shape.window), B.KVCache(torch.zeros(1), torch.zeros(1), 0)]
    st = S.BeamStack(shape, W, caches, device="cpu")
    seen = []
    for name in ("beam_qkv_gate", "beam_attn", "beam_boundary_norm", "beam_dense_mlp", "beam_route",
                 "beam_moe", "beam_paged_kv_write", "beam_paged_kv_read", "beam_paged_attn"):
        monkeypatch.setattr(B, name, lambda *a, _n=name, **k: seen.append((_n, a)))
    monkeypatch.setattr(B, "workspace_bytes", lambda *a: 100)
    monkeypatch.setattr(B, "paged_workspace_bytes", lambda *a: 5000)

    def forward(seq, pos, max_q):
        seen.clear()
        e = torch.zeros((len(seq), shape.hidden), dtype=torch.bfloat16)
        st.forward(e, torch.tensor(seq, dtype=torch.int32), torch.tensor(pos, dtype=torch.int32),
                   max(pos), max_q_per_seq=max_q)
        names = [n for n, _ in seen if n not in ("beam_boundary_norm", "beam_dense_mlp",
                                                 "beam_route", "beam_moe")]
        return names, dict(reversed(seen))     # the first call of each name

    names, args = forward([2, 0], [30, 7], 1)
    assert names == ["beam_qkv_gate", "beam_paged_kv_write", "beam_paged_attn", "beam_qkv_gate", "beam_attn"]
    stage = args["beam_qkv_gate"][9]
    assert stage.window == 1 and stage.k.shape == (2, shape.n_kv, 1, shape.head_dim)
    assert args["beam_qkv_gate"][5].tolist() == [0, 1]          # a staging row per token
    k, v, seq, pos, cache = args["beam_paged_kv_write"][:5]
    assert k.shape == (2, shape.n_kv, shape.head_dim) and k.data_ptr() == stage.k.data_ptr()
    assert seq.tolist() == [2, 0] and cache is caches[0]
    assert args["beam_paged_attn"][10].numel() >= 5000

    n = 9
    names, args = forward([2] * n + [0] * 6, list(range(30, 30 + n)) + list(range(1, 7)), n)
    assert names == ["beam_qkv_gate", "beam_paged_kv_write", "beam_paged_kv_read", "beam_attn",
                     "beam_qkv_gate", "beam_attn"]
    cache, every, first, last, longest, copy = args["beam_paged_kv_read"][:6]
    w = shape.window
    assert every.tolist() == [0, 1, 2, 3] and last.tolist() == [6, 0, 38, 0]
    assert first.tolist() == [1, 1, 30 - w + 1, 1] and longest == w - 1 + n
    assert copy.window == w and copy.k.shape[2] >= longest and copy.k.shape[2] % 128 == 0
    assert args["beam_attn"][4] is copy
    # sequence ids that name nothing do not reach the ranges
    names, args = forward([-1, 99] + [1] * 5, [50, 60, 3, 4, 5, 6, 7], 5)
    assert args["beam_paged_kv_read"][3].tolist() == [0, 7, 0, 0]


@pytest.mark.parametrize("bad", [(0, 0), (2, 0), (2, -7), (0, 39), (0, 10 ** 6), (-1, 3), (4, 3)])
@pytest.mark.parametrize("windowed", [False, True])
def test_context_of_a_chunk_with_a_bad_token(bad, windowed):
    """The ranges that a paged prefill reads back do not depend on tokens that the library flags."""
    from hybrid_attention_moe_gb300 import beam as B
    from hybrid_attention_moe_gb300 import stack as S
    st = object.__new__(S.BeamStack)
    st.shape, st.device, st._copies = synth.TINY, "cpu", {}
    kc = object.__new__(B.PagedKVCache)
    kc.page_table, kc.window = torch.zeros((4, 5), dtype=torch.int32), synth.TINY.window if windowed else 0
    seq, pos, n, most = [2] * 9 + [0] * 6, list(range(30, 39)) + list(range(1, 7)), 9, 38

    def ranges(seq, pos):
        s, p = (torch.tensor(x, dtype=torch.int32) for x in (seq, pos))
        _, every, first, last, longest = st.context(kc, s, p, most, n)
        return every.tolist(), first.tolist(), last.tolist(), longest

    assert ranges(seq + [bad[0]], pos + [bad[1]]) == ranges(seq, pos)
