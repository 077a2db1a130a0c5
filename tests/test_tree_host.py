"""Speculative decoding over the paged cache without a GPU: the oracle against closed forms and
enumeration, and the host-side argument checks of the entry points, which answer before any launch
(the 16-byte-aligned placeholder addresses are never dereferenced)."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import synth
from oracle import paged as OP
from oracle import tree as OT
from hybrid_attention_moe_gb300 import beam as B
from hybrid_attention_moe_gb300 import stack as S
from test_abi import lib  # noqa: F401  (the built library)
from test_paged_host import BAD_HANDLES, handle

P = ctypes.c_void_p
A, B_, C_ = 0x100000, 0x200000, 0x300000
WS = 1 << 28


# ------------------------------------------------------------------------ the oracle ----

def paged(n, n_kv, D, seed, window=0):
    r = np.random.default_rng(seed)
    pages = -(-n // 16)
    return OP.PagedKV("bf16", r.standard_normal((pages, n_kv, 16, D)), r.standard_normal((pages, n_kv, 16, D)),
                      np.arange(pages)[None], window=window)


@pytest.mark.parametrize("window", [0, 1, 4, 30])
def test_a_chain_is_causal_attention(window):
    c = paged(60, 2, 64, 1, window)
    q = np.random.default_rng(2).standard_normal((7, 4, 64))
    nodes = [set(range(j + 1)) for j in range(7)]
    got, mag, counts, *_ = OT.tree_attention(4, q, c, 0, 50, nodes)
    ref, rmag = OP.paged_attention(4, q, c, np.zeros(7, int), np.arange(51, 58))
    assert np.allclose(got, ref, rtol=1e-12, atol=1e-14) and np.allclose(mag, rmag, rtol=1e-12, atol=1e-14)
    assert list(counts) == [min(p, window) if window else p for p in range(51, 58)]


def test_branches_see_their_own_ancestors():
    """A branch of the tree is the chain of its nodes, moved to the front."""
    parent = [-1, 0, 1, 0, 3, 1]
    nodes = OT.masks(parent)
    assert nodes == [{0}, {0, 1}, {0, 1, 2}, {0, 3}, {0, 3, 4}, {0, 1, 5}]
    c = paged(48, 1, 64, 3)
    q = np.random.default_rng(4).standard_normal((6, 2, 64))
    got = OT.tree_attention(2, q, c, 0, 33, nodes)[0]
    d = OP.PagedKV("bf16", c.k, c.v, c.table)
    for to, src in ((1, 3), (2, 4)):
        for a in (d.k, d.v):
            a[(33 + to) // 16, :, (33 + to) % 16] = a[(33 + src) // 16, :, (33 + src) % 16]
    ref = OP.paged_attention(2, q[[0, 3, 4]], d, np.zeros(3, int), np.array([34, 35, 36]))[0]
    assert np.allclose(got[[0, 3, 4]], ref, rtol=1e-12, atol=1e-14)
    assert OT.masks([-1, 2, 0]) == [{0}, None, {0, 2}] and OT.masks([0, 0]) == [None, None]
    assert OT.bits({0, 63}) == 1 - (1 << 63) and OT.bits(None) == 0


def test_accept_follows_the_sampled_tokens():
    parent, token = [-1, 0, 0, 1, 2, 2], [9, 4, 5, 6, 6, 7]
    assert OT.accept(parent, token, [5, 6, 7, 1, 1, 3]) == ([0, 2, 5], 3)
    assert OT.accept(parent, token, [4, 6, 7, 1, 1, 3]) == ([0, 1, 3], 1)
    assert OT.accept(parent, token, [8, 6, 7, 1, 1, 3]) == ([0], 8)
    assert OT.accept([-1, 0, 0], [1, 2, 2], [2, 8, 9]) == ([0, 1], 8)   # the lowest of two
    assert OT.accept([], [], []) == ([], -1)


def test_rotation_keeps_lengths_and_scores_relative_positions():
    r = np.random.default_rng(5)
    a, b = r.standard_normal((2, 1, 1, 64))
    f = lambda x, p: OT.append_rows(x, None, [p], "rope", 1e4, 2048.0, 0.1, 1e-6, True)  # noqa: E731
    assert np.isclose((f(a, 9) ** 2).sum(), (a ** 2).sum()) and np.allclose(f(a, 1), a)
    assert np.isclose((f(a, 105) * f(b, 100)).sum(), (f(a, 6) * f(b, 1)).sum())
    s = OT.append_rows(a, None, [2048], "ssmax", 1e4, 2048.0, 0.1, 1e-6, True)
    assert np.allclose(s, a * 2 ** 0.1)
    n = OT.append_rows(a, np.ones(64), [1], "rope", 1e4, 2048.0, 0.1, 0.0, False)
    assert np.isclose((n ** 2).mean(), 1.0)


def test_kept_tokens_by_enumeration():
    """The kept set is the shortest prefix, in order of the logits, that each rule allows."""
    r = np.random.default_rng(6)
    for z in (r.standard_normal(7) * 2, np.array([1.0, 3, 3, -np.inf, 3, 0, 1])):
        for t, k, p, m in itertools.product((0.5, 1.0), (0, 1, 3, 9), (0.0, 0.4, 0.9, 1.0), (0.0, 0.3, 1.0, 2.0)):
            order = sorted(range(7), key=lambda i: (-z[i], i))[:k or 7]
            w = [np.exp((z[i] - max(z)) / t) for i in order]
            if p < 1:
                order = order[:max(1, next(n for n in range(8) if sum(w[:n]) >= p * sum(w) - 1e-15))]
            keep = [i for i in order if m == 0 or np.exp((z[i] - max(z)) / t) >= min(m, 1.0) * (1 - 1e-12)]
            assert list(OT.kept(z, t, k, p, m)) == sorted(keep), (z, t, k, p, m)
    assert list(OT.kept(np.array([1.0, 2, 2]), 0.0, 0, 1.0, 0.0)) == [1]


def test_sampled_tokens_have_their_shares():
    z, t = np.log([1.0, 4.0, 2.0, 1.0]), 1.0
    got = [OT.sample(z, u, t)[0] for u in (np.arange(800) + 0.5) / 800]
    assert [got.count(i) for i in range(4)] == [100, 400, 200, 100]
    tok, lp = OT.sample(z, 0.0, t, 2)
    assert tok == 1 and abs(lp - np.log(4 / 6)) < 1e-12 and OT.sample(z, 0.999, t, 2)[0] == 2
    assert OT.sample([np.nan, 1.0], 0.5)[0] == OT.sample([np.inf, 1.0], 0.5)[0] == OT.sample([-np.inf], 0.5)[0] == -1


# ------------------------------------------------------------------- argument checks ----

def cfg(**kw):
    c = B.LayerCfg.from_shape(synth.BEAM, B.BEAM_ATTN_NOPE_SSMAX)
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c.c())


def append(L, cf=None, z=A, stride=14336, qn=A, kn=A, seq=C_, pos=C_, slot=None, T=1, q=B_, g=B_, h=None):
    return L.beam_paged_append(cf or cfg(), P(z), stride, P(qn), P(kn), P(seq), P(pos), P(slot), T, P(q), P(g),
                               ctypes.byref(h or handle()), None)


def project(L, cf=None, u=A, w=B_, qn=A, kn=A, seq=C_, pos=C_, T=1, q=B_, g=B_, h=None, ws=A, n=WS):
    return L.beam_paged_qkv_gate(cf or cfg(), P(u), P(w), P(qn), P(kn), P(seq), P(pos), None, T, P(q), P(g),
                                 ctypes.byref(h or handle()), P(ws), n, None)


def attend(L, cf=None, q=A, g=None, bias=None, h=None, seq=C_, start=C_, base=C_, mask=C_, N=1, T=1, most=50,
           w_o=None, out=B_, ws=A, n=WS):
    return L.beam_paged_tree_attn(cf or cfg(), P(q), P(g), P(bias), ctypes.byref(h or handle()), P(seq), P(start),
                                  P(base), P(mask), N, T, most, P(w_o), P(out), P(ws), n, None)


def keep(L, h=None, seq=C_, base=C_, count=C_, path=C_, stride=8, N=1):
    return L.beam_paged_kv_keep(ctypes.byref(h or handle()), P(seq), P(base), P(count), P(path), stride, N, None)


@pytest.mark.parametrize("i", range(len(BAD_HANDLES)))
def test_bad_handles_are_refused(lib, i):  # noqa: F811
    kw, want = BAD_HANDLES[i]
    for f in (append, project, attend, keep):
        assert f(lib, h=handle(**kw)) == want


def test_append_argument_checks(lib):  # noqa: F811
    assert append(lib, T=0) == 0 and append(lib, T=0, z=None, q=None) == 0
    for kw in (dict(T=-1), dict(z=None), dict(z=A + 8), dict(seq=None), dict(pos=None), dict(q=None), dict(q=B_ + 2),
               dict(g=B_ + 4), dict(qn=None), dict(kn=None), dict(qn=A + 2), dict(stride=14328), dict(stride=14340),
               dict(g=None, stride=8184), dict(cf=cfg(n_kv=4)), dict(cf=cfg(head_dim=64)), dict(cf=cfg(kind=3)),
               dict(cf=cfg(eps=float("nan")))):
        assert append(lib, **kw) == 1, kw
    assert append(lib, cf=cfg(n_q=136)) == 2


def test_project_argument_checks(lib):  # noqa: F811
    assert project(lib, T=0) == 0
    for kw in (dict(T=-1), dict(u=None), dict(u=A + 8), dict(w=None), dict(w=B_ + 2), dict(qn=None), dict(kn=None),
               dict(seq=None), dict(pos=None), dict(q=None), dict(g=None), dict(g=B_ + 8), dict(ws=None),
               dict(ws=A + 16), dict(n=14336 * 2 - 1), dict(cf=cfg(n_kv=4)), dict(cf=cfg(hidden=5124))):
        assert project(lib, **kw) == 1, kw


def test_attention_argument_checks(lib):  # noqa: F811
    assert attend(lib, T=0) == 0 and attend(lib, T=0, N=0, q=None) == 0
    need = lib.beam_paged_tree_workspace_bytes(cfg(), 1)
    for kw in (dict(T=-1), dict(N=-1), dict(N=0), dict(most=-1), dict(q=None), dict(q=A + 8), dict(g=A), dict(bias=A),
               dict(g=A + 8, bias=A), dict(seq=None), dict(start=None), dict(base=None), dict(mask=None),
               dict(mask=C_ + 4), dict(out=None), dict(out=B_ + 8), dict(w_o=A + 8), dict(ws=None), dict(ws=A + 128),
               dict(n=0), dict(w_o=A, n=need - 256), dict(cf=cfg(n_kv=4)), dict(cf=cfg(head_dim=64))):
        assert attend(lib, **kw) == 1, kw
    assert attend(lib, cf=cfg(n_q=136)) == 2
    assert attend(lib, most=2 ** 31 - 1, N=1024, h=handle(table_stride=1 << 26)) == 2   # costs past 32 bits
    assert lib.beam_paged_tree_workspace_bytes(None, 1) == lib.beam_paged_tree_workspace_bytes(cfg(), 0) == 256
    assert need % 256 == 0 and lib.beam_paged_tree_workspace_bytes(cfg(), 65) - need == 64 * 48 * 128 * 2


def test_bookkeeping_argument_checks(lib):  # noqa: F811
    a = P(A)
    plan, acc = lib.beam_tree_plan, lib.beam_tree_accept
    assert plan(a, a, a, a, 1, 0, a, a, a, a, None) == 0 and plan(*[None] * 4, 0, 0, *[None] * 5) == 0
    good = [a, a, a, a, 1, 1, a, a, a, a, None]
    for i, x in ((0, None), (1, None), (2, None), (3, None), (4, 0), (4, -1), (5, -1), (6, None), (6, P(A + 4)), (7, None),
                 (8, None), (9, None)):
        assert plan(*good[:i], x, *good[i + 1:]) == 1, (i, x)
    assert acc(a, a, a, a, 0, 1, a, a, 4, a, None) == 0
    good = [a, a, a, a, 1, 1, a, a, 4, a, None]
    for i, x in ((0, None), (1, None), (2, None), (3, None), (4, -1), (5, -1), (6, None), (7, None), (8, 0), (9, None)):
        assert acc(*good[:i], x, *good[i + 1:]) == 1, (i, x)
    assert keep(lib, N=0) == 0
    for kw in (dict(N=-1), dict(stride=0), dict(seq=None), dict(base=None), dict(count=None), dict(path=None)):
        assert keep(lib, **kw) == 1, kw
    assert keep(lib, h=handle(n_kv=70000)) == 2


def test_sample_argument_checks(lib):  # noqa: F811
    def f(z=A, stride=100, T=1, V=100, u=A, token=A):
        return lib.beam_sample(P(z), stride, T, V, P(u), None, None, None, None, P(token), None, None)
    assert f(T=0) == 0 and f(T=0, z=None, token=None) == 0
    for kw in (dict(T=-1), dict(V=0), dict(V=-5), dict(stride=99), dict(z=None), dict(u=None), dict(token=None)):
        assert f(**kw) == 1, kw
    assert f(V=851969, stride=851969) == 2 and f(T=65536) == 2


def test_bindings_refuse_tensors_of_the_host():
    x, i = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: B.beam_sample(x, x[:, 0], i), lambda: B.beam_tree_plan(i, i, i, i, i, i, i, i),
                 lambda: B.beam_tree_accept(i, i, i, i, i, i, i)):
        with pytest.raises((B.BeamError, AssertionError, RuntimeError)):
            call()


def test_verify_needs_pages_in_every_layer():
    st = S.BeamStack(synth.TINY, [], [object()], device="cpu")
    with pytest.raises(B.BeamError):
        st.verify(torch.zeros(1, 8), None, None, None, None, 1)


def test_accept_takes_no_failed_sample_and_no_lost_root():
    assert OT.accept([-1, 0, 1], [5, -1, 6], [-1, 6, 7]) == ([0], -1)
    assert OT.accept([-1, 0], [5, -7], [-7, 1]) == ([0], -7)
    assert OT.accept([0, 0], [1, 2], [2, 3]) == OT.accept([-2, 0], [1, 2], [2, 3]) == ([], -1)


def test_logprobs_are_those_of_the_logits():
    """Of a weight of one step of 2^-44 too: 30 nats below the largest, log(1 / 2^44) would be 0.5 off."""
    for d in (1.0, 20.0, 30.0):
        tok, lp = OT.sample([-d, 0.0, -1.0], 0.0)
        assert tok == 0 and abs(lp - (-d - np.log(1 + np.exp(-1) + np.exp(-d)))) < 1e-12


def test_keep_needs_pages_in_every_layer():
    """Before the first layer's rows are moved."""
    st = S.BeamStack(synth.TINY, [], [object()], device="cpu")
    with pytest.raises(B.BeamError):
        st.keep(None, None, None, None)
