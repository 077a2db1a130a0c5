"""The bindings of a step of speculative decoding over the paged cache, without a GPU or the library."""
import pytest
import torch

import synth
from hybrid_attention_moe_gb300 import beam as B
from test_binding_host import D, N_KV, N_Q, T, cache, calls, index, z  # noqa: F401  (calls: a fixture)

WIDTH = (2 * N_Q + 2 * N_KV) * D


def cfg():
    c = B.LayerCfg.from_shape(synth.TINY, B.BEAM_ATTN_NOPE_SSMAX)
    c.n_q, c.n_kv, c.head_dim, c.hidden = N_Q, N_KV, D, 96
    return c


def append(qkv=None, q=None, g=None):
    i = index()[:2] if qkv is not None else index()
    n = i.numel()
    B.beam_paged_append(cfg(), z(T, WIDTH) if qkv is None else qkv, None, None, i, i, None, z(n, N_Q, D) if q is None else q,
                        z(n, N_Q * D) if g is None else g, cache())


def test_append_refuses_tokens_further_apart_than_an_int_says(calls):  # noqa: F811
    """The entry point takes the distance as an int, and would take the rest of one past 2^31 for it. (Tensors without
    storage: the library is not there.)"""
    def rows(step):
        return torch.empty_strided((2, WIDTH), (step, 1), dtype=torch.bfloat16, device="meta")
    for step in (1 << 31, (1 << 32) + WIDTH, (1 << 35) + 8 * WIDTH):
        with pytest.raises(B.BeamError):
            append(rows(step))
    assert not calls
    append(rows((1 << 31) - 8))
    assert calls == ["beam_paged_append"]


def project(q=None, g=None):
    B.beam_paged_qkv_gate(cfg(), z(T, 96), z(WIDTH, 96), z(D), z(D), index(), index(), None, z(T, N_Q, D) if q is None else q,
                          z(T, N_Q * D) if g is None else g, cache(), z(256, dtype=torch.uint8))


@pytest.mark.parametrize("call", [append, project])
def test_rows_are_written_into_the_documented_shapes_only(calls, call):  # noqa: F811
    """A tensor of as many elements in another order is refused, not written as something else."""
    good = [dict(), dict(q=z(T, N_Q * D)), dict(g=z(T, N_Q, D))]
    for kw in good:
        call(**kw)
    assert len(calls) == len(good)
    for kw in (dict(q=z(T, D, N_Q)), dict(q=z(N_Q, T, D)), dict(q=z(T * N_Q * D)), dict(g=z(T, D, N_Q)), dict(g=z(N_Q * D, T)),
               dict(q=z(T, N_Q, D).float()), dict(g=z(T, N_Q - 1, D))):
        with pytest.raises(B.BeamError):
            call(**kw)
    assert len(calls) == len(good)
