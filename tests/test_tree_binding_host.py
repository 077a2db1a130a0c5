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
