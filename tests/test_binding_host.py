"""The Python binding's own objects, without a GPU or the library."""
import copy
import ctypes
import dataclasses
import pickle

import pytest
import torch

import synth
from hybrid_attention_moe_gb300 import beam as B


def test_a_used_layer_cfg_copies_and_pickles():
    """As before its first use: the C struct that a call keeps is not part of it."""
    cfg = B.LayerCfg.from_shape(synth.BEAM, B.BEAM_ATTN_NOPE_SSMAX)
    fresh = copy.deepcopy(cfg)
    before = ctypes.addressof(cfg._ref()._obj)
    for made in (copy.copy(cfg), copy.deepcopy(cfg), pickle.loads(pickle.dumps(cfg)), dataclasses.replace(cfg)):
        assert made == cfg == fresh and type(made) is B.LayerCfg
        assert ctypes.addressof(made._ref()._obj) != before
        made.n_q = 24
        assert made._ref()._obj.n_q == 24 and cfg._ref()._obj.n_q == cfg.n_q == 48
    assert ctypes.addressof(cfg._ref()._obj) == before


def test_the_window_of_a_paged_cache_is_the_kernels_window():
    """Set again on a cache, it reaches the struct that the calls hand over."""
    c = object.__new__(B.PagedKVCache)
    c._c = B.PagedKVC(window=512)
    c.window = 16
    assert c.window == 16 and c._c.window == 16
    c.window = 0
    assert c.window == 0 and c._c.window == 0


@pytest.fixture
def calls(monkeypatch):
    """The paged entry points over CPU tensors: their checks run, and the library's answer is 0."""
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append(name) or 0

    monkeypatch.setattr(B, "_on_device", lambda cache: -1)
    monkeypatch.setattr(B, "_raw_stream", lambda stream, device: 0)
    monkeypatch.setattr(B, "lib", Lib)
    return seen


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


N_KV, N_Q, D, T = 2, 6, 64, 3


def cache():
    c = object.__new__(B.PagedKVCache)
    c.n_kv, c.head_dim, c.page_size, c._ref = N_KV, D, 16, None
    return c


def index():
    return z(T, dtype=torch.int32)


@pytest.mark.parametrize("shape,ok", [((T, N_KV, D), True), ((T, N_KV * D), True), ((T, D, N_KV), False),
                                      ((T, N_KV, 2, D // 2), False), ((T, N_KV * D, 1), False)])
def test_write_takes_the_documented_shapes_only(calls, shape, ok):
    """A tensor of as many elements in another order is refused, not read as something else."""
    def run(k, v):
        B.beam_paged_kv_write(k, v, index(), index(), cache())
    if ok:
        run(z(*shape), z(*shape))
        assert calls == ["beam_paged_kv_write"]
        return
    for k, v in ((z(*shape), z(*shape)), (z(T, N_KV, D), z(*shape)), (z(*shape), z(T, N_KV, D))):
        with pytest.raises(B.BeamError):
            run(k, v)
    assert not calls


@pytest.mark.parametrize("shape,ok", [((4, N_KV, 20, D), True), ((4, D, 20, N_KV), False), ((4, 20, N_KV, D), False)])
def test_read_takes_the_documented_shapes_only(calls, shape, ok):
    def run(k, v):
        B.beam_paged_kv_read(cache(), index(), index(), index(), 9, B.KVCache(k, v))
    if ok:
        run(z(*shape), z(*shape))
        assert calls == ["beam_paged_kv_read"]
        return
    for k, v in ((z(*shape), z(*shape)), (z(4, N_KV, 20, D), z(*shape))):
        with pytest.raises(B.BeamError):
            run(k, v)
    assert not calls


def attn(q=None, g=None, bias=None, w_o=None, out=None):
    cfg = B.LayerCfg.from_shape(synth.TINY, B.BEAM_ATTN_NOPE_SSMAX)
    cfg.n_q, cfg.n_kv, cfg.head_dim, cfg.hidden = N_Q, N_KV, D, 96
    B.beam_paged_attn(cfg, z(T, N_Q, D) if q is None else q, g, bias, cache(), index(), index(), 10, w_o,
                      z(T, N_Q * D) if out is None else out, z(256, dtype=torch.uint8))


def test_attn_takes_the_documented_shapes_only(calls):
    gate = dict(g=z(T, N_Q * D), bias=z(N_Q))
    proj = dict(w_o=z(96, N_Q * D), out=z(T, 96))
    good = [dict(), dict(q=z(T, N_Q * D)), dict(out=z(T, N_Q, D)), gate, dict(gate, g=z(T, N_Q, D)), proj]
    for kw in good:
        attn(**kw)
    assert calls == ["beam_paged_attn"] * len(good)
    for kw in (dict(q=z(T, D, N_Q)), dict(out=z(T, D, N_Q)), dict(out=z(N_Q * D, T)), dict(gate, g=z(T, D, N_Q)),
               dict(gate, g=z(1, T, N_Q * D)), dict(proj, w_o=z(N_Q * D, 96)), dict(proj, out=z(96, T))):
        with pytest.raises(B.BeamError):
            attn(**kw)
    assert len(calls) == len(good)


def test_a_cache_takes_the_documented_shapes_only():
    """(On the CPU every cache is refused at last; these are for their shapes.)"""
    u8, table = torch.uint8, z(1, 3, dtype=torch.int32)
    k, row, blk = z(3, 2, 16, 128, dtype=u8), z(3, 2, 2, 16, dtype=u8), z(3, 2, 2, 16, 16, dtype=u8)
    for args, name in (((k, k, table, row), "CUDA device"), ((k, k, table, row, blk), "CUDA device"),
                       ((k, k.view(3, 16, 2, 128), table, row), "v:"),
                       ((k, k, table, row.view(3, 2, 16, 2)), "row_scale"),
                       ((k, k, table, row.view(3, 2, 32)), "row_scale"),
                       ((k, k, table, row, blk.view(3, 2, 2, 256)), "block_scale"),
                       ((k, k, table, row, blk.transpose(3, 2).contiguous()), "block_scale")):
        with pytest.raises(B.BeamError, match=name):
            B.PagedKVCache(*args)
