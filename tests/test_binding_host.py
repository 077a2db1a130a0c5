"""The Python binding's own objects, without a GPU or the library."""
import copy
import ctypes
import dataclasses
import pickle

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
