"""The paged cache's Python objects and their checks on a GPU."""
import copy
import pickle

import pytest
import torch

from hybrid_attention_moe_gb300 import beam as B
from test_gpu_paged import attend, cfg_for, check_attn, ints, make_cache, randn, status

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "nvfp4"])
def test_window_set_again_and_copies(fmt):
    """Attention follows the cache's window attribute; copies of a cache are caches: a deep copy and
    a pickled one with pages of their own, a copy over the same pages with a window of its own."""
    cfg = cfg_for(6, 2, 64)
    c, k, v, s, p = make_cache(fmt, 2, 64, 32, [700, 90], 401)
    q, seq, pos = randn(402, 2, 6, 64), ints([0, 1]), ints([700, 90])
    whole = attend(cfg, c, q, seq, pos, 700)
    check_attn(cfg, c, q, seq, pos, whole)
    for w in (100, 5, 0):
        c.window = w
        out = attend(cfg, c, q, seq, pos, 700)
        check_attn(cfg, c, q, seq, pos, out)
        assert torch.equal(out, whole) == (w == 0)
    deep, same, loaded = copy.deepcopy(c), copy.copy(c), pickle.loads(pickle.dumps(c))
    same.window = 7
    assert c.window == 0 and torch.equal(attend(cfg, c, q, seq, pos, 700), whole)
    assert not torch.equal(attend(cfg, same, q, seq, pos, 700), whole)
    B.beam_paged_kv_write(v, k, s, p, c)                  # other rows into the first one's pages
    assert not torch.equal(attend(cfg, c, q, seq, pos, 700), whole)
    for x in (deep, loaded):
        assert torch.equal(attend(cfg, x, q, seq, pos, 700), whole)
    assert status() == 0
