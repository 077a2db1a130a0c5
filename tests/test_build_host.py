"""When the library counts as built."""
import os

import pytest

from hybrid_attention_moe_gb300 import build as b

DEPS = [b.__file__, os.path.join(b.ROOT, "include", "beam.h"), os.path.join(b.CSRC, "paged_tree.cuh"), os.path.join(b.CSRC, "misc.cu")]


@pytest.mark.parametrize("dep", DEPS, ids=os.path.basename)
def test_a_library_older_than_what_makes_it_is_stale(dep, tmp_path, monkeypatch):
    """Sources, headers, and the rules that say how each is compiled."""
    lib = tmp_path / "libbeam.so"
    monkeypatch.setattr(b, "LIB", str(lib))
    assert b._stale()
    lib.write_bytes(b"")
    newest = os.path.abspath(dep)
    monkeypatch.setattr(b.os.path, "getmtime", lambda p: 100.0 if os.path.abspath(p) == newest else 50.0 if p == str(lib) else 10.0)
    assert b._stale()
    monkeypatch.setattr(b.os.path, "getmtime", lambda p: 50.0 if p == str(lib) else 10.0)
    assert not b._stale()


def test_no_kernel_uses_constant_memory():
    """All units link into one module, whose constant memory every kernel's launch pays for."""
    for name in os.listdir(b.CSRC):
        with open(os.path.join(b.CSRC, name)) as f:
            code = [line.split("//")[0] for line in f]
        assert not any("__constant__" in line for line in code), name
