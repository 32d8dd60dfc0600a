"""The structs of the C ABI are read whole, so a change of their layout is a change of version:
tria_cache has had `pages` since 0.2."""
import ctypes
import re

import pytest

from kv_cache_eviction_trig_b200 import build as tbuild
from kv_cache_eviction_trig_b200 import tria
from tests.test_abi import HEADER

# bytes of each struct by version
SIZES = {"0.1": {"tria_cache": 64}, "0.2": {"tria_cache": 72, "tria_pages": 48, "tria_tree": 40}}


def test_the_version_names_the_layout():
    tbuild.build()
    version = re.search(r'#define TRIA_VERSION "([0-9.]+)"', open(HEADER).read()).group(1)
    assert version == tria.VERSION
    assert tria.tria_version() == f"tria {version} (sm_100a)"
    assert {n: ctypes.sizeof(getattr(tria, n)) for n in SIZES[version]} == SIZES[version]


def test_the_binding_refuses_a_library_of_another_version(monkeypatch):
    tbuild.build()
    monkeypatch.setattr(tria, "VERSION", "0.1")
    monkeypatch.setattr(tria, "_lib", None)
    with pytest.raises(RuntimeError, match="0.2"):
        tria.lib()
