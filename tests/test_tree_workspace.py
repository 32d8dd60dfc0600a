"""Workspace sizes of caches with pages, without a GPU."""
import pytest

from kv_cache_eviction_trig_b200 import build as tbuild
from kv_cache_eviction_trig_b200 import tria
from tests.test_abi import _cache, _cfg
from tests.test_tree_abi import _paged, _pages, _tree


@pytest.fixture(scope="module")
def L():
    tbuild.build()
    return tria.lib()


def test_a_paged_cache_needs_no_workspace_for_the_prune(L):
    """36 layers of 16 requests of 32768 slots: the calls that take pages read none of the regions
    for scores, selections and sums, which would be gigabytes."""
    cfg = _cfg(num_layers=36, batch=16, n_q_heads=32, n_kv_heads=8, budget=2048)
    starts = tuple(32768 * b for b in range(17))
    paged = _paged(_pages(block=64, n_blocks=8192, max_blocks=512), cap=8192 * 64, starts=starts)
    need = tria.tria_workspace_size(cfg, paged)
    assert need <= 4 << 20
    assert tria.tria_workspace_size(cfg, _cache(seq_start=starts, cap=starts[-1])) > 1 << 30
    tree = tria.tria_tree_workspace_size(cfg, paged, _tree(N=64))
    assert tree >= need                       # one workspace of the larger size serves all
    assert need >= 256                        # what tria_block_tables asks for
