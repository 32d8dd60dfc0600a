"""Block tables whose arrays hold what no call has written: flagged, and nothing of another
sequence is named."""
import numpy as np
import pytest
import torch

from kv_cache_eviction_trig_b200 import tria
from tests.test_gpu_tree import _lib  # noqa: F401

pytestmark = pytest.mark.gpu


def _dev(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _call(table, held, ring, state, block, lens, n_new, max_new, cap):
    B = len(lens)
    pages = tria.Pages(_dev(table), _dev(held), _dev(ring), _dev(state), block)
    cfg = tria.Config(num_layers=1, batch=B, n_q_heads=1, n_kv_heads=1, head_dim=64,
                      rope_theta=1e6, budget=64, offsets=[1])
    cache = tria.Cache(None, None, None, _dev(lens), None, [cap * b for b in range(B + 1)],
                       cap_total=len(ring) * block, pages=pages)
    ws = tria.workspace(cfg, cache)
    slots = torch.full((B, max_new), 99, dtype=torch.int32, device="cuda")
    tria.tria_block_tables(cfg, cache, _dev(n_new), slots, ws)
    torch.cuda.synchronize()
    return pages, slots.cpu().numpy(), tria.tria_get_device_error(ws)


# ids that are too large, negative, or whose slots wrap to those of block 1 in 32 bits; few
# slots and more than the first grid maps
@pytest.mark.parametrize("max_new", [20, 9000])
@pytest.mark.parametrize("bad", [6, 1000, -1, -7, (1 << 28) + 1, -(1 << 28) + 1])
def test_bad_block_ids_name_no_slot(bad, max_new):
    table = [[0, bad, 2, -1], [3, 4, -1, -1]]
    pages, slots, code = _call(table, [3, 2], [5, 1, -1, -1, -1, -1], [0, 2], 16, [14, 20], [20, 3],
                               max_new, 64)
    assert code == tria.DEVERR_PAGES
    assert slots[0, :20].tolist() == [14, 15] + [-1] * 16 + [32, 33]
    assert slots[1, :4].tolist() == [68, 69, 70, -1] and np.all(slots[:, 20:] == -1)
    assert pages.tensors[0].tolist() == table and pages.tensors[3].tolist() == [0, 2]
