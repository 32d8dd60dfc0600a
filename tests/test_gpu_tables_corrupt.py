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


def test_more_blocks_than_a_sequence_can_have():
    """Counts within the rows of a wide table, but past any segment's blocks: the sequence keeps
    what it has and gets no slots, the others are served.  (Sums of such counts over 256
    sequences would pass 32 bits.)"""
    most = tria.MAX_SEGMENT // 16
    table = np.full((3, most + 8), -1)
    table[1, 0], table[2, :most] = 7, 50 + np.arange(most)
    ring = np.full(40000, -1)
    ring[:20000] = 20000 + np.arange(20000)
    pages, slots, code = _call(table, [most + 1, 1, most], ring, [0, 20000], 16, [3, 15, 0], [1, 2, 1], 2, 64)
    assert code == tria.DEVERR_PAGES
    assert slots.tolist() == [[-1, -1], [127, 16 * 20000], [50 * 16, -1]]
    assert pages.tensors[1].tolist() == [most + 1, 2, 1]
    assert pages.tensors[3].tolist() == [1, 20000 + most - 1 - 1]
