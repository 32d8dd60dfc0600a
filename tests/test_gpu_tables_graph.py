"""Block tables in a captured graph: one and several CTAs, slots mapped by the first grid and by the second."""
import numpy as np
import pytest
import torch

import oracle
from kv_cache_eviction_trig_b200 import tria
from tests.test_gpu_tree import _lib  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,max_blocks,max_new", [(5, 40, 8), (5, 40, 3000), (70, 200, 16), (70, 200, 700)])
def test_tables_replayed_from_a_graph(B, max_blocks, max_new):
    block, rng = 16, np.random.default_rng(B + max_new)
    cap, n_blocks = max_blocks * block, int(0.7 * B * max_blocks)
    dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    pages = tria.Pages.empty(B, max_blocks, n_blocks, block)
    cfg = tria.Config(num_layers=1, batch=B, n_q_heads=1, n_kv_heads=1, head_dim=64, rope_theta=1e6,
                      budget=64, offsets=[1])
    lens, n_new = dev(np.zeros(B)), dev(np.zeros(B))
    cache = tria.Cache(None, None, None, lens, None, [cap * b for b in range(B + 1)],
                       cap_total=n_blocks * block, pages=pages)
    ws, slots = tria.workspace(cfg, cache), dev(np.zeros((B, max_new)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):            # the first call of these shapes
        tria.tria_block_tables(cfg, cache, n_new, slots, ws)
    state = [x.cpu().numpy() for x in pages.tensors]
    for _ in range(8):
        a, n = rng.integers(0, cap + 1, B), rng.integers(0, max_new + 1, B)
        a[rng.random(B) < 0.3] = 0
        lens.copy_(dev(a))
        n_new.copy_(dev(n))
        tria.tria_workspace_init(ws)
        graph.replay()
        torch.cuda.synchronize()
        want = oracle.block_tables(*state, block, a.tolist(), n.tolist(), [cap] * B, max_new)
        state = [np.asarray(x) for x in want[:4]]
        for got, ref in zip(pages.tensors, state):
            assert np.array_equal(got.cpu().numpy(), ref)
        assert np.array_equal(slots.cpu().numpy(), want[4])
    del graph
