"""The commit over as many (layer, KV head) rows as a grid has no room for with a few rows per block."""
import ctypes

import pytest
import torch

from kv_cache_eviction_trig_b200 import build as tbuild
from kv_cache_eviction_trig_b200 import tria
from tests.test_abi import FAKE, _cache, _cfg
from tests.test_tree_abi import WS, _tree


@pytest.mark.gpu
def test_commit_of_four_million_rows():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    tbuild.build()
    L, Hkv, D, N, cap = 1_400_001, 3, 8, 2, 3            # more than 64 * 65535 rows
    bf = dict(dtype=torch.bfloat16, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    k, v = torch.zeros(L, Hkv, cap, D, **bf), torch.zeros(L, Hkv, cap, D, **bf)
    kd, vd = [torch.randn(L, Hkv, 1, N, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    pos = torch.zeros(L, Hkv, cap, dtype=torch.int32, device="cuda")
    seq_len, cur = i32(1), i32(40)
    cfg = tria.Config(num_layers=L, batch=1, n_q_heads=Hkv, n_kv_heads=Hkv, head_dim=D,
                      rope_theta=1e6, budget=2, offsets=[1])
    cache = tria.Cache(k, v, pos, seq_len, cur, [0, cap])
    tree = tria.Tree(i32(-1, 0).view(1, 2), i32(2), kd, vd)
    ws = torch.empty(tria.tria_tree_workspace_size(cfg, cache, tree), dtype=torch.uint8, device="cuda")
    tria.tria_workspace_init(ws)
    tria.tria_tree_commit(cfg, cache, tree, i32(1), ws)
    torch.cuda.synchronize()
    assert tria.tria_get_device_error(ws) == 0
    assert torch.equal(k[:, :, 1:], kd[:, :, 0]) and torch.equal(v[:, :, 1:], vd[:, :, 0])
    assert not k[:, :, 0].any() and not v[:, :, 0].any()
    assert torch.equal(pos, i32(0, 41, 42).expand(L, Hkv, cap))
    assert seq_len.tolist() == [3] and cur.tolist() == [42]


def test_more_rows_than_32_bits_are_refused():
    tbuild.build()
    cfg, cache, tree = _cfg(num_layers=1 << 30), _cache(), _tree()
    assert tria.lib().tria_tree_commit(ctypes.byref(cfg.c), ctypes.byref(cache.c), ctypes.byref(tree.c),
                                       ctypes.c_void_p(FAKE), None, 0, WS, 1 << 40,
                                       None) == tria.ERR_UNSUPPORTED
