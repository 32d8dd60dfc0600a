"""The calls for drafted trees and paged caches without a GPU: what they refuse before any
launch, the binding's own checks, and the oracle's definitions of them on small cases."""
import ctypes
import re

import numpy as np
import pytest
import torch

import oracle
from kv_cache_eviction_trig_b200 import build as tbuild
from kv_cache_eviction_trig_b200 import tria
from tests.test_abi import FAKE, HEADER, _cache, _cfg, _prune


@pytest.fixture(scope="module")
def L():
    tbuild.build()
    return tria.lib()


def _tree(parent=FAKE + 0x900000, n=FAKE + 0x910000, k=FAKE + 0x920000, v=FAKE + 0x930000, N=8):
    t = tria.Tree.__new__(tria.Tree)
    t.c = tria.tria_tree(parent, n, k, v, N)
    return t


def _pages(table=FAKE + 0xa00000, held=FAKE + 0xa10000, ring=FAKE + 0xa20000,
           state=FAKE + 0xa30000, block=16, n_blocks=32, max_blocks=16):
    p = tria.Pages.__new__(tria.Pages)
    p.c = tria.tria_pages(table, held, ring, state, block, n_blocks, max_blocks)
    return p


def _paged(pages=None, cap=512, starts=(0, 256, 512), **kw):
    c = _cache(seq_start=starts, cap=cap, **kw)
    c.pages = pages or _pages()
    c.c.pages = ctypes.pointer(c.pages.c)
    return c


WS = ctypes.c_void_p(FAKE + 0x1000000)


def test_structs_match_the_header():
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    for name in ("tria_pages", "tria_tree", "tria_cache"):
        body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", text, flags=re.S).group(1)
        names = re.findall(r"([a-z_]+)\s*[;,]", body)
        assert names == [f[0] for f in getattr(tria, name)._fields_], name
    consts = dict(re.findall(r"#define (TRIA_[A-Z_]+) (\d+)\b", text))
    assert int(consts["TRIA_MAX_NODES"]) == tria.MAX_NODES
    for bit in ("TREE", "PAGES", "POOL"):
        assert int(consts["TRIA_DEVERR_" + bit]) == getattr(tria, "DEVERR_" + bit)


def test_tree_attention_rejects_bad_args(L):
    def att(cfg=_cfg(), cache=None, tree=None, layer=0, q=FAKE + 0x700000, scale=0.1,
            out=FAKE + 0x800000, ws=WS, ws_bytes=1 << 40):
        cache, tree = cache or _cache(), tree or _tree()
        return L.tria_tree_attention(ctypes.byref(cfg.c), ctypes.byref(cache.c),
                                     ctypes.byref(tree.c), layer, ctypes.c_void_p(q),
                                     ctypes.c_float(scale), ctypes.c_void_p(out), ws, ws_bytes,
                                     None)
    assert att(layer=1) == tria.ERR_INVALID_ARG
    assert att(layer=-1) == tria.ERR_INVALID_ARG
    assert att(q=FAKE + 0x700002) == tria.ERR_INVALID_ARG          # misaligned
    assert att(out=FAKE + 0x800008) == tria.ERR_INVALID_ARG
    assert att(out=0) == tria.ERR_INVALID_ARG
    assert att(scale=float("nan")) == tria.ERR_INVALID_ARG
    assert att(cache=_cache(v=0)) == tria.ERR_INVALID_ARG
    assert att(tree=_tree(parent=0)) == tria.ERR_INVALID_ARG
    assert att(tree=_tree(n=0)) == tria.ERR_INVALID_ARG
    assert att(tree=_tree(k=FAKE + 0x920008)) == tria.ERR_INVALID_ARG
    assert att(tree=_tree(N=0)) == tria.ERR_INVALID_ARG
    assert att(tree=_tree(N=257)) == tria.ERR_UNSUPPORTED
    assert att(cfg=_cfg(head_dim=96)) == tria.ERR_UNSUPPORTED
    assert att(cfg=_cfg(n_q_heads=6)) == tria.ERR_UNSUPPORTED      # G = 3
    assert att(ws_bytes=1000) == tria.ERR_WORKSPACE
    assert att(ws=ctypes.c_void_p(FAKE + 16)) == tria.ERR_WORKSPACE
    n = ctypes.c_size_t(0)
    assert L.tria_tree_workspace_size(ctypes.byref(_cfg().c), ctypes.byref(_cache().c),
                                      ctypes.byref(_tree().c), ctypes.byref(n)) == tria.OK
    assert att(ws_bytes=n.value - 1) == tria.ERR_WORKSPACE
    assert L.tria_tree_workspace_size(ctypes.byref(_cfg().c), ctypes.byref(_cache().c),
                                      ctypes.byref(_tree(N=300).c),
                                      ctypes.byref(n)) == tria.ERR_UNSUPPORTED


def test_commit_rejects_bad_args(L):
    def com(cfg=_cfg(), cache=None, tree=None, last=FAKE + 0x700000, slots=0, max_new=0,
            ws_bytes=1 << 40):
        cache, tree = cache or _cache(), tree or _tree()
        return L.tria_tree_commit(ctypes.byref(cfg.c), ctypes.byref(cache.c),
                                  ctypes.byref(tree.c), ctypes.c_void_p(last),
                                  ctypes.c_void_p(slots), max_new, WS, ws_bytes, None)
    assert com(last=0) == tria.ERR_INVALID_ARG
    assert com(last=FAKE + 2) == tria.ERR_INVALID_ARG
    assert com(cache=_cache(cur=0)) == tria.ERR_INVALID_ARG
    assert com(slots=FAKE, max_new=4) == tria.ERR_INVALID_ARG      # a slot map without pages
    assert com(cache=_paged()) == tria.ERR_INVALID_ARG             # pages without a slot map
    assert com(cache=_paged(), slots=FAKE, max_new=0) == tria.ERR_INVALID_ARG
    assert com(tree=_tree(N=300)) == tria.ERR_UNSUPPORTED
    assert com(cfg=_cfg(head_dim=100)) == tria.ERR_UNSUPPORTED
    assert com(cfg=_cfg(head_dim=512)) == tria.ERR_UNSUPPORTED
    assert com(ws_bytes=1000) == tria.ERR_WORKSPACE


def test_block_tables_rejects_bad_args(L):
    def tab(cfg=_cfg(), cache=None, n_new=FAKE + 0x700000, max_new=4, slots=FAKE + 0x800000,
            ws=WS, ws_bytes=1 << 20):
        cache = cache or _paged()
        return L.tria_block_tables(ctypes.byref(cfg.c), ctypes.byref(cache.c),
                                   ctypes.c_void_p(n_new), max_new, ctypes.c_void_p(slots), ws,
                                   ws_bytes, None)
    assert tab(cache=_cache()) == tria.ERR_INVALID_ARG             # no pages
    assert tab(n_new=0) == tria.ERR_INVALID_ARG
    assert tab(max_new=-1) == tria.ERR_INVALID_ARG
    assert tab(slots=0) == tria.ERR_INVALID_ARG
    assert tab(max_new=tria.MAX_SEGMENT + 1) == tria.ERR_UNSUPPORTED
    assert tab(ws_bytes=100) == tria.ERR_WORKSPACE
    assert tab(cache=_paged(_pages(table=0))) == tria.ERR_INVALID_ARG
    assert tab(cache=_paged(_pages(held=FAKE + 2))) == tria.ERR_INVALID_ARG
    assert tab(cache=_paged(_pages(block=8))) == tria.ERR_UNSUPPORTED
    assert tab(cache=_paged(_pages(block=48))) == tria.ERR_UNSUPPORTED
    assert tab(cache=_paged(_pages(block=512))) == tria.ERR_UNSUPPORTED
    assert tab(cache=_paged(_pages(n_blocks=31))) == tria.ERR_INVALID_ARG   # cap_total differs
    assert tab(cache=_paged(_pages(max_blocks=15))) == tria.ERR_INVALID_ARG  # rows too short
    assert tab(cache=_paged(_pages(n_blocks=1 << 27), cap=1 << 31)) == tria.ERR_UNSUPPORTED
    assert tab(cache=_paged(seq_len=0)) == tria.ERR_INVALID_ARG
    per_unit = _paged()
    per_unit.c.unit_len = FAKE + 0x400000
    assert tab(cache=per_unit) == tria.ERR_INVALID_ARG


def test_other_calls_refuse_pages(L):
    """A paged cache has no segments: the calls that read them say so."""
    cfg, cache = _cfg(), _paged()
    assert _prune(L, cfg, cache) == tria.ERR_UNSUPPORTED
    q, out = ctypes.c_void_p(FAKE + 0x700000), ctypes.c_void_p(FAKE + 0x800000)
    assert L.tria_decode_attention(ctypes.byref(cfg.c), ctypes.byref(cache.c), 0, q,
                                   ctypes.c_float(0.1), out, WS, 1 << 40, None) == tria.ERR_UNSUPPORTED
    assert L.tria_append(ctypes.byref(cfg.c), ctypes.byref(cache.c), q, out, WS, 1 << 40,
                         None) == tria.ERR_UNSUPPORTED


def test_binding_checks_shapes_and_types():
    i32, bf = dict(dtype=torch.int32), dict(dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="n_nodes"):
        tria._want(torch.zeros(3, **i32), torch.int32, (2,), "n_nodes")
    with pytest.raises(ValueError, match="k: expected"):
        tria._want(torch.zeros(2, 3), torch.bfloat16, (2, 3), "k")
    with pytest.raises(ValueError, match="CUDA"):
        tria._want(torch.zeros(2, 3, **bf), torch.bfloat16, (2, 3), "k")  # a host tensor
    tree = _tree(N=8)
    tree.shape = (1, 2, 2, 8, 64)
    with pytest.raises(ValueError, match="keys are"):
        tria._check_tree(_cfg(), tree)                                   # D = 128


# ---------------------------------------------------------------- the oracle's definitions

def test_oracle_paths():
    assert oracle.tree_path([-1, 0, 0, 2, -1], 3) == [0, 2, 3]
    assert oracle.tree_path([-1, 0, 0, 2, -1], 4) == [4]
    assert oracle.tree_path([-1, 0], -1) == []
    assert oracle.tree_path([-1, 1, 7], 2) == [2]          # out of range counts as the root


def _bits(a):
    return (torch.tensor(np.asarray(a), dtype=torch.float32).to(torch.bfloat16)
            .view(torch.int16).numpy().view(np.uint16))


def test_oracle_attention_closed_forms():
    """Equal logits average the seen values; a node sees its own branch only."""
    k, v = np.zeros((1, 1, 4, 8)), np.zeros((1, 1, 4, 8))
    v[0, 0, :, 0] = [1, 2, 3, 100]
    kd, vd = np.zeros((1, 1, 1, 3, 8)), np.zeros((1, 1, 1, 3, 8))
    vd[0, 0, 0, :, 0] = [6, 60, 12]
    q = np.ones((1, 3, 2, 8))
    out, spread, steep = oracle.tree_attention(
        _bits(k), _bits(v), [[np.arange(3)]], _bits(kd), _bits(vd), np.array([[-1, -1, 0]]), [3],
        _bits(q), 0, 0.5)
    assert np.allclose(out[0, :, 0, 0], [12 / 4, 66 / 4, 24 / 5]) and np.all(steep == 0)
    assert np.array_equal(out, spread)
    empty, _, _ = oracle.tree_attention(
        _bits(k), _bits(v), [[np.arange(0)]], _bits(kd), _bits(vd), np.array([[-1, -1, 0]]), [2],
        _bits(q), 0, 0.5)
    assert np.allclose(empty[0, :2, 1, 0], [6, 60]) and np.isnan(empty[0, 2]).all()


def test_oracle_attention_matches_decode_attention():
    """One node whose key is the cache's next token is a decode step."""
    g = np.random.default_rng(1)
    k, v = _bits(g.normal(size=(1, 2, 20, 16))), _bits(g.normal(size=(1, 2, 20, 16)))
    q = _bits(g.normal(size=(2, 1, 4, 16)))
    ref = oracle.decode_attention(k, v, [0, 8, 20], [7, 12], 0, q[:, 0], 0.3)
    kd = np.stack([k[:, :, [6]], k[:, :, [19]]], 2)
    vd = np.stack([v[:, :, [6]], v[:, :, [19]]], 2)
    out, _, _ = oracle.tree_attention(k, v, [[np.arange(6)] * 2, [np.arange(8, 19)] * 2], kd, vd,
                                      np.array([[-1], [-1]]), [1, 1], q, 0, 0.3)
    assert np.allclose(out[:, 0], ref, rtol=1e-12)


def test_oracle_block_tables_worked_example():
    """Blocks of 4: the first sequence shrinks from 3 blocks to 1, the second grows by two."""
    table = np.array([[5, 2, 7, -1], [0, -1, -1, -1], [-1] * 4], dtype=np.int32)
    ring = np.array([-1, 1, 3, 4, 6, -1, -1, -1], dtype=np.int32)
    out = oracle.block_tables(table, [3, 1, 0], ring, [1, 4], 4, [3, 4, 0], [1, 5, 30],
                              [16, 16, 16], 6)
    assert out[0].tolist() == [[5, -1, -1, -1], [0, 1, 3, -1], [-1] * 4]
    assert out[1] == [1, 3, 0] and out[3] == [3, 4]
    assert out[2].tolist() == [-1, 1, 3, 4, 6, 2, 7, -1]
    assert out[4].tolist() == [[23, -1, -1, -1, -1, -1], [4, 5, 6, 7, 12, -1], [-1] * 6]
    assert out[5] == {2: "length"}
    poor = oracle.block_tables(table, [3, 1, 0], ring, [1, 1], 4, [12, 4, 0], [0, 8, 1], [16] * 3, 8)
    assert poor[5] == {1: "pool", 2: "pool"} and poor[3] == [1, 1]
    assert np.all(poor[4] == -1) and poor[0].tolist() == table.tolist()
