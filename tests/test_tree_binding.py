"""What the binding of the calls for drafted trees and paged caches refuses before it hands
pointers to the library, without a GPU: host tensors stand in for the device's, and a library
that only counts calls for the real one."""
import ctypes

import pytest
import torch

from kv_cache_eviction_trig_b200 import tria

L, B, HQ, HKV, D, N, CAP, BLOCK = 2, 3, 4, 2, 64, 5, 96, 16


class Library:
    """Every call succeeds and is counted."""

    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return tria.OK
        return call


@pytest.fixture
def library(monkeypatch):
    L = Library()
    monkeypatch.setattr(tria, "lib", lambda: L)
    monkeypatch.setattr(tria, "_ptr", lambda t: None if t is None else ctypes.c_void_p(t.data_ptr()))
    monkeypatch.setattr(tria, "_stream", lambda s: None)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)   # where host tensors are
    return L


def _cfg(**kw):
    d = dict(num_layers=L, batch=B, n_q_heads=HQ, n_kv_heads=HKV, head_dim=D, rope_theta=1e6,
             budget=16, offsets=[1])
    return tria.Config(**{**d, **kw})


def _i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def _pages(rows=B):
    return tria.Pages(_i32(rows, CAP // BLOCK), _i32(rows), _i32(CAP // BLOCK), _i32(2), BLOCK)


def _cache(pages=None, **kw):
    d = dict(k=_bf(L, HKV, CAP, D), v=_bf(L, HKV, CAP, D), pos=_i32(L, HKV, CAP), seq_len=_i32(B),
             cur_pos=_i32(B), seq_start=[0, 32, 64, 96])
    if pages:
        d["pages"] = _pages() if pages is True else pages
    return tria.Cache(**{**d, **kw})


class Calls:
    """The three calls on one cache."""

    def __init__(self, cache, cfg=None):
        cfg = cfg or _cfg()
        b = cfg.c.batch
        tree = tria.Tree(_i32(b, N), _i32(b), _bf(L, HKV, b, N, D), _bf(L, HKV, b, N, D))
        rows, ws = _bf(b, N, HQ, D), torch.zeros(4096, dtype=torch.uint8)
        slots = _i32(b, N) if cache.pages else None
        self.attention = lambda: tria.tria_tree_attention(cfg, cache, tree, 0, rows, rows.clone(), ws)
        self.commit = lambda: tria.tria_tree_commit(cfg, cache, tree, _i32(b), ws, slot_map=slots)
        self.tables = lambda: tria.tria_block_tables(cfg, cache, _i32(b), slots, ws)
        self.all = [self.attention, self.commit] + ([self.tables] if cache.pages else [])


def _refused(library, calls, match):
    for call in calls.all:
        with pytest.raises(ValueError, match=match):
            call()
    assert library.calls == 0


@pytest.mark.parametrize("pages", [False, True])
def test_what_fits_is_passed_on(library, pages):
    calls = Calls(_cache(pages))
    for call in calls.all:
        call()
    assert library.calls == len(calls.all) == (3 if pages else 2)
    # room behind the cache is fine, and lengths per unit take the place of seq_len
    Calls(_cache(k=_bf(L, HKV, CAP + 8, D), cap_total=CAP)).commit()
    Calls(_cache(seq_len=None, unit_len=_i32(L, HKV, B))).commit()
    assert library.calls == len(calls.all) + 2


@pytest.mark.parametrize("rows", [B - 1, B + 1])
def test_pages_of_another_batch(library, rows):
    _refused(library, Calls(_cache(pages=_pages(rows))), "pages: expected tables of 3")


def test_a_configuration_of_another_batch(library):
    """The tables, lengths and segments are those of three sequences, the rest is four's."""
    _refused(library, Calls(_cache(True), _cfg(batch=4)), "seq_start")
    four = dict(seq_start=[0, 32, 64, 96, 96])
    _refused(library, Calls(_cache(True, **four), _cfg(batch=4)), "seq_len")
    four.update(seq_len=_i32(4), cur_pos=_i32(4))
    _refused(library, Calls(_cache(True, **four), _cfg(batch=4)), "pages")


@pytest.mark.parametrize("name,t", [
    ("k", _bf(L, HKV, CAP - 1, D)), ("v", _bf(L, HKV, CAP, D // 2)), ("pos", _i32(L, HKV, CAP - 1)),
    ("seq_len", _i32(B - 1)), ("seq_len", _i32(B + 1)), ("cur_pos", _i32(B - 1)),
    ("seq_len", torch.zeros(B, dtype=torch.int64)), ("k", torch.zeros(L, HKV, CAP, D)),
    ("unit_len", _i32(L, HKV, B - 1))])
@pytest.mark.parametrize("pages", [False, True])
def test_a_cache_smaller_than_the_configuration(library, pages, name, t):
    _refused(library, Calls(_cache(pages, **{name: t}, cap_total=CAP)), name + ": expected")


class Elsewhere(torch.Tensor):
    """A tensor that says it is on another device."""

    def get_device(self):
        return 1


def _elsewhere(t):
    return t.as_subclass(Elsewhere)


@pytest.mark.parametrize("name", ["k", "v", "pos", "seq_len", "cur_pos", "pages"])
def test_a_cache_on_another_device(library, name):
    c = _cache(True)
    if name == "pages":
        t = list(c.pages.tensors)
        for i in range(4):
            there = tria.Pages(*t[:i], _elsewhere(t[i]), *t[i + 1:], BLOCK)
            _refused(library, Calls(_cache(there)), "on device .*1.*, the current one is -1")
    else:
        t = c.tensors[["k", "v", "pos", "seq_len", "cur_pos"].index(name)]
        _refused(library, Calls(_cache(True, **{name: _elsewhere(t)})), "on device .*1.*, the current")


def test_arguments_on_another_device(library):
    cfg, cache, ws = _cfg(), _cache(True), torch.zeros(4096, dtype=torch.uint8)
    t = [_i32(B, N), _i32(B), _bf(L, HKV, B, N, D), _bf(L, HKV, B, N, D)]
    tree, rows, slots, last = tria.Tree(*t), _bf(B, N, HQ, D), _i32(B, N), _i32(B)
    trees = [tria.Tree(*t[:i], _elsewhere(t[i]), *t[i + 1:]) for i in range(4)]
    e = _elsewhere
    for call in ([lambda x=x: tria.tria_tree_attention(cfg, cache, x, 0, rows, rows, ws) for x in trees] +
                 [lambda x=x: tria.tria_tree_commit(cfg, cache, x, last, ws, slot_map=slots) for x in trees] +
                 [lambda: tria.tria_tree_attention(cfg, cache, tree, 0, e(rows), rows, ws),
                  lambda: tria.tria_tree_attention(cfg, cache, tree, 0, rows, e(rows), ws),
                  lambda: tria.tria_tree_attention(cfg, cache, tree, 0, rows, rows, e(ws)),
                  lambda: tria.tria_tree_commit(cfg, cache, tree, e(last), ws, slot_map=slots),
                  lambda: tria.tria_tree_commit(cfg, cache, tree, last, ws, slot_map=e(slots)),
                  lambda: tria.tria_tree_commit(cfg, cache, tree, last, e(ws), slot_map=slots),
                  lambda: tria.tria_block_tables(cfg, cache, e(last), slots, ws),
                  lambda: tria.tria_block_tables(cfg, cache, last, e(slots), ws),
                  lambda: tria.tria_block_tables(cfg, cache, last, slots, e(ws))]):
        with pytest.raises(ValueError, match="on device .*1.*, the current"):
            call()
    assert library.calls == 0
