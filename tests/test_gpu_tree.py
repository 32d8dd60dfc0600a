"""GPU parity of speculative decoding over the pruned cache against the oracle: tree
attention, the commit of accepted paths, block tables and slot maps, and a loop of them.

Tree attention: float64 reference.  The output is rounded once to bf16 (half a step is 2^-8
relative).  The softmax weights are rounded to bf16, for the product with V and for their sum
alike, each off by a share d of at most 2^-8: the output moves by sum w d (v - out), at most
2^-8 (sum w |v| + |out|).  The float32 logits are sums of D products: taken in any order,
truncated after each step, they are off by at most D 2^-23 of scale sum |q k|, and a weight's
relative error is at most twice the logits' absolute one (it and the normaliser); exponentials
and the sums with V add less than 2^-16.  Everything else (rows that are not written,
committed rows, lengths, positions, tables, slots) is exact."""
import numpy as np
import pytest
import torch

import oracle
from kv_cache_eviction_trig_b200 import tria
from tests import common

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from kv_cache_eviction_trig_b200 import build
    build.build()
    tria.lib()


def _parents(shape, B, N, rng):
    if shape == "chain":
        return np.tile(np.arange(N) - 1, (B, 1))
    if shape == "star":
        return np.full((B, N), -1)
    return np.array([[rng.integers(-1, i) if i else -1 for i in range(N)] for _ in range(B)])


class Spec:
    """A cache (segments or pages) with live lengths `lens` (or per-unit ones), drafted trees
    and queries.  Every slot, node and query row that no result may depend on holds NaN."""

    def __init__(self, *, L=1, Hq=8, Hkv=2, D=128, lens=(300,), N=8, nodes=None, block=0,
                 shape="tree", slack=40, unit_lens=None, seed=0, sharp=1.0):
        rng = np.random.default_rng(seed)
        self.L, self.Hq, self.Hkv, self.D, self.N, self.block = L, Hq, Hkv, D, N, block
        self.B = B = len(lens)
        self.lens = list(lens)
        nodes = [N] * B if nodes is None else nodes
        room = [t + slack for t in self.lens]
        if unit_lens is not None:
            room = [int(unit_lens[:, :, b].max()) + slack for b in range(B)]
        self.unit_lens = unit_lens
        pages = None
        if block:
            blocks = [-(-r // block) for r in room]
            self.starts = np.concatenate([[0], np.cumsum([x * block for x in blocks])]).tolist()
            held = [-(-t // block) for t in self.lens]
            n_blocks = sum(blocks) + 3
            order = rng.permutation(n_blocks)
            table = np.full((B, max(blocks) + 1), -1)
            at = 0
            for b in range(B):
                table[b, :held[b]] = order[at:at + held[b]]
                at += held[b]
            ring = np.concatenate([order[at:], np.full(at, -1)])
            pages = tria.Pages(*[torch.tensor(x, dtype=torch.int32, device="cuda") for x in
                                 (table, held, ring, [0, n_blocks - at])], block)
            self.table, cap = table, n_blocks * block
        else:
            self.starts = np.concatenate([[0], np.cumsum(room)]).tolist()
            cap = self.starts[-1]
        self.cap = cap
        self.slots = [[self._at(b, self._len(0, g, b)) for g in range(Hkv)] for b in range(B)]
        f = lambda *s: torch.tensor(rng.normal(size=s), dtype=torch.float32).to(torch.bfloat16)
        nan = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16)
        self.k, self.v = nan(L, Hkv, cap, D), nan(L, Hkv, cap, D)
        for l in range(L):
            for g in range(Hkv):
                for b in range(B):
                    at = self._at(b, self._len(l, g, b))
                    self.k[l, g, at], self.v[l, g, at] = f(len(at), D), f(len(at), D)
        self.kd, self.vd, self.q = nan(L, Hkv, B, N, D), nan(L, Hkv, B, N, D), nan(B, N, Hq, D)
        for b in range(B):
            self.kd[:, :, b, :nodes[b]] = f(L, Hkv, nodes[b], D)
            self.vd[:, :, b, :nodes[b]] = f(L, Hkv, nodes[b], D)
            self.q[b, :nodes[b]] = (sharp * f(nodes[b], Hq, D).float()).to(torch.bfloat16)
        self.nodes = list(nodes)
        self.parent = _parents(shape, B, N, rng)
        for b in range(B):
            self.parent[b, nodes[b]:] = 77  # not read
        dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
        self.t = dict(k=self.k.cuda(), v=self.v.cuda(),
                      pos=torch.zeros(L, Hkv, cap, dtype=torch.int32, device="cuda"),
                      seq_len=dev(self.lens), cur_pos=dev([3 * t for t in self.lens]),
                      kd=self.kd.cuda(), vd=self.vd.cuda(), q=self.q.cuda(),
                      parent=dev(self.parent), n_nodes=dev(self.nodes),
                      out=torch.full((B, N, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda"))
        unit = None if unit_lens is None else dev(unit_lens)
        self.t["unit_len"] = unit
        t = self.t
        self.pages = pages
        self.cfg = tria.Config(num_layers=L, batch=B, n_q_heads=Hq, n_kv_heads=Hkv, head_dim=D,
                               rope_theta=1e6, budget=64, offsets=[1])
        self.cache = tria.Cache(t["k"], t["v"], t["pos"], None if unit is not None else t["seq_len"],
                                t["cur_pos"], self.starts, unit_len=unit, pages=pages)
        self.tree = tria.Tree(t["parent"], t["n_nodes"], t["kd"], t["vd"])
        self.ws = tria.workspace(self.cfg, self.cache, tree=self.tree)

    def _len(self, l, g, b):
        return self.lens[b] if self.unit_lens is None else int(self.unit_lens[l, g, b])

    def _at(self, b, T):
        t = np.arange(T)
        if self.block:
            return self.table[b, t // self.block] * self.block + t % self.block
        return self.starts[b] + t

    def attend(self, layer=0, scale=None, stream=None):
        tria.tria_tree_attention(self.cfg, self.cache, self.tree, layer, self.t["q"],
                                 self.t["out"], self.ws, scale=scale, stream=stream)

    def check(self, layer=0, scale=None, skip=()):
        """The output against the oracle; rows without a node, and sequences `skip`, hold 7."""
        sc = self.D ** -0.5 if scale is None else scale
        slots = [[self._at(b, self._len(layer, g, b)) for g in range(self.Hkv)] for b in range(self.B)]
        nodes = [0 if b in skip else n for b, n in enumerate(self.nodes)]
        ref, spread, steep = oracle.tree_attention(
            common.bf16_bits(self.k), common.bf16_bits(self.v), slots, common.bf16_bits(self.kd),
            common.bf16_bits(self.vd), self.parent, nodes, common.bf16_bits(self.q), layer, sc)
        got = self.t["out"].double().cpu().numpy()
        for b in range(self.B):
            n = nodes[b]
            assert np.all(got[b, n:] == 7.0), b
            logit = 2 * self.D * 2.0 ** -23 * steep[b, :n, :, None]
            tol = 2.0 ** -7 * np.abs(ref[b, :n]) + (2.0 ** -8 + logit + 2.0 ** -16) * spread[b, :n]
            err = np.abs(got[b, :n] - ref[b, :n])
            assert np.all(err <= tol), (b, np.nanmax(err - tol), np.isnan(got[b, :n]).sum())


CASES = {
    # lengths around the tiles; one node; no node; an empty cache
    "one_node": dict(lens=[0, 1, 2, 31, 33], N=1),
    "edges": dict(lens=[127, 128, 129, 255, 256, 257, 384], N=5),
    "no_nodes": dict(lens=[0, 130, 0, 64], N=9, nodes=[9, 0, 0, 4]),
    "ragged_nodes": dict(lens=[500, 3, 77], N=37, nodes=[1, 37, 20], L=2),
    # every head dimension and group
    "d64_g1": dict(D=64, Hq=2, Hkv=2, lens=[300, 130], N=33),
    "d64_g8": dict(D=64, Hq=16, Hkv=2, lens=[515, 64], N=17),
    "d64_g16": dict(D=64, Hq=16, Hkv=1, lens=[200, 400], N=10),
    "d128_g1": dict(Hq=3, Hkv=3, lens=[301, 5], N=130),
    "d128_g2": dict(Hq=4, Hkv=2, lens=[301], N=66),
    "d128_g16": dict(Hq=32, Hkv=2, lens=[129, 700], N=19),
    "d256_g1": dict(D=256, Hq=2, Hkv=2, lens=[300, 0], N=150),
    "d256_g4": dict(D=256, Hq=8, Hkv=2, lens=[260, 41], N=40),
    "d256_g16": dict(D=256, Hq=16, Hkv=1, lens=[190], N=9),
    # trees of more than one tile of nodes: chains (every node sees all before it), stars
    "chain_256": dict(lens=[100, 0, 333], N=256, nodes=[256, 255, 129], shape="chain"),
    "star_200": dict(lens=[70], N=200, shape="star", Hq=4, Hkv=1),
    "tree_256_g8": dict(lens=[0, 260], N=256, nodes=[256, 200], Hq=8, Hkv=1, D=64),
    # pages of every size, ending inside tiles
    "pages_16": dict(lens=[0, 1, 15, 16, 17, 300], N=6, block=16),
    "pages_32": dict(lens=[129, 513], N=20, block=32, D=64),
    "pages_64": dict(lens=[64, 65, 1000], N=7, block=64, Hq=8, Hkv=1),
    "pages_128": dict(lens=[128, 127, 640], N=12, block=128, D=256, Hq=4),
    "pages_256": dict(lens=[255, 257, 900], N=31, block=256),
    # long: keys split over many blocks; steep and flat logits
    "long": dict(lens=[12001], N=4),
    "long_pages": dict(lens=[9000, 40], N=16, block=16, Hq=4, Hkv=1),
    "steep": dict(lens=[700, 2100], N=12, sharp=20.0),
    "flat": dict(lens=[700, 2100], N=12, sharp=0.0),
    "many": dict(lens=[(b * 37) % 290 for b in range(100)], N=3, Hq=4, Hkv=2, D=64),
}


@pytest.mark.parametrize("name", sorted(CASES))
def test_tree_attention_matches_oracle(name):
    s = Spec(**CASES[name])
    layer = s.L - 1
    s.attend(layer)
    torch.cuda.synchronize()
    assert tria.tria_get_device_error(s.ws) == 0
    s.check(layer)


def test_tree_attention_with_unit_lengths_and_a_scale():
    """After a prune with head budgets every (layer, KV head) holds its own keys."""
    lens = np.array([[[5, 300], [129, 0], [200, 40]], [[0, 7], [64, 130], [1, 256]]])
    s = Spec(L=2, Hq=6, Hkv=3, lens=[0, 0], unit_lens=lens, N=10, nodes=[10, 6])
    for layer in range(2):
        s.t["out"].fill_(7.0)
        s.attend(layer, scale=0.31)
        torch.cuda.synchronize()
        assert tria.tria_get_device_error(s.ws) == 0
        s.check(layer, scale=0.31)


@pytest.mark.parametrize("block", [0, 32])
def test_other_branches_do_not_leak(block):
    """Infinities and NaN in the keys and values of some nodes reach their descendants only."""
    s = Spec(lens=[200, 90], N=6, block=block)
    s.parent[:] = [-1, 0, 0, 1, 2, -1]      # node 1's branch: 1, 3
    s.t["parent"].copy_(torch.tensor(s.parent))
    s.t["vd"][:, :, 0, 1, 5] = float("inf")
    s.t["vd"][:, 1, 0, 1, 70] = float("nan")
    s.t["kd"][:, :, 1, 1] = float("nan")
    s.t["vd"][:, :, 1, 1] = float("nan")
    s.attend()
    torch.cuda.synchronize()
    assert tria.tria_get_device_error(s.ws) == 0
    got = s.t["out"].clone()
    for i in (1, 3):
        assert torch.all(got[0, i, :, 5] == float("inf"))
        assert torch.all(torch.isnan(got[0, i, 4:, 70])) and torch.isfinite(got[0, i, :4, 70]).all()
        assert torch.isnan(got[1, i]).all()
    # the finite columns of the poisoned rows are as without the poison, and so is all else
    s.t["vd"].copy_(s.vd)
    s.t["kd"].copy_(s.kd)
    s.attend()
    torch.cuda.synchronize()
    s.check()
    clean = s.t["out"]
    keep = torch.ones_like(clean, dtype=torch.bool)
    keep[0, [1, 3], :, 5] = False
    keep[0, [1, 3], 4:, 70] = False
    keep[1, [1, 3]] = False
    assert torch.equal(got[keep], clean[keep])


def test_a_nan_among_the_seen_keys_is_seen():
    s = Spec(lens=[150, 150], N=4)
    s.t["k"][0, 0, s.starts[0] + 149, 3] = float("nan")
    s.attend()
    torch.cuda.synchronize()
    assert torch.isnan(s.t["out"][0, :, :4]).all()
    assert torch.isfinite(s.t["out"][0, :, 4:]).all() and torch.isfinite(s.t["out"][1]).all()


def test_bad_sequences_are_flagged_and_skipped():
    s = Spec(lens=[100, 200, 50, 60], N=4)
    s.t["seq_len"][1] = 241                 # beyond its segment of 240
    s.t["n_nodes"][2] = 5                   # more than max_nodes
    s.attend()
    torch.cuda.synchronize()
    assert tria.tria_get_device_error(s.ws) == tria.DEVERR_SEQ_LEN | tria.DEVERR_TREE
    s.check(skip=(1, 2))
    tria.tria_workspace_init(s.ws)
    s.t["seq_len"][1], s.t["n_nodes"][2] = -1, -1
    s.t["out"].fill_(7.0)
    s.attend()
    torch.cuda.synchronize()
    assert tria.tria_get_device_error(s.ws) == tria.DEVERR_SEQ_LEN | tria.DEVERR_TREE
    s.check(skip=(1, 2))


def test_bad_parents_count_as_roots():
    s = Spec(lens=[100, 60], N=5)
    s.parent[0] = [0, 5, 2, 1, -2]          # itself, later, itself, fine, below -1
    s.t["parent"].copy_(torch.tensor(s.parent))
    s.attend()
    torch.cuda.synchronize()
    assert tria.tria_get_device_error(s.ws) == tria.DEVERR_TREE
    s.check()


def test_bad_block_ids_are_flagged():
    """The host checks no table; the kernel reads another block of the pool instead."""
    s = Spec(lens=[100, 60], N=5, block=16)
    s.pages.tensors[0][0, 2] = 10 ** 6
    s.pages.tensors[0][0, 3] = -5
    s.attend()
    torch.cuda.synchronize()
    assert tria.tria_get_device_error(s.ws) == tria.DEVERR_PAGES
    s.t["out"][0] = 7.0
    s.check(skip=(0,))


def test_another_stream_and_a_replayed_graph():
    """The same call eagerly on a stream of its own and replayed from a graph after the
    lengths, trees and queries changed on the device; two graphs share the workspace."""
    s = Spec(lens=[700, 33, 2100], N=12, block=32, slack=200)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s.attend(stream=side)
    side.synchronize()
    s.check()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.attend()
        graphs.append(g)
    s.lens, s.nodes = [650, 1, 2049], [3, 12, 7]
    s.t["seq_len"].copy_(torch.tensor(s.lens))
    s.t["n_nodes"].copy_(torch.tensor(s.nodes))
    for g in graphs * 2:
        s.t["out"].fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        s.check()
    assert tria.tria_get_device_error(s.ws) == 0
    del graphs, g


def test_repeated_calls_give_the_same_bits():
    s = Spec(lens=[5000, 900], N=16)
    s.attend()
    torch.cuda.synchronize()
    first = s.t["out"].clone()
    for _ in range(5):
        s.t["out"].fill_(7.0)
        s.attend()
        torch.cuda.synchronize()
        assert torch.equal(first, s.t["out"])


def test_offsets_past_32_bits():
    """The last sequence of a cache of more than 2^32 bytes and 2^31 elements per tensor."""
    Hkv, cap, D, N, T = 8, 2_200_000, 128, 4, 300
    big = dict(dtype=torch.bfloat16, device="cuda")
    k, v = torch.full((1, Hkv, cap, D), float("nan"), **big), torch.full((1, Hkv, cap, D), float("nan"), **big)
    starts = [cap - 2000, cap - 1000, cap]
    at = torch.arange(cap - 1000, cap - 1000 + T, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    small = [torch.randn(1, Hkv, T, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    k[:, :, at], v[:, :, at] = small
    kd, vd = [torch.randn(1, Hkv, 2, N, D, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    q = torch.randn(2, N, Hkv, D, generator=g, device="cuda").to(torch.bfloat16)
    parent = torch.tensor([[-1, 0, 1, 0]] * 2, dtype=torch.int32, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cfg = tria.Config(num_layers=1, batch=2, n_q_heads=Hkv, n_kv_heads=Hkv, head_dim=D,
                      rope_theta=1e6, budget=64, offsets=[1])
    pos = torch.zeros(1, Hkv, cap, dtype=torch.int32, device="cuda")
    cache = tria.Cache(k, v, pos, i32(0, T), i32(0, T), starts)
    tree = tria.Tree(parent, i32(0, N), kd, vd)
    ws = tria.workspace(cfg, cache, tree=tree)
    out = torch.zeros_like(q)
    tria.tria_tree_attention(cfg, cache, tree, 0, q, out, ws)
    torch.cuda.synchronize()
    assert tria.tria_get_device_error(ws) == 0
    ref, spread, _ = oracle.tree_attention(
        common.bf16_bits(small[0]), common.bf16_bits(small[1]), [[np.arange(0)] * Hkv, [np.arange(T)] * Hkv],
        common.bf16_bits(kd), common.bf16_bits(vd), parent.cpu().numpy(), [0, N], common.bf16_bits(q), 0, D ** -0.5)
    err = np.abs(out[1].double().cpu().numpy() - ref[1])
    assert np.all(err <= 2.0 ** -7 * np.abs(ref[1]) + (2.0 ** -8 + 2.0 ** -12) * spread[1])
    # the accepted path lands behind it
    last = i32(-1, 2)
    tria.tria_tree_commit(cfg, cache, tree, last, ws)
    torch.cuda.synchronize()
    assert tria.tria_get_device_error(ws) == 0
    end = cap - 1000 + T
    assert torch.equal(k[:, :, end:end + 3], kd[:, :, 1, :3]) and torch.equal(v[:, :, end:end + 3], vd[:, :, 1, :3])
    assert cache.tensors[3].tolist() == [0, T + 3]


# ---------------------------------------------------------------- commit

def _committed(s, last, slot_map=None, skip=()):
    """What the caches, positions and lengths are after the commit, by the oracle's paths."""
    t = {n: s.t[n].cpu() for n in ("k", "v", "pos", "kd", "vd")}
    seq_len = list(s.lens)
    unit = None if s.unit_lens is None else s.unit_lens.copy()
    cur = s.t["cur_pos"].tolist()
    new_cur = list(cur)
    for b in range(s.B):
        if b in skip:
            continue
        path = oracle.tree_path(s.parent[b], last[b])
        for l in range(s.L):
            for g in range(s.Hkv):
                for j, node in enumerate(path):
                    at = (int(slot_map[b, j]) if slot_map is not None
                          else s.starts[b] + s._len(l, g, b) + j)
                    t["k"][l, g, at], t["v"][l, g, at] = t["kd"][l, g, b, node], t["vd"][l, g, b, node]
                    t["pos"][l, g, at] = cur[b] + 1 + j
        if unit is not None:
            unit[:, :, b] += len(path)
        seq_len[b] += len(path)
        new_cur[b] += len(path)
    return t, (seq_len if unit is None else unit.tolist()), new_cur


def _same(a, b):
    return torch.equal(a.view(torch.int16) if a.dtype == torch.bfloat16 else a,
                       b.view(torch.int16) if b.dtype == torch.bfloat16 else b)


def _check_commit(s, last, slot_map=None, skip=(), code=0):
    want, lens, cur = _committed(s, last, None if slot_map is None else slot_map.cpu().numpy(), skip)
    dev = torch.tensor(last, dtype=torch.int32, device="cuda")
    tria.tria_tree_commit(s.cfg, s.cache, s.tree, dev, s.ws, slot_map=slot_map)
    torch.cuda.synchronize()
    assert tria.tria_get_device_error(s.ws) == code
    for n in ("k", "v", "pos"):
        assert _same(s.t[n].cpu(), want[n]), n
    assert s.t["unit_len" if s.unit_lens is not None else "seq_len"].tolist() == lens
    assert s.t["cur_pos"].tolist() == cur


@pytest.mark.parametrize("D", [64, 128, 256, 72])
def test_commit_matches_oracle(D):
    s = Spec(L=3, Hkv=5, Hq=5, D=D, lens=[10, 0, 33, 7], N=9, nodes=[9, 5, 0, 9], slack=9)
    _check_commit(s, [8, 4, -1, -1])


def test_commit_of_a_whole_chain_fills_the_segment():
    s = Spec(L=2, lens=[3, 64], N=256, shape="chain", slack=256)
    _check_commit(s, [255, 0])


def test_commit_skips_what_it_cannot_take():
    s = Spec(lens=[10, 10, 10, 10, 10], N=6, shape="chain", slack=4)
    s.t["seq_len"][3] = 15
    s.lens[3] = 15
    s.t["n_nodes"][4] = 7
    # five tokens in a room of four; a node past the count; one that fits; a bad length; a bad count
    _check_commit(s, [4, 6, 3, 0, 0], skip=(0, 1, 3, 4),
                  code=tria.DEVERR_SEGMENT_FULL | tria.DEVERR_TREE | tria.DEVERR_SEQ_LEN)


def test_commit_with_unit_lengths():
    lens = np.array([[[5, 30], [9, 0]], [[0, 7], [6, 13]]])
    s = Spec(L=2, Hq=4, Hkv=2, D=64, lens=[0, 0], unit_lens=lens, N=6, slack=3, shape="chain")
    _check_commit(s, [2, 0])
    lens = np.array([[[5, 30], [9, 0]], [[0, 7], [6, 13]]])
    s = Spec(L=2, Hq=4, Hkv=2, D=64, lens=[0, 0], unit_lens=lens, N=6, slack=3, shape="chain")
    _check_commit(s, [3, 2], skip=(0,), code=tria.DEVERR_SEGMENT_FULL)   # one unit of b = 0 is full


def test_commit_into_pages():
    s = Spec(L=2, lens=[14, 0, 31], N=8, shape="chain", block=16, slack=64)
    slots = torch.tensor([[5, 0, 90, 91, 2], [7, -1, 8, 9, 10], [40, 41, 42, 43, s.cap]],
                         dtype=torch.int32, device="cuda")
    _check_commit(s, [3, 1, 4], slot_map=slots, skip=(1, 2), code=tria.DEVERR_PAGES)
    s = Spec(L=2, lens=[14, 0, 31], N=8, shape="chain", block=16, slack=64)
    _check_commit(s, [5, 0, 3], slot_map=slots, skip=(0,), code=tria.DEVERR_PAGES)  # six tokens, five slots


# ---------------------------------------------------------------- block tables

def _tables_case(B, block, max_blocks, n_blocks, lens, held, n_new, max_new, seed, head=0):
    rng = np.random.default_rng(seed)
    order = rng.permutation(n_blocks)
    table = np.full((B, max_blocks), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    ring = np.full(n_blocks, -1, dtype=np.int32)
    ring[(head + np.arange(n_blocks - at)) % n_blocks] = order[at:]
    return dict(table=table, held=np.array(held, dtype=np.int32), ring=ring,
                state=np.array([head, n_blocks - at], dtype=np.int32), block=block,
                lens=list(lens), n_new=list(n_new), caps=[max_blocks * block] * B, max_new=max_new)


def _run_tables(c, steps=1, next_step=None):
    dev = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    B = len(c["lens"])
    pages = tria.Pages(dev(c["table"]), dev(c["held"]), dev(c["ring"]), dev(c["state"]), c["block"])
    starts = np.concatenate([[0], np.cumsum(c["caps"])]).tolist()
    cfg = tria.Config(num_layers=1, batch=B, n_q_heads=1, n_kv_heads=1, head_dim=64,
                      rope_theta=1e6, budget=64, offsets=[1])
    seq_len = dev(c["lens"])
    cache = tria.Cache(None, None, None, seq_len, None, starts,
                       cap_total=len(c["ring"]) * c["block"], pages=pages)
    ws = tria.workspace(cfg, cache)
    for step in range(steps):
        if step:
            c = {**c, **next_step(step)}
            seq_len.copy_(dev(c["lens"]))
        slot_map = torch.full((B, c["max_new"]), 99, dtype=torch.int32, device="cuda") if c["max_new"] else None
        tria.tria_workspace_init(ws)
        tria.tria_block_tables(cfg, cache, dev(c["n_new"]), slot_map, ws)
        torch.cuda.synchronize()
        want = oracle.block_tables(c["table"], c["held"], c["ring"], c["state"], c["block"],
                                   c["lens"], c["n_new"], c["caps"], c["max_new"])
        table, held, ring, state = [x.cpu().numpy() for x in pages.tensors]
        assert np.array_equal(table, want[0]) and held.tolist() == want[1]
        assert np.array_equal(ring, want[2]) and state.tolist() == want[3]
        if slot_map is not None:
            assert np.array_equal(slot_map.cpu().numpy(), want[4])
        bits = {"length": tria.DEVERR_SEQ_LEN, "full": tria.DEVERR_SEGMENT_FULL, "pool": tria.DEVERR_POOL}
        assert tria.tria_get_device_error(ws) == sum({bits[w] for w in want[5].values()})
        assert seq_len.tolist() == c["lens"]
        c = {**c, "table": want[0], "held": want[1], "ring": want[2], "state": want[3]}
    return c


@pytest.mark.parametrize("B,block,max_new", [(1, 16, 1), (3, 32, 40), (16, 16, 16), (31, 64, 300),
                                             (200, 128, 5), (256, 16, 64), (2, 256, 70000)])
def test_block_tables_match_oracle_over_steps(B, block, max_new):
    """Twelve steps of lengths that grow, shrink, start and end at random, in a pool that at
    times is too small; the ring wraps."""
    rng = np.random.default_rng(B)
    max_blocks = max(6, 2 * max_new // block)
    cap = max_blocks * block
    n_blocks = max(4, int(0.6 * B * max_blocks))

    def step(_):
        n_new = rng.integers(0, max_new + 1, B)
        lens = rng.integers(0, cap + 1, B)
        lens[rng.random(B) < 0.2] = 0
        return dict(lens=[int(x) for x in lens], n_new=[int(x) for x in n_new])
    first = step(0)
    c = _tables_case(B, block, max_blocks, n_blocks, first["lens"], [0] * B, first["n_new"], max_new,
                     seed=B, head=n_blocks - 2)
    _run_tables(c, 12, step)


def test_block_tables_edge_requests():
    c = _tables_case(6, 16, 4, 24, lens=[16, 17, 64, -1, 60, 0], held=[1, 2, 4, 2, 4, 3],
                     n_new=[0, 15, 0, 3, 5, 0], max_new=20, seed=1)
    c = _run_tables(c)
    assert list(c["held"]) == [1, 2, 4, 2, 4, 0]
    c = {**c, "lens": [65, 3, 0, 1, 1, 0], "n_new": [0, 21, -1, 0, 0, 0]}
    _run_tables(c)
    _run_tables({**c, "lens": [1] * 6, "n_new": [0] * 6, "max_new": 0})


def test_block_tables_refuse_a_corrupt_pool():
    """A ring state or a held count out of range is flagged and no block changes hands."""
    dev = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cfg = tria.Config(num_layers=1, batch=2, n_q_heads=1, n_kv_heads=1, head_dim=64,
                      rope_theta=1e6, budget=64, offsets=[1])
    for state, held, gone in [([9, 4], [2, 1], True), ([-1, 4], [2, 1], True), ([0, 9], [2, 1], True),
                              ([0, -1], [2, 1], True), ([0, 8], [2, 1], True), ([0, 5], [2, 5], False)]:
        pages = tria.Pages(dev([[0, 1, -1, -1], [2, -1, -1, -1]]), dev(held),
                           dev([3, 4, 5, 6, 7, -1, -1, -1]), dev(state), 16)
        cache = tria.Cache(None, None, None, dev([3, 3]), None, [0, 64, 128], cap_total=128, pages=pages)
        ws = tria.workspace(cfg, cache)
        slots = torch.zeros(2, 40, dtype=torch.int32, device="cuda")
        tria.tria_block_tables(cfg, cache, dev([2, 40]), slots, ws)
        torch.cuda.synchronize()
        assert tria.tria_get_device_error(ws) & tria.DEVERR_PAGES
        assert torch.all(slots[1] == -1)
        if gone:
            assert pages.tensors[0].tolist() == [[0, 1, -1, -1], [2, -1, -1, -1]]
            assert pages.tensors[1].tolist() == held and pages.tensors[3].tolist() == state
            assert slots[0, :3].tolist() == [3, 4, -1]   # it holds the block of these tokens
        else:  # the other sequence is served
            assert pages.tensors[1].tolist() == [1, 5] and pages.tensors[3].tolist() == [0, 6]


# ---------------------------------------------------------------- the calls together

def _draw_trees(rng, L, Hkv, B, N, D):
    f = lambda *s: torch.tensor(rng.normal(size=s), dtype=torch.float32).to(torch.bfloat16)
    nodes = rng.integers(0, N + 1, B)
    return dict(parent=torch.tensor(_parents("tree", B, N, rng), dtype=torch.int32),
                n_nodes=torch.tensor(nodes, dtype=torch.int32), kd=f(L, Hkv, B, N, D),
                vd=f(L, Hkv, B, N, D),
                last=torch.tensor([rng.integers(-1, n) if n else -1 for n in nodes], dtype=torch.int32))


def test_speculative_loop_over_pages_matches_oracle_and_its_graph():
    """Twelve steps of: blocks for a tree's tokens, the trees' attention in every layer, the
    accepted paths into the cache; requests end and start in between.  The first steps run
    eagerly, the others from one captured graph."""
    L, Hkv, Hq, D, B, N, block, steps = 2, 2, 4, 64, 3, 10, 16, 12
    rng = np.random.default_rng(5)
    caps, n_blocks = [160, 96, 160], 20          # 26 blocks would hold them all
    starts = np.concatenate([[0], np.cumsum(caps)]).tolist()
    bf, i32 = dict(dtype=torch.bfloat16, device="cuda"), dict(dtype=torch.int32, device="cuda")
    cap = n_blocks * block
    t = dict(k=torch.full((L, Hkv, cap, D), float("nan"), **bf), v=torch.full((L, Hkv, cap, D), float("nan"), **bf),
             pos=torch.zeros(L, Hkv, cap, **i32), seq_len=torch.zeros(B, **i32), cur_pos=torch.zeros(B, **i32),
             parent=torch.zeros(B, N, **i32), n_nodes=torch.zeros(B, **i32), last=torch.zeros(B, **i32),
             n_new=torch.zeros(B, **i32), slots=torch.zeros(B, N, **i32),
             kd=torch.zeros(L, Hkv, B, N, D, **bf), vd=torch.zeros(L, Hkv, B, N, D, **bf),
             q=torch.zeros(L, B, N, Hq, D, **bf), out=torch.zeros(L, B, N, Hq, D, **bf))
    pages = tria.Pages.empty(B, max(caps) // block, n_blocks, block)
    cfg = tria.Config(num_layers=L, batch=B, n_q_heads=Hq, n_kv_heads=Hkv, head_dim=D,
                      rope_theta=1e6, budget=64, offsets=[1])
    cache = tria.Cache(t["k"], t["v"], t["pos"], t["seq_len"], t["cur_pos"], starts, pages=pages)
    tree = tria.Tree(t["parent"], t["n_nodes"], t["kd"], t["vd"])
    ws = tria.workspace(cfg, cache, tree=tree)

    def step():
        tria.tria_block_tables(cfg, cache, t["n_new"], t["slots"], ws)
        for layer in range(L):
            tria.tria_tree_attention(cfg, cache, tree, layer, t["q"][layer], t["out"][layer], ws)
        tria.tria_tree_commit(cfg, cache, tree, t["last"], ws, slot_map=t["slots"])

    state = [x.cpu().numpy() for x in pages.tensors]
    graph, lens, cur, served = None, [0, 0, 0], [0, 0, 0], 0
    kept = {(b, l, g): [] for b in range(B) for l in range(L) for g in range(Hkv)}   # (k, v) rows
    for n in range(steps):
        if n in (5, 9):                          # a request ends, a new one takes its place
            lens[n % B], cur[n % B] = 0, 0
            t["seq_len"][n % B], t["cur_pos"][n % B] = 0, 0
            for l in range(L):
                for g in range(Hkv):
                    kept[n % B, l, g] = []
        d = _draw_trees(rng, L, Hkv, B, N, D)
        q = torch.tensor(rng.normal(size=(L, B, N, Hq, D)), dtype=torch.float32).to(torch.bfloat16)
        for name, x in (*d.items(), ("q", q)):
            t[name].copy_(x)
        t["n_new"].copy_(d["n_nodes"])
        t["out"].fill_(7.0)
        if graph is None and n >= 3:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        tria.tria_workspace_init(ws)
        graph.replay() if graph is not None else step()
        torch.cuda.synchronize()
        want = oracle.block_tables(*state, block, lens, d["n_nodes"].tolist(), caps, N)
        state = [np.asarray(x) for x in want[:4]]
        for got, ref in zip(pages.tensors, state):
            assert np.array_equal(got.cpu().numpy(), ref)
        assert np.array_equal(t["slots"].cpu().numpy(), want[4])
        # the attention, from the rows that were committed so far
        nodes, parent = d["n_nodes"].tolist(), d["parent"].numpy()
        for l in range(L):
            k = torch.zeros(1, Hkv, sum(lens) + 1, D, dtype=torch.bfloat16)
            v, at, slots = torch.zeros_like(k), 0, []
            for b in range(B):
                for g in range(Hkv):
                    for j, (kr, vr) in enumerate(kept[b, l, g]):
                        k[0, g, at + j], v[0, g, at + j] = kr, vr
                slots.append([np.arange(at, at + lens[b])] * Hkv)
                at += lens[b]
            ref, spread, steep = oracle.tree_attention(
                common.bf16_bits(k), common.bf16_bits(v), slots, common.bf16_bits(d["kd"][l:l + 1]),
                common.bf16_bits(d["vd"][l:l + 1]), parent, nodes, common.bf16_bits(q[l]), 0, D ** -0.5)
            got = t["out"][l].double().cpu().numpy()
            for b in range(B):
                m = nodes[b]
                assert np.all(got[b, m:] == 7.0)
                logit = 2 * D * 2.0 ** -23 * steep[b, :m, :, None]
                tol = 2.0 ** -7 * np.abs(ref[b, :m]) + (2.0 ** -8 + logit + 2.0 ** -16) * spread[b, :m]
                assert np.all(np.abs(got[b, :m] - ref[b, :m]) <= tol), (n, l, b)
        # the commit
        code = 0
        for b in range(B):
            path = oracle.tree_path(parent[b], int(d["last"][b]))
            if b in want[5]:
                code |= {"pool": tria.DEVERR_POOL, "full": tria.DEVERR_SEGMENT_FULL}[want[5][b]]
                if path:
                    code |= tria.DEVERR_SEGMENT_FULL if lens[b] + len(path) > caps[b] else 0
                    code |= tria.DEVERR_PAGES    # its slots are -1
                continue
            served += len(path)
            for l in range(L):
                for g in range(Hkv):
                    for j, node in enumerate(path):
                        kept[b, l, g].append((d["kd"][l, g, b, node], d["vd"][l, g, b, node]))
                        assert int(t["pos"][l, g, want[4][b, j]]) == cur[b] + 1 + j
            lens[b] += len(path)
            cur[b] += len(path)
        assert tria.tria_get_device_error(ws) == code, n
        assert t["seq_len"].tolist() == lens and t["cur_pos"].tolist() == cur
    assert served > 40
    del graph


def test_speculative_loop_with_the_windowed_prune():
    """Segments: trees of drafted tokens, accepted paths, and the prune back to the budget once
    a window of them has joined; every step against the oracle run from the state before it."""
    from tests.test_gpu_decode import _check_windowed, _problem, _state
    from tests.test_gpu_parity import Case, small
    budget, W, N, steps = 48, 16, 9, 14
    wl = small("speculative", L=2, B=3, Hq=4, Hkv=2, D=64, theta=1e4, seq_lens=[40, 60, 63],
               budget=budget, slack=40, offsets=range(1, 33))
    a = Case(wl)
    cfg = tria.Config.from_workload(wl, prune_window=W)
    rng = np.random.default_rng(8)
    L, Hkv, B, D = 2, 2, 3, 64
    d = _draw_trees(rng, L, Hkv, B, N, D)
    t = {n: x.cuda() for n, x in d.items()}
    tree = tria.Tree(t["parent"], t["n_nodes"], t["kd"], t["vd"])
    ws = tria.workspace(cfg, a.cache, tree=tree)
    q, out = torch.zeros(B, N, 4, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, N, 4, D, dtype=torch.bfloat16, device="cuda")
    sel = torch.empty((L, Hkv, B, budget), dtype=torch.int32, device="cuda")
    pruned = 0
    for _ in range(steps):
        d = _draw_trees(rng, L, Hkv, B, N, D)
        for n, x in d.items():
            t[n].copy_(x)
        q.copy_(torch.tensor(rng.normal(size=q.shape), dtype=torch.float32))
        before = _state(a)
        sel.fill_(-7)
        tria.tria_tree_attention(cfg, a.cache, tree, 1, q, out, ws)
        tria.tria_tree_commit(cfg, a.cache, tree, t["last"], ws)
        torch.cuda.synchronize()
        joined = _state(a)
        tria.tria_prune(cfg, a.stats, a.cache, ws, sel_out=sel)
        torch.cuda.synchronize()
        assert tria.tria_get_device_error(ws) == 0
        # attention over the keys before the step
        starts = a.host["seq_start"]
        slots = [[starts[b] + np.arange(before["seq_len"][b])] * Hkv for b in range(B)]
        ref, spread, steep = oracle.tree_attention(
            before["k"], before["v"], slots, common.bf16_bits(d["kd"]), common.bf16_bits(d["vd"]),
            d["parent"].numpy(), d["n_nodes"].tolist(), common.bf16_bits(q), 1, D ** -0.5)
        got = out.double().cpu().numpy()
        for b in range(B):
            m = int(d["n_nodes"][b])
            logit = 2 * D * 2.0 ** -23 * steep[b, :m, :, None]
            tol = 2.0 ** -7 * np.abs(ref[b, :m]) + (2.0 ** -8 + logit + 2.0 ** -16) * spread[b, :m]
            assert np.all(np.abs(got[b, :m] - ref[b, :m]) <= tol), b
        # the commit, then the prune of what it left
        want = {n: before[n].copy() for n in ("k", "v", "pos", "seq_len", "cur_pos")}
        kd, vd = common.bf16_bits(d["kd"]), common.bf16_bits(d["vd"])
        for b in range(B):
            for j, node in enumerate(oracle.tree_path(d["parent"][b].tolist(), int(d["last"][b]))):
                at = starts[b] + want["seq_len"][b]
                want["k"][:, :, at], want["v"][:, :, at] = kd[:, :, b, node], vd[:, :, b, node]
                want["pos"][:, :, at] = want["cur_pos"][b] + 1
                want["seq_len"][b] += 1
                want["cur_pos"][b] += 1
        for n in want:
            assert np.array_equal(joined[n], want[n]), n
        ref = oracle.prune_window(_problem(a, want["k"], want["pos"], want["seq_len"], want["cur_pos"]),
                                  want["v"], W)
        _check_windowed(a, W, want, _state(a), sel.cpu().numpy(), ref)
        pruned += int(np.sum(want["seq_len"] >= budget + W))
    assert pruned == 2  # by the lengths alone


def test_two_calls_at_once():
    """Two streams with workspaces of their own: the CTAs of a call wait for one another, and
    never for the other call's."""
    a, b = Spec(lens=[5000, 700], N=16, seed=1), Spec(lens=[3000, 90, 2000], N=9, seed=2, block=16, Hq=4)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(25):
        a.attend(stream=streams[0])
        b.attend(stream=streams[1])
    torch.cuda.synchronize()
    for s in (a, b):
        assert tria.tria_get_device_error(s.ws) == 0
        s.check()


def test_largest_batch_and_shapes():
    """256 sequences (some empty, some without nodes), and 256 nodes of 16 heads at D = 256."""
    rng = np.random.default_rng(4)
    s = Spec(lens=rng.integers(0, 200, 256).tolist(), N=4, nodes=rng.integers(0, 5, 256).tolist(),
             Hq=2, Hkv=1, D=64, block=16)
    s.attend()
    torch.cuda.synchronize()
    assert tria.tria_get_device_error(s.ws) == 0
    s.check()
    s = Spec(lens=[140], N=256, Hq=16, Hkv=1, D=256)
    s.attend()
    torch.cuda.synchronize()
    assert tria.tria_get_device_error(s.ws) == 0
    s.check()


def test_a_cache_without_slots():
    s = Spec(lens=[0, 0], slack=0, N=3)
    assert s.cap == 0
    s.t["k"] = torch.zeros(1, 2, 1, 128, dtype=torch.bfloat16, device="cuda")
    s.cache = tria.Cache(s.t["k"], s.t["k"], torch.zeros(4, dtype=torch.int32, device="cuda"),
                         s.t["seq_len"], s.t["cur_pos"], s.starts, cap_total=0)
    s.attend()
    torch.cuda.synchronize()
    assert tria.tria_get_device_error(s.ws) == 0
    s.check()


def test_jumping_maxima():
    """Logits that grow along the keys by less and by far more than the running maximum allows
    without a change of scale, in both halves of a tile and between tiles; -0 and huge values."""
    s = Spec(lens=[1500, 640], N=6, Hq=4, Hkv=2)
    grow = torch.ones(1500)
    grow[130:] = 8.0                       # inside a tile, in its second half
    grow[400:] = 30.0
    grow[900] = 600.0
    for b, T in enumerate(s.lens):
        at = torch.tensor(s._at(b, T))
        s.k[:, :, at] = (s.k[:, :, at].float() * grow[:T].view(1, 1, T, 1)).to(torch.bfloat16)
    s.t["k"].copy_(s.k)
    s.attend()
    torch.cuda.synchronize()
    assert tria.tria_get_device_error(s.ws) == 0
    s.check()


def test_binding_refuses_strides_and_shapes():
    s = Spec(lens=[20], N=3, Hq=4, Hkv=2, D=64)
    with pytest.raises(ValueError, match="contiguous"):
        tria.tria_tree_attention(s.cfg, s.cache, s.tree, 0, s.t["q"].transpose(1, 2).contiguous().transpose(1, 2),
                                 s.t["out"], s.ws)
    with pytest.raises(ValueError, match="q: expected"):
        tria.tria_tree_attention(s.cfg, s.cache, s.tree, 0, s.t["q"][:, :2].contiguous(), s.t["out"], s.ws)
    with pytest.raises(ValueError, match="out: expected"):
        tria.tria_tree_attention(s.cfg, s.cache, s.tree, 0, s.t["q"], s.t["out"].float(), s.ws)
    with pytest.raises(ValueError, match="last: expected"):
        tria.tria_tree_commit(s.cfg, s.cache, s.tree, torch.zeros(2, dtype=torch.int32, device="cuda"), s.ws)
    with pytest.raises(tria.TriaError, match="WORKSPACE"):
        tria.tria_tree_attention(s.cfg, s.cache, s.tree, 0, s.t["q"], s.t["out"], s.ws[:1 << 20])
