"""Tree attention over the forms where a CTA walks many key tiles: one and two M tiles, every
head dimension, segments, pages and per-unit lengths, and logits that make the running maximum
change.  The reference and the tolerances are those of test_gpu_tree.py."""
import numpy as np
import pytest
import torch

import oracle
from kv_cache_eviction_trig_b200 import tria
from tests import common
from tests.test_gpu_tree import Spec, _lib  # noqa: F401

pytestmark = pytest.mark.gpu

TILE = 128


def _many_tiles(s, layer=0, per_cta=2):
    """A CTA takes at least `per_cta` key tiles: the grid is at most the number of SMs."""
    G = s.Hq // s.Hkv
    m_tiles = 2 if s.D < 256 and s.N * G > TILE else 1
    tiles = sum(-(-s.nodes[b] * G // (m_tiles * TILE)) *
                (-(-s._len(layer, g, b) // TILE) - (-s.nodes[b] // TILE))
                for b in range(s.B) for g in range(s.Hkv))
    assert tiles > per_cta * torch.cuda.get_device_properties(0).multi_processor_count
    return m_tiles


def _run(s, layer=0, scale=None):
    s.t["out"].fill_(7.0)
    s.attend(layer, scale=scale)
    torch.cuda.synchronize()
    assert tria.tria_get_device_error(s.ws) == 0
    s.check(layer, scale=scale)


def _ladder(s, step):
    """Keys whose logits climb in both halves of every tile: dimension 0 of the queries is 16,
    that of the keys grows by `step` at the 10th and at the 74th key of a tile, and the other
    dimensions add little."""
    for b, T in enumerate(s.lens):
        at = torch.tensor(s._at(b, T))
        t = torch.arange(T)
        level = step * (2 * (t // TILE) + (t % TILE >= 10).long() + (t % TILE >= 74).long()).float()
        rows = 0.3 * s.k[:, :, at].float()
        rows[..., 0] = level
        s.k[:, :, at] = rows.to(torch.bfloat16)
        s.q[b, :s.nodes[b], :, 0] = 16.0
        top = step * 2.0 * (T // TILE + 1)
        s.kd[:, :, b, :s.nodes[b], 0] = top
    s.t["k"].copy_(s.k)
    s.t["q"].copy_(s.q)
    s.t["kd"].copy_(s.kd)


# A step of 5 is 10.2 powers of two at D = 128 and 14.4 at D = 64 (the other dimensions move it
# by at most about 2): past the 8 that a maximum may lag behind, in both halves of each tile.  What came before
# then keeps a weight of 2^-10 or so per key, 60 keys of it: a change of scale that is lost
# moves the result by several per cent, ten times the tolerance.
@pytest.mark.parametrize("D,block", [(128, 0), (64, 0), (128, 32), (64, 256)])
def test_two_m_tiles_rescaled_in_both_halves_of_a_tile(D, block):
    s = Spec(D=D, Hq=32, Hkv=8, lens=[2400, 2100, 640], N=40, nodes=[40, 33, 36], block=block)
    assert _many_tiles(s) == 2
    _ladder(s, 5.0)
    _run(s)


# Each kernel (head dimension, M tiles) over many key tiles per CTA: rings that go round, both phases of every
# barrier, changes of unit in the middle of a share, parts over several CTAs; keys that climb slowly
# (the maximum lags behind them, within 2^8) or fast, and zeros of both signs.
KERNELS = {"d64": dict(D=64, N=7), "d64 two M tiles": dict(D=64, N=13), "d128": dict(D=128, N=7),
           "d128 two M tiles": dict(D=128, N=13), "d256": dict(D=256, N=7), "d256 more rows": dict(D=256, N=11)}


@pytest.mark.parametrize("layout", ["segments", "pages of 16", "pages of 256", "unit lengths"])
@pytest.mark.parametrize("name", sorted(KERNELS))
def test_many_tiles_per_cta(name, layout):
    kw = dict(Hq=128, Hkv=8, nodes=[KERNELS[name]["N"], 5, KERNELS[name]["N"] - 1], **KERNELS[name])
    if layout == "segments":
        s = Spec(lens=[8100, 7000, 9300], **kw)
    elif layout == "unit lengths":
        lens = np.random.default_rng(3).integers(1000, 5000, (1, 8, 3))
        lens[0, 2, 1], lens[0, 5, 0], lens[0, 7, 2] = 0, 1, 128
        s = Spec(lens=[0, 0, 0], unit_lens=lens, **kw)
        s.lens = [int(lens[0, :, b].max()) for b in range(3)]        # for the keys below
    else:
        s = Spec(lens=[4100, 1, 5333], block=int(layout.split()[-1]), **kw)
    assert _many_tiles(s, per_cta=10 if layout == "segments" else 3) == (2 if "two" in name else 1)
    _ladder(s, 5.0 if layout in ("segments", "pages of 256") else 0.7)
    for x in ("k", "v", "kd", "vd", "q"):
        zero = getattr(s, x)[..., 1::7]
        zero[:] = torch.where(torch.isnan(zero), zero, torch.where(zero < 0, -0.0, 0.0).to(zero.dtype))
        s.t[x].copy_(getattr(s, x))
    _run(s)


@pytest.mark.parametrize("block", [0, 64])
@pytest.mark.parametrize("shape", ["tree", "chain"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_many_large_trees(D, shape, block):
    """Tiles of nodes in the middle of a CTA's share, two of them per tree, with infinities and
    NaN in values of some nodes of either tile: they reach those nodes' descendants, and no
    other row."""
    rng = np.random.default_rng(D + block)
    s = Spec(D=D, Hq=8, Hkv=8, lens=rng.integers(0, 300, 24).tolist(), N=200, shape=shape, block=block,
             nodes=rng.integers(0, 201, 24).tolist(), seed=block)
    assert _many_tiles(s) == (1 if D == 256 else 2)
    for b in range(0, 24, 2):
        for node in rng.integers(0, 200, 3):
            if node < s.nodes[b]:
                s.vd[0, rng.integers(8), b, node, rng.integers(D)] = float("inf")
                s.vd[0, rng.integers(8), b, node, rng.integers(D)] = float("nan")
    s.t["vd"].copy_(s.vd)
    s.t["out"].fill_(7.0)
    s.attend()
    torch.cuda.synchronize()
    assert tria.tria_get_device_error(s.ws) == 0
    slots = [[s._at(b, s.lens[b])] * s.Hkv for b in range(s.B)]
    ref, spread, steep = oracle.tree_attention(
        common.bf16_bits(s.k), common.bf16_bits(s.v), slots, common.bf16_bits(s.kd),
        common.bf16_bits(s.vd), s.parent, s.nodes, common.bf16_bits(s.q), 0, D ** -0.5)
    got = s.t["out"].double().cpu().numpy()
    poisoned = 0
    for b, n in enumerate(s.nodes):
        g, r = got[b, :n], ref[b, :n]
        assert np.all(got[b, n:] == 7.0)
        fine = np.isfinite(r)
        poisoned += np.sum(~fine)
        assert np.array_equal(np.isnan(g), np.isnan(r)) and np.array_equal(g[np.isinf(r)], r[np.isinf(r)]), b
        tol = (2.0 ** -7 * np.abs(r) + (2.0 ** -8 + 2 * D * 2.0 ** -23 * steep[b, :n, :, None] + 2.0 ** -16) *
               spread[b, :n])
        assert np.all(np.abs(g[fine] - r[fine]) <= tol[fine]), b
    assert poisoned > 0                      # (of the reference: some node was poisoned)


# Logits so large that they are one key's, or a few equal keys', in float32 and in float64 alike.
# The queries have one dimension, so a logit before its scale is a product of two bf16 numbers
# and exact in float32; two different ones of a row are more than 2^-8 of the largest apart,
# millions of powers of two here.  What is left is the rounding of the weights and of the output.
HUGE = {
    "2^33": (17, 16, "mixed"),
    "2^60": (30, 30, "mixed"),
    "2^33 negative": (17, 16, "negative"),
    "2^60 negative": (30, 30, "negative"),
    "2^60 climbing": (30, 30, "climbing"),
    "2^127 climbing": (64, 63, "climbing"),       # from -3e38 to 3e38: the difference is not finite
}


@pytest.mark.parametrize("D,N,block", [(64, 6, 0), (64, 70, 64), (128, 6, 32), (128, 70, 0), (256, 6, 0)])
@pytest.mark.parametrize("name", sorted(HUGE))
def test_huge_finite_logits(name, D, N, block):
    qe, ke, kind = HUGE[name]
    s = Spec(D=D, Hq=16, Hkv=4, lens=[700, 3, 2600], N=N, nodes=[N, N - 1, N - 3], block=block, seed=qe + D)
    rng = np.random.default_rng(ke)

    def bf16(x):  # of 8 bits, at most 1.98 in size
        return np.clip(np.round(x * 64), -127, 127) / 64

    for b, T in enumerate(s.lens):
        n = s.nodes[b]
        at = torch.tensor(s._at(b, T))
        k = bf16(rng.uniform(-1.99, 1.99, (s.L, s.Hkv, T + n)))
        q = bf16(rng.uniform(0.5, 1.99, (n, s.Hq)))
        if kind == "climbing":
            k = np.concatenate([np.sort(k[..., :T]), k[..., T:]], -1)
            k[..., 0], k[..., T - 1], q[:] = -127 / 64, 127 / 64, 1.0
        if kind == "negative":
            k = -np.maximum(np.abs(k), 0.5)
        k = torch.tensor(k * 2.0 ** ke, dtype=torch.float32).to(torch.bfloat16)
        s.k[:, :, at, 0], s.kd[:, :, b, :n, 0] = k[..., :T], k[..., T:]
        s.q[b, :n] = 0.0
        s.q[b, :n, :, 0] = torch.tensor(q * 2.0 ** qe, dtype=torch.float32).to(torch.bfloat16)
    for x in ("k", "kd", "q"):
        s.t[x].copy_(getattr(s, x))
    s.attend()
    torch.cuda.synchronize()
    assert tria.tria_get_device_error(s.ws) == 0
    slots = [[s._at(b, s.lens[b])] * s.Hkv for b in range(s.B)]
    ref, spread, _ = oracle.tree_attention(
        common.bf16_bits(s.k), common.bf16_bits(s.v), slots, common.bf16_bits(s.kd),
        common.bf16_bits(s.vd), s.parent, s.nodes, common.bf16_bits(s.q), 0, s.D ** -0.5)
    got = s.t["out"].double().cpu().numpy()
    for b, n in enumerate(s.nodes):
        tol = 2.0 ** -7 * np.abs(ref[b, :n]) + (2.0 ** -8 + 2.0 ** -16) * spread[b, :n]
        assert np.all(np.abs(got[b, :n] - ref[b, :n]) <= tol), b


@pytest.mark.parametrize("D,N,lens", [(64, 6, [300, 0, 20000]), (128, 6, [300, 0, 9000]), (256, 6, [300, 0, 9000]),
                                      (64, 70, [300, 0, 9000]), (128, 70, [300, 0, 20000])])
def test_logits_of_minus_infinity(D, N, lens):
    """A key of -inf has no weight beside a finite one; where a row sees nothing else, the softmax
    is 0 / 0.  Sequence by sequence: all cached keys are -inf, node 1 is finite (its
    descendants are its own); no cached key, node 1 is finite; all cached keys are -inf but the last."""
    s = Spec(D=D, Hq=8, Hkv=2, lens=lens, N=N)
    s.q[..., 1:] = 0.0
    s.q[..., 0] = s.q[..., 0].float().abs().to(torch.bfloat16) + 0.5
    for b, T in enumerate(lens):
        at = torch.tensor(s._at(b, T), dtype=torch.long)
        s.k[:, :, at, 0] = float("-inf")
        s.kd[:, :, b, :, 0] = float("-inf")
    s.kd[:, :, 0, 1, 0] = s.kd[:, :, 1, 1, 0] = 0.25
    s.k[:, :, s.starts[2] + lens[2] - 1, 0] = -3.0
    for x in ("k", "kd", "q"):
        s.t[x].copy_(getattr(s, x))
    s.attend()
    torch.cuda.synchronize()
    assert tria.tria_get_device_error(s.ws) == 0
    got = s.t["out"].float().cpu()
    for b in range(3):
        for i in range(N):
            path = oracle.tree_path(s.parent[b], i)
            if b < 2 and 1 not in path:
                assert torch.isnan(got[b, i]).all(), (b, i)
                continue
            seen = s.vd[0, :, b, 1] if b < 2 else s.v[0, :, s.starts[2] + lens[2] - 1]
            assert torch.equal(got[b, i], seen.float().repeat_interleave(4, 0)), (b, i)


def test_a_bad_unit_length_skips_that_unit():
    """Per-unit lengths: the heads of the other units are served; later units and sequences too."""
    lens = np.array([[[300, 700, 64], [129, 900, 1000], [200, 40, 300]]])
    s = Spec(Hq=12, Hkv=3, lens=[0, 0, 0], unit_lens=lens, N=9)
    _run(s)
    good = s.t["out"].clone()
    s.t["unit_len"][0, 1, 0], s.t["unit_len"][0, 2, 1], s.t["unit_len"][0, 0, 2] = -1, 10 ** 6, 1041
    s.t["out"].fill_(7.0)
    s.attend()
    torch.cuda.synchronize()
    assert tria.tria_get_device_error(s.ws) == tria.DEVERR_SEQ_LEN
    for b, g in ((0, 1), (1, 2), (2, 0)):
        heads = slice(4 * g, 4 * g + 4)
        assert torch.all(s.t["out"][b, :, heads] == 7.0)
        s.t["out"][b, :, heads] = good[b, :, heads]
    s.check()


@pytest.mark.parametrize("D,N", [(64, 4), (128, 200)])
def test_no_nodes_at_all(D, N):
    s = Spec(D=D, lens=[300, 0], N=N, nodes=[0, 0])
    _run(s)
