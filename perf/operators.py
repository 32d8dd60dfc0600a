"""Measured cases of the speculative decode step over the pruned cache.

Three operators work together there:

* ``tree``    attention of the nodes of a drafted token tree over the cached keys and over
              their own ancestors in the tree (the cache in segments, or in pages);
* ``tables``  block tables and slot maps of a paged cache, brought up to date on the GPU
              from the requests' lengths (blocks taken from and given back to a pool);
* ``commit``  the accepted path of the tree joins the cache.

``own`` false: plain torch operations in float32 (float64 where noted).  ``own`` true: the
calls of the framework.  Shapes come from the workloads of this repository (the tiny, the
8B-shaped, the ragged serving and the long one) and its budgets of 512, 2048 and 4096 keys.
"""
from __future__ import annotations

import math

import torch

own = False


# ---------------------------------------------------------------- cases

def listed():
    return [
        # the tiny workload after its prune: 512 keys, a small tree; launch latency counts
        dict(name="tree tiny", op="tree", B=1, Hq=4, Hkv=2, D=64, N=8, t_lo=512, t_hi=512,
             block=0, chain=False),
        # one request of the 8B-shaped model right after a prune to the default budget
        dict(name="tree 8B budget", op="tree", B=1, Hq=32, Hkv=8, D=128, N=32, t_lo=2048,
             t_hi=2048, block=0, chain=False),
        # a serving batch between two prunes (2048 to 2176 keys each), in pages of 16
        dict(name="tree batch paged", op="tree", B=16, Hq=32, Hkv=8, D=128, N=16, t_lo=2048,
             t_hi=2176, block=16, chain=False),
        # the 8B-shaped layer before its first prune, a large tree
        dict(name="tree 8B 32K", op="tree", B=1, Hq=32, Hkv=8, D=128, N=64, t_lo=32768,
             t_hi=32768, block=0, chain=False),
        # the ragged serving batch before its first prune, in pages of 64
        dict(name="tree ragged paged", op="tree", B=16, Hq=32, Hkv=8, D=128, N=32, t_lo=8192,
             t_hi=32768, block=64, chain=False),
        # the long workload (8 query heads per KV head), a tree of 16
        dict(name="tree long", op="tree", B=4, Hq=64, Hkv=8, D=128, N=16, t_lo=131072,
             t_hi=131072, block=0, chain=False),
        # a chunk of 255 prompt tokens (a chain) over odd prefixes: bound by the products
        dict(name="tree chunk", op="tree", B=4, Hq=64, Hkv=8, D=128, N=255, t_lo=4097,
             t_hi=9001, block=0, chain=True),
        # a decode step of a serving batch: most requests stay inside their last block
        dict(name="tables decode", op="tables", B=16, block=16, max_len=2304, n_lo=1, n_hi=16,
             full=False),
        # 256 requests, some just pruned from long prompts, some just admitted with one
        dict(name="tables admit", op="tables", B=256, block=64, max_len=32768, n_lo=0, n_hi=8192,
             full=True),
        # one request of the 8B-shaped model accepts part of a tree
        dict(name="commit 8B", op="commit", L=36, B=1, Hkv=8, D=128, N=32, room=2304, block=0),
        # a serving batch accepts its paths, in pages of 16
        dict(name="commit batch paged", op="commit", L=36, B=64, Hkv=8, D=128, N=64, room=160,
             block=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tree", "tree", "tree", "tables", "commit"])
    while True:
        if op == "tree":
            G = rng.choice([1, 2, 4, 8, 16])
            Hkv = rng.choice([1, 2, 4, 8])
            hi = _log(rng, 1, 131072)
            c = dict(op=op, B=_log(rng, 1, 64), Hq=G * Hkv, Hkv=Hkv,
                     D=rng.choice([64, 128, 128, 256]), N=_log(rng, 1, 256),
                     t_lo=rng.randint(max(0, hi // 4), hi), t_hi=hi,
                     block=rng.choice([0, 16, 32, 64, 128]), chain=rng.random() < 0.3)
            w = work(c)
            # no dearer than the dearest listed case, and its plain logits fit
            if (w["bytes"] <= 2.2e9 and w["flops"] <= 2.2e11
                    and c["B"] * c["Hq"] * c["N"] * (hi + c["N"]) <= 6e8
                    and c["B"] * Hkv * (hi + c["N"]) * c["D"] <= 6e8):
                return c
        elif op == "tables":
            B = _log(rng, 1, 256)
            max_len = _log(rng, 64, 32768)
            return dict(op=op, B=B, block=rng.choice([16, 32, 64, 128]), max_len=max_len,
                        n_lo=0, n_hi=_log(rng, 1, max(1, max_len // 4)), full=rng.random() < 0.5)
        else:
            c = dict(op=op, L=_log(rng, 1, 36), B=_log(rng, 1, 64), Hkv=rng.choice([1, 2, 4, 8]),
                     D=rng.choice([64, 128, 256]), N=_log(rng, 1, 256),
                     room=0, block=rng.choice([0, 16, 32, 64]))
            c["room"] = c["N"] + _log(rng, 32, 2304)
            if c["L"] * c["B"] * c["Hkv"] * c["D"] * c["room"] <= 6e8:
                return c


# ---------------------------------------------------------------- inputs

def _ints(g, lo, hi, n, device="cpu"):
    """n whole numbers of [lo, hi]; the largest of the range among them."""
    x = torch.randint(lo, hi + 1, (n,), generator=g)
    x[n // 2] = hi
    return x.to(torch.int32).to(device)


def _parents(g, B, N, chain):
    """Drafted trees: node i hangs below an earlier node, or below the last cached token (-1)."""
    if chain:
        return (torch.arange(N) - 1).repeat(B, 1).to(torch.int32)
    up = torch.rand(B, N, generator=g)
    return (torch.floor(up * (torch.arange(N) + 1)) - 1).to(torch.int32)


def _tables(g, need, max_blocks, n_blocks):
    """Block tables that hold need[b] blocks each, in shuffled order, and the ring of free blocks."""
    B = need.numel()
    order = torch.randperm(n_blocks, generator=g).to(torch.int32)
    table = torch.full((B, max_blocks), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        n = int(need[b])
        table[b, :n] = order[at:at + n]
        at += n
    ring = torch.full((n_blocks,), -1, dtype=torch.int32)
    ring[:n_blocks - at] = order[at:]
    return table, ring, torch.tensor([0, n_blocks - at], dtype=torch.int32)


def prepare(case, seed):
    return {"tree": _prepare_tree, "tables": _prepare_tables, "commit": _prepare_commit}[
        case["op"]](case, seed)


def _gpu(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _handles(s, case, L, Hq):
    """The configuration, cache, tree and workspace that a program keeps between calls."""
    if not own:
        return
    from kv_cache_eviction_trig_b200 import tria
    B = case["B"]
    s["tria"] = tria
    s["cfg"] = tria.Config(num_layers=L, batch=B, n_q_heads=Hq, n_kv_heads=s["Hkv"],
                           head_dim=s["D"], rope_theta=1e6, budget=2048, offsets=[1])
    pages = None
    if case["block"]:
        pages = tria.Pages(s["table"], s["held"], s["ring"], s["state"], case["block"])
    s["cache"] = tria.Cache(s["k"], s["v"], s["pos"], s["seq_len"], s["cur_pos"], s["starts"],
                            pages=pages)
    tree = None
    if "parent" in s:
        tree = s["tree"] = tria.Tree(s["parent"], s["n_nodes"], s["kd"], s["vd"])
    s["ws"] = tria.workspace(s["cfg"], s["cache"], tree=tree)


def _layout(s, g, lens, room, block):
    """Segments, or pages in a pool that holds every request's most: where each request's keys live."""
    B = lens.numel()
    s["block"] = block
    if not block:
        s["starts"] = [b * room for b in range(B + 1)]
        s["slots"] = B * room
        return
    blocks = (room + block - 1) // block
    s["starts"] = [b * blocks * block for b in range(B + 1)]
    need = (lens.long() + block - 1) // block
    n_blocks = B * blocks
    s["need"], s["blocks"], s["n_blocks"] = need, blocks, n_blocks
    s["slots"] = n_blocks * block
    table, ring, state = _tables(g, need, blocks, n_blocks)
    s["table"], s["ring"], s["state"] = table.cuda(), ring.cuda(), state.cuda()
    s["held"] = need.to(torch.int32).cuda()


def _prepare_tree(case, seed):
    g, gg = torch.Generator().manual_seed(seed), _gpu(seed)
    B, Hq, Hkv, D, N = (case[n] for n in ("B", "Hq", "Hkv", "D", "N"))
    lens = _ints(g, case["t_lo"], case["t_hi"], B)
    s = dict(op="tree", Hkv=Hkv, D=D, N=N, t_hi=case["t_hi"])
    _layout(s, g, lens, case["t_hi"] + 128, case["block"])
    s["seq_len"] = lens.cuda()
    s["cur_pos"] = (2 * lens).cuda()
    # keys and queries gather around a centre per head, as pre-RoPE vectors do
    centre = torch.randn(Hkv, D, generator=gg, device="cuda")
    s["k"] = torch.empty(1, Hkv, s["slots"], D, dtype=torch.bfloat16, device="cuda")
    s["v"] = torch.empty_like(s["k"])
    for h in range(Hkv):
        s["k"][0, h] = (0.5 * centre[h] + torch.randn(s["slots"], D, generator=gg, device="cuda")).to(torch.bfloat16)
        s["v"][0, h] = torch.randn(s["slots"], D, generator=gg, device="cuda").to(torch.bfloat16)
    s["pos"] = torch.zeros(1, Hkv, s["slots"], dtype=torch.int32, device="cuda")
    s["kd"] = (0.5 * centre.view(1, Hkv, 1, 1, D)
               + torch.randn(1, Hkv, B, N, D, generator=gg, device="cuda")).to(torch.bfloat16)
    s["vd"] = torch.randn(1, Hkv, B, N, D, generator=gg, device="cuda").to(torch.bfloat16)
    qc = 0.5 * centre.repeat_interleave(Hq // Hkv, 0)
    s["q"] = (qc + 1.5 * torch.randn(B, N, Hq, D, generator=gg, device="cuda")).to(torch.bfloat16)
    s["parent"] = _parents(g, B, N, case["chain"]).cuda()
    s["n_nodes"] = _ints(g, (N + 1) // 2, N, B, "cuda")
    s["out"] = torch.zeros(B, N, Hq, D, dtype=torch.bfloat16, device="cuda")
    _handles(s, case, 1, Hq)
    return s


def _prepare_tables(case, seed):
    g = torch.Generator().manual_seed(seed)
    B, block, top = case["B"], case["block"], case["max_len"]
    # what each request holds now, its length in this step and in the next: where full, a
    # third of the requests were pruned to an eighth and a third starts with a new prompt
    held_len = _ints(g, 0, top - case["n_hi"], B)
    n1, n2 = _ints(g, case["n_lo"], case["n_hi"], B), _ints(g, case["n_lo"], case["n_hi"], B)
    len1 = torch.minimum(held_len + _ints(g, 0, block, B), torch.tensor(top - case["n_hi"])).to(torch.int32)
    if case["full"]:
        kind = torch.randint(0, 3, (B,), generator=g)
        len1 = torch.where(kind == 0, len1 // 8, len1).to(torch.int32)
        held_len = torch.where(kind == 1, torch.zeros_like(held_len), held_len)
        len1 = torch.where(kind == 1, torch.zeros_like(len1), len1)
    need = (held_len.long() + block - 1) // block
    max_blocks = (top + block - 1) // block
    n_blocks = B * max_blocks
    table, ring, state = _tables(g, need, max_blocks, n_blocks)
    s = dict(op="tables", block=block, n_blocks=n_blocks, Hkv=1, D=64, max_new=case["n_hi"])
    s["table"], s["ring"], s["state"] = table.cuda(), ring.cuda(), state.cuda()
    s["held"] = need.to(torch.int32).cuda()
    s["steps"] = []
    s["slot_map"] = [torch.zeros(B, case["n_hi"], dtype=torch.int32, device="cuda") for _ in range(2)]
    s["starts"] = [b * max_blocks * block for b in range(B + 1)]
    for i, (t, n) in enumerate(((len1, n1), (held_len, n2))):
        s["seq_len"], s["cur_pos"] = t.to(torch.int32).cuda(), t.to(torch.int32).cuda()
        s["steps"].append(dict(seq_len=s["seq_len"], n_new=n.cuda(), slot_map=s["slot_map"][i]))
        if own:
            s["k"] = s["v"] = s["pos"] = None
            from kv_cache_eviction_trig_b200 import tria
            s["tria"] = tria
            s["cfg"] = tria.Config(num_layers=1, batch=B, n_q_heads=1, n_kv_heads=1, head_dim=64,
                                   rope_theta=1e6, budget=2048, offsets=[1])
            pages = tria.Pages(s["table"], s["held"], s["ring"], s["state"], block)
            s["steps"][-1]["cache"] = tria.Cache(None, None, None, s["seq_len"], s["cur_pos"],
                                                 s["starts"], cap_total=n_blocks * block, pages=pages)
    if own:
        s["ws"] = s["tria"].workspace(s["cfg"], s["steps"][0]["cache"])
    return s


def _prepare_commit(case, seed):
    g, gg = torch.Generator().manual_seed(seed), _gpu(seed)
    L, B, Hkv, D, N, room = (case[n] for n in ("L", "B", "Hkv", "D", "N", "room"))
    lens = _ints(g, 0, room - N, B)
    s = dict(op="commit", Hkv=Hkv, D=D, N=N)
    # in pages, the blocks of the tokens to come are held already
    _layout(s, g, lens + N, room, case["block"])
    s["k"] = torch.zeros(L, Hkv, s["slots"], D, dtype=torch.bfloat16, device="cuda")
    s["v"] = torch.zeros_like(s["k"])
    s["pos"] = torch.zeros(L, Hkv, s["slots"], dtype=torch.int32, device="cuda")
    s["kd"] = torch.randn(L, Hkv, B, N, D, generator=gg, device="cuda").to(torch.bfloat16)
    s["vd"] = torch.randn(L, Hkv, B, N, D, generator=gg, device="cuda").to(torch.bfloat16)
    # lengths and positions side by side: every pass starts from the same ones
    s["start"] = torch.stack([lens, 2 * lens]).to(torch.int32).cuda()
    s["now"] = s["start"].clone()
    s["seq_len"], s["cur_pos"] = s["now"][0], s["now"][1]
    s["parent"] = _parents(g, B, N, False).cuda()
    s["n_nodes"] = _ints(g, (N + 1) // 2, N, B, "cuda")
    # the last accepted node; a request in eight accepts none
    last = torch.floor(torch.rand(B, generator=g) * s["n_nodes"].cpu()).to(torch.int32)
    s["last"] = torch.where(torch.rand(B, generator=g) < 0.125, torch.full_like(last, -1), last).cuda()
    s["slot_map"] = None
    if case["block"]:
        t = lens.long().view(B, 1) + torch.arange(N)
        at = s["table"].cpu().long().gather(1, t // case["block"])
        s["slot_map"] = (at * case["block"] + t % case["block"]).to(torch.int32).cuda()
    _handles(s, case, L, Hkv)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return {"tree": _run_tree, "tables": _run_tables, "commit": _run_commit}[s["op"]](s)


def _ancestors(parent, n_nodes):
    """[B][N][N]: whether node j is node i or one of its ancestors.  The sum of the powers of
    the parent relation, which the inverse of a unit triangular matrix gives exactly."""
    B, N = parent.shape
    node = torch.arange(N, device=parent.device)
    real = node < n_nodes.view(B, 1)
    up = (parent.unsqueeze(2) == node) & real.unsqueeze(2)
    eye = torch.eye(N, device=parent.device, dtype=torch.float64).expand(B, N, N)
    reach = torch.linalg.solve_triangular(eye - up.double(), eye, upper=False) > 0.5
    return reach & real.unsqueeze(2)


def _slots(s, t):
    """Slots [B][len(t)] of the cached tokens t of every request."""
    if s["block"]:
        at = s["table"].long()[:, t // s["block"]]
        return at.clamp_min(0) * s["block"] + t % s["block"]
    starts = torch.tensor(s["starts"][:-1], device=t.device).view(-1, 1)
    return starts + t


def _run_tree(s):
    if own:
        s["tria"].tria_tree_attention(s["cfg"], s["cache"], s["tree"], 0, s["q"], s["out"], s["ws"])
        return s["out"]
    q, out = s["q"], s["out"]
    B, N, Hq, D = q.shape
    Hkv = s["Hkv"]
    G = Hq // Hkv
    t = torch.arange(s["t_hi"], device=q.device)
    live = t < s["seq_len"].view(B, 1)                                   # [B][T]
    at = torch.where(live, _slots(s, t), 0)
    k = torch.cat([s["k"][0][:, at], s["kd"][0]], 2).float()             # [Hkv][B][T + N][D]
    v = torch.cat([s["v"][0][:, at], s["vd"][0]], 2).float()
    reach = _ancestors(s["parent"], s["n_nodes"])                        # [B][N][N]
    seen = torch.cat([live.unsqueeze(1).expand(B, N, -1), reach], 2)     # [B][N][T + N]
    held = torch.cat([live, torch.arange(N, device=q.device) < s["n_nodes"].view(B, 1)], 1)
    v = torch.where(held.unsqueeze(-1), v, 0.0)
    qf = q.float().view(B, N, Hkv, G, D).permute(2, 0, 1, 3, 4).reshape(Hkv, B, N * G, D)
    x = (qf @ k.transpose(2, 3)) * D ** -0.5
    x = x.view(Hkv, B, N, G, -1).masked_fill_(~seen.view(1, B, N, 1, -1), -math.inf)
    x = (x - x.amax(-1, keepdim=True).clamp_min(-3e38)).exp_()
    total = x.sum(-1, keepdim=True)
    o = (x.view(Hkv, B, N * G, -1) @ v).view(Hkv, B, N, G, D) / total
    o = o.permute(1, 2, 0, 3, 4).reshape(B, N, Hq, D).to(torch.bfloat16)
    rows = torch.arange(N, device=q.device) < s["n_nodes"].view(B, 1)    # the others stay as they were
    out.copy_(torch.where(rows.view(B, N, 1, 1), o, out))
    return out


def _run_tables(s):
    for step in s["steps"]:
        if own:
            s["tria"].tria_block_tables(s["cfg"], step["cache"], step["n_new"], step["slot_map"],
                                        s["ws"])
        else:
            _update_tables(s, step)
    return s["table"], s["held"], s["ring"], s["state"], s["slot_map"]


def _update_tables(s, step):
    table, held, ring, state = s["table"], s["held"], s["ring"], s["state"]
    block, n_blocks = s["block"], s["n_blocks"]
    B, max_blocks = table.shape
    n_new = step["n_new"].long()
    end = step["seq_len"].long() + n_new
    need = (end + block - 1) // block
    old = held.long()
    j = torch.arange(max_blocks, device=table.device)
    # given back: what lies past the need, in the order of requests and places
    back = (j >= need.view(B, 1)) & (j < old.view(B, 1))
    to = (state[0].long() + state[1].long() + back.view(-1).cumsum(0) - 1) % n_blocks
    ring[to[back.view(-1)]] = table[back]
    free = state[1].long() + back.sum()
    # taken: from the ring's head, the same order, while the pool covers the demand so far
    short = (need - old).clamp_min(0)
    ok = (short.cumsum(0) <= free) | (short == 0)
    take = (j >= old.view(B, 1)) & (j < need.view(B, 1)) & ok.view(B, 1)
    got = ring[(state[0].long() + take.view(-1).cumsum(0) - 1) % n_blocks].view(B, max_blocks)
    table.copy_(torch.where(take, got, torch.where(back, -1, table)))
    held.copy_(torch.where(ok, need, old))
    used = take.sum()
    state.copy_(torch.stack([(state[0] + used) % n_blocks, free - used]))
    i = torch.arange(step["slot_map"].shape[1], device=table.device)
    t = step["seq_len"].long().view(B, 1) + i
    at = table.long().gather(1, (t // block).clamp_max(max_blocks - 1)) * block + t % block
    step["slot_map"].copy_(torch.where((i < n_new.view(B, 1)) & ok.view(B, 1), at, -1))


def _run_commit(s):
    s["now"].copy_(s["start"])
    if own:
        s["tria"].tria_tree_commit(s["cfg"], s["cache"], s["tree"], s["last"], s["ws"],
                                   slot_map=s["slot_map"])
        return s["k"], s["v"], s["pos"], s["now"]
    B, N = s["parent"].shape
    reach = _ancestors(s["parent"], s["n_nodes"])
    last = s["last"].long()
    on = reach[torch.arange(B, device=last.device), last.clamp_min(0)] & (last >= 0).view(B, 1)
    b, node = on.nonzero(as_tuple=True)                                  # in the path's order
    step = on.cumsum(1)[b, node] - 1
    if s["block"]:
        slot = s["slot_map"].long()[b, step]
    else:
        slot = torch.tensor(s["starts"], device=b.device)[b] + s["seq_len"].long()[b] + step
    s["k"][:, :, slot] = s["kd"][:, :, b, node]
    s["v"][:, :, slot] = s["vd"][:, :, b, node]
    s["pos"][:, :, slot] = (s["cur_pos"][b] + 1 + step).to(torch.int32)
    s["now"].add_(on.sum(1).to(torch.int32))
    return s["k"], s["v"], s["pos"], s["now"]


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    B = case["B"]
    if case["op"] == "tree":
        Hq, Hkv, D, N = case["Hq"], case["Hkv"], case["D"], case["N"]
        # the lengths are spread evenly over their range, three quarters of the nodes are there
        T, n = (case["t_lo"] + case["t_hi"]) / 2, 0.75 * N
        seen = T + (n / 2 if case["chain"] else math.log(n + 1) + 1)
        return {"bytes": 4 * B * Hkv * D * (T + n) + 4 * B * n * Hq * D + 4 * B * (n + 2),
                "flops": 4 * B * n * Hq * D * seen}
    if case["op"] == "tables":
        # two calls; a request's lengths and holdings, the blocks that change hands, the slots
        moved = case["max_len"] / case["block"] / 4 if case["full"] else case["n_hi"] / case["block"]
        one = B * (5 * 4 + 4 * case["n_hi"] + 12 * moved)
        return {"bytes": 2 * one, "flops": 2 * B * case["n_hi"]}
    n = math.log(0.75 * case["N"] + 1) + 1  # the depth of a random tree's node
    rows = case["L"] * B * case["Hkv"] * n
    return {"bytes": rows * (8 * case["D"] + 4) + B * (case["N"] * 4 + 20), "flops": rows}


# ---------------------------------------------------------------- in 64 bits

def _path(parent, i):
    """Node i and its ancestors, from the root on."""
    out = []
    while i >= 0:
        out.append(i)
        i = parent[i]
    return out[::-1]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return _exact_tables(s)
    parent, n_nodes = s["parent"].tolist(), s["n_nodes"].tolist()
    lens = s["seq_len"].tolist()
    if case["op"] == "commit":
        now = s["start"].clone()
        for b in range(case["B"]):
            last = int(s["last"][b])
            path = _path(parent[b], last) if last >= 0 else []
            for i, node in enumerate(path):
                at = int(s["slot_map"][b, i]) if s["block"] else s["starts"][b] + lens[b] + i
                s["k"][:, :, at] = s["kd"][:, :, b, node]
                s["v"][:, :, at] = s["vd"][:, :, b, node]
                s["pos"][:, :, at] = 2 * lens[b] + 1 + i
            now[:, b] += len(path)
        return s["k"].double(), s["v"].double(), s["pos"], now
    B, N, Hq, D = s["q"].shape
    G = Hq // s["Hkv"]
    out = torch.zeros(B, N, Hq, D, dtype=torch.float64, device="cuda")
    for b in range(B):
        n, T = n_nodes[b], lens[b]
        mask = torch.full((n, T + n), -math.inf, dtype=torch.float64)
        mask[:, :T] = 0.0
        for i in range(n):
            mask[i, [T + j for j in _path(parent[b], i)]] = 0.0
        mask = mask.cuda()
        t = torch.arange(T)
        if s["block"]:
            at = (s["table"][b].cpu().long()[t // s["block"]] * s["block"] + t % s["block"]).cuda()
        else:
            at = (s["starts"][b] + t).cuda()
        for g in range(s["Hkv"]):
            k = torch.cat([s["k"][0, g, at], s["kd"][0, g, b, :n]]).double()
            v = torch.cat([s["v"][0, g, at], s["vd"][0, g, b, :n]]).double()
            for h in range(g * G, (g + 1) * G):
                x = torch.softmax(s["q"][b, :n, h].double() @ k.T / math.sqrt(D) + mask, 1)
                out[b, :n, h] = x @ v
    return out


def _exact_tables(s):
    table, held, ring = s["table"].tolist(), s["held"].tolist(), s["ring"].tolist()
    head, count = s["state"].tolist()
    block, n = s["block"], s["n_blocks"]
    maps = []
    for step in s["steps"]:
        lens, new = step["seq_len"].tolist(), step["n_new"].tolist()
        need = [-(-(t + m) // block) for t, m in zip(lens, new)]
        for b in range(len(lens)):
            for j in range(need[b], held[b]):
                ring[(head + count) % n] = table[b][j]
                table[b][j] = -1
                count += 1
            held[b] = min(held[b], need[b])
        wanted, pool, slots = 0, count, []
        for b in range(len(lens)):
            wanted += need[b] - held[b]
            served = held[b] == need[b] or wanted <= pool
            while served and held[b] < need[b]:
                table[b][held[b]] = ring[head]
                head, count, held[b] = (head + 1) % n, count - 1, held[b] + 1
            row = [-1] * step["slot_map"].shape[1]
            for i in range(new[b] if served else 0):
                row[i] = table[b][(lens[b] + i) // block] * block + (lens[b] + i) % block
            slots.append(row)
        maps.append(torch.tensor(slots, dtype=torch.int32))
    whole = [torch.tensor(x, dtype=torch.int32) for x in (table, held, ring, [head, count])]
    return (*whole, maps)
