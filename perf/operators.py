"""Measured cases of the decoder's attention and draft-tree operators.

Three operators of one decoding step around the beam search:

- ``cross``: attention of every beam's queries over the encoder's states of its sentence
  (the beams of a sentence share its keys and values; sentences have lengths of their own);
- ``tree``: attention of a tree of drafted tokens over its row's key / value cache and over the
  drafted tokens on its own branch (one node is the ordinary single-token step);
- ``commit``: the longest branch of the tree that the model's own choices confirm, its keys
  and values appended to the cache of every layer, and the next token.

``own`` selects what ``run`` computes with: elementary torch operations in 32 bits, or the
framework's entry points.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
EOS = 2
VOCAB = 40000

# The most that a case may read, write and compute (the largest listed ones).
MOST_BYTES = 6.0e8
MOST_FLOPS = {"f16": 2.8e11, "bf16": 2.8e11, "f32": 8.0e9}


def _cross(name, dtype, batch, k, q_len, heads, kv_heads, dim, src_min, src_max, order="bhsd"):
    """src lengths spread evenly over [src_min, src_max]; order: how the keys lie in memory
    ("bhsd": the cache's [batch, heads, src, dim]; "bshd": as a projection writes them)."""
    return {"name": name, "op": "cross", "dtype": dtype, "batch": batch, "k": k, "q_len": q_len, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "len_min": src_min, "len_max": src_max, "order": order}


def _tree(name, dtype, rows, nodes, heads, kv_heads, dim, len_min, len_max):
    return {"name": name, "op": "tree", "dtype": dtype, "rows": rows, "nodes": nodes, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "len_min": len_min, "len_max": len_max}


def _commit(name, dtype, layers, rows, nodes, heads, dim, max_len):
    return {"name": name, "op": "commit", "dtype": dtype, "layers": layers, "rows": rows, "nodes": nodes,
            "heads": heads, "dim": dim, "max_len": max_len}


def listed():
    return [
        # a small translation request, fp32 engine: sentences of up to 17 pieces; latency counts
        _cross("cross_small_f32", "f32", 4, 4, 1, 16, 16, 64, 3, 17),
        # the decode benchmark's batch: 256 sentences of 24 to 128 pieces, 4 beams
        _cross("cross_batch_f16", "f16", 256, 4, 1, 16, 16, 64, 24, 128),
        # long documents, 8 beams, shared key heads, keys as the projection writes them
        _cross("cross_long_bf16", "bf16", 8, 8, 1, 32, 8, 128, 5001, 8191, "bshd"),
        # scoring whole target texts against their sources (one query per target token)
        _cross("cross_score_f16", "f16", 32, 1, 509, 16, 16, 128, 1500, 2048),
        # a forced prefix in front of a beam search, head size of the benchmark
        _cross("cross_prefix_bf16", "bf16", 24, 4, 100, 16, 16, 64, 700, 1021),
        # the ordinary single-token step of a small request
        _tree("tree_step_small_f16", "f16", 4, 1, 16, 16, 64, 1, 63),
        # the single-token step of the decode benchmark's cache (1024 beams, up to 64 positions)
        _tree("tree_step_batch_f16", "f16", 1024, 1, 16, 16, 64, 48, 63),
        # a small tree of drafts for a batch of sequences of a few hundred tokens
        _tree("tree_draft_f16", "f16", 128, 13, 16, 16, 64, 300, 999),
        # a full tree of drafts, shared key heads: compute and memory in balance
        _tree("tree_full_bf16", "bf16", 32, 64, 32, 8, 128, 1025, 4000),
        # one sequence with a long cache: few rows, the length has to be split
        _tree("tree_long_bf16", "bf16", 1, 16, 32, 8, 128, 131000, 131000),
        # the step's append of a small request (one node: the token itself)
        _commit("commit_small_f16", "f16", 6, 4, 1, 16, 64, 64),
        # a batch's drafted trees appended to six layers
        _commit("commit_batch_f16", "f16", 6, 256, 31, 16, 64, 100),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    while True:
        op = rng.choice(["cross", "cross", "tree", "tree", "commit"])
        dtype = rng.choice(["f16", "bf16", "f16", "bf16", "f32"])
        heads = rng.choice([4, 8, 12, 16, 32])
        kv_heads = heads // rng.choice([1, 1, 2, 4])
        dim = rng.choice([32, 64, 64, 80, 96, 128, 128, 256])
        if op == "cross":
            q_len = 1 if rng.random() < 0.6 else _log_int(rng, 2, 1024)
            top = _log_int(rng, 1, 8191)
            case = _cross("", dtype, _log_int(rng, 1, 256), rng.choice([1, 2, 3, 4, 5, 8]), q_len, heads, kv_heads,
                          dim, _log_int(rng, 1, top), top, rng.choice(["bhsd", "bshd"]))
        elif op == "tree":
            top = _log_int(rng, 1, 131000)
            nodes = 1 if rng.random() < 0.35 else _log_int(rng, 2, 64)
            case = _tree("", dtype, _log_int(rng, 1, 1024), nodes, heads, kv_heads, dim, _log_int(rng, 1, top), top)
        else:
            nodes = 1 if rng.random() < 0.25 else _log_int(rng, 2, 64)
            case = _commit("", dtype, rng.randint(1, 12), _log_int(rng, 1, 512), nodes, kv_heads, dim,
                           rng.randint(nodes, 200))
            cache = case["layers"] * case["rows"] * kv_heads * case["max_len"] * dim * SIZES[dtype]
            if cache > 5.0e8:
                continue
        w = work(case)
        if w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS[dtype]:
            del case["name"]
            return case


# ---------------------------------------------------------------- what a case consists of
def _lengths(n, lo, hi):
    """n lengths spread evenly over [lo, hi] (the seed only decides whose is which)."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _tree_shape(i, nodes):
    """Parents of tree i: a chain, a binary or a ternary tree; every fourth tree is a quarter
    smaller and leaves its last places empty (-2)."""
    width = 1 + i % 3
    used = nodes - nodes // 4 if i % 4 == 3 else nodes
    return [-1 if n == 0 else (n - 1) // width if n < used else -2 for n in range(nodes)]


def _branch(parents, leaf):
    b = []
    while leaf >= 0:
        b.append(leaf)
        leaf = parents[leaf]
    return b[::-1]


def _commit_plan(rows, nodes):
    """For every row its tree and the branch that the model confirms."""
    plan = []
    for i in range(rows):
        parents = _tree_shape(i, nodes)
        used = sum(p >= -1 for p in parents)
        plan.append((parents, _branch(parents, (i * 7 + 3) % used)))
    return plan


def work(case):
    e = SIZES[case["dtype"]]
    if case["op"] == "cross":
        n = case["batch"] * case["k"] * case["q_len"] * case["heads"] * case["dim"]
        kv = sum(_lengths(case["batch"], case["len_min"], case["len_max"]))
        return {"bytes": 2 * n * e + 2 * kv * case["kv_heads"] * case["dim"] * e + 4 * case["batch"],
                "flops": 4.0 * case["k"] * case["q_len"] * case["heads"] * case["dim"] * kv}
    if case["op"] == "tree":
        rows, nodes = case["rows"], case["nodes"]
        lens = _lengths(rows, case["len_min"], case["len_max"])
        seen = 0  # (query, key) pairs
        keys = 0
        shapes = {}
        for i in range(rows):
            if i % 12 not in shapes:
                t = _tree_shape(i, nodes)
                shapes[i % 12] = (sum(p >= -1 for p in t), sum(len(_branch(t, n)) for n in range(nodes) if t[n] >= -1))
            used, pairs = shapes[i % 12]
            seen += used * lens[i] + pairs
            keys += lens[i] + used
        return {"bytes": (2 * rows * nodes * case["heads"] + 2 * keys * case["kv_heads"]) * case["dim"] * e
                + 4 * rows * (nodes + 1),
                "flops": 4.0 * seen * case["heads"] * case["dim"]}
    moved = sum(len(b) for _, b in _commit_plan(case["rows"], case["nodes"]))
    return {"bytes": 4 * moved * case["layers"] * case["heads"] * case["dim"] * e + 4 * case["rows"] * (4 * case["nodes"] + 4),
            "flops": 0.0}


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32 if dtype == "f32" else DTYPES[dtype])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    dt = case["dtype"]
    st = {"case": case}

    def ints(values, dtype=torch.int32):
        return torch.tensor(values, dtype=dtype, device="cuda")

    if case["op"] == "cross":
        b, k, t, h, d = case["batch"], case["k"], case["q_len"], case["heads"], case["dim"]
        st["q"] = _normal(gen, (b, k, t, h, d), dt)
        if case["order"] == "bhsd":
            st["key"] = _normal(gen, (b, case["kv_heads"], case["len_max"], d), dt)
            st["value"] = _normal(gen, (b, case["kv_heads"], case["len_max"], d), dt)
        else:
            st["key"] = _normal(gen, (b, case["len_max"], case["kv_heads"], d), dt).transpose(1, 2)
            st["value"] = _normal(gen, (b, case["len_max"], case["kv_heads"], d), dt).transpose(1, 2)
        lens = _lengths(b, case["len_min"], case["len_max"])
        rng.shuffle(lens)
        st["src_len"] = ints(lens)
        if own:
            import serving_ls_beam_gb300 as lsb

            st["out"] = torch.empty_like(st["q"])
            st["ws"] = torch.empty(lsb.ls_cross_attention_workspace_size(b, k, t, h, case["kv_heads"], case["len_max"], d),
                                   dtype=torch.uint8, device="cuda")
            lsb.check(lsb.ls_workspace_init(st["ws"]))
        return st
    rows, nodes, d = case["rows"], case["nodes"], case["dim"]
    if case["op"] == "tree":
        h, hk, n = case["heads"], case["kv_heads"], case["len_max"]
        st["q"] = _normal(gen, (rows, nodes, h, d), dt)
        st["cache_key"] = _normal(gen, (rows, hk, n, d), dt)
        st["cache_value"] = _normal(gen, (rows, hk, n, d), dt)
        st["draft_key"] = _normal(gen, (rows, nodes, hk, d), dt)
        st["draft_value"] = _normal(gen, (rows, nodes, hk, d), dt)
        both = list(zip(_lengths(rows, case["len_min"], n), [_tree_shape(i, nodes) for i in range(rows)]))
        rng.shuffle(both)
        st["cache_len"] = ints([x for x, _ in both])
        st["parent"] = ints([x for _, x in both])
        if own:
            import serving_ls_beam_gb300 as lsb

            st["out"] = torch.empty_like(st["q"])
            st["ws"] = torch.empty(lsb.ls_tree_attention_workspace_size(rows, nodes, h, hk, n, d), dtype=torch.uint8,
                                   device="cuda")
            lsb.check(lsb.ls_workspace_init(st["ws"]))
        return st
    layers, h, n = case["layers"], case["heads"], case["max_len"]
    for name in ("cache_key", "cache_value"):
        st[name] = _normal(gen, (layers, rows, h, n, d), dt)
    for name in ("draft_key", "draft_value"):
        st[name] = _normal(gen, (layers, rows, nodes, h, d), dt)
    plan = _commit_plan(rows, nodes)
    rng.shuffle(plan)
    parent, token, target, lens = [], [], [], []
    for parents, branch in plan:
        # siblings' tokens differ, as drafts do; the model agrees along the branch and then not
        toks = [3 + (rng.randrange(1000) * 64 + i) % (VOCAB - 4) for i in range(nodes)]
        want = [3 + (rng.randrange(1000) * 64 + i + 64 * 1000) % (VOCAB - 4) for i in range(nodes)]
        children = {}
        for i, p in enumerate(parents):
            children.setdefault(p, set()).add(toks[i])
        for a in range(nodes):
            while want[a] in children.get(a, ()):
                want[a] = 3 + (want[a] + 1) % (VOCAB - 4)
        for a, b in zip(branch, branch[1:]):
            want[a] = toks[b]
        parent.append(parents)
        token.append(toks)
        target.append(want)
        lens.append(rng.randint(0, n - len(branch)))
    st["parent"], st["token"], st["target"], st["cache_len"] = ints(parent), ints(token), ints(target), ints(lens)
    st["finished"] = torch.zeros(rows, dtype=torch.uint8, device="cuda")
    st["out_len"] = torch.empty(rows, dtype=torch.int32, device="cuda")
    st["out_path"] = torch.empty((rows, nodes), dtype=torch.int32, device="cuda")
    st["out_count"] = torch.empty(rows, dtype=torch.int32, device="cuda")
    st["out_token"] = torch.empty(rows, dtype=torch.int32, device="cuda")
    st["out_finished"] = torch.empty(rows, dtype=torch.uint8, device="cuda")
    return st


# ---------------------------------------------------------------- plain forms
def _softmax_parts(x):
    """exp(x - max) and its sums along the last axis; rows of -inf give zeros."""
    m = x.amax(dim=-1, keepdim=True)
    p = torch.exp(x - torch.where(m == -math.inf, torch.zeros_like(m), m))
    return p, p.sum(dim=-1, keepdim=True)


def _plain_cross(st):
    q, key, value = st["q"], st["key"].float(), st["value"].float()
    b, k, t, h, d = q.shape
    hk, n = key.shape[1], key.shape[2]
    g = h // hk
    # [b, hk, (k, t, g), d]: every query that reads one head of one sentence
    x = q.float().view(b, k * t, hk, g, d).transpose(1, 2).reshape(b, hk, k * t * g, d)
    s = torch.matmul(x, key.transpose(2, 3)) * (1.0 / math.sqrt(d))
    past = torch.arange(n, device=q.device)[None, :] >= st["src_len"][:, None]
    s.masked_fill_(past[:, None, None, :], -math.inf)
    p, z = _softmax_parts(s)
    del s
    o = torch.matmul(p, value) / z
    o = torch.where(z == 0, torch.zeros_like(o), o)
    return o.view(b, hk, k * t, g, d).transpose(1, 2).reshape(b, k, t, h, d).to(q.dtype)


def _tree_sees(parent):
    """[rows, nodes, nodes]: node i sees node j (itself or an ancestor); empty places see nothing."""
    rows, nodes = parent.shape
    up = parent.long()
    there = up >= -1
    sees = torch.eye(nodes, dtype=torch.bool, device=parent.device).expand(rows, nodes, nodes) & there[:, :, None]
    up = up.clamp(min=-1)
    steps = 1
    while steps < nodes:  # pointer doubling: after each round sees covers twice the ancestors
        at = up.clamp(min=0)
        more = torch.gather(sees, 1, at[:, :, None].expand(rows, nodes, nodes)) & (up >= 0)[:, :, None]
        sees = sees | more
        up = torch.where(up >= 0, torch.gather(up, 1, at), up)
        steps *= 2
    return sees, there


def _plain_tree(st):
    q = st["q"]
    rows, nodes, h, d = q.shape
    key, value = st["cache_key"].float(), st["cache_value"].float()
    dk, dv = st["draft_key"].float().transpose(1, 2), st["draft_value"].float().transpose(1, 2)
    hk, n = key.shape[1], key.shape[2]
    g = h // hk
    x = q.float().view(rows, nodes, hk, g, d).transpose(1, 2).reshape(rows, hk, nodes * g, d)
    scale = 1.0 / math.sqrt(d)
    sees, there = _tree_sees(st["parent"])
    s = torch.empty((rows, hk, nodes * g, n + nodes), device=q.device)
    s[..., :n] = torch.matmul(x, key.transpose(2, 3)) * scale
    s[..., n:] = torch.matmul(x, dk.transpose(2, 3)) * scale
    past = torch.arange(n, device=q.device)[None, :] >= st["cache_len"][:, None]
    s[..., :n].masked_fill_(past[:, None, None, :], -math.inf)
    s[..., n:].masked_fill_(~sees.repeat_interleave(g, dim=1)[:, None], -math.inf)
    s.masked_fill_(~there.repeat_interleave(g, dim=1)[:, None, :, None], -math.inf)
    p, z = _softmax_parts(s)
    del s
    o = (torch.matmul(p[..., :n], value) + torch.matmul(p[..., n:], dv)) / z
    o = torch.where(z == 0, torch.zeros_like(o), o)
    return o.view(rows, hk, nodes, g, d).transpose(1, 2).reshape(rows, nodes, h, d).to(q.dtype)


def _plain_commit(st):
    parent, token, target = st["parent"].long(), st["token"], st["target"]
    rows, nodes = parent.shape
    cache_len = st["cache_len"].long()
    max_len = st["cache_key"].shape[3]
    dev = parent.device
    node = torch.arange(nodes, device=dev)
    at = parent.clamp(min=0)
    fits = (parent >= 0) & (parent < node) & (token == torch.gather(target, 1, at)) & (token != EOS)
    # of siblings that fit, the first
    twin = (parent[:, :, None] == parent[:, None, :]) & fits[:, :, None] & fits[:, None, :]
    fits &= ~(twin & (node[None, :] < node[:, None])).any(dim=2)
    on = torch.where(node == 0, parent == -1, fits)
    steps = 1
    while steps < nodes:
        on = on & torch.gather(on, 1, at)
        at = torch.gather(at, 1, at)
        steps *= 2
    on = on & (st["finished"] == 0)[:, None]
    place = torch.cumsum(on, dim=1) - 1
    on = on & (place < (max_len - cache_len)[:, None])
    count = on.sum(dim=1)
    path = torch.full((rows, nodes + 1), -1, dtype=torch.int64, device=dev)
    path.scatter_(1, torch.where(on, place, torch.full_like(place, nodes)), node.expand(rows, nodes))
    path = path[:, :nodes]
    last = torch.gather(path, 1, (count - 1).clamp(min=0)[:, None]).clamp(min=0)
    nxt = torch.where(count > 0, torch.gather(target, 1, last)[:, 0], token[:, 0])
    nxt = torch.where(st["finished"] != 0, torch.full_like(nxt, EOS), nxt)
    st["out_finished"].copy_((st["finished"] != 0) | ((count > 0) & (nxt == EOS)))
    st["out_len"].copy_(cache_len + count)
    st["out_path"].copy_(path)
    st["out_count"].copy_(count)
    st["out_token"].copy_(nxt)
    # node i of row r goes to position cache_len + its place on the branch; the others write
    # back what stands at position 0 of their own row's free part or is there already
    pos = torch.where(on, cache_len[:, None] + place, torch.zeros_like(place))
    r = torch.arange(rows, device=dev)[:, None].expand(rows, nodes)
    for cache, draft in ((st["cache_key"], st["draft_key"]), (st["cache_value"], st["draft_value"])):
        for layer in range(cache.shape[0]):
            there = cache[layer].transpose(1, 2)  # [rows, max_len, heads, dim]
            old = there[r, pos]
            # places that are not on the branch all hold position 0: they write what it will hold
            first = torch.where(((cache_len == 0) & on[:, 0])[:, None, None], draft[layer][:, 0], there[:, 0])
            new = torch.where(on[:, :, None, None], draft[layer], first[:, None].expand_as(old))
            there[r, pos] = new
    return _commit_outputs(st)


def _commit_outputs(st):
    return {n: st[n] for n in ("cache_key", "cache_value", "out_len", "out_path", "out_count", "out_token", "out_finished")}


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if not own:
        return {"cross": _plain_cross, "tree": _plain_tree, "commit": _plain_commit}[op](state)
    import serving_ls_beam_gb300 as lsb

    if op == "cross":
        lsb.check(lsb.ls_cross_attention(state["q"], state["key"], state["value"], state["src_len"], state["out"],
                                         state["ws"]))
        return state["out"]
    if op == "tree":
        lsb.check(lsb.ls_tree_attention(state["q"], state["cache_key"], state["cache_value"], state["cache_len"],
                                        state["draft_key"], state["draft_value"], state["parent"], state["out"],
                                        state["ws"]))
        return state["out"]
    lsb.check(lsb.ls_tree_commit(state["cache_key"], state["cache_value"], state["cache_len"], state["draft_key"],
                                 state["draft_value"], state["parent"], state["token"], state["target"],
                                 state["finished"], EOS, state["out_len"], state["out_path"], state["out_count"],
                                 state["out_token"], state["out_finished"]))
    return _commit_outputs(state)


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "commit":
        return None  # copies and whole numbers
    d = case["dim"]
    if case["op"] == "cross":
        q = st["q"].reshape(case["batch"], -1, case["heads"], d)
        lens = st["src_len"].tolist()
    else:
        q = st["q"]
        lens = st["cache_len"].tolist()
        parents = st["parent"].tolist()
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    group = case["heads"] // case["kv_heads"]
    for r in range(q.shape[0]):
        n = lens[r]
        if case["op"] == "cross":
            ks, vs = st["key"][r, :, :n].double(), st["value"][r, :, :n].double()
            hidden = None
        else:
            ks = torch.cat([st["cache_key"][r, :, :n].double(), st["draft_key"][r].double().transpose(0, 1)], dim=1)
            vs = torch.cat([st["cache_value"][r, :, :n].double(), st["draft_value"][r].double().transpose(0, 1)], dim=1)
            nodes = case["nodes"]
            rowmask = torch.ones((nodes, n + nodes), dtype=torch.bool)
            for i in range(nodes):
                if parents[r][i] >= -1:
                    rowmask[i, :n] = False
                    for a in _branch(parents[r], i):
                        rowmask[i, n + a] = False
            hidden = rowmask.to(q.device)
        if ks.shape[1] == 0:
            continue
        # [heads, queries, dim] against the heads' shared keys
        x = q[r].double().permute(1, 0, 2)
        for h in range(case["kv_heads"]):
            s = torch.einsum("gqd,nd->gqn", x[h * group:(h + 1) * group], ks[h]) / math.sqrt(d)
            if hidden is not None:
                s = s.masked_fill(hidden, -math.inf)
            top = s.max(dim=2, keepdim=True).values
            e = torch.exp(s - top.nan_to_num(neginf=0.0))
            total = e.sum(dim=2, keepdim=True)
            o = torch.einsum("gqn,nd->gqd", e, vs[h]) / torch.where(total == 0, 1.0, total)
            out[r, :, h * group:(h + 1) * group] = o.permute(1, 0, 2)
    return out.reshape(st["q"].shape)
