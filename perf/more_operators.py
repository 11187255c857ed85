"""Measured cases of the paged cache and of sampling with filters.

Four operators of a decoding step on a cache held in pages:

- ``write``: new tokens' keys and values into the pages, quantised to 8 bits per head vector or as they are;
- ``read``: positions of the cache back as dense tensors;
- ``attend``: attention of one new token per row over its row's pages;
- ``sample``: one token per row by temperature, top-k, top-p and min-p at the caller's uniforms.

``own`` selects what ``run`` computes with: elementary torch operations, or the framework's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
          "i8": torch.int8}
SIZES = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1, "i8": 1}

# The most that a drawn case may read and write, and the dense elements that its plain form may lay out.
MOST_BYTES = {"write": 2.0e8, "read": 2.5e8, "attend": 1.2e9, "sample": 8.2e7}
MOST_DENSE = 1.1e9


def _write(name, dtype, cache, rows, tokens, heads, dim, page, count_min, start_max, order="head"):
    """count_min..tokens new tokens per row at starts of up to start_max; order: how a page lies in memory
    ("head": [head, position, dim]; "token": [position, head, dim])."""
    return {"name": name, "op": "write", "dtype": dtype, "cache": cache, "rows": rows, "tokens": tokens, "heads": heads,
            "dim": dim, "page": page, "count_min": count_min, "start_max": start_max, "order": order}


def _read(name, dtype, cache, rows, heads, dim, page, len_min, len_max, order="head"):
    return {"name": name, "op": "read", "dtype": dtype, "cache": cache, "rows": rows, "heads": heads, "dim": dim,
            "page": page, "len_min": len_min, "len_max": len_max, "order": order}


def _attend(name, dtype, cache, rows, heads, kv_heads, dim, page, len_min, len_max, order="head"):
    return {"name": name, "op": "attend", "dtype": dtype, "cache": cache, "rows": rows, "q_heads": heads,
            "heads": kv_heads, "dim": dim, "page": page, "len_min": len_min, "len_max": len_max, "order": order}


def _sample(name, dtype, rows, vocab, top_k, top_p, min_p, t_min, t_max, spread, bias=False):
    """top_k 0, top_p 1, min_p 0: that filter is off; temperatures in [t_min, t_max], logits of deviation spread."""
    return {"name": name, "op": "sample", "dtype": dtype, "rows": rows, "vocab": vocab, "top_k": top_k, "top_p": top_p,
            "min_p": min_p, "t_min": t_min, "t_max": t_max, "spread": spread, "bias": bias}


def listed():
    return [
        # one decode step of a small request: eight new tokens into 8-bit pages, latency counts
        _write("write_step_e4m3", "f16", "e4m3", 8, 1, 16, 64, 16, 1, 60),
        # one decode step of the decode benchmark's 1024 beams
        _write("write_batch_i8", "f16", "i8", 1024, 1, 16, 64, 16, 1, 63),
        # a batch of prompts of different lengths stored at once
        _write("write_prompt_e4m3", "bf16", "e4m3", 16, 2048, 8, 128, 64, 1201, 100),
        # a short cache handed to another kernel
        _read("read_small_e4m3", "f16", "e4m3", 4, 16, 64, 16, 1, 199),
        # long contexts brought back from 8-bit pages
        _read("read_batch_i8", "bf16", "i8", 16, 8, 128, 64, 1001, 4000),
        # the single-token step of a small request
        _attend("attend_small_f16", "f16", "f16", 4, 16, 16, 64, 16, 1, 63),
        # a middling batch on int8 pages, as many key heads as query heads, pages as a projection writes them
        _attend("attend_i8", "f16", "i8", 64, 16, 16, 64, 32, 300, 999, "token"),
        # a large batch of long contexts, shared key heads, 8-bit pages
        _attend("attend_batch_e4m3", "bf16", "e4m3", 256, 32, 8, 128, 64, 501, 4000),
        # one sequence with a long cache: its length has to be split
        _attend("attend_long_bf16", "bf16", "bf16", 1, 32, 8, 128, 128, 131000, 131000),
        # a small request: the usual short candidate list
        _sample("sample_small_f32", "f32", 4, 40000, 50, 0.9, 0.0, 0.7, 0.7, 2.0),
        # the decode benchmark's rows, settings of their own for each
        _sample("sample_batch_f16", "f16", 1024, 40000, 64, 0.95, 0.02, 0.5, 1.2, 2.0),
        # a large vocabulary with no top-k: the nucleus may be thousands of tokens
        _sample("sample_nucleus_bf16", "bf16", 64, 120000, 0, 0.95, 0.0, 0.8, 1.1, 2.5),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng: random.Random):
    while True:
        op = rng.choice(["write", "read", "attend", "attend", "sample", "sample"])
        dtype = rng.choice(["f16", "bf16", "f16", "bf16", "f32"])
        if op == "sample":
            case = _sample("", dtype, _log_int(rng, 1, 1024), _log_int(rng, 500, 260000),
                           0 if rng.random() < 0.5 else _log_int(rng, 1, 3000),
                           1.0 if rng.random() < 0.35 else round(rng.uniform(0.3, 0.99), 3),
                           0.0 if rng.random() < 0.6 else round(rng.uniform(0.005, 0.2), 4), 0.5, rng.choice([0.5, 1.0, 1.5]),
                           round(rng.uniform(0.7, 3.0), 2), rng.random() < 0.2)
        else:
            cache = rng.choice(["e4m3", "i8", "e4m3", "i8", dtype])
            kv = rng.choice([1, 2, 4, 8, 12, 16])
            dim = rng.choice([32, 64, 64, 80, 96, 128, 128, 192, 256])
            page = rng.choice([1, 8, 16, 16, 24, 32, 64, 128])
            order = rng.choice(["head", "head", "token"])
            rows = _log_int(rng, 1, 1024)
            if op == "write":
                tokens = 1 if rng.random() < 0.5 else _log_int(rng, 2, 4096)
                case = _write("", dtype, cache, rows, tokens, kv, dim, page, rng.randint(1, tokens), _log_int(rng, 1, 500),
                              order)
            else:
                top = _log_int(rng, 1, 131000)
                low = _log_int(rng, 1, top)
                if op == "read":
                    case = _read("", dtype, cache, rows, kv, dim, page, low, top, order)
                else:
                    case = _attend("", dtype, cache, rows, kv * rng.choice([1, 1, 2, 4, 5, 8]), kv, dim, page, low, top, order)
            held = sum(_rows_of(case)[1])
            longest = max(_rows_of(case)[1])
            if held * kv * dim > MOST_DENSE / 2 or rows * longest * kv * dim > MOST_DENSE:
                continue
        if work(case)["bytes"] <= MOST_BYTES[op]:
            del case["name"]
            return case


# ---------------------------------------------------------------- what a case consists of
def _spread(n, lo, hi):
    """n whole numbers spread evenly over [lo, hi] (the seed only decides whose is which)."""
    if n == 1:
        return [hi]
    return [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _rows_of(case):
    """(starts, ends, counts): what each row writes and holds, before the seed's shuffle."""
    if case["op"] == "write":
        counts = _spread(case["rows"], case["count_min"], case["tokens"])
        starts = [(i * 37 + 11) % (case["start_max"] + 1) for i in range(case["rows"])]
        return starts, [s + c for s, c in zip(starts, counts)], counts
    lens = _spread(case["rows"], case["len_min"], case["len_max"])
    return [0] * case["rows"], lens, lens


def work(case):
    if case["op"] == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * SIZES[case["dtype"]] + case["rows"] * 28 + (4 * case["vocab"] if case["bias"] else 0),
                "flops": 2.0 * n}
    _, _, counts = _rows_of(case)
    e, ec = SIZES[case["dtype"]], SIZES[case["cache"]]
    vectors = 2 * sum(counts) * case["heads"]
    held = vectors * (case["dim"] * ec + (4 if ec == 1 else 0))
    if case["op"] == "attend":
        io = 2 * case["rows"] * case["q_heads"] * case["dim"] * e
        return {"bytes": held + io + 4 * case["rows"], "flops": 4.0 * sum(counts) * case["q_heads"] * case["dim"]}
    return {"bytes": held + vectors * case["dim"] * e + 8 * case["rows"], "flops": 2.0 * vectors * case["dim"] if ec == 1 else 0.0}


def _quantised(x, cache):
    """(codes, scales) of head vectors x [..., dim]: a scale per vector."""
    a = x.float().abs().amax(dim=-1)
    if cache == "e4m3":
        m, e = torch.frexp(a)  # a = m 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
        e = torch.where(m <= 0.875, e - 9, e - 8)
        e = torch.where(a == 0, torch.full_like(e, -126), e.clamp(min=-126))
        s = ((e + 127) << 23).view(torch.float32)  # 2^e by its bits
        return (x.double() / s.double()[..., None]).float().to(torch.float8_e4m3fn), s
    s = (a / 127.0).clamp(min=2.0 ** -126)
    return torch.round(x.double() / s.double()[..., None]).to(torch.int8), s


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32 if dtype == "f32" else DTYPES[dtype])


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    rng = random.Random(seed)
    st = {"case": case}

    def ints(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    if case["op"] == "sample":
        rows, vocab = case["rows"], case["vocab"]
        # a bulk of unlikely tokens and a few likely ones
        x = torch.randn((rows, vocab), generator=gen, device="cuda") * case["spread"]
        likely = torch.randint(vocab, (rows, 24), generator=gen, device="cuda")
        x.scatter_add_(1, likely, torch.rand((rows, 24), generator=gen, device="cuda") * 4.0 * case["spread"])
        st["logits"] = x.to(DTYPES[case["dtype"]])
        st["bias"] = torch.randn(vocab, generator=gen, device="cuda") * 0.3 if case["bias"] else None
        st["u"] = torch.rand(rows, generator=gen, device="cuda")
        st["temperature"] = case["t_min"] + (case["t_max"] - case["t_min"]) * torch.rand(rows, generator=gen, device="cuda")
        full = lambda v, dt: torch.full((rows,), v, dtype=dt, device="cuda")  # noqa: E731
        st["top_k"] = full(case["top_k"], torch.int32) if case["top_k"] else None
        st["top_p"] = full(case["top_p"], torch.float32) if case["top_p"] < 1.0 else None
        st["min_p"] = full(case["min_p"], torch.float32) if case["min_p"] > 0.0 else None
        st["token"] = torch.empty(rows, dtype=torch.int32, device="cuda")
        st["logprob"] = torch.empty(rows, device="cuda")
        return st

    rows, heads, dim, page, cache = case["rows"], case["heads"], case["dim"], case["page"], case["cache"]
    starts, ends, counts = _rows_of(case)
    both = list(zip(starts, ends, counts))
    rng.shuffle(both)
    starts, ends, counts = (list(x) for x in zip(*both))
    # every row its pages, in an order of their own; a spare page that no row has takes the plain form's padding
    need = [-(-n // page) for n in ends]
    order = list(range(sum(need)))
    rng.shuffle(order)
    st["table"] = torch.full((rows, max(need)), -1, dtype=torch.int32)
    at = 0
    for r, n in enumerate(need):
        st["table"][r, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
        at += n
    st["table"] = st["table"].cuda()
    shape = (at + 1, heads, page, dim) if case["order"] == "head" else (at + 1, page, heads, dim)
    for name in ("key", "value"):
        pages = torch.empty(shape, dtype=DTYPES[cache], device="cuda")
        scale = torch.empty((at + 1, heads, page), device="cuda") if SIZES[cache] == 1 else None
        view = pages if case["order"] == "head" else pages.transpose(1, 2)
        step = max(1, (1 << 27) // (heads * page * dim))
        for i in range(0, at + 1, step):
            # channels differ in size, as a projection's do
            part = _normal(gen, (min(step, at + 1 - i), heads, page, dim), case["dtype"])
            part = part * torch.linspace(0.5, 1.5, dim, device="cuda", dtype=part.dtype)
            if scale is None:
                view[i:i + step] = part
            else:
                view[i:i + step], scale[i:i + step] = _quantised(part, cache)
        st[name + "_pages"], st[name + "_scale"] = view, scale
    if case["op"] == "write":
        # as a projection writes them: [rows, tokens, heads, dim]
        st["key"] = _normal(gen, (rows, case["tokens"], heads, dim), case["dtype"])
        st["value"] = _normal(gen, (rows, case["tokens"], heads, dim), case["dtype"])
        st["start"], st["count"] = ints(starts), ints(counts)
    elif case["op"] == "read":
        st["start"], st["count"] = ints(starts), ints(counts)
        for name in ("key", "value"):  # what lies behind a row's last position stays as it is
            st["out_" + name] = torch.zeros((rows, case["len_max"], heads, dim), dtype=DTYPES[case["dtype"]], device="cuda")
    else:
        st["q"] = _normal(gen, (rows, case["q_heads"], dim), case["dtype"])
        st["len"] = ints(ends)
    if own:
        import serving_ls_beam_gb300 as lsb

        whole = lambda t: None if t is None else t[:at]  # noqa: E731
        st["pages"] = lsb.ls_pages(whole(st["key_pages"]), whole(st["value_pages"]), st["table"], whole(st["key_scale"]),
                                   whole(st["value_scale"]))
        size = lsb.ls_paged_attention_workspace_size(rows, case.get("q_heads", heads), heads, dim)
        st["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        lsb.check(lsb.ls_workspace_init(st["ws"]))
        if case["op"] == "attend":
            st["out"] = torch.empty_like(st["q"])
    return st


# ---------------------------------------------------------------- plain forms
def _places(st, n):
    """(page, place in the page) [rows, n] of positions start..start + n of every row; past count: the spare page."""
    page = st["key_pages"].shape[2]
    i = torch.arange(n, device="cuda")[None, :]
    pos = st["start"].long()[:, None] + i
    slot = (pos // page).clamp(max=st["table"].shape[1] - 1)
    at = torch.gather(st["table"].long(), 1, slot)
    there = i < st["count"].long()[:, None]
    return torch.where(there, at, torch.full_like(at, st["key_pages"].shape[0] - 1)), pos % page, there


def _plain_write(st):
    cache = st["case"]["cache"]
    at, place, _ = _places(st, st["key"].shape[1])
    for name in ("key", "value"):
        pages, scale, x = st[name + "_pages"], st[name + "_scale"], st[name]
        if scale is None:
            pages[at, :, place] = x
        else:
            codes, s = _quantised(x, cache)
            raw = pages.view(torch.uint8)
            raw[at, :, place] = codes.view(torch.uint8)
            scale[at, :, place] = s
    return _write_outputs(st)


def _write_outputs(st):
    out = {}
    for name in ("key_pages", "value_pages", "key_scale", "value_scale"):
        if st[name] is not None:
            out[name] = st[name][:-1]
    return out


def _plain_read(st):
    out = {}
    for name in ("key", "value"):
        to = st["out_" + name]
        at, place, there = _places(st, to.shape[1])
        pages, scale = st[name + "_pages"], st[name + "_scale"]
        if scale is None:
            x = pages[at, :, place]
        else:
            x = pages.view(torch.uint8)[at, :, place].view(pages.dtype).float() * scale[at, :, place][..., None]
        to.copy_(torch.where(there[:, :, None, None], x.to(to.dtype), to))
        out[name] = to
    return out


def _dense(st, name):
    """A cache's pages laid out as [rows, heads, positions, dim] in 32 bits."""
    at = st["table"].long().clamp(min=0)
    rows, pages = at.shape
    _, heads, page, dim = st[name + "_pages"].shape
    x = st[name + "_pages"].view(torch.uint8) if st[name + "_scale"] is not None else st[name + "_pages"]
    x = x[at].view(st[name + "_pages"].dtype).float()
    if st[name + "_scale"] is not None:
        x = x * st[name + "_scale"][at][..., None]
    return x.transpose(1, 2).reshape(rows, heads, pages * page, dim)


def _plain_attend(st):
    q = st["q"].float()
    rows, heads, dim = q.shape
    key = _dense(st, "key")
    kv, n = key.shape[1], key.shape[2]
    s = torch.matmul(q.view(rows, kv, heads // kv, dim), key.transpose(2, 3)) * (1.0 / math.sqrt(dim))
    del key
    past = torch.arange(n, device=q.device)[None, :] >= st["len"][:, None]
    s.masked_fill_(past[:, None, None, :], -math.inf)
    m = s.amax(dim=-1, keepdim=True)
    p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
    z = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p, _dense(st, "value"))
    return torch.where(z == 0, torch.zeros_like(o), o / z).view(rows, heads, dim).to(st["q"].dtype)


def _plain_sample(st):
    # in 64 bits: what is kept and drawn hangs on values next to a border
    x = st["logits"].float()
    if st["bias"] is not None:
        x = x + st["bias"]
    x = x.double()
    w = torch.exp((x - x.amax(dim=1, keepdim=True)) / st["temperature"].double()[:, None])
    vocab = w.shape[1]
    x, by = torch.sort(x, dim=1, descending=True, stable=True)
    w = torch.gather(w, 1, by)
    keep = torch.ones_like(w, dtype=torch.bool)
    if st["top_k"] is not None:
        keep &= torch.arange(vocab, device=w.device)[None, :] < st["top_k"][:, None]
    if st["top_p"] is not None:
        up = torch.cumsum(torch.where(keep, w, torch.zeros_like(w)), dim=1)
        keep &= up - w < st["top_p"].double()[:, None] * up[:, -1:]
    if st["min_p"] is not None:
        keep &= w >= st["min_p"].double()[:, None]
    w = torch.where(keep, w, torch.zeros_like(w))
    w = torch.zeros_like(w).scatter_(1, by, w)  # back in the vocabulary's order
    up = torch.cumsum(w, dim=1)
    token = (up <= st["u"].double()[:, None] * up[:, -1:]).sum(dim=1).clamp(max=vocab - 1)
    picked = torch.gather(w, 1, token[:, None])[:, 0]
    st["token"].copy_(token)
    st["logprob"].copy_(torch.log(picked / up[:, -1]))
    return {"token": st["token"], "logprob": st["logprob"]}


# ---------------------------------------------------------------- one pass
def run(state):
    op = state["case"]["op"]
    if not own:
        return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend, "sample": _plain_sample}[op](state)
    import serving_ls_beam_gb300 as lsb

    if op == "write":
        lsb.check(lsb.ls_paged_write(state["key"], state["value"], state["start"], state["count"], state["pages"],
                                     state["ws"]))
        return _write_outputs(state)
    if op == "read":
        lsb.check(lsb.ls_paged_read(state["pages"], state["start"], state["count"], state["out_key"], state["out_value"],
                                    state["ws"]))
        return {"key": state["out_key"], "value": state["out_value"]}
    if op == "attend":
        lsb.check(lsb.ls_paged_attention(state["q"], state["pages"], state["len"], state["out"], state["ws"]))
        return state["out"]
    lsb.check(lsb.ls_sample_filtered(state["logits"], state["bias"], state["u"], state["temperature"], state["top_k"],
                                     state["top_p"], state["min_p"], state["token"], state["logprob"]))
    return {"token": state["token"], "logprob": state["logprob"]}


# ---------------------------------------------------------------- the definition in 64 bits
def _power_of_two(e):
    """2^e in float64, by its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _rounded_e4m3(x):
    """float64 values to the nearest of 4 bits of significand and exponents from -6 (subnormal below), ties to even."""
    _, e = torch.frexp(x)
    step = _power_of_two((e - 1).clamp(min=-6) - 3)
    return torch.round(x / step) * step


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "sample":
        return _exact_sample(st)
    table, page, cache = st["table"].tolist(), case["page"], case["cache"]

    def positions(name, r, lo, hi):
        """[hi - lo, heads, dim] of row r's positions lo..hi."""
        p0, p1 = lo // page, -(-hi // page)
        at = torch.tensor(table[r][p0:p1], dtype=torch.long, device="cuda")
        x = st[name + "_pages"].contiguous().view(torch.uint8 if SIZES[cache] == 1 else DTYPES[cache]).index_select(0, at)
        x = x.view(DTYPES[cache]).to(torch.float64)
        if st[name + "_scale"] is not None:
            x = x * st[name + "_scale"].index_select(0, at).double().unsqueeze(3)
        x = x.permute(0, 2, 1, 3).reshape(-1, case["heads"], case["dim"])
        return x[lo - p0 * page:hi - p0 * page]

    if case["op"] == "attend":
        out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
        for name in ("key", "value"):
            st[name + "_pages"] = st[name + "_pages"].contiguous()
        for r, n in enumerate(st["len"].tolist()):
            if n == 0:
                continue
            q = st["q"][r].double().view(case["heads"], -1, case["dim"])
            s = torch.einsum("hgd,nhd->hgn", q, positions("key", r, 0, n)) / math.sqrt(case["dim"])
            p = torch.softmax(s, dim=-1)
            out[r] = torch.einsum("hgn,nhd->hgd", p, positions("value", r, 0, n)).reshape(out[r].shape)
        return out
    starts, counts = st["start"].tolist(), st["count"].tolist()
    if case["op"] == "read":
        res = {}
        for name in ("key", "value"):
            st[name + "_pages"] = st[name + "_pages"].contiguous()
            res[name] = st["out_" + name].double()
            for r, (s, c) in enumerate(zip(starts, counts)):
                res[name][r, :c] = positions(name, r, s, s + c)
        return res
    # write: scales and, where they are not whole numbers, codes
    res = {}
    for name in ("key", "value"):
        codes = None if cache == "i8" else st[name + "_pages"].to(torch.float64)
        scale = None if st[name + "_scale"] is None else st[name + "_scale"].double()
        for r, (s, c) in enumerate(zip(starts, counts)):
            n = torch.arange(s, s + c, device="cuda")
            at, place = st["table"][r].long()[n // page], n % page
            x = st[name][r, :c].double()
            if scale is not None:
                top = x.abs().amax(dim=-1)
                if cache == "e4m3":
                    e = torch.floor(torch.log2(top / 448.0)).clamp(min=-126.0)
                    for _ in range(2):  # the logarithm's own rounding
                        e = torch.where(_power_of_two(e) * 448.0 < top, e + 1.0, e)
                    unit = _power_of_two(e)
                    codes[at, :, place] = _rounded_e4m3(x / unit.unsqueeze(2))
                else:
                    unit = (top / 127.0).clamp(min=2.0 ** -126)
                scale[at, :, place] = unit
            else:
                codes[at, :, place] = x
        res[name + "_pages"] = None if codes is None else codes[:-1]
        if scale is not None:
            res[name + "_scale"] = scale[:-1]
    return res


def _exact_sample(st):
    x = st["logits"].float()
    if st["bias"] is not None:
        x = x + st["bias"]
    x = x.cpu().numpy()
    host = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    temp, top_k, top_p, min_p, u = (host(st[n]) for n in ("temperature", "top_k", "top_p", "min_p", "u"))
    out = np.empty(len(x))
    for r in range(len(x)):
        row = x[r].astype(np.float64)
        z = (row - row.max()) / float(temp[r])
        ids = np.lexsort((np.arange(len(row)), -row))  # best first, ties by the smaller index
        n = len(row) if top_k is None else min(len(row), int(top_k[r]))
        p = np.exp(z[ids[:n]])
        if top_p is not None:
            n = int(np.searchsorted(np.cumsum(p), float(top_p[r]) * p.sum(), side="left")) + 1
        if min_p is not None:
            n = min(n, int((p >= float(min_p[r])).sum()))
        kept = np.sort(ids[:n])
        p = np.exp(z[kept])
        c = np.cumsum(p)
        j = min(int(np.searchsorted(c, float(u[r]) * c[-1], side="right")), len(kept) - 1)
        out[r] = z[kept[j]] - math.log(c[-1])
    return {"token": None, "logprob": torch.from_numpy(out)}
