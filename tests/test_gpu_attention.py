"""Cross attention and the draft tree's attention on the GPU against their float64 definitions:
types, head layouts, lengths from none to several blocks, strides and odd sizes, trees with empty
places, anything in the places that are not read; every kernel forced wherever it applies."""
import numpy as np
import pytest

import attention_plain as ap

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import serving_ls_beam_gb300 as lsb  # noqa: E402

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
KERNELS = [None, "atsimt", "atmma,atwarps=1", "atmma,atwarps=4", "atmma,atwarps=4,atsplits=3",
           "attc", "attc,atsplits=3"]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lsb.load_library()
    return torch.device("cuda:0")


@pytest.fixture(params=KERNELS)
def kernel(request, monkeypatch):
    if request.param:
        monkeypatch.setenv("LS_BEAM_DEBUG", request.param)
    return request.param


def tensor(g, shape, dtype, dev, spread=1.0):
    return torch.from_numpy(g.normal(size=shape, scale=spread).astype(np.float32)).to(DT[dtype]).to(dev)


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def workspace(size, dev):
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    lsb.check(lsb.ls_workspace_init(ws))
    return ws


def run_cross(q, k, v, lens, scale=None, out=None, status=0):
    B, K, T, H, D = q.shape
    ws = workspace(lsb.ls_cross_attention_workspace_size(B, K, T, H, k.shape[1], k.shape[2], D), q.device)
    out = torch.full_like(q, float("nan")) if out is None else out
    lens = torch.as_tensor(lens, dtype=torch.int32, device=q.device)
    lsb.check(lsb.ls_cross_attention(q, k, v, lens, out, ws, scale))
    assert lsb.ls_read_status(ws) == status
    return out


def close(out, want, bound):
    got = f64(out)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:3].tolist(), got[bad][:3], want[bad][:3], bound[bad][:3])


def check_cross(dev, dtype, B, K, T, H, HK, S, D, lens, seed=0, spread=1.0, scale=None):
    g = np.random.default_rng(seed)
    q = tensor(g, (B, K, T, H, D), dtype, dev, spread)
    k, v = tensor(g, (B, HK, S, D), dtype, dev), tensor(g, (B, HK, S, D), dtype, dev)
    for b, n in enumerate(lens):  # anything past the lengths
        k[b, :, n:] = float("nan")
        v[b, :, n:] = float("inf") if b % 2 else float("nan")
    out = run_cross(q, k, v, lens, scale)
    kz, vz = f64(k), f64(v)
    want, bound = ap.cross(f64(q), kz, vz, lens, D ** -0.5 if scale is None else scale, dtype)
    close(out, want, bound)


# (batch, k, q_len, heads, kv_heads, max_src, dim, lens)
CROSS = [
    (1, 1, 1, 1, 1, 1, 64, [1]),
    (3, 4, 1, 4, 4, 40, 64, [40, 0, 17]),           # an empty sentence
    (2, 4, 1, 8, 2, 300, 64, [300, 257]),           # 16 queries per key head
    (2, 5, 1, 12, 4, 129, 128, [128, 129]),         # 15 queries
    (2, 8, 1, 8, 2, 200, 128, [31, 200]),           # 32 queries
    (1, 3, 1, 6, 2, 77, 80, [77]),
    (2, 2, 3, 4, 2, 65, 96, [1, 65]),
    (1, 2, 1, 2, 1, 50, 256, [49]),
    (2, 1, 40, 4, 4, 100, 64, [99, 64]),            # 40 queries
    (1, 1, 130, 4, 2, 200, 64, [190]),              # 260 queries
    (2, 2, 70, 2, 2, 333, 128, [333, 128]),         # 140 queries
    (1, 1, 300, 2, 1, 150, 32, [150]),
    (2, 3, 7, 2, 1, 20, 8, [20, 3]),
    (1, 4, 1, 2, 2, 2000, 64, [1999]),              # a long source, split
    (1, 1, 20, 2, 1, 3001, 128, [3001]),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", CROSS)
def test_cross(dev, kernel, shape, dtype):
    B, K, T, H, HK, S, D, lens = shape
    check_cross(dev, dtype, B, K, T, H, HK, S, D, lens, seed=S)


# more problems than any launch has CTAs, of every kind in turn: no key, one block, one tile and a
# bit, several; one tile of queries, a tile and a bit, several
@pytest.mark.parametrize("T,D", [(1, 64), (12, 128), (40, 64), (150, 64), (150, 128), (300, 64)])
def test_cross_many_problems(dev, kernel, T, D):
    B, H, S = (120, 8, 300) if T < 100 else (50, 4, 300)
    g = np.random.default_rng(T + D)
    dtype = "f16" if T % 4 else "bf16"
    q = tensor(g, (B, 1, T, H, D), dtype, dev)
    k, v = tensor(g, (B, H, S, D), dtype, dev), tensor(g, (B, H, S, D), dtype, dev)
    lens = [[0, 1, 128, 129, 300, 17, 256, 257, 100][b % 9] if b % 5 else int(g.integers(0, S + 1)) for b in range(B)]
    out = run_cross(q, k, v, lens)
    pick = sorted({0, T // 2, T - 1, min(T - 1, 127), min(T - 1, 128)})  # a few of the queries, every problem
    want, bound = ap.cross(f64(q)[:, :, pick], f64(k), f64(v), lens, D ** -0.5, dtype)
    close(out[:, :, pick], want, bound)


@pytest.mark.parametrize("nodes,heads,D", [(1, 8, 64), (10, 8, 128), (33, 8, 64), (64, 16, 128)])
def test_tree_many_problems(dev, kernel, nodes, heads, D):
    R, HK, S = 150, 4, 270
    g = np.random.default_rng(nodes)
    dtype = "bf16"
    kinds = ["forest", "chain", "ragged", "empty", "forest"]
    parent = np.stack([random_parents(g, nodes, kinds[r % 5] if nodes > 1 else "chain") for r in range(R)])
    q = tensor(g, (R, nodes, heads, D), dtype, dev)
    ck, cv = tensor(g, (R, HK, S, D), dtype, dev), tensor(g, (R, HK, S, D), dtype, dev)
    dk, dv = tensor(g, (R, nodes, HK, D), dtype, dev), tensor(g, (R, nodes, HK, D), dtype, dev)
    for r in range(R):
        for i in range(nodes):
            if not ap.branch(parent[r], i):
                dv[r, i] = float("nan")  # some rows meet values to clear, their neighbours do not
    lens = [[0, 128, 270, 60, 129][r % 5] if r % 3 else int(g.integers(0, S + 1)) for r in range(R)]
    out = run_tree(q, ck, cv, lens, dk, dv, parent)
    pick = sorted({0, nodes // 2, nodes - 1})
    full_out = f64(out)
    for r in range(0, R, 2):
        for i in pick:
            br = ap.branch(parent[r], i)
            for h in range(0, heads, 3):
                kh = h // (heads // HK)
                if not br:
                    assert not full_out[r, i, h].any()
                    continue
                ks = np.concatenate([f64(ck[r, kh, :lens[r]]), f64(dk[r, br, kh])])
                vs = np.concatenate([f64(cv[r, kh, :lens[r]]), f64(dv[r, br, kh])])
                want, bound = ap.one_query(f64(q[r, i, h]), ks, vs, D ** -0.5, dtype)
                assert (np.abs(full_out[r, i, h] - want) <= bound).all(), (r, i, h)


def test_waits_that_run_out_are_reported(dev, monkeypatch):
    """A wait limit of zero: calls end with the status set (their result is unspecified), and the
    next call with the ordinary limit is right."""
    g = np.random.default_rng(4)
    for T, D in ((1, 64), (200, 64), (200, 128)):
        q = tensor(g, (2, 1, T, 2, D), "f16", dev)
        k, v = tensor(g, (2, 2, 500, D), "f16", dev), tensor(g, (2, 2, 500, D), "f16", dev)
        monkeypatch.setenv("LS_BEAM_DEBUG", "spin=0," + ("attc" if T > 1 else "atmma"))
        run_cross(q, k, v, [500, 300], status=lsb.LS_ERR_TIMEOUT)
        monkeypatch.delenv("LS_BEAM_DEBUG")
        out = run_cross(q, k, v, [500, 300])
        want, bound = ap.cross(f64(q)[:, :, :2], f64(k), f64(v), [500, 300], D ** -0.5, "f16")
        close(out[:, :, :2], want, bound)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_cross_odd_head_sizes(dev, dtype):
    for d in (1, 7, 33, 65, 100, 255):
        check_cross(dev, dtype, 2, 3, 1, 2, 2, 37, d, [37, 5], seed=d)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_cross_sharp_and_negative_scales(dev, kernel, dtype):
    """Large scores (the running maximum moves by a lot) and a negative scale."""
    check_cross(dev, dtype, 2, 4, 1, 4, 2, 260, 64, [260, 131], spread=30.0)
    check_cross(dev, dtype, 1, 1, 150, 2, 2, 260, 64, [259], spread=30.0)
    check_cross(dev, dtype, 2, 4, 1, 4, 2, 100, 64, [100, 31], scale=-0.3)
    check_cross(dev, dtype, 1, 2, 80, 2, 2, 100, 64, [100], scale=0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,T", [(64, 1), (128, 1), (64, 100)])
def test_cross_rising_scores(dev, kernel, dtype, D, T):
    """Scores that rise from key to key: the maximum changes in every block."""
    S = 700
    q = torch.ones((1, 2, T, 2, D), device=dev).to(DT[dtype])
    k = (torch.arange(S, device=dev).view(1, 1, S, 1) / 64).expand(1, 2, S, D).to(DT[dtype]).contiguous()
    v = tensor(np.random.default_rng(3), (1, 2, S, D), dtype, dev)
    for kk in (k, k.flip(2).contiguous()):
        out = run_cross(q, kk, v, [S])
        want, bound = ap.cross(f64(q), f64(kk), f64(v), [S], D ** -0.5, dtype)
        close(out, want, bound)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_cross_strided_views(dev, kernel, dtype):
    """Keys as a projection writes them, slices of a wider tensor, rows that share one key tensor."""
    g = np.random.default_rng(9)
    B, K, T, H, HK, S, D = 3, 2, 2, 4, 2, 45, 64
    wide = tensor(g, (B, S, 2, HK, D), dtype, dev)
    k, v = wide[:, :, 0].transpose(1, 2), wide[:, :, 1].transpose(1, 2)
    qw = tensor(g, (B * K, T, 3 * H, D), dtype, dev)
    q = qw[:, :, H:2 * H].unflatten(0, (B, K))
    ow = torch.full((B * K, T, H, 2 * D), float("nan"), dtype=DT[dtype], device=dev)
    out = ow[..., :D].unflatten(0, (B, K))
    lens = [45, 44, 1]
    run_cross(q, k, v, lens, out=out)
    want, bound = ap.cross(f64(q), f64(k), f64(v), lens, D ** -0.5, dtype)
    close(out, want, bound)
    assert torch.isnan(ow[..., D:]).all()
    one_k, one_v = k[:1].expand(B, -1, -1, -1), v[:1].expand(B, -1, -1, -1)
    out2 = run_cross(q.contiguous(), one_k, one_v, lens)
    want, bound = ap.cross(f64(q), f64(one_k), f64(one_v), lens, D ** -0.5, dtype)
    close(out2, want, bound)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_cross_odd_alignment(dev, dtype):
    """Tensors that start one element past an aligned address, and odd row strides."""
    g = np.random.default_rng(11)
    B, K, T, H, HK, S, D = 2, 2, 1, 2, 2, 40, 64
    k = tensor(g, (B, HK, S, D + 1), dtype, dev)[..., 1:]
    v = tensor(g, (B, HK, S, D + 1), dtype, dev)[..., :D]
    q = tensor(g, (B * K * T * H * D + 1,), dtype, dev)[1:].view(B, K, T, H, D)
    o = torch.full((B * K * T * H * D + 1,), float("nan"), dtype=DT[dtype], device=dev)
    out = run_cross(q, k, v, [40, 33], out=o[1:].view(B, K, T, H, D))
    want, bound = ap.cross(f64(q), f64(k), f64(v), [40, 33], D ** -0.5, dtype)
    close(out, want, bound)
    assert torch.isnan(o[0])


def test_cross_lengths_out_of_range_are_clamped_and_reported(dev, kernel):
    g = np.random.default_rng(2)
    q = tensor(g, (2, 2, 1, 2, 64), "f16", dev)
    k, v = tensor(g, (2, 2, 30, 64), "f16", dev), tensor(g, (2, 2, 30, 64), "f16", dev)
    out = run_cross(q, k, v, [31, -4], status=lsb.LS_ERR_INTERNAL)
    want, bound = ap.cross(f64(q), f64(k), f64(v), [30, 0], 0.125, "f16")
    close(out, want, bound)
    empty = run_cross(q, k[:, :, :0], v[:, :, :0], [0, 0])
    assert not empty.any()


# ---------------------------------------------------------------- trees
def random_parents(g, nodes, kind):
    if kind == "chain":
        p = np.arange(-1, nodes - 1)
    elif kind == "forest":
        p = np.array([-1] + [g.integers(-1, i) for i in range(1, nodes)])
    elif kind == "ragged":  # empty places at the end and in the middle
        p = np.array([-1] + [g.integers(0, i) for i in range(1, nodes)])
        p[nodes - nodes // 4:] = -2
        if nodes > 6:
            p[3] = -5
    else:  # "empty": no node at all
        p = np.full(nodes, -2)
    return p.astype(np.int32)


def run_tree(q, ck, cv, lens, dk, dv, parent, status=0, out=None):
    R, N, H, D = q.shape
    ws = workspace(lsb.ls_tree_attention_workspace_size(R, N, H, ck.shape[1], ck.shape[2], D), q.device)
    out = torch.full_like(q, float("nan")) if out is None else out
    lens = torch.as_tensor(lens, dtype=torch.int32, device=q.device)
    parent = torch.as_tensor(parent, dtype=torch.int32, device=q.device)
    lsb.check(lsb.ls_tree_attention(q, ck, cv, lens, dk, dv, parent, out, ws))
    assert lsb.ls_read_status(ws) == status
    return out


# (rows, nodes, heads, kv_heads, max_len, dim, lens)
TREES = [
    (1, 1, 1, 1, 1, 64, [0]),                # the very first token: nothing in the cache
    (3, 1, 4, 4, 64, 64, [0, 63, 64]),
    (4, 1, 8, 2, 200, 128, [1, 31, 32, 200]),
    (4, 13, 4, 4, 100, 64, [100, 0, 33, 64]),
    (4, 16, 8, 2, 70, 128, [70, 69, 1, 0]),  # 64 queries per key head
    (4, 64, 4, 2, 150, 64, [150, 128, 5, 0]),
    (4, 33, 8, 2, 130, 128, [130, 127, 5, 64]),
    (2, 7, 2, 2, 90, 80, [90, 17]),
    (4, 5, 4, 1, 40, 256, [40, 39, 2, 0]),
    (1, 16, 4, 1, 3000, 64, [2999]),         # a long cache, split
    (1, 64, 4, 1, 2500, 128, [2500]),
    (2, 1, 2, 1, 5000, 128, [5000, 1]),
]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", TREES)
def test_tree(dev, kernel, shape, dtype):
    R, N, H, HK, S, D, lens = shape
    g = np.random.default_rng(S + N)
    kinds = ["forest", "chain", "ragged", "empty"]
    parent = np.stack([random_parents(g, N, kinds[(r + (N == 1)) % (4 if N > 1 else 3)]) for r in range(R)])
    q = tensor(g, (R, N, H, D), dtype, dev)
    ck, cv = tensor(g, (R, HK, S, D), dtype, dev), tensor(g, (R, HK, S, D), dtype, dev)
    dk, dv = tensor(g, (R, N, HK, D), dtype, dev), tensor(g, (R, N, HK, D), dtype, dev)
    for r in range(R):
        ck[r, :, lens[r]:] = float("inf")
        cv[r, :, lens[r]:] = float("nan")
        for i in range(N):
            if not ap.branch(parent[r], i):
                dk[r, i] = float("nan")
                dv[r, i] = float("inf")
                q[r, i] = float("nan")
    out = run_tree(q, ck, cv, lens, dk, dv, parent)
    want, bound = ap.tree(f64(q), f64(ck), f64(cv), lens, f64(dk), f64(dv), parent, D ** -0.5, dtype)
    close(out, want, bound)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("nodes,heads", [(6, 2), (20, 8), (40, 8)])
def test_tree_other_branches_do_not_matter(dev, kernel, dtype, nodes, heads):
    """Infinities and NaN in a node's values reach the nodes under it and no other."""
    g = np.random.default_rng(nodes)
    R, HK, S, D = 2, 2, 40, 64
    parent = np.stack([random_parents(g, nodes, "forest"), random_parents(g, nodes, "forest")])
    parent[:, 2] = 0
    q, ck, cv = tensor(g, (R, nodes, heads, D), dtype, dev), tensor(g, (R, HK, S, D), dtype, dev), \
        tensor(g, (R, HK, S, D), dtype, dev)
    dk, dv = tensor(g, (R, nodes, HK, D), dtype, dev), tensor(g, (R, nodes, HK, D), dtype, dev)
    dv[0, 2, :, 5] = float("inf")
    dv[0, 2, :, 6] = float("nan")
    dv[1, nodes - 1, 1, D - 1] = float("-inf")
    out = f64(run_tree(q, ck, cv, [S, 3], dk, dv, parent))
    clean = dv.clone()
    clean[0, 2, :, 5:7] = 0
    clean[1, nodes - 1, 1, D - 1] = 0
    want, bound = ap.tree(f64(q), f64(ck), f64(cv), [S, 3], f64(dk), f64(clean), parent, D ** -0.5, dtype)
    hit = np.zeros(want.shape, bool)
    for i in range(nodes):
        if 2 in ap.branch(parent[0], i):
            assert (out[0, i, :, 5] == np.inf).all() and np.isnan(out[0, i, :, 6]).all()
            hit[0, i, :, 5:7] = True
    assert (out[1, nodes - 1, heads // 2:, D - 1] == -np.inf).all()
    hit[1, nodes - 1, heads // 2:, D - 1] = True
    assert (np.abs(out - want) <= bound)[~hit].all()


def test_tree_invalid_parents_are_reported(dev, kernel):
    g = np.random.default_rng(5)
    R, N, H, S, D = 1, 5, 2, 10, 64
    q = tensor(g, (R, N, H, D), "bf16", dev)
    ck, cv = tensor(g, (R, H, S, D), "bf16", dev), tensor(g, (R, H, S, D), "bf16", dev)
    dk, dv = tensor(g, (R, N, H, D), "bf16", dev), tensor(g, (R, N, H, D), "bf16", dev)
    parent = np.array([[-1, 0, 3, 1, 2]])  # node 2's parent does not come before it; node 4 is under it
    out = run_tree(q, ck, cv, [7], dk, dv, parent, status=lsb.LS_ERR_INTERNAL)
    want, bound = ap.tree(f64(q), f64(ck), f64(cv), [7], f64(dk), f64(dv), parent, D ** -0.5, "bf16")
    close(out, want, bound)
    assert not out[0, 2].any() and not out[0, 4].any()


def test_tree_strided_views(dev, kernel):
    """One layer of a cache, and queries, keys and values as slices of one projection's output."""
    g = np.random.default_rng(6)
    L, R, N, H, HK, S, D = 2, 3, 4, 4, 2, 30, 64
    cache_k, cache_v = tensor(g, (L, R, HK, S, D), "f16", dev), tensor(g, (L, R, HK, S, D), "f16", dev)
    qkv = tensor(g, (R, N, H + 2 * HK, D), "f16", dev)
    q, dk, dv = qkv[:, :, :H], qkv[:, :, H:H + HK], qkv[:, :, H + HK:]
    parent = np.stack([random_parents(g, N, "forest") for _ in range(R)])
    out = run_tree(q, cache_k[1], cache_v[1], [30, 29, 0], dk, dv, parent,
                   out=torch.full((R, N, H, D), float("nan"), dtype=torch.float16, device=dev))
    want, bound = ap.tree(f64(q), f64(cache_k[1]), f64(cache_v[1]), [30, 29, 0], f64(dk), f64(dv), parent, 0.125, "f16")
    close(out, want, bound)


@pytest.mark.parametrize("T", [1, 100])
def test_same_workspace_and_other_streams(dev, kernel, T):
    """Calls of several shapes share one workspace; a call on a side stream is ordered by it."""
    g = np.random.default_rng(8)
    ws = workspace(lsb.ls_cross_attention_workspace_size(1, 4, T, 8, 1, 1, 128), dev)
    side = torch.cuda.Stream()
    for B, K, H, HK, S, D in ((1, 4, 8, 1, 2000, 128), (3, 2, 4, 2, 50, 64), (1, 1, 2, 1, 999, 128), (1, 4, 8, 1, 1500, 128)):
        q = tensor(g, (B, K, T, H, D), "bf16", dev)
        k, v = tensor(g, (B, HK, S, D), "bf16", dev), tensor(g, (B, HK, S, D), "bf16", dev)
        lens = torch.full((B,), S, dtype=torch.int32, device=dev)
        out = torch.empty_like(q)
        side.wait_stream(torch.cuda.current_stream())
        lsb.check(lsb.ls_cross_attention(q, k, v, lens, out, ws, stream=side))
        torch.cuda.current_stream().wait_stream(side)
        sample = (slice(None), slice(None), slice(0, 3))
        want, bound = ap.cross(f64(q)[sample], f64(k), f64(v), [S] * B, D ** -0.5, "bf16")
        close(out[sample], want, bound)
        again = torch.empty_like(q)
        lsb.check(lsb.ls_cross_attention(q, k, v, lens, again, ws))
        assert torch.equal(out, again)  # the same bits every time


@pytest.mark.parametrize("T", [1, 20, 150])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_cross_offsets_past_32_bits(dev, kernel, dtype, T):
    """Keys a megabyte apart and sentences gigabytes apart: byte offsets of more than 2^32 within a
    row, element offsets of more than 2^31 between rows."""
    g = np.random.default_rng(T)
    B, H, S, D = 2, 1, 700, 64
    es = 4 if dtype == "f32" else 2
    pos = (1 << 23) // es  # 8 MB from key to key: 5.6 GB a row
    big = torch.empty(B * S * pos + D, dtype=DT[dtype], device=dev)
    k = torch.as_strided(big, (B, H, S, D), (S * pos, D, pos, 1))
    v = torch.as_strided(big, (B, H, S, D), (S * pos, D, pos, 1), 4 * D)
    k.copy_(tensor(g, (B, H, S, D), dtype, dev))
    v.copy_(tensor(g, (B, H, S, D), dtype, dev))
    q = tensor(g, (B, 1, T, H, D), dtype, dev)
    lens = [700, 601]
    out = run_cross(q, k, v, lens)
    pick = sorted({0, T - 1})
    want, bound = ap.cross(f64(q)[:, :, pick], f64(k), f64(v), lens, D ** -0.5, dtype)
    close(out[:, :, pick], want, bound)


@pytest.mark.parametrize("T", [1, 40])
def test_graph_capture(dev, kernel, T):
    g = np.random.default_rng(12)
    q = tensor(g, (1, 2, T, 4, 64), "f16", dev)
    k, v = tensor(g, (1, 2, 900, 64), "f16", dev), tensor(g, (1, 2, 900, 64), "f16", dev)
    lens = torch.full((1,), 900, dtype=torch.int32, device=dev)
    out, ws = torch.zeros_like(q), workspace(lsb.ls_cross_attention_workspace_size(1, 2, T, 4, 2, 900, 64), dev)
    lsb.check(lsb.ls_cross_attention(q, k, v, lens, out, ws))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lsb.check(lsb.ls_cross_attention(q, k, v, lens, out, ws))
    first = out.clone()
    out.zero_()
    lens.fill_(450)
    graph.replay()
    want, bound = ap.cross(f64(q), f64(k), f64(v), [450], 0.125, "f16")
    close(out, want, bound)
    assert not torch.equal(out, first)
