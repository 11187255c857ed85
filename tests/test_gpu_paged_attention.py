"""Attention of one new token over a paged cache on the GPU against its float64 definition: types, head layouts, page sizes,
lengths from none to many parts, strides and odd sizes, anything in the places that are not read."""
import numpy as np
import pytest

import paged_plain as pp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import serving_ls_beam_gb300 as lsb  # noqa: E402

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
KERNELS = [None, "pgsimt", "pgwarps=1", "pgwarps=4", "pgwarps=1,pgworkers=2", "pgwarps=4,pgworkers=5"]


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


def f64(t):
    return t.double().cpu().numpy()


def workspace(size, dev):
    ws = torch.empty(size, dtype=torch.uint8, device=dev)
    lsb.check(lsb.ls_workspace_init(ws))
    return ws


class Cache:
    """Rows of given lengths in pages; what lies past a length, and in pages that no row has, may hold anything."""

    def __init__(self, g, dev, cache, heads, dim, page, lens, order="head", odd=0, spread=1.0):
        need = [-(-n // page) for n in lens]
        num = sum(need) + 2
        perm = g.permutation(num - 1) + 1  # (page 0 is no row's)
        table = np.full((len(lens), max(max(need), 1) + 1), 1 << 30, np.int32)  # entries past the pages in use: not looked up
        at = 0
        for r, n in enumerate(need):
            table[r, :n] = perm[at:at + n]
            at += n
        self.lens, self.page, self.dim, self.coded = lens, page, dim, cache in ("e4m3", "i8")
        self.table = torch.from_numpy(table).to(dev)
        shape = (num, heads, page, dim + odd) if order == "head" else (num, page, heads, dim + odd)
        for name in ("key", "value"):
            x = g.normal(size=(num, heads, page, dim), scale=spread).astype(np.float32)
            used = np.zeros((num, page), bool)
            for r, n in enumerate(lens):
                for i in range(n):
                    used[table[r, i // page], i % page] = True
            scale = None
            t = torch.from_numpy(x)
            if self.coded:
                codes, s = pp.quantise(x.astype(np.float64), cache)
                s = s * 2.0 ** g.integers(-3, 3, s.shape)
                t = torch.from_numpy(codes.astype(np.float32))
                scale = torch.from_numpy(s.astype(np.float32))
                scale[torch.from_numpy(~used)[:, None, :].expand(scale.shape)] = float("nan")
            t = t.to(DT[cache])
            hide = torch.from_numpy(~used)[:, None, :, None].expand(t.shape)
            if cache == "e4m3":
                t.view(torch.uint8)[hide] = 0x7f  # NaN
            elif cache != "i8":
                t[hide] = float("nan") if name == "key" else float("inf")
            full = torch.zeros(shape, dtype=torch.float32).to(DT[cache]) if not self.coded else torch.zeros(shape, dtype=torch.uint8).view(DT[cache])
            view = full if order == "head" else full.transpose(1, 2)
            if self.coded:
                view.view(torch.uint8)[..., :dim] = t.view(torch.uint8)
            else:
                view[..., :dim] = t
            full = full.to(dev)
            view = full if order == "head" else full.transpose(1, 2)
            setattr(self, name, view[..., :dim])
            setattr(self, name + "_scale", None if scale is None else scale.to(dev))

    def pages(self):
        return lsb.ls_pages(self.key, self.value, self.table, self.key_scale, self.value_scale)

    def row(self, name, r):
        """[heads, n, dim] and the scales [heads, n] of row r."""
        n = max(self.lens[r], 0)
        t, table = f64(getattr(self, name)) if not hasattr(self, "_" + name) else getattr(self, "_" + name), self.table.cpu().numpy()
        setattr(self, "_" + name, t)
        pos = np.arange(n)
        at, place = table[r, pos // self.page], pos % self.page
        x = t[at, :, place].transpose(1, 0, 2)
        if not self.coded:
            return x, np.ones(x.shape[:2])
        s = f64(getattr(self, name + "_scale"))[at, :, place].T
        return x * s[:, :, None], s


def check(dev, dtype, cache, heads, kv, dim, page, lens, order="head", seed=0, scale=None, odd=0, spread=1.0, pick=None, status=0, change=None):
    g = np.random.default_rng(seed)
    c = Cache(g, dev, cache, kv, dim, page, lens, order, odd, spread)
    q = torch.from_numpy(g.normal(size=(len(lens), heads, dim + odd)).astype(np.float32)).to(DT[dtype]).to(dev)[..., :dim]
    out = torch.full((len(lens), heads, dim + odd), float("nan"), dtype=DT[dtype], device=dev)[..., :dim]
    ws = workspace(lsb.ls_paged_attention_workspace_size(len(lens), heads, kv, dim), dev)
    length = torch.tensor(lens, dtype=torch.int32, device=dev)
    if change:
        change(c, length)
    for _ in range(2):  # the second call finds the workspace as the first left it
        out.fill_(float("nan"))
        lsb.check(lsb.ls_paged_attention(q, c.pages(), length, out, ws, scale))
    assert lsb.ls_read_status(ws) == status
    got, q64 = f64(out), f64(q)
    for r in pick if pick is not None else range(len(lens)):
        (ks, _), (vs, sv) = c.row("key", r), c.row("value", r)
        for h in range(heads):
            k = h // (heads // kv)
            want, bound = pp.attend(q64[r, h], ks[k], vs[k], sv[k], dim ** -0.5 if scale is None else scale, dtype, cache)
            bad = ~(np.abs(got[r, h] - want) <= bound)
            assert not bad.any(), (r, h, np.argwhere(bad)[:3].tolist(), got[r, h][bad][:3], want[bad][:3], bound[bad][:3])
    return out


# (heads, kv_heads, dim, page, lens, order)
SHAPES = [
    (1, 1, 64, 16, [1], "head"),
    (4, 4, 64, 16, [40, 0, 17, 16, 1, 15], "head"),   # an empty row
    (8, 2, 128, 64, [300, 257, 3], "token"),
    (10, 2, 128, 8, [129, 8, 9], "head"),             # five queries per key head
    (16, 1, 64, 32, [200, 31], "head"),               # sixteen
    (40, 2, 96, 16, [77, 33], "head"),                # twenty: more than an item has
    (9, 1, 256, 24, [50, 49], "token"),
    (2, 2, 256, 128, [300], "head"),
    (3, 3, 80, 1, [33, 70], "head"),                  # a page per position
    (6, 3, 48, 5, [64, 11], "token"),                 # pages that end inside a block
    (2, 1, 33, 16, [40, 100], "head"),                # odd head sizes
    (2, 2, 1, 7, [20, 3], "token"),
    (4, 1, 200, 16, [65], "head"),
    (2, 1, 64, 16, [5000], "head"),                   # many parts
    (8, 8, 32, 100, [2, 1000, 0, 350], "head"),
]


@pytest.mark.parametrize("dtype,cache", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f32", "e4m3"), ("f16", "e4m3"),
                                         ("bf16", "e4m3"), ("f32", "i8"), ("f16", "i8"), ("bf16", "i8")])
@pytest.mark.parametrize("shape", SHAPES)
def test_attention(dev, kernel, shape, dtype, cache):
    heads, kv, dim, page, lens, order = shape
    check(dev, dtype, cache, heads, kv, dim, page, lens, order, seed=dim)


@pytest.mark.parametrize("dtype,cache", [("f32", "f32"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "i8")])
def test_many_rows(dev, kernel, dtype, cache):
    """More items than any launch has workers, of every length in turn; long rows among short ones."""
    g = np.random.default_rng(3)
    lens = [[0, 1, 16, 17, 64, 5, 33, 128, 100][r % 9] if r % 5 else int(g.integers(0, 200)) for r in range(700)]
    lens[11], lens[500] = 1500, 900
    check(dev, dtype, cache, 8, 4, 64, 16, lens, seed=4, pick=[0, 1, 2, 3, 4, 5, 6, 7, 8, 10, 11, 12, 350, 499, 500, 501, 698, 699])


@pytest.mark.parametrize("dtype,cache", [("f32", "i8"), ("f16", "f16"), ("bf16", "e4m3")])
def test_long_rows(dev, kernel, dtype, cache):
    """Rows cut into parts at any block, the parts of several rows with one worker."""
    check(dev, dtype, cache, 4, 2, 128, 64, [20000, 1, 0, 7777, 13001], seed=5)


@pytest.mark.parametrize("dtype,cache", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("bf16", "e4m3"), ("f16", "i8")])
def test_scales(dev, kernel, dtype, cache):
    """No scale, a negative one, large scores (one key has all the weight), and one far under the others' values."""
    check(dev, dtype, cache, 4, 2, 64, 16, [100, 37], scale=0.0)
    check(dev, dtype, cache, 4, 2, 64, 16, [100, 37], scale=-0.3)
    check(dev, dtype, cache, 4, 2, 64, 16, [100, 37], scale=4.0, spread=3.0)


@pytest.mark.parametrize("dtype,cache", [("f32", "f32"), ("f16", "f16"), ("bf16", "bf16"), ("f32", "e4m3"), ("f16", "e4m3"), ("bf16", "i8")])
def test_unaligned(dev, dtype, cache):
    """Strides that are no multiples of 16 bytes."""
    check(dev, dtype, cache, 4, 2, 64, 16, [100, 37, 0], odd=1)


@pytest.mark.parametrize("dtype,cache", [("f32", "f32"), ("f16", "f16"), ("bf16", "e4m3"), ("f16", "i8")])
def test_out_of_range(dev, kernel, dtype, cache):
    """Lengths outside the table's places are clamped; a page that does not exist is left out: both are reported."""
    def lengths(c, length):
        length[0], length[1] = -5, 1 << 30
        c.lens = [0, 32, 9]
        c.table = c.table[:, :2].contiguous()
    check(dev, dtype, cache, 4, 2, 64, 16, [3, 32, 9], status=5, change=lengths)

    g = np.random.default_rng(8)
    c = Cache(g, dev, cache, 2, 64, 16, [70, 40])
    q = torch.from_numpy(g.normal(size=(2, 4, 64)).astype(np.float32)).to(DT[dtype]).to(dev)
    length = torch.tensor([70, 40], dtype=torch.int32, device=dev)
    ws = workspace(lsb.ls_paged_attention_workspace_size(2, 4, 2, 64), dev)
    c.table[0, 1], c.table[0, 3], c.table[1, 0], c.table[1, 1], c.table[1, 2] = -1, 1 << 20, -7, -7, -7
    out = torch.empty_like(q)
    lsb.check(lsb.ls_paged_attention(q, c.pages(), length, out, ws))
    assert lsb.ls_read_status(ws) == 5
    assert torch.equal(out[1], torch.zeros_like(out[1]))  # nothing is left of this row
    keep = np.r_[0:16, 32:48, 64:70]
    c.table[0, 1] = c.table[0, 3] = c.table[0, 0]
    for h in range(4):
        (ks, _), (vs, sv) = c.row("key", 0), c.row("value", 0)
        want, bound = pp.attend(f64(q)[0, h], ks[h // 2][keep], vs[h // 2][keep], sv[h // 2][keep], 0.125, dtype, cache)
        assert (np.abs(f64(out)[0, h] - want) <= bound).all()


@pytest.mark.parametrize("cache", ["e4m3", "i8"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_values_of_very_different_scales(dev, kernel, dtype, cache):
    """A key with nearly all the weight whose values are 2^-20 of the others': the weights' rounding must not lose them."""
    g = np.random.default_rng(9)
    c = Cache(g, dev, cache, 1, 64, 16, [90])
    at = c.table.cpu().numpy()[0]
    q = torch.ones((1, 1, 64), device=dev, dtype=DT[dtype])
    c.key.view(torch.uint8)[int(at[2]), 0, 5] = torch.full((64,), 16.0, device=dev).to(DT[cache]).view(torch.uint8)
    c.key_scale[int(at[2]), 0, 5] = 0.0625 if cache == "e4m3" else 1 / 16  # q . k = 64
    c.value_scale[int(at[2]), 0, 5] = 2.0 ** -26
    length = torch.tensor([90], dtype=torch.int32, device=dev)
    ws = workspace(lsb.ls_paged_attention_workspace_size(1, 1, 1, 64), dev)
    out = torch.empty_like(q)
    lsb.check(lsb.ls_paged_attention(q, c.pages(), length, out, ws, 1.0))
    (ks, _), (vs, sv) = c.row("key", 0), c.row("value", 0)
    want, bound = pp.attend(f64(q)[0, 0], ks[0], vs[0], sv[0], 1.0, dtype, cache)
    assert (np.abs(f64(out)[0, 0] - want) <= bound).all()


def test_shared_pages_and_views(dev, kernel):
    """Rows that share the pages of a common beginning, one table row for all (stride 0), queries and results as slices
    of larger tensors."""
    g = np.random.default_rng(10)
    c = Cache(g, dev, "e4m3", 2, 64, 16, [100])
    rows = 5
    big = torch.from_numpy(g.normal(size=(rows, 3, 4, 64)).astype(np.float32)).to(torch.bfloat16).to(dev)
    q = big[:, 1]
    res = torch.full((rows, 2, 4, 64), float("nan"), dtype=torch.bfloat16, device=dev)
    pages = lsb.ls_pages(c.key, c.value, c.table.expand(rows, -1), c.key_scale, c.value_scale)
    lens = [100, 1, 50, 0, 99]
    length = torch.tensor(lens, dtype=torch.int32, device=dev)
    ws = workspace(lsb.ls_paged_attention_workspace_size(rows, 4, 2, 64), dev)
    lsb.check(lsb.ls_paged_attention(q, pages, length, res[:, 0], ws))
    assert lsb.ls_read_status(ws) == 0
    assert torch.isnan(res[:, 1]).all()
    (ks, _), (vs, sv) = c.row("key", 0), c.row("value", 0)
    for r, n in enumerate(lens):
        for h in range(4):
            want, bound = pp.attend(f64(q)[r, h], ks[h // 2][:n], vs[h // 2][:n], sv[h // 2][:n], 0.125, "bf16", "e4m3")
            assert (np.abs(f64(res)[r, 0, h] - want) <= bound).all()


def test_repeats_are_equal(dev, kernel):
    """The parts are joined in the order of the keys, whichever comes last."""
    g = np.random.default_rng(11)
    c = Cache(g, dev, "f16", 2, 64, 16, [4000, 100, 2500])
    q = torch.from_numpy(g.normal(size=(3, 8, 64)).astype(np.float32)).half().to(dev)
    ws = workspace(lsb.ls_paged_attention_workspace_size(3, 8, 2, 64), dev)
    length = torch.tensor(c.lens, dtype=torch.int32, device=dev)
    outs = [torch.empty_like(q) for _ in range(20)]
    pages = c.pages()
    for o in outs:
        lsb.check(lsb.ls_paged_attention(q, pages, length, o, ws))
    for o in outs[1:]:
        assert torch.equal(o, outs[0])


def test_captured(dev):
    """Captured, and replayed with other lengths and another table in the same tensors."""
    g = np.random.default_rng(12)
    a, b = Cache(g, dev, "e4m3", 2, 128, 16, [700, 30, 0]), Cache(g, dev, "e4m3", 2, 128, 16, [10, 600, 333])
    q = torch.from_numpy(g.normal(size=(3, 16, 128)).astype(np.float32)).bfloat16().to(dev)
    ws = workspace(lsb.ls_paged_attention_workspace_size(3, 16, 2, 128), dev)
    wide = max(a.table.shape[1], b.table.shape[1])
    num = max(a.key.shape[0], b.key.shape[0])
    key = torch.zeros((num, 2, 16, 128), dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
    value = key.clone()
    ks, vs = torch.zeros((num, 2, 16), device=dev), torch.zeros((num, 2, 16), device=dev)
    table, length = torch.zeros((3, wide), dtype=torch.int32, device=dev), torch.zeros(3, dtype=torch.int32, device=dev)
    out = torch.empty_like(q)
    pages = lsb.ls_pages(key, value, table, ks, vs)

    def fill(c):
        n = c.key.shape[0]
        key.view(torch.uint8)[:n].copy_(c.key.view(torch.uint8))
        value.view(torch.uint8)[:n].copy_(c.value.view(torch.uint8))
        ks[:n].copy_(c.key_scale)
        vs[:n].copy_(c.value_scale)
        table[:, :c.table.shape[1]].copy_(c.table)
        length.copy_(torch.tensor(c.lens, dtype=torch.int32))

    fill(a)
    lsb.check(lsb.ls_paged_attention(q, pages, length, out, ws))
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        lsb.check(lsb.ls_paged_attention(q, pages, length, out, ws))
    for c in (b, a, b):
        fill(c)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        lsb.check(lsb.ls_paged_attention(q, c.pages(), torch.tensor(c.lens, dtype=torch.int32, device=dev), out, ws))
        assert torch.equal(got, out)
    assert lsb.ls_read_status(ws) == 0
