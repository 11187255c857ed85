"""Writing into and reading from a paged cache on the GPU, bit by bit against the definition: types, head sizes, layouts,
page sizes, ragged counts, positions and pages out of range, what must stay as it was."""
import numpy as np
import pytest

import paged_plain as pp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import serving_ls_beam_gb300 as lsb  # noqa: E402

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lsb.load_library()
    return torch.device("cuda:0")


def workspace(dev):
    ws = torch.empty(1024, dtype=torch.uint8, device=dev)
    lsb.check(lsb.ls_workspace_init(ws))
    return ws


def raw(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


class Cache:
    """Pages of random bytes (of finite values where they are not 8-bit ones), for `rows` rows of up to `length` positions."""

    def __init__(self, g, dev, cache, rows, heads, dim, page, length, order="head", spare=2, odd=0):
        need = -(-length // page)
        num = rows * need + spare
        self.table = torch.from_numpy(g.permutation(num)[:rows * need].reshape(rows, need).astype(np.int32)).to(dev)
        self.coded = cache in ("e4m3", "i8")
        shape = (num, heads, page, dim + odd) if order == "head" else (num, page, heads, dim + odd)
        self.key, self.value, self.key_scale, self.value_scale = None, None, None, None
        for name in ("key", "value"):
            t = torch.from_numpy(g.normal(size=shape).astype(np.float32)).to(dev)
            t = (t * 50).round().to(DT[cache]) if cache == "i8" else t.to(DT[cache])
            t = t if order == "head" else t.transpose(1, 2)
            setattr(self, name, t[..., :dim])
            if self.coded:
                s = torch.from_numpy(2.0 ** g.integers(-9, 3, (num, heads, page)).astype(np.float32)).to(dev)
                if cache == "i8":
                    s *= 1.37
                setattr(self, name + "_scale", s)
        self.page, self.num = page, num

    def pages(self):
        return lsb.ls_pages(self.key, self.value, self.table, self.key_scale, self.value_scale)

    def where(self, r, n):
        return pp.place(self.table.cpu().numpy(), self.page, self.num, r, n)


def values(g, shape, dtype, dev, odd=0):
    x = g.normal(size=shape[:-1] + (shape[-1] + odd,)) * 2.0 ** g.integers(-6, 7, shape[:-1] + (1,))
    x.reshape(-1, x.shape[-1])[::7] = 0.0
    return torch.from_numpy(x.astype(np.float32)).to(DT[dtype]).to(dev)[..., :shape[-1]]


def check_write(dev, dtype, cache, rows, tokens, heads, dim, page, start, count, order="head", seed=0, status=0, odd=0, spoil=None):
    g = np.random.default_rng(seed)
    length = max(s + tokens for s in start)
    c = Cache(g, dev, cache, rows, heads, dim, page, max(length, 1), order, odd=odd)
    if spoil:
        spoil(c)
    key, value = values(g, (rows, tokens, heads, dim), dtype, dev, odd), values(g, (rows, tokens, heads, dim), dtype, dev, odd)
    want = {n: getattr(c, n).contiguous().clone() for n in ("key", "value", "key_scale", "value_scale") if getattr(c, n) is not None}
    for name, x in (("key", key), ("value", value)):
        x64 = x.float().cpu().numpy().astype(np.float64)
        for r in range(rows):
            for i in range(min(count[r] if count is not None else tokens, tokens)):
                at = c.where(r, start[r] + i)
                if at is None:
                    continue
                if c.coded:
                    codes, s = pp.quantise(x64[r, i], cache)
                    want[name][at[0], :, at[1]] = torch.from_numpy(codes.astype(np.float32)).to(DT[cache]).to(dev)
                    want[name + "_scale"][at[0], :, at[1]] = torch.from_numpy(s.astype(np.float32)).to(dev)
                else:
                    want[name][at[0], :, at[1]] = x[r, i]
    ws = workspace(dev)
    ints = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    lsb.check(lsb.ls_paged_write(key, value, ints(start), ints(count), c.pages(), ws))
    assert lsb.ls_read_status(ws) == status
    for n, t in want.items():
        got = getattr(c, n)
        # (a zero keeps its sign in e4m3, the definition's has none)
        same = raw(got) == raw(t)
        if cache == "e4m3" and n in ("key", "value"):
            same |= (raw(got) & 0x7f) + (raw(t) & 0x7f) == 0
        assert same.all(), (n, np.argwhere(~same)[:5].tolist())


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cache", ["same", "e4m3", "i8"])
@pytest.mark.parametrize("heads,dim,page,order", [(4, 64, 16, "head"), (3, 128, 64, "token"), (2, 256, 8, "head"), (5, 32, 1, "head"),
                                                  (1, 80, 24, "token"), (2, 1, 16, "head"), (2, 200, 16, "head"), (3, 33, 5, "token")])
def test_write(dev, dtype, cache, heads, dim, page, order):
    check_write(dev, dtype, dtype if cache == "same" else cache, 4, 9, heads, dim, page, [0, 5, 31, 64], [9, 1, 0, 7], order, seed=dim)


@pytest.mark.parametrize("cache", ["f16", "e4m3", "i8"])
def test_write_single_tokens(dev, cache):
    check_write(dev, "f16", cache, 37, 1, 16, 64, 16, [7 * i % 90 for i in range(37)], None, seed=3)


@pytest.mark.parametrize("cache", ["bf16", "e4m3", "i8"])
def test_write_out_of_range(dev, cache):
    """Counts outside [0, tokens], positions outside the table and pages that do not exist: left out, and reported."""
    check_write(dev, "bf16", cache, 3, 4, 2, 64, 8, [0, 3, 9], [4, -1, 4], status=5)
    check_write(dev, "bf16", cache, 3, 4, 2, 64, 8, [0, 3, 9], [4, 4, 9], status=5)
    check_write(dev, "bf16", cache, 2, 4, 2, 64, 8, [-2, 3], None, status=5)

    def shorter(c):
        c.table = c.table[:, :1].contiguous()
    check_write(dev, "bf16", cache, 2, 4, 2, 64, 8, [6, 3], None, status=5, spoil=shorter)

    def bad(c):
        c.table[0, 1], c.table[1, 0] = -1, c.num
    check_write(dev, "bf16", cache, 2, 4, 2, 64, 8, [6, 3], None, status=5, spoil=bad)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cache", ["same", "e4m3", "i8"])
def test_write_unaligned_rows(dev, dtype, cache):
    """Strides that are no multiples of 16 bytes."""
    check_write(dev, dtype, dtype if cache == "same" else cache, 2, 3, 2, 64, 16, [0, 5], None, odd=1)


def test_write_extremes(dev):
    """The largest and smallest elements of each type, all equal ones, and values at the borders between codes."""
    g = np.random.default_rng(1)
    for dtype, cache in [("f32", "e4m3"), ("f32", "i8"), ("bf16", "e4m3"), ("bf16", "i8"), ("f16", "e4m3"), ("f16", "i8")]:
        top = float(torch.finfo(DT[dtype]).max)
        rows = [np.zeros(64), np.full(64, top), np.full(64, -top), np.full(64, 2.0 ** -24 if dtype == "f16" else 2.0 ** -133),
                np.linspace(-127, 127, 64), np.arange(64) - 31.5, np.concatenate([[448.0], (np.arange(63) + 0.5) / 8]),
                np.concatenate([[127.0], np.arange(63) + 0.5]), np.concatenate([[12.7], g.integers(-127, 127, 63) / 10 + 0.05]),
                g.normal(size=64), np.full(64, 449.0 * 2.0 ** 3), np.full(64, 448.0 * 2.0 ** 3)]
        x = torch.from_numpy(np.array(rows, np.float64)).to(DT[dtype]).to(dev).view(1, len(rows), 1, 64)
        c = Cache(g, dev, cache, 1, 1, 64, 16, len(rows))
        ws = workspace(dev)
        lsb.check(lsb.ls_paged_write(x, x.clone(), torch.zeros(1, dtype=torch.int32, device=dev), None, c.pages(), ws))
        assert lsb.ls_read_status(ws) == 0
        codes, s = pp.quantise(x.double().cpu().numpy()[0, :, 0], cache)
        for i in range(len(rows)):
            at = c.where(0, i)
            assert np.array_equal(c.key[at[0], 0, at[1]].float().cpu().numpy(), codes[i].astype(np.float32)), (dtype, cache, i)
            assert float(c.key_scale[at[0], 0, at[1]]) == s[i], (dtype, cache, i)


def check_read(dev, dtype, cache, rows, tokens, heads, dim, page, start, count, order="head", seed=0, status=0, odd=0, spoil=None):
    g = np.random.default_rng(seed)
    c = Cache(g, dev, cache, rows, heads, dim, page, max(max((start or [0] * rows)[r] + tokens for r in range(rows)), 1), order, odd=odd)
    if spoil:
        spoil(c)
    outs = [values(g, (rows, tokens, heads, dim), dtype, dev, odd) for _ in range(2)]
    want = [o.clone() for o in outs]
    for w, name in zip(want, ("key", "value")):
        codes, scale = getattr(c, name), getattr(c, name + "_scale")
        for r in range(rows):
            for i in range(min(count[r] if count is not None else tokens, tokens)):
                at = c.where(r, (start[r] if start else 0) + i)
                if at is not None:
                    x = codes[at[0], :, at[1]]
                    w[r, i] = (x.float() * scale[at[0], :, at[1]][:, None]).to(DT[dtype]) if c.coded else x
    ws = workspace(dev)
    ints = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    lsb.check(lsb.ls_paged_read(c.pages(), ints(start), ints(count), outs[0], outs[1], ws))
    assert lsb.ls_read_status(ws) == status
    for o, w in zip(outs, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("cache", ["same", "e4m3", "i8"])
@pytest.mark.parametrize("heads,dim,page,order", [(4, 64, 16, "head"), (3, 128, 64, "token"), (2, 256, 8, "head"), (1, 80, 1, "head"),
                                                  (2, 1, 16, "token"), (2, 100, 7, "head")])
def test_read(dev, dtype, cache, heads, dim, page, order):
    check_read(dev, dtype, dtype if cache == "same" else cache, 4, 21, heads, dim, page, [0, 5, 31, 3], [21, 1, 0, 20], order, seed=dim)
    check_read(dev, dtype, dtype if cache == "same" else cache, 2, 5, heads, dim, page, None, None, order, seed=dim, odd=1)


def test_read_out_of_range(dev):
    for cache in ("f16", "e4m3"):
        check_read(dev, "f16", cache, 3, 4, 2, 64, 8, [0, 3, 9], [4, -7, 5], status=5)
        check_read(dev, "f16", cache, 2, 4, 2, 64, 8, [-3, 2], None, status=5)

        def bad(c):
            c.table[0, 0], c.table[1, 0] = c.num, -5
        check_read(dev, "f16", cache, 2, 12, 2, 64, 8, None, None, status=5, spoil=bad)


def test_positions_near_the_end_of_32_bits(dev):
    g = np.random.default_rng(0)
    c = Cache(g, dev, "e4m3", 2, 2, 64, 8, 16)
    before = raw(c.key)
    x = values(g, (2, 4, 2, 64), "f16", dev)
    ws = workspace(dev)
    start = torch.tensor([2 ** 31 - 2, -2 ** 31], dtype=torch.int32, device=dev)
    lsb.check(lsb.ls_paged_write(x, x.clone(), start, None, c.pages(), ws))
    assert lsb.ls_read_status(ws) == 5 and np.array_equal(before, raw(c.key))


def test_no_pages_and_no_workspace(dev):
    key = torch.empty((0, 2, 16, 64), dtype=torch.float16, device=dev)
    table = torch.zeros((3, 0), dtype=torch.int32, device=dev)
    x = torch.zeros((3, 2, 2, 64), dtype=torch.float16, device=dev)
    ws = workspace(dev)
    pages = lsb.ls_pages(key, key.clone(), table)
    lsb.check(lsb.ls_paged_write(x, x.clone(), torch.zeros(3, dtype=torch.int32, device=dev), None, pages, ws))
    assert lsb.ls_read_status(ws) == 5
    lsb.check(lsb.ls_paged_write(x, x.clone(), torch.zeros(3, dtype=torch.int32, device=dev), None, pages))
    lsb.check(lsb.ls_paged_read(pages, None, torch.zeros(3, dtype=torch.int32, device=dev), x, x.clone(), ws))
    assert lsb.ls_read_status(ws) == 0


def test_past_4_gib(dev):
    """Pages whose bytes lie past 32 bits of offset."""
    g = np.random.default_rng(7)
    heads, page, dim = 8, 64, 128
    num = (5 << 30) // (heads * page * dim)
    key = torch.zeros((num, heads, page, dim), dtype=torch.float8_e4m3fn, device=dev)
    value = torch.zeros_like(key)
    ks, vs = torch.zeros((num, heads, page), device=dev), torch.zeros((num, heads, page), device=dev)
    table = torch.tensor([[num - 1, 0], [3, num - 2]], dtype=torch.int32, device=dev)
    pages = lsb.ls_pages(key, value, table, ks, vs)
    x = values(g, (2, 70, heads, dim), "bf16", dev)
    y = values(g, (2, 70, heads, dim), "bf16", dev)
    ws = workspace(dev)
    lsb.check(lsb.ls_paged_write(x, y, torch.tensor([1, 2], dtype=torch.int32, device=dev), None, pages, ws))
    back = [torch.zeros_like(x), torch.zeros_like(x)]
    lsb.check(lsb.ls_paged_read(pages, torch.tensor([1, 2], dtype=torch.int32, device=dev), None, back[0], back[1], ws))
    assert lsb.ls_read_status(ws) == 0
    for a, b in zip(back, (x, y)):
        codes, s = pp.quantise(b.double().cpu().numpy(), "e4m3")
        want = torch.from_numpy(codes * s[..., None]).to(torch.bfloat16)
        assert torch.equal(a.cpu(), want)
