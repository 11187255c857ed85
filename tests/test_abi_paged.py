"""Host-side checks of the paged cache's and the filtered sampler's entry points (no GPU): workspace sizes and every
refusal, all found before any CUDA call."""
import pytest

E, UNSUPPORTED = 1, 2
P = 4096  # never dereferenced


@pytest.fixture(scope="module")
def lsb():
    from serving_ls_beam_gb300 import _build

    _build.build()
    import serving_ls_beam_gb300 as m

    m.load_library()
    return m


def view(lsb, data=P, row=64, pos=64, head=8):
    return lsb._View(data, 0, row, pos, head)


def pages(lsb, dtype=3, key=None, value=None, ks=None, vs=None, table=P, table_row=4, num=8, size=16, most=4, heads=2, dim=8):
    v = lambda x, data: x if x is not None else view(lsb, data=data)  # noqa: E731
    return lsb._Pages(v(key, P), v(value, 2 * P), v(ks, 3 * P), v(vs, 4 * P), table, table_row, dtype, num, size, most, heads, dim)


def test_workspace_size(lsb):
    size = lsb.ls_paged_attention_workspace_size
    assert size(4, 16, 16, 64) > 0
    assert size(4, 16, 16, 64) == size(4000, 16, 16, 64)  # rows do not matter
    assert size(4, 16, 16, 64) < size(4, 32, 16, 64) < size(4, 32, 16, 128)
    assert size(4, 16, 1, 64) == size(4, 160, 1, 64)  # more than 16 queries per key head share what 16 have
    assert size(4, 16, 5, 64) == size(4, 16, 16, 257) == size(-1, 16, 16, 64) == size(4, 0, 1, 64) == size(4, 16, 16, 0) == 0


def bad_pages(lsb, written):
    yield pages(lsb, dtype=5)
    yield pages(lsb, dtype=0)  # f32 pages with f16 tensors
    yield pages(lsb, num=-1)
    yield pages(lsb, size=0)
    yield pages(lsb, most=-1)
    yield pages(lsb, heads=0)
    yield pages(lsb, dim=0)
    yield pages(lsb, dim=257)
    yield pages(lsb, key=view(lsb, data=None))
    yield pages(lsb, value=view(lsb, data=None))
    yield pages(lsb, dtype=1, key=view(lsb, data=P + 1))
    yield pages(lsb, key=view(lsb, row=-1))
    yield pages(lsb, key=view(lsb, pos=1 << 62))
    yield pages(lsb, ks=view(lsb, data=None))
    yield pages(lsb, vs=view(lsb, data=P + 2))
    yield pages(lsb, table=None)
    yield pages(lsb, table=P + 2)
    yield pages(lsb, table_row=-1)
    if written:
        yield pages(lsb, key=view(lsb, row=0))
        yield pages(lsb, value=view(lsb, pos=0))
        yield pages(lsb, ks=view(lsb, head=0))
        yield pages(lsb, value=view(lsb, data=P))  # one tensor given as both
        yield pages(lsb, vs=view(lsb, data=3 * P))


def test_write_and_read_refusals(lsb):
    L = lsb.load_library()

    def write(g=None, key=None, value=None, dtype=1, start=P, count=P, rows=2, tokens=3, ws=None):
        v = view(lsb)
        return L.ls_paged_write(key or v, value or v, dtype, start, count, g or pages(lsb), rows, tokens, ws, None)

    def read(g=None, key=None, value=None, dtype=1, start=P, count=P, rows=2, tokens=3, ws=None):
        return L.ls_paged_read(g or pages(lsb), start, count, key or view(lsb), value or view(lsb, data=2 * P), dtype, rows, tokens,
                               ws, None)

    for i, g in enumerate(bad_pages(lsb, True)):
        assert write(g) == E, i
    for i, g in enumerate(bad_pages(lsb, False)):
        assert read(g) == E, i
    for call in (write, read):
        assert call(dtype=3) == E and call(dtype=-1) == E and call(dtype=7) == E
        assert call(rows=-1) == E and call(tokens=-1) == E
        assert call(key=view(lsb, data=None)) == E and call(value=view(lsb, data=P + 1)) == E
        assert call(key=view(lsb, head=-2)) == E and call(value=view(lsb, row=1 << 62)) == E
        assert call(start=P + 1) == E and call(count=P + 2) == E and call(ws=P + 64) == E
        assert call(rows=0) == 0 and call(tokens=0) == 0
        assert call(rows=1 << 20, tokens=1 << 20) == UNSUPPORTED
        assert call(pages(lsb, size=1 << 20, most=1 << 12)) == UNSUPPORTED
    assert write(start=None) == E
    assert read(key=view(lsb, pos=0)) == E and read(value=view(lsb, data=P)) == E


def test_attention_refusals(lsb):
    L = lsb.load_library()

    def call(g=None, q=None, out=None, lens=P, dtype=1, scale=1.0, rows=2, heads=4, ws=P, size=1 << 30):
        return L.ls_paged_attention(q or view(lsb), g or pages(lsb), lens, dtype, scale, rows, heads, out or view(lsb), ws, size, None)

    for i, g in enumerate(bad_pages(lsb, False)):
        assert call(g) == E, i
    assert call(dtype=3) == E and call(dtype=9) == E and call(rows=-1) == E
    assert call(heads=3) == E and call(heads=0) == E
    assert call(scale=float("nan")) == E and call(scale=float("-inf")) == E
    assert call(lens=None) == E and call(lens=P + 1) == E
    assert call(q=view(lsb, data=None)) == E and call(out=view(lsb, data=P + 1)) == E
    assert call(out=view(lsb, row=0)) == E and call(out=view(lsb, head=0)) == E
    assert call(ws=None) == E and call(ws=P + 16) == E and call(size=4096) == E
    assert call(rows=0) == 0
    assert call(rows=1 << 30) == UNSUPPORTED
    assert call(pages(lsb, heads=1), rows=(1 << 31) - 1000, heads=1) == UNSUPPORTED  # the walks over rows go on by up to 128
    assert call(pages(lsb, size=1 << 16, most=1 << 15)) == UNSUPPORTED


def test_sample_refusals(lsb):
    L = lsb.load_library()

    def call(logits=P, dtype=1, stride=100, bias=None, u=P, t=P, k=P, p=P, m=P, rows=2, vocab=100, token=P, logprob=P, ws=None):
        return L.ls_sample_filtered(logits, dtype, stride, bias, u, t, k, p, m, rows, vocab, token, logprob, ws, None)

    assert call(dtype=3) == E and call(dtype=-1) == E
    assert call(rows=-1) == E and call(vocab=0) == E and call(vocab=(1 << 28) + 1, stride=1 << 29) == E
    assert call(logits=None) == E and call(logits=P + 1) == E and call(stride=99) == E and call(stride=1 << 62) == E
    assert call(u=None) == E and call(token=None) == E and call(ws=P + 8) == E
    for name in ("bias", "u", "t", "k", "p", "m", "token", "logprob"):
        assert call(**{name: P + 1}) == E, name
    assert call(rows=0) == 0
    assert call(rows=1 << 30) == UNSUPPORTED


def test_python_shape_checks(lsb):
    torch = pytest.importorskip("torch")
    f = lambda *s, dt=torch.float16: torch.zeros(s, dtype=dt)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    c = lambda *s: f(*s).to(torch.float8_e4m3fn)  # noqa: E731
    s = lambda *s_: f(*s_, dt=torch.float32)  # noqa: E731
    g = lsb.ls_pages(c(8, 2, 16, 64), c(8, 2, 16, 64), i(3, 4), s(8, 2, 16), s(8, 2, 16))
    h = lsb.ls_pages(f(8, 2, 16, 64), f(8, 2, 16, 64), i(3, 4))
    for bad in (lambda: lsb.ls_pages(c(8, 2, 16, 64), c(8, 2, 16, 64), i(3, 4)),
                lambda: lsb.ls_pages(f(8, 2, 16, 64), f(8, 2, 16, 64), i(3, 4), s(8, 2, 16), s(8, 2, 16)),
                lambda: lsb.ls_pages(f(8, 2, 16, 64), f(8, 2, 16, 32), i(3, 4)),
                lambda: lsb.ls_pages(f(8, 2, 16, 64), f(8, 2, 16, 64), i(3, 4).long()),
                lambda: lsb.ls_pages(f(8, 2, 64, 16).transpose(2, 3), f(8, 2, 16, 64), i(3, 4)),
                lambda: lsb.ls_pages(f(8, 2, 16, 64), f(8, 2, 16, 64), i(4, 3).t()),
                lambda: lsb.ls_pages(c(8, 2, 16, 64), c(8, 2, 16, 64), i(3, 4), s(8, 2, 15), s(8, 2, 16)),
                lambda: lsb.ls_paged_write(f(3, 1, 2, 64), f(3, 1, 2, 32), i(3), None, g),
                lambda: lsb.ls_paged_write(f(2, 1, 2, 64), f(2, 1, 2, 64), i(3), None, g),
                lambda: lsb.ls_paged_write(f(3, 1, 2, 64), f(3, 1, 2, 64), i(2), None, g),
                lambda: lsb.ls_paged_write(f(3, 1, 2, 64).float(), f(3, 1, 2, 64).float(), i(3), None, h),
                lambda: lsb.ls_paged_read(g, i(3), i(3).long(), f(3, 1, 2, 64), f(3, 1, 2, 64)),
                lambda: lsb.ls_paged_attention(f(3, 5, 64), g, i(3), f(3, 5, 64), i(4)),
                lambda: lsb.ls_paged_attention(f(3, 4, 64), g, i(2), f(3, 4, 64), i(4)),
                lambda: lsb.ls_paged_attention(f(3, 4, 64).bfloat16(), h, i(3), f(3, 4, 64).bfloat16(), i(4)),
                lambda: lsb.ls_sample_filtered(f(3, 9), None, s(3), s(2), None, None, None, i(3)),
                lambda: lsb.ls_sample_filtered(f(3, 9), s(8), s(3), None, None, None, None, i(3)),
                lambda: lsb.ls_sample_filtered(f(3, 9), None, s(3), None, s(3), None, None, i(3)),
                lambda: lsb.ls_sample_filtered(f(9, 3).t(), None, s(3), None, None, None, None, i(3))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        lsb.ls_pages(f(8, 2, 16, 64).double(), f(8, 2, 16, 64).double(), i(3, 4))
    with pytest.raises(TypeError):
        lsb.ls_paged_write(f(3, 1, 2, 64).double(), f(3, 1, 2, 64).double(), i(3), None, g)
