"""Host-side checks of the attention and commit entry points (no GPU): workspace sizes and
every refusal, all found before any CUDA call."""
import ctypes

import pytest

E, UNSUPPORTED = 1, 2


@pytest.fixture(scope="module")
def lsb():
    from serving_ls_beam_gb300 import _build

    _build.build()
    import serving_ls_beam_gb300 as m

    m.load_library()
    return m


P = 4096  # never dereferenced


def view(lsb, data=P, row=64, pos=64, head=8, layer=0):
    return lsb._View(data, layer, row, pos, head)


def test_workspace_sizes(lsb):
    cross, tree = lsb.ls_cross_attention_workspace_size, lsb.ls_tree_attention_workspace_size
    assert cross(4, 4, 1, 16, 16, 100, 64) > 0
    assert cross(4, 4, 1, 16, 16, 100, 64) == cross(400, 4, 1, 16, 16, 100000, 64)  # rows and length do not matter
    assert cross(4, 4, 1, 16, 16, 100, 64) < cross(4, 8, 1, 16, 16, 100, 64) <= cross(4, 8, 500, 16, 16, 100, 64)
    assert cross(4, 4, 1, 16, 16, 100, 64) < cross(4, 4, 1, 16, 16, 100, 65)
    assert cross(4, 1, 4, 16, 16, 100, 64) == tree(4, 4, 16, 16, 100, 64)
    assert cross(4, 4, 1, 16, 5, 100, 64) == 0
    assert cross(4, 0, 1, 16, 16, 100, 64) == 0
    assert cross(4, 4, 1, 16, 16, 100, 257) == 0
    assert tree(4, 0, 16, 16, 100, 64) == 0 and tree(4, 65, 16, 16, 100, 64) == 0


def test_cross_refusals(lsb):
    L = lsb.load_library()
    big = 1 << 30

    def call(q=None, key=None, value=None, dtype=1, lens=P, scale=1.0, b=2, k=4, t=1, h=8, hk=8, n=16, d=8, out=None,
             ws=P, size=big):
        vs = [x if x is not None else view(lsb) for x in (q, key, value, out)]
        return L.ls_cross_attention(vs[0], vs[1], vs[2], dtype, lens, scale, b, k, t, h, hk, n, d, vs[3], ws, size, None)

    assert call(dtype=7) == E
    assert call(b=-1) == E and call(k=0) == E and call(t=-1) == E and call(n=-1) == E
    assert call(h=8, hk=3) == E and call(hk=0) == E
    assert call(d=0) == E and call(d=257) == E
    assert call(scale=float("nan")) == E and call(scale=float("inf")) == E
    assert call(lens=None) == E and call(lens=P + 2) == E
    assert call(ws=None) == E and call(ws=P + 16) == E and call(size=256) == E
    assert call(q=view(lsb, data=None)) == E and call(key=view(lsb, data=None)) == E
    assert call(value=view(lsb, data=P + 1)) == E and call(out=view(lsb, data=None)) == E
    assert call(q=view(lsb, row=-1)) == E and call(key=view(lsb, pos=1 << 62)) == E
    assert call(out=view(lsb, row=0)) == E and call(out=view(lsb, head=0)) == E
    assert call(b=0) == 0 and call(t=0) == 0
    assert call(b=1 << 30, k=8) == UNSUPPORTED
    assert call(b=1, k=1 << 30, t=1 << 30, h=8, hk=1) == UNSUPPORTED  # queries that no 64-bit product holds
    assert lsb.ls_cross_attention_workspace_size(1, 1 << 30, 1 << 30, 1 << 10, 1, 5, 64) == 0


def test_tree_refusals(lsb):
    L = lsb.load_library()

    def call(nodes=4, rows=2, h=8, hk=8, n=16, d=8, dtype=2, lens=P, parent=P, ws=P, dk=None, scale=1.0, size=1 << 30):
        v = view(lsb)
        return L.ls_tree_attention(v, v, v, lens, dk if dk is not None else v, v, parent, dtype, scale, rows, nodes, h, hk,
                                   n, d, v, ws, size, None)

    assert call(nodes=0) == E and call(nodes=65) == E and call(rows=-1) == E
    assert call(h=6, hk=4) == E and call(d=300) == E and call(dtype=-1) == E and call(n=-2) == E
    assert call(lens=None) == E and call(parent=None) == E and call(parent=P + 1) == E
    assert call(dk=view(lsb, data=None)) == E and call(ws=None) == E and call(size=0) == E
    assert call(scale=float("nan")) == E
    assert call(rows=0) == 0


def test_commit_refusals(lsb):
    L = lsb.load_library()

    def call(ck=P, cv=2 * P, lens=P, dtype=1, parent=P, token=P, target=P, layers=1, rows=2, nodes=4, heads=2, n=8, d=8,
             out_len=2 * P, path=P, count=P, tok=P, ws=None, dk=None):
        v = view(lsb)
        return L.ls_tree_commit(ck, cv, lens, dk if dk is not None else v, v, dtype, parent, token, target, None, 2, layers,
                                rows, nodes, heads, n, d, out_len, path, count, tok, None, ws, None)

    assert call(ck=None) == E and call(cv=P) == E  # one cache given as both
    assert call(ck=P + 1) == E and call(dtype=3) == E
    assert call(nodes=0) == E and call(nodes=65) == E and call(rows=-1) == E and call(layers=-1) == E
    assert call(heads=-1) == E and call(n=-1) == E and call(d=-1) == E
    for name in ("lens", "parent", "token", "target", "path", "count", "tok"):
        assert call(**{name: None}) == E, name
    assert call(out_len=P) == E  # cache_len itself
    assert call(ws=P + 8) == E and call(dk=view(lsb, data=None)) == E
    assert call(rows=0) == 0


def test_python_shape_checks(lsb):
    torch = pytest.importorskip("torch")
    f = lambda *s, dt=torch.float16: torch.zeros(s, dtype=dt)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    ws = torch.zeros(16, dtype=torch.uint8)
    q, k = f(2, 4, 1, 8, 64), f(2, 8, 5, 64)
    with pytest.raises(ValueError):
        lsb.ls_cross_attention(q, k, f(2, 8, 6, 64), i(2), q, ws)
    with pytest.raises(ValueError):
        lsb.ls_cross_attention(q, k, k, i(3), q, ws)
    with pytest.raises(ValueError):
        lsb.ls_cross_attention(q, k, k.float(), i(2), q, ws)
    with pytest.raises(ValueError):
        lsb.ls_cross_attention(q, k, k, i(2).long(), q, ws)
    with pytest.raises(ValueError):  # batch and k do not form one dimension
        lsb.ls_cross_attention(f(4, 2, 1, 8, 64).transpose(0, 1), k, k, i(2), q, ws)
    with pytest.raises(ValueError):  # the last dimension is not contiguous
        lsb.ls_cross_attention(f(2, 4, 1, 64, 8).transpose(3, 4), k, k, i(2), q, ws)
    with pytest.raises(TypeError):
        lsb.ls_cross_attention(q.double(), k.double(), k.double(), i(2), q.double(), ws)
    t = f(2, 3, 8, 64)
    with pytest.raises(ValueError):
        lsb.ls_tree_attention(t, k, k, i(2), f(2, 4, 8, 64), f(2, 4, 8, 64), i(2, 3), t, ws)
    c, d = f(1, 2, 8, 5, 64), f(1, 2, 3, 8, 64)
    with pytest.raises(ValueError):
        lsb.ls_tree_commit(c.transpose(2, 3), c.transpose(2, 3), i(2), d, d, i(2, 3), i(2, 3), i(2, 3), None, 2, i(2),
                           i(2, 3), i(2), i(2))
