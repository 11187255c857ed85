"""The paged cache's and the filters' definitions against other ways to the same values (no GPU)."""
import numpy as np
import pytest

import paged_plain as pp

torch = pytest.importorskip("torch")


def test_e4m3_is_the_types_rounding():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    held = np.unique(codes[np.isfinite(codes)])
    assert held.max() == 448.0
    x = np.concatenate([held, (held[1:] + held[:-1]) / 2, np.random.default_rng(0).uniform(-448, 448, 4000),
                        np.random.default_rng(1).normal(size=4000) * 2.0 ** -6])
    assert np.array_equal(pp.e4m3_round(x), torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy())


@pytest.mark.parametrize("cache,most,step", [("e4m3", 448.0, 2.0 ** -4), ("i8", 127.0, 0.5 / 127)])
def test_quantised_values_are_near(cache, most, step):
    x = np.random.default_rng(2).normal(size=(300, 64)).astype(np.float32).astype(np.float64)
    x *= 2.0 ** np.random.default_rng(3).integers(-40, 40, (300, 1))
    x[0] = 0
    x[1] = 2.0 ** -140
    codes, s = pp.quantise(x, cache)
    assert np.abs(codes).max() <= most and (s >= 2.0 ** -126).all()
    a = np.abs(x).max(axis=1, keepdims=True)
    off = np.abs(codes * s[:, None] - x)[2:]
    assert (off <= (step * np.abs(x[2:]) + 2.0 ** -10 * s[2:, None] if cache == "e4m3" else 1.0001 * step * a[2:])).all()
    if cache == "e4m3":  # the least power of two that holds the largest element
        assert (a[2:, 0] <= 448 * s[2:]).all() and (a[2:, 0] > 224 * s[2:]).all()


def test_sample_by_hand():
    x = np.log(np.array([0.1, 0.4, 0.2, 0.3]))
    draw = lambda u, k=0, p=1.0, m=0.0, t=1.0: pp.sample(x, t, k, p, m, u)[0]  # noqa: E731
    assert [draw(u) for u in (0.0, 0.05, 0.15, 0.55, 0.75, 0.999)] == [0, 0, 1, 2, 3, 3]
    assert [draw(u, k=2) for u in (0.0, 0.5, 0.6, 0.99)] == [1, 1, 3, 3]  # 4/7 and 3/7
    assert {draw(u, p=0.75) for u in np.linspace(0, 0.999, 50)} == {1, 2, 3}
    assert {draw(u, p=0.65) for u in np.linspace(0, 0.999, 50)} == {1, 3}
    assert {draw(u, m=0.6) for u in np.linspace(0, 0.999, 50)} == {1, 3}
    assert {draw(u, m=1.0) for u in np.linspace(0, 0.999, 50)} == {1}
    assert {draw(u, k=3, p=0.7) for u in np.linspace(0, 0.999, 50)} == {1, 3}  # 0.7 of the first three's 0.9
    assert draw(0.9, t=0.0) == 1
    assert abs(pp.sample(x, 1.0, 2, 1.0, 0.0, 0.0)[1] - np.log(4 / 7)) < 1e-12
    assert pp.sample(np.full(3, -np.inf), 1.0, 0, 1.0, 0.0, 0.5)[0] == -1
    assert pp.sample(np.array([1.0, 1.0, 1.0]), 1.0, 2, 1.0, 0.0, 0.75)[0] == 1  # ties: the smaller tokens


def test_attend_against_torch():
    g = np.random.default_rng(5)
    q, k, v = g.normal(size=16), g.normal(size=(40, 16)), g.normal(size=(40, 16))
    o, bound = pp.attend(q, k, v, np.ones(40), 0.25, "f32", "f32")
    t = torch.softmax(torch.from_numpy(k @ q * 0.25), 0) @ torch.from_numpy(v)
    assert np.allclose(o, t.numpy(), atol=1e-12) and (bound > 0).all()
