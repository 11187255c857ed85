"""One key that outweighs every other, and a long flat tail under it: the tail's small weights have to
count, above all where the large one's value is zero and the tail makes up the whole output.

Error bound of an output element, from the arithmetic (u: the type's unit roundoff, e = 2^-24, weights p_n
relative to the largest, L = sum_n p_n, W = sum_n p_n |v_n| / L):

- scores and exponents as in attention_plain: a weight is off by 2 ds relatively, the sums by (n + 16) e,
  each in numerator and denominator;
- weights rounded to the type: u W.  In f16 a row's largest weight is 2^7 or more in the scale in which they
  are rounded, and f16 rounds to multiples of 2^-24 below its normal numbers: at most 2^-25 a key there,
  2^-32 of the largest weight, so 2^-32 sum_n |v_n| / L together;
- the output's own rounding: u |o|, and 2^-25 for f16's subnormal numbers."""
import numpy as np
import pytest

import attention_plain as ap

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_attention import DT, KERNELS, f64, run_cross, run_tree  # noqa: E402

import serving_ls_beam_gb300 as lsb  # noqa: E402


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


def expected(q, keys, values, scale, dtype):
    n, dim = keys.shape
    s = keys @ q * scale
    p = np.exp(s - s.max())
    L, u = p.sum(), ap.UNIT[dtype]
    o, W = p @ values / L, p @ np.abs(values) / L
    ds = (dim + 2) * ap.E * abs(scale) * (np.abs(keys) @ np.abs(q)).max() + 8 * ap.E * np.abs(s).max() + 2.0 ** -21
    bound = (2 * ds + 2 * (n + 16) * ap.E + u) * W + u * np.abs(o)
    if dtype == "f16":
        bound = bound + 2.0 ** -32 * np.abs(values).sum(axis=0) / L + 2.0 ** -25
    return o, 1.0001 * bound + 1e-30


def close(got, want, bound, where):
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (where, int(bad.sum()), got[bad][:3], want[bad][:3], bound[bad][:3])


def rows(g, n, dim, depth, sink, dev, dtype, heads=2):
    """Keys whose scores lie about `depth` powers of two below the key `sink`'s (against q = [4, 0, ..], scale 1)."""
    k = np.zeros((1, heads, n, dim), np.float32)
    k[..., 0] = g.normal(size=(1, heads, n), scale=0.02)
    k[:, :, sink, 0] = depth * np.log(2.0) / 4
    k[..., 1:] = g.normal(size=(1, heads, n, dim - 1))
    v = (1 + 0.25 * g.normal(size=(1, heads, n, dim))).astype(np.float32)
    v[:, 1, sink] = 3.0
    v[:, 0, sink] = 0.0  # the first head's output is the tail alone
    return torch.from_numpy(k).to(DT[dtype]).to(dev), torch.from_numpy(v).to(DT[dtype]).to(dev)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("depth", [18.0, 25.1, 30.0])
@pytest.mark.parametrize("n,sink", [(400, 0), (400, 399), (5000, 2600)])
@pytest.mark.parametrize("T,D", [(1, 64), (3, 128), (12, 64), (40, 128), (200, 64), (2, 256)])
def test_sink_and_flat_tail(dev, kernel, T, D, n, sink, depth, dtype):
    g = np.random.default_rng(n + T)
    k, v = rows(g, n, D, depth, sink, dev, dtype)
    q = torch.zeros((1, 1, T, 2, D), dtype=DT[dtype], device=dev)
    q[..., 0] = 4.0
    out = f64(run_cross(q, k, v, [n], 1.0))
    assert (out == out[:, :, :1]).all()  # equal queries, equal results
    for h in range(2):
        want, bound = expected(f64(q)[0, 0, 0, h], f64(k)[0, h], f64(v)[0, h], 1.0, dtype)
        close(out[0, 0, 0, h], want, bound, h)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("nodes,D", [(1, 64), (6, 64), (40, 128)])
def test_drafted_sink(dev, kernel, nodes, D, dtype):
    """The outweighing key is a drafted token, the last that a row reads; the tail is its cache."""
    g = np.random.default_rng(nodes)
    n = 3000
    k, v = rows(g, n + nodes, D, 25.1, n, dev, dtype)
    dk, dv = k[:, :, n:].transpose(1, 2), v[:, :, n:].transpose(1, 2)
    q = torch.zeros((1, nodes, 2, D), dtype=DT[dtype], device=dev)
    q[..., 0] = 4.0
    scale = D ** -0.5  # run_tree's
    q *= D ** 0.5 if D == 64 else 8.0  # 8 is exact; at 128 the tail lies 25.1 / 1.41 deep
    out = f64(run_tree(q, k[:, :, :n], v[:, :, :n], [n], dk, dv, np.arange(-1, nodes - 1)[None]))
    for i in {0, nodes // 2, nodes - 1}:
        for h in range(2):
            want, bound = expected(f64(q)[0, i, h], f64(k)[0, h, :n + i + 1], f64(v)[0, h, :n + i + 1], scale, dtype)
            close(out[0, i, h], want, bound, (i, h))
