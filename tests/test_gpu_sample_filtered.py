"""Sampling with filters on the GPU against its float64 definition: the token itself, wherever it does not hang on less than
the kernel's error bound, and the log-probability."""
import numpy as np
import pytest

import paged_plain as pp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import serving_ls_beam_gb300 as lsb  # noqa: E402

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
KERNELS = [None, "sfcluster=1", "sfcluster=2", "sfcluster=8"]


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


def workspace(dev):
    ws = torch.empty(1024, dtype=torch.uint8, device=dev)
    lsb.check(lsb.ls_workspace_init(ws))
    return ws


def run(dev, logits, u, t=None, k=None, p=None, m=None, bias=None, status=0):
    rows = logits.shape[0]
    token = torch.full((rows,), -9, dtype=torch.int32, device=dev)
    logprob = torch.full((rows,), float("nan"), device=dev)
    f = lambda v, dt=torch.float32: None if v is None else torch.as_tensor(np.broadcast_to(np.asarray(v), (rows,)).copy()).to(dt).to(dev)  # noqa: E731
    ws = workspace(dev)
    lsb.check(lsb.ls_sample_filtered(logits, bias, f(u), f(t), f(k, torch.int32), f(p), f(m), token, logprob, ws))
    assert lsb.ls_read_status(ws) == status
    return token.cpu().numpy(), logprob.cpu().numpy()


def check(dev, logits, u, t=None, k=None, p=None, m=None, bias=None, rows=None):
    token, logprob = run(dev, logits, u, t, k, p, m, bias)
    x = logits.float() if bias is None else logits.float() + bias
    x = x.cpu().numpy().astype(np.float64)
    n = logits.shape[0]
    at = lambda v, r, off: off if v is None else float(np.float32(np.broadcast_to(np.asarray(v), (n,))[r]))  # noqa: E731
    unsure = 0
    for r in rows if rows is not None else range(n):
        want, lp, sure = pp.sample(x[r], at(t, r, 1.0), int(at(k, r, 0)), at(p, r, 1.0), at(m, r, 0.0), at(u, r, 0.0))
        if not sure:
            unsure += 1
            continue
        assert token[r] == want, (r, token[r], want, x[r][token[r]], x[r][want])
        assert logprob[r] == lp or abs(logprob[r] - lp) <= 2.0 ** -21 * (1 + abs(lp)), (r, logprob[r], lp)
    assert unsure <= max(1, n // 50)


def normal(g, rows, vocab, dtype, dev, spread=2.0):
    return torch.from_numpy(g.normal(size=(rows, vocab), scale=spread).astype(np.float32)).to(DT[dtype]).to(dev)


FILTERS = [dict(), dict(k=1), dict(k=7), dict(k=50, p=0.9), dict(p=0.9), dict(p=0.3), dict(m=0.05), dict(k=300, p=0.8, m=0.01),
           dict(k=1500), dict(k=900, p=0.95), dict(p=0.99, m=0.001), dict(m=1.0), dict(k=10 ** 6, p=1.0, m=0.0)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("f", FILTERS)
@pytest.mark.parametrize("vocab", [1, 3, 33, 1000, 5003, 40000])
def test_filters(dev, kernel, dtype, f, vocab):
    g = np.random.default_rng(vocab)
    rows = 12 if vocab < 40000 else 5
    check(dev, normal(g, rows, vocab, dtype, dev), g.random(rows), t=g.uniform(0.3, 1.6, rows), **f)


def test_settings_of_each_row(dev, kernel):
    g = np.random.default_rng(1)
    rows = 60
    check(dev, normal(g, rows, 3001, "f16", dev), g.random(rows), t=g.choice([0.0, 0.2, 1.0, 3.0], rows),
          k=g.choice([0, 1, 40, 200, 5000], rows), p=g.choice([0.1, 0.7, 1.0], rows), m=g.choice([0.0, 0.02, 0.5], rows))


@pytest.mark.parametrize("f", [dict(), dict(k=40, p=0.9), dict(p=0.95)])
def test_many_rows(dev, f):
    g = np.random.default_rng(2)
    check(dev, normal(g, 1100, 2000, "bf16", dev), g.random(1100), **f, rows=range(0, 1100, 7))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("f", [dict(), dict(k=3), dict(k=700, p=0.5), dict(p=0.9), dict(k=20000), dict(p=0.9999)])
def test_ties(dev, kernel, dtype, f):
    """Equal values, few and many (more than the list holds): the smaller tokens come first."""
    g = np.random.default_rng(3)
    x = np.zeros((6, 30000), np.float32)
    x[1] = g.integers(0, 3, 30000)
    x[2] = g.integers(-40, 2, 30000) / 4
    x[3, ::2] = -np.inf
    x[4] = -7.25
    x[5, 17:25] = 3.0
    x[5, 100:] = -np.inf
    check(dev, torch.from_numpy(x).to(DT[dtype]).to(dev), g.random(6), **f)


@pytest.mark.parametrize("f", [dict(), dict(k=2), dict(p=0.5), dict(m=0.2), dict(k=600, p=0.7)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_masked_rows(dev, kernel, dtype, f):
    """-inf, NaN and the type's lowest value in masked places; rows with one token left, and with none."""
    g = np.random.default_rng(4)
    x = g.normal(size=(8, 1501)).astype(np.float32)
    low = float(torch.finfo(DT[dtype]).min)
    x[0] = -np.inf
    x[1] = np.nan
    x[2] = -np.inf
    x[2, 1500] = -3.0
    x[3, 5:] = low
    x[4] = low
    x[5, ::3] = np.nan
    x[6, :1400] = -np.inf
    x[7] = np.nan
    x[7, 0] = 0.0
    check(dev, torch.from_numpy(x).to(DT[dtype]).to(dev), g.random(8), **f)


def test_uniforms_at_the_ends(dev, kernel):
    x = torch.zeros((3, 1000), device=dev)
    x[:, 0] = x[:, 999] = -np.inf
    token, logprob = run(dev, x, [0.0, 1 - 2.0 ** -24, 0.5])
    assert token.tolist() == [1, 998, 500] and np.allclose(logprob, -np.log(998), rtol=1e-6)


def test_temperatures(dev, kernel):
    """From none (the first largest) over very small to very large."""
    g = np.random.default_rng(5)
    t = np.array([0.0, 1e-30, 1e-3, 0.05, 1.0, 30.0, 1e6, 1e30, 3e38, np.inf])
    x = normal(g, len(t), 4000, "f32", dev, 3.0)
    x[:, 77] = x[:, 1234] = x.max() + 1
    for f in (dict(), dict(k=20), dict(p=0.9), dict(m=0.9)):
        check(dev, x, g.random(len(t)), t=t, **f)
    assert run(dev, x, 0.999, t=0.0)[0].tolist() == [77] * len(t)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_bias_and_strided_rows(dev, kernel, dtype):
    g = np.random.default_rng(6)
    big = normal(g, 9, 1237, dtype, dev)
    bias = torch.from_numpy(g.normal(size=1111).astype(np.float32)).to(dev)
    bias[5] = -np.inf
    for lead in range(5):  # rows that begin at any element of a 16-byte vector
        check(dev, big[:, lead:lead + 1111], g.random(9), k=30, p=0.9, bias=bias)
        check(dev, big[:, lead:lead + 1111], g.random(9), p=0.8, bias=None)


@pytest.mark.parametrize("vocab,dtype", [(260001, "f32"), (700001, "bf16"), (2200003, "f32")])
@pytest.mark.parametrize("f", [dict(), dict(k=64), dict(p=0.9), dict(k=5000, p=0.9)])
def test_large_vocabularies(dev, vocab, dtype, f):
    """Rows that fill a cluster's shared memory, and rows that do not fit it."""
    g = np.random.default_rng(7)
    check(dev, normal(g, 2, vocab, dtype, dev), g.random(2), **f)


def test_out_of_range_settings(dev):
    """Reported; a temperature counts as 0, a filter as off."""
    g = np.random.default_rng(8)
    x = normal(g, 3, 500, "f32", dev)
    want = x.argmax(dim=1).cpu().tolist()
    assert run(dev, x, 0.9, t=[-1.0, np.nan, 0.0], status=5)[0].tolist() == want
    plain = run(dev, x, 0.3)[0].tolist()
    assert run(dev, x, 0.3, p=[0.0, -1.0, np.nan], status=5)[0].tolist() == plain
    assert run(dev, x, 0.3, m=[-0.1, 1.1, np.nan], status=5)[0].tolist() == plain
    assert run(dev, x, 0.3, k=[-1, -5, 0], status=5)[0].tolist() == plain
    assert run(dev, x, [1.0, -0.1, np.nan], status=5)[0][1] == run(dev, x, 0.0)[0][1]


def test_infinite_logits_end(dev):
    """Not supported: any token or -1, and no fault."""
    x = torch.zeros((2, 1000), device=dev)
    x[0, 3] = float("inf")
    x[1] = float("inf")
    for f in (dict(), dict(k=5), dict(p=0.5), dict(k=400, p=0.5)):
        token, _ = run(dev, x, 0.5, **f)
        assert ((token >= -1) & (token < 1000)).all()


def test_the_draw_does_not_depend_on_the_split(dev, monkeypatch):
    """The same bits from one CTA per row and from eight."""
    g = np.random.default_rng(9)
    x = normal(g, 40, 30011, "f16", dev)
    u = g.random(40)
    for f in (dict(), dict(k=64, p=0.9), dict(p=0.97), dict(k=2000, p=0.9, m=0.001)):
        got = []
        for c in (1, 2, 4, 8):
            monkeypatch.setenv("LS_BEAM_DEBUG", f"sfcluster={c}")
            got.append(run(dev, x, u, **f))
        for tok, lp in got[1:]:
            assert np.array_equal(tok, got[0][0]) and np.array_equal(lp, got[0][1])


def test_frequencies(dev):
    """Over a fine grid of uniforms every token comes as often as its probability says."""
    g = np.random.default_rng(10)
    x = torch.from_numpy(g.normal(size=40).astype(np.float32)).to(dev)
    n = 20000
    token, _ = run(dev, x.expand(n, 40).contiguous(), (np.arange(n) + 0.5) / n, t=0.8, k=20)
    p = np.exp(x.double().cpu().numpy() / np.float32(0.8))
    p[np.argsort(-p)[20:]] = 0
    p /= p.sum()
    assert np.abs(np.bincount(token, minlength=40) / n - p).max() <= 1.0 / n + 1e-6


def test_captured(dev):
    g = np.random.default_rng(11)
    x, y = normal(g, 6, 9000, "f16", dev), normal(g, 6, 9000, "f16", dev)
    buf, u = x.clone(), torch.rand(6, device=dev)
    token, logprob = torch.empty(6, dtype=torch.int32, device=dev), torch.empty(6, device=dev)
    top_p = torch.full((6,), 0.9, device=dev)
    call = lambda: lsb.check(lsb.ls_sample_filtered(buf, None, u, None, None, top_p, None, token, logprob))  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for z in (y, x):
        buf.copy_(z)
        graph.replay()
        torch.cuda.synchronize()
        got = token.clone(), logprob.clone()
        call()
        assert torch.equal(got[0], token) and torch.equal(got[1], logprob)


@pytest.mark.parametrize("dtype,vocab", [("f32", 40000), ("bf16", 120000)])
@pytest.mark.parametrize("p", [1e-6, 0.02, 0.5, 0.99])
def test_nucleus_of_long_rows(dev, kernel, dtype, vocab, p):
    g = np.random.default_rng(vocab + 9)
    check(dev, normal(g, 6, vocab, dtype, dev, 2.5), g.random(6), t=[0.05, 0.3, 1.0, 1.0, 2.0, 4.0], p=p)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("p", [1e-30, 0.05, 0.9, 0.9999, 0.99999, 1.0 - 2.0 ** -24])
@pytest.mark.parametrize("k", [0, 3000])
def test_nucleus_does_not_depend_on_the_split(dev, monkeypatch, dtype, p, k):
    g = np.random.default_rng(31)
    logits, u = normal(g, 24, 33001, dtype, dev, 2.5), g.random(24)
    t = np.resize([0.02, 0.5, 1.0, 1.3, 30.0, 1e30, np.inf, 3e38], 24)
    got = []
    for split in ("sfcluster=1", "sfcluster=2", "sfcluster=8"):
        monkeypatch.setenv("LS_BEAM_DEBUG", split)
        got.append(run(dev, logits, u, t=t, p=p, k=k or None))
    for token, logprob in got[1:]:
        assert (token == got[0][0]).all() and (logprob == got[0][1]).all()
