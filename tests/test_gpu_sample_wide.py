"""Filtered sampling from logits that lie far apart, at high temperatures: candidates far below the largest logit count there."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_sample_filtered import DT, check, dev, kernel  # noqa: E402,F401


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [90, 1000, 5003])
@pytest.mark.parametrize("k", [2, 50, 300, 1000])
@pytest.mark.parametrize("p", [None, 0.9])
def test_wide_logits_at_high_temperatures(dev, kernel, dtype, vocab, k, p):  # noqa: F811
    """A few leading logits, the others 40 to 1000 below them."""
    g = np.random.default_rng(vocab + k)
    cases = [(gap, t) for gap in (40.0, 50.0, 60.0, 300.0, 1000.0) for t in (1.0, 2.0, 5.0, 30.0, 1e3, 1e6, 1e30, np.inf)]
    x = np.empty((len(cases), vocab), np.float32)
    for r, (gap, _) in enumerate(cases):
        x[r] = -gap - g.uniform(0, 5, vocab)
        x[r, g.permutation(vocab)[:1 + r % 3]] = g.uniform(-1, 0, 1 + r % 3)
    check(dev, torch.from_numpy(x).to(DT[dtype]).to(dev), g.random(len(cases)), t=[t for _, t in cases], k=k, p=p)


def test_the_probability_of_a_lone_leader(dev):  # noqa: F811
    """One logit at 0 and 999 at -60, 50 candidates at a temperature of 30: probability 1 / (1 + 49 e^-2) = 0.131."""
    from test_gpu_sample_filtered import run

    n = 2000
    x = torch.full((n, 1000), -60.0, device=dev)
    x[:, 700] = 0.0
    token, logprob = run(dev, x, (np.arange(n) + 0.5) / n, t=30.0, k=50)
    want = 1.0 / (1.0 + 49.0 * np.exp(-2.0))
    assert abs((token == 700).mean() - want) <= 1.0 / n + 1e-6
    assert np.allclose(logprob[token == 700], np.log(want), rtol=1e-6)
    assert set(token[token != 700]) == set(range(49))  # ties: the smaller tokens
