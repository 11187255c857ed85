"""Filtered sampling at an infinite temperature: the finite logits that the filters keep are equally likely, whatever min_p."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_sample_filtered import DT, dev, kernel, run  # noqa: E402,F401


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [1, 200, 1000, 2048, 5003])
@pytest.mark.parametrize("k", [None, 1, 5, 300, 900, 3000])
@pytest.mark.parametrize("m", [None, 1e-30, 0.5, 1.0])
def test_min_p_at_an_infinite_temperature(dev, kernel, dtype, vocab, k, m):  # noqa: F811
    g = np.random.default_rng(vocab)
    x = torch.from_numpy(g.normal(size=(5, vocab), scale=3.0).astype(np.float32)).to(DT[dtype])
    x[2:, 1::3] = -float("inf")
    x[3, 5:] = float("nan")
    u = np.array([0.0, 0.3, 0.999, 0.5, 1 - 2.0 ** -24], np.float32)
    token, logprob = run(dev, x.to(dev), u, t=np.inf, k=k, m=m)
    x = x.double().numpy()
    for r in range(5):
        order = np.lexsort((np.arange(vocab), -np.where(np.isnan(x[r]), -np.inf, x[r])))
        order = order[np.isfinite(x[r][order])][:k]
        kept = np.sort(order)
        assert token[r] == kept[int(float(u[r]) * len(kept))], (r, token[r])
        assert abs(logprob[r] + np.log(len(kept))) <= 2.0 ** -21 * (1 + np.log(len(kept)))
