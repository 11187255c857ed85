"""Rows in parts of which some are empty: the infinite values of a row's drafted tokens reach the nodes under
them, whatever parts a thread block worked on before and after."""
import numpy as np
import pytest

import attention_plain as ap

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_attention import f64, run_tree, tensor  # noqa: E402


@pytest.mark.parametrize("parts", ["attc,atsplits=2", "atmma,atwarps=4,atsplits=2", "attc"])
@pytest.mark.parametrize("nodes,heads,D", [(64, 4, 64), (20, 4, 64), (64, 4, 128)])
def test_infinite_drafts_between_empty_parts(monkeypatch, parts, nodes, heads, D):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    monkeypatch.setenv("LS_BEAM_DEBUG", parts)
    dev = torch.device("cuda:0")
    g = np.random.default_rng(nodes + D)
    R, S = 76 * 6, 300  # two parts a row over 152 blocks: a block's rows are 76 apart
    lens = [S if (r // 76) % 2 == 0 else 0 for r in range(R)]  # every other one of them leaves its second part empty
    parent = np.array([-1] + [int(g.integers(-1, i)) for i in range(1, nodes)])
    branches = [ap.branch(parent, i) for i in range(nodes)]
    q = tensor(g, (R, nodes, heads, D), "bf16", dev)
    ck, cv = tensor(g, (R, 1, S, D), "bf16", dev), tensor(g, (R, 1, S, D), "bf16", dev)
    dk, dv = tensor(g, (R, nodes, 1, D), "bf16", dev), tensor(g, (R, nodes, 1, D), "bf16", dev)
    bad = nodes // 3
    dv[:, bad, 0, 5] = float("inf")
    out = f64(run_tree(q, ck, cv, lens, dk, dv, np.stack([parent] * R)))
    under = np.zeros(out.shape, bool)
    under[:, [i for i in range(nodes) if bad in branches[i]], :, 5] = True
    assert (out[under] == np.inf).all() and np.isfinite(out[~under]).all()
    for r in range(0, R, 37):
        for i in (0, bad, nodes - 1):
            ks = np.concatenate([f64(ck[r, 0, :lens[r]]), f64(dk[r, branches[i], 0])])
            vs = np.concatenate([f64(cv[r, 0, :lens[r]]), f64(dv[r, branches[i], 0])])
            want, bound = ap.one_query(f64(q[r, i, 1]), ks, np.where(np.isfinite(vs), vs, 0.0), D ** -0.5, "bf16")
            ok = ~under[r, i, 1]
            assert (np.abs(out[r, i, 1] - want) <= bound)[ok].all(), (r, i)
