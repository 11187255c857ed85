"""The f32 attention kernels at the places where their tiles end: queries, keys and head sizes
around every multiple that they are built of, streamed and tiled, whole and in parts."""
import numpy as np
import pytest

import attention_plain as ap

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_attention import check_cross, close, f64, random_parents, run_cross, run_tree, tensor  # noqa: E402

import serving_ls_beam_gb300 as lsb  # noqa: E402

KERNELS = [None, "attc", "attc,atsplits=2", "attc,atsplits=3", "atmma,atwarps=1", "atmma,atwarps=4", "atmma,atwarps=4,atsplits=2"]
LENS = [0, 1, 3, 15, 16, 17, 31, 32, 33, 48, 49, 63, 64, 65, 130, 200]


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


@pytest.mark.parametrize("dim", [4, 32, 36, 64, 68, 96, 100, 128, 132, 200, 256])
def test_head_sizes(dev, kernel, dim):
    check_cross(dev, "f32", len(LENS), 1, 3, 8, 2, 200, dim, LENS, seed=dim)


@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("queries", [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 31, 32, 33, 65])
def test_queries(dev, kernel, queries, dim):
    check_cross(dev, "f32", len(LENS), 1, queries, 2, 2, 200, dim, LENS, seed=queries)


@pytest.mark.parametrize("dim", [32, 80, 128, 256])
@pytest.mark.parametrize("nodes", [1, 2, 9, 17, 40, 64])
def test_trees(dev, kernel, nodes, dim):
    """The drafted tokens begin and end anywhere in a tile; some see nothing, with NaN in their place."""
    g = np.random.default_rng(nodes * dim)
    R, H, HK, S = len(LENS), 4, 2, 200
    kinds = ["forest", "chain", "ragged", "empty"]
    parent = np.stack([random_parents(g, nodes, kinds[r % (4 if nodes > 1 else 2)]) for r in range(R)])
    q = tensor(g, (R, nodes, H, dim), "f32", dev)
    ck, cv = tensor(g, (R, HK, S, dim), "f32", dev), tensor(g, (R, HK, S, dim), "f32", dev)
    dk, dv = tensor(g, (R, nodes, HK, dim), "f32", dev), tensor(g, (R, nodes, HK, dim), "f32", dev)
    for r in range(R):
        ck[r, :, LENS[r]:] = float("nan")
        cv[r, :, LENS[r]:] = float("inf")
        for i in range(nodes):
            if not ap.branch(parent[r], i):
                q[r, i] = dk[r, i] = float("nan")
                dv[r, i] = float("-inf")
    out = run_tree(q, ck, cv, LENS, dk, dv, parent)
    want, bound = ap.tree(f64(q), f64(ck), f64(cv), LENS, f64(dk), f64(dv), parent, dim ** -0.5, "f32")
    close(out, want, bound)


@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
def test_scales(dev, kernel, scale):
    check_cross(dev, "f32", 4, 2, 10, 4, 2, 130, 64, [130, 65, 64, 1], scale=scale)
    check_cross(dev, "f32", 4, 1, 2, 4, 2, 130, 256, [130, 65, 64, 1], scale=scale)


def test_strided_views(dev, kernel):
    """Keys as a projection writes them, queries and results as parts of wider tensors."""
    g = np.random.default_rng(3)
    B, T, H, S, D = 3, 20, 4, 77, 256
    wide = tensor(g, (B, 1, T, 3, H, D), "f32", dev)
    q, k = wide[:, :, :, 1], tensor(g, (B, S, 2, 2, D), "f32", dev)
    out = torch.full_like(wide, float("nan"))
    run_cross(q, k[:, :, 0].transpose(1, 2), k[:, :, 1].transpose(1, 2), [77, 5, 64], out=out[:, :, :, 2])
    want, bound = ap.cross(f64(q), f64(k[:, :, 0].transpose(1, 2)), f64(k[:, :, 1].transpose(1, 2)), [77, 5, 64], D ** -0.5, "f32")
    close(out[:, :, :, 2], want, bound)
    assert torch.isnan(out[:, :, :, :2]).all()
