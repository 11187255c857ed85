"""Attention of so many rows that a row's number plus a launch's stride passes 2^31: the last rows are
answered and the walk over them ends.  The rows share one query and one set of keys, so that the outputs
(16 bytes a row) and the lengths are all that takes memory."""
import numpy as np
import pytest

import attention_plain as ap

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_attention import DT, f64, tensor, workspace  # noqa: E402

import serving_ls_beam_gb300 as lsb  # noqa: E402


# one warp to a row: the stride is a few thousand rows; four: it is the number of rows
@pytest.mark.parametrize("dtype,dim", [("bf16", 8), ("f32", 4)])
@pytest.mark.parametrize("kernel,rows", [("atmma,atwarps=1", 2**31 - 1), ("atmma,atwarps=4", 2**30 + 1000)])
def test_rows_up_to_the_limit(monkeypatch, kernel, rows, dtype, dim):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev = torch.device("cuda:0")
    if torch.cuda.mem_get_info(dev)[0] < 26 * rows:
        pytest.skip("not enough free memory")
    monkeypatch.setenv("LS_BEAM_DEBUG", kernel)
    g = np.random.default_rng(dim)
    S = 8
    q, k, v = tensor(g, (1, 1, 1, 1, dim), dtype, dev), tensor(g, (1, 1, S, dim), dtype, dev), tensor(g, (1, 1, S, dim), dtype, dev)
    lens = torch.zeros(rows, dtype=torch.int32, device=dev)
    at = sorted({0, 1, 4095, rows // 2, 2**30 - 1, 2**30, rows - 2000, rows - 2, rows - 1})
    lens[torch.tensor(at, device=dev)] = S
    out = torch.full((rows, 1, 1, 1, dim), float("nan"), dtype=DT[dtype], device=dev)
    ws = workspace(lsb.ls_cross_attention_workspace_size(rows, 1, 1, 1, 1, S, dim), dev)
    lsb.check(lsb.ls_cross_attention(q.expand(rows, 1, 1, 1, dim), k.expand(rows, 1, S, dim), v.expand(rows, 1, S, dim), lens,
                                     out, ws))
    assert lsb.ls_read_status(ws) == lsb.LS_OK
    want, bound = ap.one_query(f64(q).reshape(dim), f64(k)[0, 0], f64(v)[0, 0], dim ** -0.5, dtype)
    words, found = out.view(torch.int64).view(rows, 2), []
    for a in range(0, rows, 2**27):  # every other row is zero
        found += (words[a:a + 2**27].ne(0).any(dim=1).nonzero().view(-1) + a).tolist()
        assert len(found) <= len(at)
    assert found == at
    for r in at:
        assert (np.abs(f64(out[r]).reshape(dim) - want) <= bound).all(), r
