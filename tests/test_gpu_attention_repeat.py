"""The same call gives the same bits, whatever ran before it: nothing that a kernel finds in its shared
memory reaches a result.  Tiles that are not full of queries, after calls that leave large and infinite
values behind."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_attention import DT, KERNELS, run_cross  # noqa: E402

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


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,D", [(1, 64), (5, 64), (12, 64), (40, 64), (5, 128), (12, 128), (18, 128), (40, 128), (150, 128),
                                 (3, 256), (9, 256), (20, 256)])
def test_queries_past_the_last(dev, kernel, T, D, dtype):
    g = torch.Generator(device=dev).manual_seed(T * D)
    B, H, S = 300, 2, 333

    def tensor(*shape):
        return torch.randn(shape, generator=g, device=dev).to(DT[dtype])

    q = tensor(B, 1, 1, H, D).expand(B, 1, T, H, D).contiguous()
    k, v = tensor(B, H, S, D), tensor(B, H, S, D)
    k *= torch.linspace(0.2, 4, S, device=dev).view(1, 1, S, 1).to(DT[dtype])  # maxima that grow along a row
    lens = [S - b % 40 for b in range(B)]
    bits = torch.int32 if dtype == "f32" else torch.int16
    first = run_cross(q, k, v, lens)
    assert torch.equal(first.view(bits), first[:, :, :1].expand_as(first).contiguous().view(bits))  # equal queries
    # calls whose queries fill their tiles with something else
    for fill in (30.0, float("inf"), -7.0):
        full = torch.full((B, 1, 256, H, D), fill, dtype=DT[dtype], device=dev)
        run_cross(full[:, :, :32], k, v, lens)
        run_cross(full, k, v, lens)
        again = run_cross(q, k, v, lens)
        assert torch.equal(first.view(bits), again.view(bits)), fill
