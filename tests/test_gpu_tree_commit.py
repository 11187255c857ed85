"""The draft tree's commit on the GPU against its definition: whole numbers and copied bytes,
equal everywhere, nothing else of the caches touched."""
import numpy as np
import pytest

import attention_plain as ap

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import serving_ls_beam_gb300 as lsb  # noqa: E402

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EOS = 2


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lsb.load_library()
    return torch.device("cuda:0")


def run(dev, dtype, L, R, N, H, S, D, parent, token, target, lens, finished=None, eos=EOS, status=0, dk=None, dv=None):
    g = torch.Generator(device=dev).manual_seed(R * 100 + N)

    def rnd(*s):
        return torch.randn(s, generator=g, device=dev).to(DT[dtype])

    ck, cv = rnd(L, R, H, S, D), rnd(L, R, H, S, D)
    dk = rnd(L, R, N, H, D) if dk is None else dk
    dv = rnd(L, R, N, H, D) if dv is None else dv
    want_k, want_v = ck.clone(), cv.clone()
    i32 = lambda a: torch.as_tensor(np.asarray(a), dtype=torch.int32, device=dev)  # noqa: E731
    out = {n: torch.full((R,), -77, dtype=torch.int32, device=dev) for n in ("len", "count", "token")}
    path = torch.full((R, N), -77, dtype=torch.int32, device=dev)
    fin = torch.full((R,), 9, dtype=torch.uint8, device=dev)
    ws = torch.empty(256, dtype=torch.uint8, device=dev)
    lsb.check(lsb.ls_workspace_init(ws))
    fd = None if finished is None else torch.as_tensor(finished, dtype=torch.uint8, device=dev)
    lsb.check(lsb.ls_tree_commit(ck, cv, i32(lens), dk, dv, i32(parent), i32(token), i32(target), fd, eos, out["len"], path,
                                 out["count"], out["token"], fin, ws))
    assert lsb.ls_read_status(ws) == status
    ref = ap.commit(lens, parent, token, target, finished, eos, S)
    for r, (p, nxt, f) in enumerate(ref):
        assert path[r].tolist() == p + [-1] * (N - len(p)), r
        assert out["count"][r].item() == len(p) and out["len"][r].item() == lens[r] + len(p)
        assert out["token"][r].item() == nxt and fin[r].item() == f
        for i, n in enumerate(p):
            want_k[:, r, :, lens[r] + i] = dk[:, r, n]
            want_v[:, r, :, lens[r] + i] = dv[:, r, n]
    bits = torch.int32 if dtype == "f32" else torch.int16
    assert torch.equal(ck.view(bits), want_k.view(bits)) and torch.equal(cv.view(bits), want_v.view(bits))
    return ref


def random_trees(g, R, N, vocab):
    parent = np.stack([[-1] + [int(g.integers(0, i)) for i in range(1, N)] for _ in range(R)]).astype(np.int32)
    return parent, g.integers(0, vocab, (R, N)).astype(np.int32), g.integers(0, vocab, (R, N)).astype(np.int32)


# (dtype, layers, rows, nodes, heads, max_len, dim)
SHAPES = [("f16", 6, 4, 1, 16, 64, 64), ("f16", 2, 33, 31, 4, 70, 64), ("bf16", 3, 9, 64, 2, 65, 80),
          ("f32", 1, 17, 12, 3, 20, 7), ("f16", 2, 5, 8, 3, 9, 5), ("bf16", 1, 3, 64, 1, 40, 256)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("vocab", [3, 6])
def test_commit(dev, shape, vocab):
    """A tiny vocabulary: many confirmed nodes, equal siblings, end tokens, rows that run full."""
    dtype, L, R, N, H, S, D = shape
    g = np.random.default_rng(N * 10 + vocab)
    parent, token, target = random_trees(g, R, N, vocab)
    if N > 4:
        parent[::3, N - 2] = -2  # an empty place
    lens = g.integers(0, S, R)
    lens[0] = S - 1
    finished = (g.random(R) < 0.2).astype(np.uint8)
    ref = run(dev, dtype, L, R, N, H, S, D, parent, token, target, lens, finished, eos=EOS)
    run(dev, dtype, L, R, N, H, S, D, parent, token, target, lens, None, eos=-1)
    assert N < 12 or max(len(p) for p, _, _ in ref) > 1  # the larger trees do confirm drafts


def test_chain_of_all_nodes_and_no_room(dev):
    N = 64
    parent = np.tile(np.arange(-1, N - 1), (3, 1))
    token = np.tile(np.arange(100, 100 + N), (3, 1))
    target = token + 1
    ref = run(dev, "f16", 2, 3, N, 2, 80, 64, parent, token, target, [0, 16, 50])
    assert [len(p) for p, _, _ in ref] == [64, 64, 30]


def test_reported_rows_append_nothing(dev):
    parent, token, target = np.array([[-1, 0]] * 2), np.array([[5, 6]] * 2), np.array([[6, 7]] * 2)
    run(dev, "f16", 1, 2, 2, 2, 8, 64, parent, token, target, [8, 3], status=lsb.LS_ERR_INTERNAL)  # full
    run(dev, "f16", 1, 2, 2, 2, 8, 64, np.array([[-2, 0], [-1, 0]]), token, target, [1, 3], status=lsb.LS_ERR_INTERNAL)
    run(dev, "f16", 1, 2, 2, 2, 8, 64, parent, token, target, [8, 3], finished=[1, 0])  # a finished row may be full


def test_only_confirmed_drafts_are_read_and_strides(dev):
    g = torch.Generator(device=dev).manual_seed(1)
    L, R, N, H, D = 2, 3, 5, 2, 64
    both = torch.randn((R, N, L, 2, H, D), generator=g, device=dev).half()
    parent, token, target = np.array([[-1, 0, 0, 1, 2]] * R), np.array([[9, 4, 5, 6, 7]] * R), np.array([[5, 0, 7, 0, 3]] * R)
    both[:, [1, 3]] = float("nan")
    d = both.permute(2, 0, 1, 3, 4, 5)
    ref = run(dev, "f16", L, R, N, H, 12, D, parent, token, target, [0, 4, 9], dk=d[:, :, :, 0], dv=d[:, :, :, 1])
    assert ref[0][0] == [0, 2, 4]
