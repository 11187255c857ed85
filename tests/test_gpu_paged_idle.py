"""Rows of PagedDecoder without a sequence, over several steps: nothing is written or reported for them, and the sequences that
come to them later are computed from their own positions alone."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import serving_ls_beam_gb300 as lsb  # noqa: E402
from serving_ls_beam_gb300.paged import PagedDecoder  # noqa: E402
from test_gpu_paged_decode import DIM, EOS, HEADS, KV, LAYERS, NAMES, PAGE, ROWS, VOCAB, Model, Shadow, dev  # noqa: E402,F401


@pytest.mark.parametrize("dtype,cache", [(torch.float16, None), (torch.bfloat16, torch.float8_e4m3fn), (torch.float32, torch.int8)])
def test_idle_rows(dev, dtype, cache):  # noqa: F811
    model = Model(dev, dtype, 11)
    dec = PagedDecoder(LAYERS, ROWS, HEADS, KV, DIM, PAGE, 40, 8, EOS, dtype, cache, dev)
    shadow = Shadow(NAMES[cache or dtype])
    g = torch.Generator(device=dev).manual_seed(12)
    lens = [None] * ROWS  # None: no sequence
    token = torch.randint(3, VOCAB, (ROWS,), generator=g, device=dev, dtype=torch.int32)

    def admit(counts):
        most = max(counts.values())
        count = torch.tensor([counts.get(r, 0) for r in range(ROWS)], dtype=torch.int32, device=dev)
        x = model.embed[torch.randint(3, VOCAB, (ROWS, max(most, 1)), generator=g, device=dev)]
        for r, n in counts.items():
            dec.reserve(r, n + 1)
            lens[r] = n
            for i in range(LAYERS):
                shadow.rows[i][r] = ([], [], [])
        for i in range(LAYERS):
            _, k, v = model.qkv(i, x)
            dec.store(i, k, v, count)
            for r, n in counts.items():
                for j in range(n):
                    shadow.add(i, r, k[r, j], v[r, j])
        dec.advance(count)

    def steps(n):
        nonlocal token
        for _ in range(n):
            for r in range(ROWS):
                if lens[r] is not None:
                    dec.reserve(r, lens[r] + 1)
            x = model.embed[token.long()]
            for i in range(LAYERS):
                q, k, v = model.qkv(i, x)
                out = dec.attention(i, q, k, v)
                for r in range(ROWS):
                    if lens[r] is None:
                        assert (out[r] == 0).all()
                    else:
                        shadow.add(i, r, k[r], v[r])
                        shadow.check(i, r, q[r], out[r], NAMES[dtype])
                x = x + out.view(ROWS, -1) @ model.o[i].T
            logits = x @ model.out.T
            logits[:, EOS] = -1000.0
            for r in range(ROWS):
                if lens[r] is None:
                    logits[r] = float("nan") if r % 2 else 0.0
                    logits[r, EOS] = 1000.0
            token = dec.finish(logits, torch.rand(ROWS, generator=g, device=dev)).clone()
            for r in range(ROWS):
                if lens[r] is None:
                    assert int(token[r]) == EOS
                else:
                    lens[r] += 1
            assert dec.length.tolist() == [n or 0 for n in lens]
            assert lsb.ls_read_status(dec.workspace) == 0

    steps(2)  # no sequence at all
    admit({1: 17, 4: 0})
    steps(4)
    admit({0: 7, 2: 20})
    steps(4)
    dec.release(4)
    lens[4] = None
    steps(3)
    admit({4: 0, 3: 1})
    steps(3)
