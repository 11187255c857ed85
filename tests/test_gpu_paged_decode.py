"""Decoding over pages from end to end: prompts of different lengths, steps that cross pages, rows that finish, leave and are
replaced; every attention and every draw against the float64 definitions, on caches of every type, and captured."""
import numpy as np
import pytest

import paged_plain as pp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import serving_ls_beam_gb300 as lsb  # noqa: E402
from serving_ls_beam_gb300.paged import PagedDecoder  # noqa: E402

LAYERS, ROWS, HEADS, KV, DIM, VOCAB, EOS, PAGE = 2, 5, 8, 2, 64, 300, 2, 16
NAMES = {torch.float16: "f16", torch.bfloat16: "bf16", torch.float32: "f32", torch.float8_e4m3fn: "e4m3", torch.int8: "i8"}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lsb.load_library()
    return torch.device("cuda:0")


class Model:
    """A decoder with random weights: its projections by torch on the GPU."""

    def __init__(self, dev, dtype, seed):
        g = torch.Generator().manual_seed(seed)
        w = lambda *s: (torch.randn(s, generator=g) * s[-1] ** -0.5).to(dtype).to(dev)  # noqa: E731
        self.width = HEADS * DIM
        self.embed = torch.randn((VOCAB, self.width), generator=g).to(dtype).to(dev)
        self.q = [w(HEADS * DIM, self.width) for _ in range(LAYERS)]
        self.k = [w(KV * DIM, self.width) for _ in range(LAYERS)]
        self.v = [w(KV * DIM, self.width) for _ in range(LAYERS)]
        self.o = [w(self.width, HEADS * DIM) for _ in range(LAYERS)]
        self.out = w(VOCAB, self.width) * 3

    def qkv(self, i, x):
        lead = x.shape[:-1]
        return ((x @ self.q[i].T).view(*lead, HEADS, DIM), (x @ self.k[i].T).view(*lead, KV, DIM),
                (x @ self.v[i].T).view(*lead, KV, DIM))


def held(x, cache):
    """What the cache holds of x [.., dim], and the scales."""
    x = x.double().cpu().numpy()
    if cache not in ("e4m3", "i8"):
        return x, np.ones(x.shape[:-1])
    codes, s = pp.quantise(x, cache)
    return codes * s[..., None], s


class Shadow:
    """The caches as float64 arrays, row by row."""

    def __init__(self, cache):
        self.cache = cache
        self.rows = [[([], [], []) for _ in range(ROWS)] for _ in range(LAYERS)]

    def add(self, layer, r, k, v):
        ks, _ = held(k, self.cache)
        vs, sv = held(v, self.cache)
        for a, b in zip(self.rows[layer][r], (ks, vs, sv)):
            a.append(b)

    def check(self, layer, r, q, out, dtype):
        ks, vs, sv = (np.array(a) for a in self.rows[layer][r])
        for h in range(HEADS):
            g = h // (HEADS // KV)
            want, bound = pp.attend(q[h].double().cpu().numpy(), ks[:, g], vs[:, g], sv[:, g], DIM ** -0.5, dtype, self.cache)
            assert (np.abs(out[h].double().cpu().numpy() - want) <= bound).all(), (layer, r, h)


@pytest.mark.parametrize("dtype,cache", [(torch.float16, None), (torch.float16, torch.float8_e4m3fn), (torch.bfloat16, torch.int8),
                                         (torch.float32, torch.float8_e4m3fn)])
def test_decode(dev, dtype, cache):
    model = Model(dev, dtype, 1)
    dec = PagedDecoder(LAYERS, ROWS, HEADS, KV, DIM, PAGE, 40, 8, EOS, dtype, cache, dev)
    name, kind = NAMES[dtype], NAMES[cache or dtype]
    shadow = Shadow(kind)
    g = torch.Generator(device=dev).manual_seed(2)
    counts = [0, 1, 16, 33, 20]
    prompt = torch.randint(3, VOCAB, (ROWS, 33), generator=g, device=dev)
    count = torch.tensor(counts, dtype=torch.int32, device=dev)
    for r in range(ROWS):
        dec.reserve(r, counts[r])
    x = model.embed[prompt]
    for i in range(LAYERS):
        _, k, v = model.qkv(i, x)
        dec.store(i, k, v, count)
        for r in range(ROWS):
            for n in range(counts[r]):
                shadow.add(i, r, k[r, n], v[r, n])
    dec.advance(count)
    token = torch.randint(3, VOCAB, (ROWS,), generator=g, device=dev, dtype=torch.int32)
    settings = dict(temperature=torch.tensor([0.0, 0.7, 1.0, 1.3, 1.0], device=dev),
                    top_k=torch.tensor([0, 20, 0, 0, 3], dtype=torch.int32, device=dev),
                    top_p=torch.tensor([1.0, 0.9, 0.8, 1.0, 1.0], device=dev), min_p=torch.tensor([0.0, 0.0, 0.0, 0.05, 0.0], device=dev))
    live = [1] * ROWS
    lens = list(counts)
    for step in range(22):
        if step == 9:  # row 3 leaves, a new sequence takes its place
            before = len(dec.free)
            pages = len(dec.held[3])
            dec.release(3)
            assert len(dec.free) == before + pages
            lens[3], live[3] = 0, 1
            for i in range(LAYERS):
                shadow.rows[i][3] = ([], [], [])
        for r in range(ROWS):
            dec.reserve(r, lens[r] + 1)
        x = model.embed[token.long()]
        for i in range(LAYERS):
            q, k, v = model.qkv(i, x)
            out = dec.attention(i, q, k, v)
            for r in range(ROWS):
                if live[r]:
                    shadow.add(i, r, k[r], v[r])
                if lens[r] + live[r]:
                    shadow.check(i, r, q[r], out[r], name)
            x = x + out.view(ROWS, -1) @ model.o[i].T
        logits = x @ model.out.T
        if step == 5:
            logits[1, EOS] = 1000.0  # row 1 ends
        u = torch.rand(ROWS, generator=g, device=dev)
        token = dec.finish(logits, u, **settings).clone()
        for r in range(ROWS):
            if not live[r]:
                assert int(token[r]) == EOS
                continue
            want, lp, sure = pp.sample(logits[r].double().cpu().numpy(), *(float(settings[n][r]) if n != "top_k" else int(settings[n][r])
                                       for n in ("temperature", "top_k", "top_p", "min_p")), float(u[r]))
            if sure:
                assert int(token[r]) == want and abs(float(dec.logprob[r]) - lp) <= 2.0 ** -21 * (1 + abs(lp))
            lens[r] += 1
            live[r] = int(int(token[r]) != EOS)
        assert dec.length.tolist() == lens and dec.live.tolist() == live
    assert not live[1] and lsb.ls_read_status(dec.workspace) == 0
    # the whole cache back
    most = max(lens)
    for i in range(LAYERS):
        k = torch.full((ROWS, most, KV, DIM), 7.0, dtype=torch.float32 if cache else dtype, device=dev)
        v = k.clone()
        dec.restore(i, k, v)
        for r in range(ROWS):
            n = lens[r]
            for got, want in ((k, 0), (v, 1)):
                if n:
                    assert np.array_equal(got[r, :n].double().cpu().numpy(),
                                          np.array(shadow.rows[i][r][want]).astype(np.float32).astype(np.float64))
                assert (got[r, n:] == 7.0).all()


def test_captured_steps_on_another_stream(dev):
    """A captured step replayed, with pages reserved between, does what the eager one does; the work goes where it is told."""
    def run(captured):
        model = Model(dev, torch.float16, 3)
        dec = PagedDecoder(LAYERS, ROWS, HEADS, KV, DIM, PAGE, 40, 8, EOS, torch.float16, torch.float8_e4m3fn, dev)
        g = torch.Generator(device=dev).manual_seed(4)
        token = torch.randint(3, VOCAB, (ROWS,), generator=g, device=dev, dtype=torch.int32)
        u, top_p = torch.empty(ROWS, device=dev), torch.full((ROWS,), 0.9, device=dev)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())

        def step(stream):
            x = model.embed[token.long()]
            for i in range(LAYERS):
                q, k, v = model.qkv(i, x)
                x = x + dec.attention(i, q, k, v, stream).view(ROWS, -1) @ model.o[i].T
            token.copy_(dec.finish(x @ model.out.T, u, top_p=top_p, stream=stream))

        seen = []
        with torch.cuda.stream(side):
            for r in range(ROWS):
                dec.reserve(r, 1)
            u.fill_(0.5)
            step(side)  # warm up
            for r in range(ROWS):
                dec.release(r)
            token.copy_(torch.arange(5, 5 + ROWS, dtype=torch.int32, device=dev))
            graph = None
            if captured:
                side.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    step(side)
                for r in range(ROWS):  # (the capture ran nothing)
                    dec.release(r)
            for n in range(20):
                for r in range(ROWS):
                    dec.reserve(r, n + 1)
                u.copy_(torch.rand(ROWS, generator=g, device=dev))
                if graph:
                    graph.replay()
                else:
                    step(side)
                seen.append((token.clone(), dec.logprob.clone(), dec.attended.clone(), dec.length.clone()))
        side.synchronize()
        assert lsb.ls_read_status(dec.workspace) == 0
        return seen

    for a, b in zip(run(False), run(True)):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_reserve_refusals(dev):
    dec = PagedDecoder(1, 2, 4, 4, 64, 16, 5, 4, EOS, device=dev)
    dec.reserve(0, 64)
    with pytest.raises(ValueError):
        dec.reserve(0, 65)  # more than a row may have
    with pytest.raises(ValueError):
        dec.reserve(1, 17)  # more than there is
    assert len(dec.free) == 1 and dec.held[1] == []
    dec.reserve(1, 16)
    dec.release(0)
    dec.reserve(1, 64)
    assert sorted(dec.held[1] + dec.free) == [0, 1, 2, 3, 4] and dec.table[1].tolist() == dec.held[1]
