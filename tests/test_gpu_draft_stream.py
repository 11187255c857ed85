"""DraftTreeDecoder on a stream of the caller's, and captured in a CUDA graph: the same tokens, lengths and
caches as on the current stream."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import serving_ls_beam_gb300 as lsb  # noqa: E402
from serving_ls_beam_gb300.draft import DraftTreeDecoder  # noqa: E402

L, R, N, H, HK, D, S, V, EOS = 2, 3, 4, 4, 2, 64, 64, 50, 1
PARENT = [-1, 0, 0, 1]


class Program:
    """A decoder of fixed random projections whose every step is made of device operations alone."""

    def __init__(self, dtype=torch.float16):
        if not torch.cuda.is_available():
            pytest.skip("no CUDA device")
        g = torch.Generator(device="cuda").manual_seed(3)

        def r(*s):
            return torch.randn(s, generator=g, device="cuda").div(s[0] ** 0.5).to(dtype)

        w = H * D
        self.emb, self.out = r(V, w) * 7, r(w, V)
        self.proj = [(r(w, H * D), r(w, HK * D), r(w, HK * D), r(H * D, w)) for _ in range(L)]
        self.dec = DraftTreeDecoder(L, R, N, H, HK, D, S, V, EOS, dtype=dtype)
        self.dec.cache_key.zero_()
        self.dec.cache_value.zero_()
        self.parent = torch.tensor([PARENT] * R, dtype=torch.int32, device="cuda")
        self.start = torch.tensor([3, 9, 20], dtype=torch.int32, device="cuda")
        self.token = torch.zeros((R, N), dtype=torch.int32, device="cuda")
        self.guess = torch.tensor([0, 11, 5, 17], dtype=torch.int32, device="cuda")

    def reset(self):
        self.dec.reset()
        self.dec.next_token.copy_(self.start)

    def step(self, stream=None, handle=None):
        """stream: of the library's calls, given as `handle`; torch's operations stay on the current one, and the two
        are ordered both ways around every call."""
        def call(f, *args):
            if stream is None:
                return f(*args)
            stream.wait_stream(torch.cuda.current_stream())
            y = f(*args, stream=handle)
            torch.cuda.current_stream().wait_stream(stream)
            return y

        self.token.copy_((self.dec.next_token[:, None] + self.guess) % V)
        x = self.emb[self.token.long()]
        for i, (q, k, v, o) in enumerate(self.proj):
            y = call(self.dec.self_attention, i, (x @ q).view(R, N, H, D), (x @ k).view(R, N, HK, D),
                     (x @ v).view(R, N, HK, D), self.parent)
            x = x + y.reshape(R, N, H * D) @ o
        call(self.dec.finish, x @ self.out, self.token, self.parent)

    def state(self):
        d = self.dec
        return [t.clone() for t in (d.next_token, d.length(), d.path, d.count, d.finished[d.cur], d.cache_key, d.cache_value)]


def eager(steps):
    p = Program()
    p.reset()
    states = []
    for _ in range(steps):
        p.step()
        states.append(p.state())
    return states


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("integer", [False, True])
def test_a_stream_of_the_callers(integer):
    """The stream, or its handle as the C calls take it."""
    want = eager(6)
    assert int(want[-1][1].sum()) > 0
    p = Program()
    p.reset()
    side = torch.cuda.Stream()
    for n in range(6):
        p.step(side, side.cuda_stream if integer else side)
        assert same(p.state(), want[n]), n


def test_two_steps_captured():
    """The two sets of lengths alternate: two captured steps, replayed, go on as single ones do."""
    want = eager(8)
    p = Program()
    p.reset()
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        p.step()
        p.step()
    torch.cuda.current_stream().wait_stream(warm)
    assert same(p.state(), want[1])
    p.reset()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.step()
        p.step()
    for n in range(4):
        graph.replay()
        assert same(p.state()[:5], want[2 * n + 1][:5]), n
    assert same(p.state(), want[7])
    assert lsb.ls_read_status(p.dec.workspace) == lsb.LS_OK
