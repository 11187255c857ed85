"""Rows without a sequence in PagedDecoder (no GPU: the library's calls are recorded in place of run): they hold nothing, write
nothing and do not move, and the next sequence begins at position 0."""
import pytest

torch = pytest.importorskip("torch")

from serving_ls_beam_gb300 import paged  # noqa: E402

EOS = 2


class Calls:
    def __init__(self):
        self.writes, self.reads, self.draws = [], [], None


@pytest.fixture
def calls(monkeypatch):
    c = Calls()

    def write(key, value, start, count, pages, workspace=None, stream=None):
        n = torch.full_like(start, key.shape[1]) if count is None else count
        c.writes.append((start.tolist(), n.tolist()))
        return 0

    def attend(q, pages, length, out, workspace, scale=None, stream=None):
        c.reads.append(length.tolist())
        return 0

    def sample(logits, bias, u, t, k, p, m, token, logprob=None, workspace=None, stream=None):
        token.copy_(torch.tensor(c.draws, dtype=torch.int32))
        return 0

    monkeypatch.setattr(paged, "ls_paged_write", write)
    monkeypatch.setattr(paged, "ls_paged_attention", attend)
    monkeypatch.setattr(paged, "ls_sample_filtered", sample)
    monkeypatch.setattr(paged, "ls_workspace_init", lambda w, stream=None: 0)
    monkeypatch.setattr(paged, "ls_paged_attention_workspace_size", lambda *a: 256)
    return c


def step(dec, calls, draws):
    x = torch.zeros(dec.rows, 4, 8)
    calls.draws = draws
    dec.attention(0, x, x, x)
    return dec.finish(torch.zeros(dec.rows, 5), torch.zeros(dec.rows)).tolist()


def decoder(rows=3):
    return paged.PagedDecoder(1, rows, 4, 4, 8, 16, 20, 4, EOS, torch.float32, device="cpu")


def test_idle_rows_do_not_move(calls):
    dec = decoder()
    dec.reserve(0, 8)
    for n in range(3):
        assert step(dec, calls, [7, 7, EOS]) == [7, EOS, EOS]
        assert calls.writes[-1] == ([n, 0, 0], [1, 0, 0]) and calls.reads[-1] == [n + 1, 0, 0]
    assert dec.length.tolist() == [3, 0, 0] and dec.live.tolist() == [1, 0, 0]
    # sequences come to both idle rows: one with a prompt, one without
    dec.reserve(1, 3)
    dec.reserve(2, 1)
    x = torch.zeros(3, 2, 4, 8)
    count = torch.tensor([0, 2, 0], dtype=torch.int32)
    dec.store(0, x, x, count)
    assert calls.writes[-1] == ([3, 0, 0], [0, 2, 0])
    dec.advance(count)
    assert dec.length.tolist() == [3, 2, 0]
    assert step(dec, calls, [8, 9, 10]) == [8, 9, 10]
    assert calls.writes[-1] == ([3, 2, 0], [1, 1, 1]) and calls.reads[-1] == [4, 3, 1]
    assert dec.length.tolist() == [4, 3, 1]


def test_a_released_row_is_idle(calls):
    dec = decoder()
    for r in range(3):
        dec.reserve(r, 4)
    step(dec, calls, [7, 7, 7])
    dec.release(1)
    assert len(dec.free) == 18
    for _ in range(2):
        assert step(dec, calls, [7, 7, 7]) == [7, EOS, 7]
        assert calls.writes[-1][1] == [1, 0, 1] and calls.reads[-1][1] == 0
    dec.reserve(1, 1)
    assert step(dec, calls, [7, 7, 7]) == [7, 7, 7]
    assert calls.writes[-1] == ([3, 0, 3], [1, 1, 1]) and dec.length.tolist() == [4, 1, 4]


def test_more_pages_do_not_revive_a_finished_row(calls):
    dec = decoder()
    dec.reserve(0, 1)
    assert step(dec, calls, [EOS, 7, 7]) == [EOS, EOS, EOS]
    dec.reserve(0, 40)
    assert step(dec, calls, [7, 7, 7]) == [EOS, EOS, EOS] and dec.length.tolist() == [1, 0, 0]


def test_a_prompt_for_all_rows_leaves_idle_ones_out(calls):
    dec = decoder()
    dec.reserve(0, 8)
    dec.reserve(2, 8)
    x = torch.zeros(3, 5, 4, 8)
    dec.store(0, x, x)
    assert calls.writes[-1] == ([0, 0, 0], [5, 0, 5])
    dec.advance(5)
    assert dec.length.tolist() == [5, 0, 5]


def test_nothing_to_draw_ends_a_row(calls):
    dec = decoder()
    for r in range(3):
        dec.reserve(r, 8)
    assert step(dec, calls, [7, -1, 7]) == [7, -1, 7]
    assert dec.live.tolist() == [1, 0, 1]
    assert step(dec, calls, [7, 7, 7]) == [7, EOS, 7] and dec.length.tolist() == [2, 1, 2]
