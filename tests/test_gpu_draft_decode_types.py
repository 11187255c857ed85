"""Decoding with drafted trees in 16 bits: every chosen token against the float64 model of
test_gpu_draft_decode, from the same tokens before it.

Margin: a logit is a sum over the normalised state with weights of 6 / sqrt(W), so a relative error x of the
state's elements moves it by about 6 x.  Some 30 roundings lie one after the other on the way (weights and
activations of two layers), each of one unit u or less; all in one direction they make x = 30 u and 180 u of a
logit, twice that of the difference of two.  A chosen token's exact logit lies within 360 u of the best."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_draft_decode import ROWS, V, logits64, model, run  # noqa: E402, F401

MARGIN = {torch.float16: 360 * 2.0 ** -11, torch.bfloat16: 360 * 2.0 ** -8}


def check(m, seqs, margin):
    """Every token within the margin of the best; how many had no rival within it, and the tokens."""
    sure = total = 0
    for r, s in enumerate(seqs):
        for n in range(1, len(s)):
            logits = logits64(m, r, torch.tensor(s[:n], device="cuda"))[-1]
            top = logits.topk(2).values
            assert (top[0] - logits[s[n]]).item() <= margin, (r, n, s)
            sure += int((top[0] - top[1]).item() > margin)
            total += 1
    return sure, total


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_sixteen_bit_tokens(model, dtype):  # noqa: F811
    steps = 20
    single, _ = run(model, dtype, 1, steps, lambda r, s: ([s[-1]], [-1]))
    sure, total = check(model, single, MARGIN[dtype])
    assert total >= 3 * ROWS and sure >= total // 4
    g = np.random.default_rng(5)

    def drafts(r, s):
        """A branch of what the single-token search chose (one guess in four wrong), a random one, an empty place."""
        right = (single[r][len(s):len(s) + 4] + [5] * 4)[:4]
        if g.random() < 0.25:
            right[1] = (right[1] + 1) % V
        rnd = [int(t) for t in g.integers(3, V, 3)]
        return [s[-1]] + rnd[:1] + right + rnd[1:] + [0], [-1, 0, 0, 2, 3, 4, 1, 6, -2]

    tree, rounds = run(model, dtype, 9, steps, drafts)
    sure, total = check(model, tree, MARGIN[dtype])
    assert total >= 3 * ROWS and sure >= total // 4
    assert rounds < 0.8 * max(len(s) - 1 for s in tree)  # confirmed drafts save steps
