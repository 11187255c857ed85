"""Decoding with drafted trees through the three operators together, as a program uses them: a small
random decoder with cross attention.  The tokens must be those of decoding one token at a time, and
both those of the plain float64 model, wherever that model's choice is clear."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import serving_ls_beam_gb300 as lsb  # noqa: E402
from serving_ls_beam_gb300.draft import DraftTreeDecoder  # noqa: E402

L, H, HK, D, V, EOS = 2, 4, 2, 64, 97, 2
W = H * D
BATCH, BEAMS, SRC = 3, 2, 23
ROWS = BATCH * BEAMS
CLEAR = 0.02  # a choice whose two best logits are closer is not compared (f32 sums differ by about 1e-4)


@pytest.fixture(scope="module")
def model():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    lsb.load_library()
    g = torch.Generator().manual_seed(7)

    def r(*s):
        return (torch.randn(s, generator=g, dtype=torch.float64) / s[0] ** 0.5).cuda()

    m = {"emb": r(V, W) * V ** 0.5, "pos": r(200, W) * 200 ** 0.5 * 0.5, "out": r(W, V) * 6,
         "layers": [{n: r(W, H * D) if n in ("q", "cq", "o", "co") else r(W, HK * D) for n in ("q", "k", "v", "o", "cq", "co")}
                    for _ in range(L)]}
    m["enc"] = [(torch.randn((BATCH, HK, SRC, D), generator=g, dtype=torch.float64).cuda(),
                 torch.randn((BATCH, HK, SRC, D), generator=g, dtype=torch.float64).cuda()) for _ in range(L)]
    m["src_len"] = [SRC, 5, 14]
    m["start"] = torch.arange(3, 3 + ROWS)
    return m


def norm(x):
    return x / x.pow(2).mean(-1, keepdim=True).sqrt()


def attend64(q, k, v):
    """q [t, H, D] over k, v [n, HK, D]; causal where they are of one length."""
    k, v = k.repeat_interleave(H // HK, 1), v.repeat_interleave(H // HK, 1)
    s = torch.einsum("thd,nhd->htn", q, k) * D ** -0.5
    if q.shape[0] == k.shape[0]:
        s = s.masked_fill(torch.triu(torch.ones(s.shape[1:], dtype=torch.bool, device=s.device), 1), -np.inf)
    return torch.einsum("htn,nhd->thd", torch.softmax(s, -1), v)


def logits64(m, row, tokens):
    x = m["emb"][tokens] + m["pos"][: len(tokens)]
    b = row // BEAMS
    for i, p in enumerate(m["layers"]):
        y = norm(x)
        t = len(tokens)
        x = x + attend64((y @ p["q"]).view(t, H, D), (y @ p["k"]).view(t, HK, D), (y @ p["v"]).view(t, HK, D)).reshape(t, W) @ p["o"]
        k, v = (e[b, :, : m["src_len"][b]].transpose(0, 1) for e in m["enc"][i])
        y = norm(x)
        q = (y @ p["cq"]).view(t, H, D)
        x = x + torch.cat([attend64(q[j:j + 1], k, v)
                           for j in range(t)]).reshape(t, W) @ p["co"]
    return norm(x) @ m["out"]


def run(m, dtype, nodes, steps, drafts):
    """Greedy decoding; drafts(row tokens so far) -> (tokens, parents) of `nodes` nodes, node 0 the last token."""
    f = {k: (v.to(dtype) if torch.is_tensor(v) else v) for k, v in m.items()}
    f["layers"] = [{k: v.to(dtype) for k, v in p.items()} for p in m["layers"]]
    enc = [(k.to(dtype), v.to(dtype)) for k, v in m["enc"]]
    dec = DraftTreeDecoder(L, ROWS, nodes, H, HK, D, 64, V, EOS, dtype=dtype, beams=BEAMS)
    dec.reset(enc, torch.tensor(m["src_len"], dtype=torch.int32, device="cuda"))
    seqs = [[int(t)] for t in m["start"]]
    rounds = 0
    while any(len(s) < steps and s[-1] != EOS for s in seqs) and rounds < steps:
        rounds += 1
        guess = [drafts(r, s) for r, s in enumerate(seqs)]
        token = torch.tensor([g[0] for g in guess], dtype=torch.int32, device="cuda")
        parent = torch.tensor([g[1] for g in guess], dtype=torch.int32, device="cuda")
        depth = []
        for _, par in guess:
            d = []
            for p in par:
                d.append(0 if p < 0 else d[p] + 1)
            depth.append(d)
        at = dec.length()[:, None].long() + torch.tensor(depth, device="cuda")
        x = f["emb"][token.long()] + f["pos"][at]
        for i, p in enumerate(f["layers"]):
            y = norm(x)
            o = dec.self_attention(i, (y @ p["q"]).view(ROWS, nodes, H, D), (y @ p["k"]).view(ROWS, nodes, HK, D),
                                   (y @ p["v"]).view(ROWS, nodes, HK, D), parent)
            x = x + o.reshape(ROWS, nodes, W) @ p["o"]
            o = dec.cross_attention(i, (norm(x) @ p["cq"]).view(ROWS, nodes, H, D))
            x = x + o.reshape(ROWS, nodes, W) @ p["co"]
        nxt = dec.finish((norm(x) @ f["out"]).contiguous(), token, parent)
        assert lsb.ls_read_status(dec.workspace) == lsb.LS_OK
        path, count = dec.path.cpu().numpy(), dec.count.cpu().numpy()
        tok, end = nxt.cpu().numpy(), dec.finished[dec.cur].cpu().numpy()
        for r in range(ROWS):
            if seqs[r][-1] == EOS:
                continue
            seqs[r] += [guess[r][0][n] for n in path[r][1:count[r]]] + [int(tok[r])]
            assert (seqs[r][-1] == EOS) == bool(end[r])
        assert all(int(n) == len(s) - 1 for n, s in zip(dec.length().cpu(), seqs))
    return seqs, rounds


def test_drafted_trees_decode_what_single_tokens_do(model):
    steps = 24
    single, _ = run(model, torch.float32, 1, steps, lambda r, s: ([s[-1]], [-1]))
    g = np.random.default_rng(3)
    # the plain model's greedy sequences, as far as its choices are clear
    clear = []
    for r in range(ROWS):
        s, n = [int(model["start"][r])], 1
        while len(s) < steps and s[-1] != EOS:
            top = logits64(model, r, torch.tensor(s, device="cuda"))[-1].topk(2)
            if (top.values[0] - top.values[1]).item() < CLEAR:
                break
            s.append(int(top.indices[0]))
            n = len(s)
        clear.append(s[:n])
        assert single[r][:n] == s[:n], r
    assert sum(len(c) for c in clear) > ROWS * 4  # most choices are compared

    def drafts(r, s):
        """Two branches: what the single-token search says (wrong after a while) and a random one; an empty place."""
        right = single[r][len(s):len(s) + 4]
        right = (right + [5] * 4)[:4]
        if g.random() < 0.5:
            right[2] = (right[2] + 1) % V
        rnd = [int(t) for t in g.integers(3, V, 3)]
        return [s[-1]] + rnd[:1] + right + rnd[1:] + [0], [-1, 0, 0, 2, 3, 4, 1, 6, -2]

    tree, rounds = run(model, torch.float32, 9, steps, drafts)
    for r in range(ROWS):
        n = len(clear[r])
        assert tree[r][:n] == clear[r], (r, tree[r], clear[r])
    assert rounds < steps * 0.7  # confirmed drafts save steps


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_sixteen_bit_types_run(model, dtype):
    seqs, rounds = run(model, dtype, 5, 12, lambda r, s: ([s[-1], 7, 8, 9, 10], [-1, 0, 0, 1, -2]))
    assert rounds <= 12 and all(len(s) >= 2 for s in seqs)


def test_rows_that_do_not_divide_by_beams_are_refused():
    with pytest.raises(ValueError):
        DraftTreeDecoder(1, 5, 1, 1, 1, 64, 8, 10, 2, device="cpu", beams=2)
