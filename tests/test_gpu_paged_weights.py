"""The softmax weights of 16-bit paged attention lose less on the way to the values than the result in its own rounding, also
where values of both signs nearly cancel.

Bound: that of f32 arithmetic (paged_plain.attend), the result's rounding, and a weight in two pieces of its type, each off
by half a step: 2^-22 of it in f16, 2^-16 in bf16 (bf16 queries over 8-bit pages: one piece in f16, 2^-11); in f16 a piece is
a whole number of 2^-24, of weights whose largest is 2^7 at least: 2^-32 of it for each."""
import numpy as np
import pytest

import paged_plain as pp

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import serving_ls_beam_gb300 as lsb  # noqa: E402
from test_gpu_paged_attention import DT, Cache, dev, f64, kernel, workspace  # noqa: E402,F401


@pytest.mark.parametrize("dtype,cache", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3"), ("f16", "i8"), ("bf16", "i8")])
@pytest.mark.parametrize("heads,kv,dim,page,lens", [(4, 4, 64, 16, [3, 40, 700]), (8, 2, 128, 64, [2, 90, 3000]), (12, 1, 96, 8, [33, 500]),
                                                    (2, 1, 256, 16, [5, 260])])
def test_weights(dev, kernel, dtype, cache, heads, kv, dim, page, lens):  # noqa: F811
    g = np.random.default_rng(dim)
    c = Cache(g, dev, cache, kv, dim, page, lens)
    q = torch.from_numpy(g.normal(size=(len(lens), heads, dim)).astype(np.float32)).to(DT[dtype]).to(dev)
    out = torch.empty_like(q)
    ws = workspace(lsb.ls_paged_attention_workspace_size(len(lens), heads, kv, dim), dev)
    lsb.check(lsb.ls_paged_attention(q, c.pages(), torch.tensor(lens, dtype=torch.int32, device=dev), out, ws))
    assert lsb.ls_read_status(ws) == 0
    half = cache != "bf16"
    wu = 2.0 ** -16 if not half else 2.0 ** -22 if dtype == "f16" else 2.0 ** -11
    for r in range(len(lens)):
        (ks, _), (vs, sv) = c.row("key", r), c.row("value", r)
        for h in range(heads):
            k, v, s = ks[h * kv // heads], vs[h * kv // heads], sv[h * kv // heads]
            x = f64(q)[r, h]
            want, bound = pp.attend(x, k, v, s, dim ** -0.5, "f32", cache)
            p = np.exp(k @ x * dim ** -0.5)
            p /= p.sum()
            bound = bound + pp.UNIT[dtype] * np.abs(want) + wu * (p @ np.abs(v))
            if half:
                top = (p * s).max() * (np.abs(v) / s[:, None]).max()
                bound = bound + 2 * len(p) * 2.0 ** -32 * top
            if dtype == "f16":
                bound = bound + 2.0 ** -25
            bad = ~(np.abs(f64(out)[r, h] - want) <= 1.0001 * bound)
            assert not bad.any(), (r, h, np.abs(f64(out)[r, h] - want)[bad][:3], bound[bad][:3])
