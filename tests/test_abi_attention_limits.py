"""Counts that 32 or 64 bits do not hold, and outputs that are inputs, are refused by the attention and commit
entry points (no GPU: all of it is found on the host).  Each call runs in a process of its own, with the pointer checks off, so that
an abort would be a failed test and nothing else."""
import subprocess
import sys

import pytest

INVALID, UNSUPPORTED = 1, 2

CALL = """
import os
os.environ["LS_BEAM_DEBUG"] = "nocheck"
import serving_ls_beam_gb300 as lsb
L, P = lsb.load_library(), 4096  # an address that no refused call looks behind
def view(row=64, pos=64, head=8):
    return lsb._View(P, 0, row, pos, head)
def cross(b=2, k=4, t=1, h=8, hk=8, n=16, d=8, size=1 << 40):
    return L.ls_cross_attention(view(), view(), view(), 1, P, 1.0, b, k, t, h, hk, n, d, view(), P, size, None)
def tree(rows=2, nodes=4, h=8, hk=8, n=16, d=8, size=1 << 40):
    return L.ls_tree_attention(view(), view(), view(), P, view(), view(), P, 2, 1.0, rows, nodes, h, hk, n, d, view(), P,
                               size, None)
def commit(rows=2, layers=1, nodes=4, heads=2, n=8, d=8, out_len=2 * P, finished=None, out_finished=None):
    return L.ls_tree_commit(P, 2 * P, P, view(), view(), 1, P, P, P, finished, 2, layers, rows, nodes, heads, n, d, out_len,
                            P, P, P, out_finished, None, None)
print("status", EXPR)
"""


@pytest.fixture(scope="module")
def call():
    from serving_ls_beam_gb300 import _build

    _build.build()

    def run(expr):
        r = subprocess.run([sys.executable, "-c", CALL.replace("EXPR", expr)], capture_output=True, text=True, timeout=120)
        assert r.returncode == 0, (expr, r.returncode, r.stderr[-400:])
        return int(r.stdout.split()[-1])

    return run


def test_queries_per_key_of_a_tree(call):
    """nodes * group past 31 bits: products that wrap to 0 (a division by it) and to a small count (64)."""
    assert call("tree(nodes=4, h=1 << 30, hk=1)") == UNSUPPORTED
    assert call("tree(nodes=64, h=1 << 27, hk=1)") == UNSUPPORTED
    assert call("tree(nodes=64, h=(1 << 26) + 1, hk=1)") == UNSUPPORTED
    assert call("tree(nodes=64, h=(1 << 26) + 1, hk=1, size=0)") == UNSUPPORTED  # and no workspace is looked at
    assert call("cross(k=1 << 26, t=64, h=8, hk=1)") == UNSUPPORTED
    assert call("tree(size=0)") == INVALID


def test_queries_of_a_call(call):
    """Rows x key heads x queries per key past 31 bits, also where 64 bits do not hold the product (2^64, 2^64 + 2^14)."""
    assert call("cross(b=1 << 30, k=1, t=1 << 14, h=1 << 20, hk=1 << 20)") == UNSUPPORTED
    assert call("cross(b=(1 << 30) + 1, k=1, t=1 << 14, h=1 << 20, hk=1 << 20)") == UNSUPPORTED
    assert call("cross(b=1 << 20, k=1, t=1 << 11, h=1, hk=1)") == UNSUPPORTED
    assert call("tree(rows=1 << 30, nodes=64, h=1 << 28, hk=1 << 28)") == UNSUPPORTED
    assert call("tree(rows=1 << 30, nodes=2, h=1, hk=1)") == UNSUPPORTED
    # rows long enough to be cut in parts: the number of parts is divided by that product
    assert call("cross(b=1 << 30, k=1, t=1 << 14, h=1 << 20, hk=1 << 20, n=1 << 16)") == UNSUPPORTED
    assert call("tree(rows=1 << 30, nodes=64, h=1 << 28, hk=1 << 28, n=1 << 16)") == UNSUPPORTED


def test_elements_of_a_commit(call):
    """nodes x heads x head_dim elements past 2^30, also where 64 bits do not hold the product."""
    assert call("commit(nodes=8, heads=1 << 30, d=1 << 30)") == UNSUPPORTED
    assert call("commit(nodes=64, heads=(1 << 31) - 1, d=(1 << 31) - 1)") == UNSUPPORTED
    assert call("commit(nodes=64, heads=1 << 14, d=(1 << 9) + 1)") == UNSUPPORTED
    assert call("commit(layers=65536)") == UNSUPPORTED


def test_positions_of_a_row(call):
    """Lengths whose sums with the drafted tokens and a block's keys 32 bits would not hold."""
    for n in ((1 << 31) - 1, (1 << 31) - 64, (1 << 31) - 1023):
        assert call(f"cross(n={n})") == UNSUPPORTED
        assert call(f"tree(n={n})") == UNSUPPORTED
        assert call(f"cross(n={n}, b=0)") == 0 and call(f"tree(n={n}, rows=0)") == 0


def test_outputs_that_every_layer_reads(call):
    """A layer's block may run after the first one's results are written."""
    assert call("commit(out_len=P)") == INVALID  # cache_len itself
    assert call("commit(layers=6, finished=3 * P, out_finished=3 * P)") == INVALID
    assert call("commit(layers=1, finished=3 * P + 1, out_finished=3 * P + 1)") == INVALID
