"""Pins of the float64 definitions that the attention tests compare against (no GPU): closed
forms, so that a wrong scale, index, mask or group would show."""
import numpy as np

import attention_plain as ap


def test_equal_scores_average_the_values():
    g = np.random.default_rng(0)
    v = g.normal(size=(1, 2, 5, 3))
    q = np.zeros((1, 2, 1, 4, 3))
    k = g.normal(size=(1, 2, 5, 3))
    out, _ = ap.cross(q, k, v, [4], 0.5, "f32")
    for h in range(4):
        np.testing.assert_allclose(out[0, 1, 0, h], v[0, h // 2, :4].mean(0), atol=1e-12)


def test_a_large_score_selects_its_key():
    k = np.zeros((2, 1, 6, 2))
    k[:, 0, 3, 0] = 1.0
    v = np.arange(24, dtype=float).reshape(2, 1, 6, 2)
    q = np.zeros((2, 1, 1, 1, 2))
    q[..., 0] = 1000.0
    out, _ = ap.cross(q, k, v, [6, 3], 1.0, "f32")
    np.testing.assert_allclose(out[0, 0, 0, 0], v[0, 0, 3])
    np.testing.assert_allclose(out[1, 0, 0, 0], v[1, 0, :3].mean(0))  # key 3 is past the length
    assert not ap.cross(q, k, v, [0, 0], 1.0, "f32")[0].any()


def test_scale_by_two_keys():
    q, k, v = np.ones((1, 1, 1, 1, 1)), np.array([0.0, 1.0]).reshape(1, 1, 2, 1), np.array([0.0, 1.0]).reshape(1, 1, 2, 1)
    out, _ = ap.cross(q, k, v, [2], 3.0, "f32")
    np.testing.assert_allclose(out.ravel(), [1 / (1 + np.exp(-3.0))])


def test_branches():
    parents = [-1, 0, 0, 1, -2, 4, 7, -1]
    assert [ap.branch(parents, i) for i in range(8)] == [[0], [1, 0], [2, 0], [3, 1, 0], [], [], [], [7]]


def test_tree_sees_its_branch_only():
    q = np.zeros((1, 4, 1, 1))
    ck, cv = np.zeros((1, 1, 3, 1)), np.array([6.0, 9.0, 100.0]).reshape(1, 1, 3, 1)
    dk, dv = np.zeros((1, 4, 1, 1)), np.array([3.0, 5.0, 7.0, np.nan]).reshape(1, 4, 1, 1)
    out, _ = ap.tree(q, ck, cv, [2], dk, dv, np.array([[-1, 0, 0, -2]]), 1.0, "f32")
    np.testing.assert_allclose(out.ravel(), [(6 + 9 + 3) / 3, (6 + 9 + 3 + 5) / 4, (6 + 9 + 3 + 7) / 4, 0])


def test_one_node_is_causal_attention_over_the_cache_and_itself():
    g = np.random.default_rng(1)
    q, c, v = g.normal(size=(1, 1, 2, 4)), g.normal(size=(1, 2, 7, 4)), g.normal(size=(1, 2, 7, 4))
    full, _ = ap.cross(q[:, None], c, v, [7], 0.7, "f32")
    out, _ = ap.tree(q, c[:, :, :6], v[:, :, :6], [6], c[:, None, :, 6], v[:, None, :, 6], np.array([[-1]]), 0.7, "f32")
    np.testing.assert_allclose(out[0, 0], full[0, 0, 0], atol=1e-12)


def test_commit_by_hand():
    parent = np.array([[-1, 0, 0, 1, 2, 2]])
    token = np.array([[5, 10, 11, 12, 13, 13]])
    target = np.array([[11, 0, 13, 0, 17, 18]])
    assert ap.commit([3], parent, token, target, None, 2, 100) == [([0, 2, 4], 17, 0)]
    assert ap.commit([98], parent, token, target, None, 2, 100) == [([0, 2], 13, 0)]  # two places left
    assert ap.commit([100], parent, token, target, None, 2, 100) == [([], 5, 0)]
    assert ap.commit([3], parent, token, target, [1], 2, 100) == [([], 2, 1)]
    assert ap.commit([3], parent, token, target, None, 13, 100) == [([0, 2], 13, 1)]  # 13 is the end token
