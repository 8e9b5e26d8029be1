"""Pins of the paged cache's oracle on cases worked out by hand."""
import numpy as np

import oracle.kv_oracle as KV


def test_plan_by_hand():
    # page size 4: request 0 continues page 9 at place 3 and takes page 5; request 1 takes page 2; request 2 nothing
    p = KV.plan([3, 0, 8], [2, 4, 0], [5, 2, 7], [[9, -1], [-1, -1], [1, 3]], 4, 8, [-1, 0, -1, 0, 0, 2], 1)
    assert p["table"].tolist() == [[9, 5], [2, -1], [1, 3]]
    assert p["cu_new"].tolist() == [0, 2, 6, 6] and p["taken"] == 2
    assert p["slots"].tolist() == [39, 20, 8, 9, 10, 11, -1, -1]
    assert p["positions"].tolist() == [3, 4, 0, 1, 1, 2, 0, 0]
    assert p["mask"][:, 0].tolist() == [1, 3, 1, 3, 5, 13, 0, 0]


def test_attend_by_hand():
    # equal scores: the average of what is seen; a query along one key with a large scale: that key's value
    k = np.zeros((3, 1, 2))
    v = np.array([[[1.0, 0]], [[3.0, 2]], [[100.0, -9]]])
    seen = np.array([[True, True, False], [False, False, False]])
    out, w = KV.attend(np.ones((2, 2, 2)), k, v, seen, 1.0)
    assert np.allclose(out[0], [[2, 1], [2, 1]]) and not out[1].any() and np.allclose(w[0], [[2, 1], [2, 1]])
    k[1, 0] = [1, 0]
    out, _ = KV.attend(np.array([[[1.0, 0]]]), k, v, np.ones((1, 3), bool), 1000.0)
    assert np.allclose(out[0, 0], [3, 2])
    out, _ = KV.attend(np.array([[[np.log(3.0), 0]]]), k, v, np.array([[True, True, False]]), 1.0)
    assert np.allclose(out[0, 0], [0.25 * 1 + 0.75 * 3, 0.75 * 2])


def test_visible():
    assert KV.visible(2, 2).tolist() == [[True, True, True, False], [True] * 4]
    assert KV.visible(1, 2, [[1], [2]]).tolist() == [[True, True, False], [True, False, True]]


def test_hidden_values_do_not_matter():
    rng = np.random.default_rng(0)
    q, k, v = rng.normal(size=(1, 2, 4)), rng.normal(size=(5, 2, 4)), rng.normal(size=(5, 2, 4))
    seen = np.array([[True, False, True, True, False]])
    a, _ = KV.attend(q, k, v, seen, 0.5)
    k[1], v[4] = np.nan, np.inf
    b, _ = KV.attend(q, k, v, seen, 0.5)
    assert np.array_equal(a, b)
