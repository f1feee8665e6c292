"""The oracle of the 8-bit token and channel operators: closed forms and hand-worked cases."""
import numpy as np
import pytest

from oracle import token8


def test_select_by_hand():
    l = np.log(np.array([[1.0, 4.0, 2.0, 1.0], [1.0, 1.0, 1.0, 1.0]]))
    ids, w, bad = token8.select(l, 2)
    assert ids.tolist() == [[1, 2], [0, 1]] and np.allclose(w, [[4 / 6, 2 / 6], [0.5, 0.5]]) and not bad.any()
    ids, w, _ = token8.select(l, 2, renorm=False, scaling=3.0)
    assert np.allclose(w, [[1.5, 0.75], [0.75, 0.75]])
    # a bias ranks and does not weigh
    ids, w, _ = token8.select(l[:1], 2, bias=[1.0, 0, 0, 0], renorm=False)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, [[1 / 8, 4 / 8]])


def test_select_groups():
    v = np.array([[0.9, 0.1, 0.6, 0.5]])
    l = np.log(v / (1 - v))
    assert token8.select(l, 1, softmax=False, groups=2, keep=1, top2=True)[0].tolist() == [[2]]   # 1.1 over 1.0
    assert token8.select(l, 1, softmax=False, groups=2, keep=1, top2=False)[0].tolist() == [[0]]
    # equal groups: the lower; excluded experts add nothing
    assert token8.select(np.zeros((1, 4)), 2, softmax=False, groups=2, keep=1)[0].tolist() == [[0, 1]]
    ids, w, _ = token8.select(np.array([[0.0, -np.inf, -np.inf, -np.inf]]), 2, softmax=False, groups=2, keep=1)
    assert ids.tolist() == [[0, -1]] and w.tolist() == [[1.0, 0.0]]
    ids, w, bad = token8.select(np.array([[0.0, np.nan], [0.0, np.inf], [-np.inf, -np.inf]]), 1)
    assert bad.tolist() == [True, True, False] and (ids == -1).all() and (w == 0).all()


def test_group_by_hand():
    idx = np.array([[2, 0], [0, -1], [2, 5]])
    off, rows, slots = token8.group(idx, 4)
    assert off.tolist() == [0, 2, 2, 4, 4] and rows.tolist() == [0, 1, 0, 2] and slots.tolist() == [[2, 0], [1, -1], [3, -1]]
    off, rows, slots = token8.group(idx, 4, 0, 2)
    assert off.tolist() == [0, 2, 4] and rows.tolist() == [0, 1, 0, 2]
    assert token8.group(idx, 4, 1, 2)[0].tolist() == [0, 0, 0]


def test_quantize_by_hand():
    q, s = token8.quantize([[127.0, 0.5, 1.5, -2.5], [0.0, 0.0, 0.0, 0.0], [np.inf, 1.0, 0.0, 0.0], [2.0 ** -101, 0, 0, 0]])
    assert q.tolist() == [[127, 0, 2, -2], [0] * 4, [0] * 4, [0] * 4] and s[0] == 1.0 and s[1] == 0.0 and np.isnan(s[2]) and s[3] == 0.0
    assert token8.swiglu([[0.0, 100.0, 3.0, 2.0]]).tolist() == [[0.0, 200.0]]


def test_sums_and_combine():
    x, w = np.array([[1, -2], [3, 4]]), np.array([[[1, 1]], [[2, -1]]])
    assert token8.sums(x, w, [0, 1, 3], [1, 0, 1]).tolist() == [[7], [4], [2]]
    assert token8.sums(x, w, [0, 1, 1], [1, 0, 7]).tolist() == [[7], [0], [0]]
    assert token8.sums(x, w, [1, 0, 9], [1, 0, 7]).tolist() == [[0], [4], [0]]      # ascending, row 7 does not exist
    y, mag = token8.combine(np.array([[1.0], [10.0]]), np.array([[1, -1], [0, 1]]), np.array([[0.5, np.nan], [2.0, -0.1]]), [[3.0], [0.0]])
    assert y.tolist() == [[8.0], [1.0]] and mag.tolist() == [[8.0], [3.0]]


@pytest.mark.parametrize("seed", range(3))
def test_select_without_groups_is_plain_topk(seed):
    l = np.random.default_rng(seed).standard_normal((5, 37))
    ids, w, _ = token8.select(l, 6, softmax=bool(seed % 2))
    assert (ids == np.argsort(-l, axis=-1, kind="stable")[:, :6]).all() and np.allclose(w.sum(-1), 1.0)
