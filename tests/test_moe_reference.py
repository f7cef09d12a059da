"""The routing reference of the GPU tests on inputs whose groups are decided by
hand, so that a reference that keeps another group cannot pass."""
import numpy as np

import moe_ref


def kept(score, bias=None, **kw):
    """The experts chosen with softmax scores `score` (of sum 1), two of one kept group of two."""
    ids, _, off, rows = moe_ref.route(np.log(np.array([score])), bias, 2, groups=2, groups_kept=1, **kw)
    assert off.tolist() == np.r_[0, np.cumsum([e in ids for e in range(4)])].tolist()
    assert sorted(rows.tolist()) == [0, 1]
    return ids.tolist()


def test_one_or_two_largest_of_a_group():
    # group 0 has the largest score, group 1 the larger sum
    score = [0.41, 0.04, 0.25, 0.30]
    assert kept(score, group_top=1) == [[0, 1]]
    assert kept(score, group_top=2) == [[3, 2]]
    # a bias that turns either around
    assert kept(score, np.array([0, 0, 0.125, 0.125]), group_top=1) == [[3, 2]]
    assert kept(score, np.array([0, 0.25, 0, 0]), group_top=2) == [[0, 1]]


def test_equal_groups_keep_the_lower():
    for top in (1, 2):
        assert kept([0.125, 0.375, 0.375, 0.125], group_top=top) == [[1, 0]]
        assert kept([0.25, 0.25, 0.25, 0.25], group_top=top) == [[0, 1]]


def test_a_group_of_one_expert_left():
    z = np.array([[1.0, -np.inf, 0.9, 0.8]])
    # sigmoids 0.73 alone against 0.71 + 0.69
    for top, want in ((1, [[0, -1]]), (2, [[2, 3]])):
        ids, w, _, _ = moe_ref.route(z, None, 2, "sigmoid", groups=2, groups_kept=1, group_top=top)
        assert ids.tolist() == want and (w > 0).tolist() == [[i >= 0 for i in want[0]]]
