"""Group-limited routing where experts are masked: the oracle (oracle/layer.py) on cases worked by hand (CPU only).

A group's score is the sum of its group_top largest scores, of the experts that can be chosen.  A group with one of them
has that one's score, a group with none comes after all others."""
import math

import numpy as np
import pytest

from oracle import layer as ol

INF = np.inf


def logit(p):
    return math.log(p / (1 - p))


def masked(E, at):
    """Logits of E experts of which only those in `at` can be chosen."""
    l = np.full((1, E), -INF)
    for e, v in at.items():
        l[0, e] = v
    return l


def test_the_only_expert_left_is_found():
    b = np.full(8, -INF)
    b[3] = 0
    for group_top in (1, 2):
        for score in ("softmax", "sigmoid"):
            ids, w = ol.route(np.zeros((1, 8)), 2, score, bias=b, n_groups=4, topk_groups=1, group_top=group_top)
            assert ids.tolist() == [[3, -1]] and w[0].tolist() == [1, 0]


def test_groups_of_one_candidate_are_ordered_by_it():
    for group_top in (1, 2):
        ids, _ = ol.route(masked(8, {1: 0, 3: 9, 6: 3}), 2, n_groups=4, topk_groups=1, group_top=group_top)
        assert ids.tolist() == [[3, -1]]
        ids, _ = ol.route(masked(8, {1: 0, 3: 9, 6: 3}), 2, n_groups=4, topk_groups=2, group_top=group_top)
        assert ids.tolist() == [[3, 6]]


@pytest.mark.parametrize("pair,first", [(0.3, 5), (0.48, 0)])
def test_one_candidate_against_a_pair(pair, first):
    """0.9 alone against twice 0.3 (0.6) and twice 0.48 (0.96)."""
    l = masked(6, {0: logit(pair), 1: logit(pair), 5: logit(0.9)})
    ids, _ = ol.route(l, 2, "sigmoid", n_groups=2, topk_groups=1, group_top=2)
    assert ids[0, 0] == first


def test_one_negative_key_against_a_pair():
    """Keys are s + b: -0.5 alone against -0.3 twice (-0.6): sums, whatever their sign."""
    l = np.zeros((1, 4))                                     # sigmoid 0.5
    ids, _ = ol.route(l, 2, "sigmoid", bias=np.array([-0.8, -0.8, -1.0, -INF]), n_groups=2, topk_groups=1, group_top=2)
    assert ids.tolist() == [[2, -1]]


def test_an_empty_group_is_last():
    l = masked(8, {4: 0, 5: 0, 6: 0})
    for group_top in (1, 2):
        ids, _ = ol.route(l, 3, "sigmoid", bias=np.full(8, -7.0), n_groups=4, topk_groups=2, group_top=group_top)
        assert ids.tolist() == [[4, 5, 6]]
    # and of equal ones the lower comes first
    ids, _ = ol.route(masked(8, {2: 1, 4: 1}), 2, n_groups=4, topk_groups=1, group_top=2)
    assert ids.tolist() == [[2, -1]]
