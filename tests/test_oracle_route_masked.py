"""The plain form of routing with experts masked by a logit of -infinity. No GPU."""
import numpy as np
import pytest

from oracle import step as st

INF = np.inf


def test_worked_masks():
    x = np.array([[-INF, -3.0, -2.0, -1.0]], dtype=np.float32)
    bias = np.array([0.5, 0.0, 0.0, 0.0], dtype=np.float32)
    idx, w = st.route_experts(x, 2, "sigmoid", bias)
    assert idx.tolist() == [[3, 2]] and (w > 0).all()
    assert st.route_experts(x, 4, "sigmoid", bias)[0].tolist() == [[3, 2, 1, 0]]
    # softmax: the scores of 0 and 1 beside 200 round to 0 in fp32
    x = np.array([[200.0, -INF, 0.0, 1.0]], dtype=np.float32)
    assert st.route_experts(x, 4, "softmax", np.zeros(4, dtype=np.float32))[0].tolist() == [[0, 2, 3, 1]]


def test_worked_groups():
    # {-inf, -inf} with a large bias against {0.1, 0.2}; then a group with one expert left
    x = np.array([[-INF, -INF, -2.0, -1.5]], dtype=np.float32)
    bias = np.array([5.0, 5.0, 0.0, 0.0], dtype=np.float32)
    for top in (1, 2):
        assert st.route_experts(x, 2, "sigmoid", bias, 2, 1, top)[0].tolist() == [[3, 2]]
    x[0, 0] = 3.0
    assert st.route_experts(x, 2, "sigmoid", bias, 2, 1, 1)[0].tolist() == [[0, 1]]
    assert st.route_experts(x, 2, "sigmoid", bias, 2, 1, 2)[0].tolist() == [[3, 2]]  # the sum is -infinity


def test_nan_stays_behind_masks():
    x = np.array([[0.0, -INF, 1.0, np.nan]], dtype=np.float32)
    bias = np.array([0.0, np.nan, 0.0, 0.0], dtype=np.float32)
    # sigmoid: expert 1 is masked, its bias is NaN: a NaN comes after every number, the lower id first
    assert st.route_experts(x, 4, "sigmoid", bias)[0].tolist() == [[2, 0, 1, 3]]
    # softmax: one NaN among a token's logits makes all its scores NaN, masked or not
    with np.errstate(invalid="ignore"):
        assert st.route_experts(x, 4, "softmax", bias)[0].tolist() == [[0, 1, 2, 3]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_values_that_are_not_masked_are_untouched(score):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 8)).astype(np.float32)
    bias = rng.standard_normal(8).astype(np.float32)
    s = st.sigmoid(x) if score == "sigmoid" else st.softmax(x)
    np.testing.assert_array_equal(st.choice_values(x, score, bias), (s + bias.astype(np.float64)).astype(np.float32))


def test_groups_with_one_expert_left():
    """Groups whose sum of two is -infinity are ranked by their largest value: one with an expert that is not masked
    comes before one without."""
    x = np.array([[-INF, -INF, -INF, 2.0, 1.0, -INF]], dtype=np.float32)
    for score in ("sigmoid", "softmax"):
        for bias in (None, np.zeros(6, dtype=np.float32), np.array([9, 9, 0, 0, 0, 0], dtype=np.float32)):
            assert st.route_experts(x, 2, score, bias, 3, 1, 2)[0].tolist() == [[3, 2]]
            assert st.route_experts(x, 2, score, bias, 3, 2, 2)[0].tolist() == [[3, 4]]
    # and after every group with two
    x[0, 0:2] = -20.0
    assert st.route_experts(x, 2, "sigmoid", np.zeros(6, dtype=np.float32), 3, 1, 2)[0].tolist() == [[0, 1]]
    # equal ones by their ids; by a bias of -infinity as by a mask
    x = np.array([[1.0, 0.0, 1.0, 0.0]], dtype=np.float32)
    bias = np.array([0, -INF, 0, -INF], dtype=np.float32)
    assert st.route_experts(x, 1, "sigmoid", bias, 2, 1, 2)[0].tolist() == [[0]]
    x[0, 2] = 1.5
    assert st.route_experts(x, 1, "sigmoid", bias, 2, 1, 2)[0].tolist() == [[2]]
