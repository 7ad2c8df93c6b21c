"""The plain forms of routing by scores, RMS norm and AdamW, pinned by hand-worked
examples, brute force, differences and the formats' own definitions. No GPU."""
import itertools

import numpy as np
import pytest

from oracle import step as st


def test_worked_sigmoid_router():
    # sigmoids 0.5, 0.75, 0.9, 0.25; the bias lifts expert 3 over expert 2
    x = np.log(np.array([[1.0, 3.0, 9.0, 1 / 3]]))
    bias = np.array([0.0, 0.0, -0.5, 0.5], dtype=np.float32)
    idx, w = st.route_experts(x, 2, "sigmoid", bias)
    assert idx.tolist() == [[1, 3]]  # c: 0.5, 0.75, 0.4, 0.75 (a tie: the lower id)
    np.testing.assert_allclose(w, [[0.75, 0.25]], rtol=1e-6)
    idx, w = st.route_experts(x, 2, "sigmoid", bias, renormalize=False, scale=2.0)
    np.testing.assert_allclose(w, [[1.5, 0.5]], rtol=1e-6)


def test_worked_groups():
    # two groups: {0.9, 0.1} and {0.6, 0.5}; by their largest the first wins, by their two largest the second
    s = np.array([0.9, 0.1, 0.6, 0.5])
    x = np.log(s / (1 - s))[None]
    assert st.route_experts(x, 2, "sigmoid", None, 2, 1, 1)[0].tolist() == [[0, 1]]
    assert st.route_experts(x, 2, "sigmoid", None, 2, 1, 2)[0].tolist() == [[2, 3]]
    assert st.route_experts(x, 2, "sigmoid", None, 2, 2, 2)[0].tolist() == [[0, 2]]


def test_ties_nans_and_infinities():
    x = np.zeros((1, 6), dtype=np.float32)
    assert st.route_experts(x, 6, "softmax")[0].tolist() == [[0, 1, 2, 3, 4, 5]]
    x[0] = [np.nan, -np.inf, 1.0, -0.0, 0.0, np.inf]
    assert st.route_experts(x, 6, "softmax")[0].tolist() == [[5, 2, 3, 4, 1, 0]]
    assert st.route_experts(x, 4, "softmax", None, 3, 2, 1)[0].tolist() == [[5, 2, 3, 4]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_choice_against_brute_force(score):
    """Among all sets of top_groups groups and k experts of theirs, the one whose sorted
    values are largest."""
    rng = np.random.default_rng(3)
    E, groups, top_groups, k = 8, 4, 2, 3
    for _ in range(20):
        x = rng.standard_normal((1, E)).astype(np.float32)
        bias = (0.3 * rng.standard_normal(E)).astype(np.float32)
        c = st.choice_values(x, score, bias, groups, 2)[0]
        best = max(itertools.combinations(range(groups), top_groups),
                   key=lambda gs: sorted((c[2 * g] + c[2 * g + 1] for g in gs), reverse=True))
        pool = [e for g in best for e in (2 * g, 2 * g + 1)]
        want = max(itertools.permutations(pool, k), key=lambda es: [c[e] for e in es])
        assert st.route_experts(x, k, score, bias, groups, top_groups, 2)[0][0].tolist() == list(want)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_route_gradient_against_differences(score, renormalize):
    rng = np.random.default_rng(5)
    T, E, k, h = 3, 7, 3, 1e-6
    x = rng.standard_normal((T, E))
    u = rng.standard_normal((T, k))
    idx = np.argsort(-x, axis=1)[:, :k]

    def value(z):  # the weights of the same ids
        if score == "sigmoid":
            s = np.take_along_axis(st.sigmoid(z), idx, 1)
            w = s / s.sum(axis=1, keepdims=True) if renormalize else s
        else:
            picked = np.take_along_axis(z, idx, 1)
            w = st.softmax(picked) if renormalize else np.take_along_axis(st.softmax(z), idx, 1)
        return (u * w).sum() * 2.5

    got = st.route_experts_backward(x, idx, u, score, renormalize, 2.5)
    for t, e in itertools.product(range(T), range(E)):
        d = np.zeros((T, E))
        d[t, e] = h
        assert abs((value(x + d) - value(x - d)) / (2 * h) - got[t, e]) < 1e-8


def test_rms_gradient_against_differences():
    rng = np.random.default_rng(6)
    T, d, h, eps = 3, 5, 1e-6, 1e-3
    x, w, dy, ds = (rng.standard_normal(n) for n in ((T, d), d, (T, d), (T, d)))
    value = lambda x, w: (dy * st.rms_norm(x, w, eps)[0]).sum() + (ds * x).sum()  # noqa: E731
    _, s, rstd = st.rms_norm(x, w, eps)
    dx, dw = st.rms_norm_backward(dy, s, w, rstd, ds)
    for i in itertools.product(range(T), range(d)):
        e = np.zeros((T, d))
        e[i] = h
        assert abs((value(x + e, w) - value(x - e, w)) / (2 * h) - dx[i]) < 1e-7
    for j in range(d):
        e = np.zeros(d)
        e[j] = h
        assert abs((value(x, w + e) - value(x, w - e)) / (2 * h) - dw[j]) < 1e-7


def test_worked_rms():
    y, _, rstd = st.rms_norm(np.array([[3.0, 4.0]]), np.array([1.0, 2.0]), 0.0)
    r = np.sqrt(2) / 5  # the mean square of (3, 4) is 12.5
    np.testing.assert_allclose(rstd, [r])
    np.testing.assert_allclose(y, [[3 * r, 8 * r]])


def test_worked_adamw():
    # the first step moves every element by lr * sign(g) (eps aside), after the decay
    p, m, v = st.adamw([1.0, -2.0], [0.5, -1e-3], [0, 0], [0, 0], 1, 0.1, (0.9, 0.99), 1e-12, 0.5)
    np.testing.assert_allclose(p, [1.0 * 0.95 - 0.1, -2.0 * 0.95 + 0.1], rtol=1e-7)
    np.testing.assert_allclose(m, [0.05, -1e-4])
    np.testing.assert_allclose(v, [0.0025, 1e-8])


def test_adamw_against_torch():
    torch = pytest.importorskip("torch")
    rng = np.random.default_rng(7)
    start = rng.standard_normal(50)
    q = torch.nn.Parameter(torch.tensor(start))
    opt = torch.optim.AdamW([q], lr=0.03, betas=(0.8, 0.9), eps=1e-3, weight_decay=0.2)
    p, m, v = start, np.zeros(50), np.zeros(50)
    for t in range(1, 6):
        g = rng.standard_normal(50)
        q.grad = torch.tensor(g)
        opt.step()
        p, m, v = st.adamw(p, g, m, v, t, 0.03, (0.8, 0.9), 1e-3, 0.2)
        np.testing.assert_allclose(p, q.detach().numpy(), rtol=1e-12)


def test_e4m3_against_torch():
    torch = pytest.importorskip("torch")
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(st.from_e4m3(codes), want)
    a = np.concatenate([np.linspace(-448, 448, 20001), np.geomspace(1e-4, 448, 5000), st.E4M3,
                        (st.E4M3[1:] + st.E4M3[:-1]) / 2]).astype(np.float32)
    got = torch.from_numpy(a).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(st.to_e4m3(a), got)


def test_state_codes():
    a = np.zeros(300, dtype=np.float32)
    a[:3] = [448.0, 224.0, -1e-9]
    a[200] = np.nan
    a[299] = 1e-30
    codes, scale = st.encode_state(a)
    assert scale.shape == (3,) and scale[0] == 1.0 and np.isnan(scale[1]) and not codes[128:256].any()
    np.testing.assert_array_equal(st.decode_state(codes, scale)[:3], [448.0, 224.0, 0.0])
    # a root above 0 is never 0
    codes, scale = st.encode_state(np.abs(a), root=True)
    assert st.decode_state(codes, scale)[2] == 2.0 ** -9 and codes[3] == 0
    np.testing.assert_allclose(st.decode_state(codes, scale)[299], 1e-30, rtol=1e-6)
