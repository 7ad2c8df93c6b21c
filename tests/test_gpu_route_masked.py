"""Routing with experts masked by a logit of -infinity, under a bias that would lift them, and
with biases of +infinity: ids against the plain form bit for bit, and against what the mask
promises."""
import numpy as np
import pytest

from oracle import step as st

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import token_dispatch_grouped_amd as moe  # noqa: E402

dev = torch.device("cuda:0")


def _gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def _inputs(T, E, seed):
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((T, E)) + 0.5 * rng.standard_normal(E)).astype(np.float32)
    return rng, x, (0.05 * rng.standard_normal(E)).astype(np.float32)


def _route(x, bias, k, score, groups, top_groups, group_score):
    """Ids of one call, checked against calls of a few tokens (another path, where the first searches
    fp32 values) and, for some rows, against the plain form."""
    router = moe.Router(score, _gpu(bias), groups, top_groups, group_score, True, 1.0)
    lx = _gpu(x)
    idx, w = moe.route_experts(lx, k, router)
    few = torch.cat([moe.route_experts(lx[at:at + 1000], k, router)[0] for at in range(0, x.shape[0], 1000)])
    torch.cuda.synchronize()
    assert torch.equal(idx, few)
    ids = idx.cpu().numpy()
    at = np.unique(np.r_[0:24, np.random.default_rng(1).integers(0, x.shape[0], 40)]) % x.shape[0]
    with np.errstate(invalid="ignore", over="ignore"):
        want, _ = st.route_experts(x[at], k, score, bias, groups, top_groups, 2 if group_score == "top2" else 1)
    np.testing.assert_array_equal(ids[at], want)
    return ids, w.cpu().numpy()


# one wave a token (k > 16), sorted in fp64, and searched as fp32 values first (many tokens)
SHAPES = [(37, 32, 1, 1, 20), (203, 60, 1, 1, 4), (120, 64, 8, 3, 6), (1000, 256, 1, 1, 8), (16391, 128, 1, 1, 8),
          (16391, 256, 8, 4, 8), (16391, 256, 1, 1, 8), (8209, 512, 8, 4, 8)]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,groups,top_groups,k", SHAPES)
def test_masked_experts_come_after_all_others(T, E, groups, top_groups, k, score):
    """A bias of half a score on every masked expert, or none at all, does not bring it before an
    expert that is not masked."""
    rng, x, bias = _inputs(T, E, seed=T + E)
    out = rng.random((T, E)) < 0.3
    out[0], out[1] = False, True
    out[2], out[2, E // 2] = True, False
    x[out] = -np.inf
    x[3], x[3, 1], x[3, 2] = 0.0, 200.0, -np.inf  # softmax: every other score rounds to 0
    bias += 0.5 * (np.arange(E) % 3 == 0).astype(np.float32)
    for b in (bias, np.zeros(E, dtype=np.float32)):
        for group_score in ("top2", "max"):
            print(f"case T={T} E={E} groups={groups} k={k} {score} {group_score}", flush=True)
            ids, w = _route(x, b, k, score, groups, top_groups, group_score)
            if groups > 1:
                continue
            masked = np.isneginf(np.take_along_axis(x, ids, 1))
            # once a masked expert is chosen, every later one is masked, and none that is not was left
            assert (np.diff(masked.astype(int), axis=1) >= 0).all()
            rows = masked.any(axis=1)
            assert ((~masked[rows]).sum(axis=1) == np.isfinite(x[rows]).sum(axis=1)).all()
            alone = np.isfinite(x).sum(axis=1) >= 1
            assert not np.nan_to_num(w[alone])[masked[alone]].any()


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("T,E,groups,top_groups,k", SHAPES)
def test_biases_of_infinity(T, E, groups, top_groups, k, score):
    """+infinity puts experts, and so their groups, before all others; several of them tie."""
    rng, x, bias = _inputs(T, E, seed=T + E + 1)
    size = E // groups
    for high in ([size], [size, size + 1], [size, 2 * size + 1, E - 1], list(range(size, size + 3)) + [E - 1]):
        b = bias.copy()
        b[[e % E for e in high]] = np.inf
        b[3] = -np.inf
        for group_score in ("top2", "max"):
            print(f"case T={T} E={E} groups={groups} k={k} {score} {group_score} {high}", flush=True)
            ids, _ = _route(x, b, k, score, groups, top_groups, group_score)
            if k >= len(high) and top_groups >= len({e % E // size for e in high}):
                assert (ids[:, :len(high)] == np.array(sorted({e % E for e in high}))).all()


def test_a_masked_expert_passes_no_gradient_under_a_bias():
    _, x, bias = _inputs(40, 24, seed=2)
    x[:, 5] = x[:, 20] = -np.inf
    bias[5] = 3.0
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            router = moe.Router(score, _gpu(bias), renormalize=renormalize)
            lx = _gpu(x)
            for k in (4, 22):
                idx, w = moe.route_experts(lx, k, router)
                g = moe.route_experts_backward(lx, idx, torch.randn(40, k, device=dev), router)
                torch.cuda.synchronize()
                assert not ((idx == 5) | (idx == 20)).any()
                assert torch.isfinite(w).all() and torch.isfinite(g).all() and not g[:, [5, 20]].any()


# as SHAPES, and more than 64 groups
GROUPS = [(37, 32, 8, 3, 9), (203, 60, 6, 2, 4), (120, 64, 32, 3, 6), (1000, 256, 8, 4, 8), (500, 1024, 128, 9, 12), (16391, 256, 8, 2, 8),
          (16391, 256, 4, 1, 4), (16391, 128, 2, 1, 8), (8209, 512, 16, 4, 8), (8209, 1024, 8, 3, 16), (32771, 128, 4, 2, 8)]


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("by", ["logit", "bias"])
@pytest.mark.parametrize("T,E,groups,top_groups,k", GROUPS)
def test_groups_with_few_experts_left(T, E, groups, top_groups, k, by, score):
    """Groups with none, one or two experts that are not masked: one with any comes before one with none, and the
    groups that stay hold as many of them as there are, up to top_groups."""
    rng, x, bias = _inputs(T, E, seed=T + E + 2)
    size = E // groups
    left = rng.choice([0, 0, 1, 1, 1, 2], (T, groups) if by == "logit" else (1, groups))
    order = rng.random((left.shape[0], groups, size)).argsort(axis=2).argsort(axis=2)
    out = (order >= left[:, :, None]).reshape(left.shape[0], E)
    if by == "logit":
        x[out] = -np.inf
    else:
        bias[out[0]] = -np.inf
    left, out = np.broadcast_to(left, (T, groups)), np.broadcast_to(out, (T, E))
    for b in (bias, None) if by == "logit" else (bias,):
        print(f"case T={T} E={E} groups={groups} of which {top_groups} k={k} {score} by {by} bias={b is not None}", flush=True)
        if b is None:
            router = moe.Router(score, None, groups, top_groups, "top2", True, 1.0)
            idx, _ = moe.route_experts(_gpu(x), k, router)
            torch.cuda.synchronize()
            ids = idx.cpu().numpy()
            with np.errstate(invalid="ignore"):
                want, _ = st.route_experts(x[:64], k, score, None, groups, top_groups, 2)
            np.testing.assert_array_equal(ids[:64], want)
        else:
            ids, _ = _route(x, b, k, score, groups, top_groups, "top2")
        if k >= 2 * top_groups:  # every expert that is left in the groups that stay is chosen
            chosen = (~np.take_along_axis(out, ids, 1)).sum(axis=1)
            twos, ones = (left == 2).sum(axis=1), (left == 1).sum(axis=1)
            best = 2 * np.minimum(twos, top_groups) + np.minimum(ones, np.maximum(top_groups - twos, 0))
            np.testing.assert_array_equal(chosen, best)
