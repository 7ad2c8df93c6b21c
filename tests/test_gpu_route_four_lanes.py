"""Routing of so many tokens that four lanes share one with 16 or 32 values each: ids as in calls of few tokens
bit for bit and, for some rows, against the plain form."""
import numpy as np
import pytest

from oracle import step as st

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import token_dispatch_grouped_amd as moe  # noqa: E402

dev = torch.device("cuda:0")
U = 2.0 ** -24
T = 32771


@pytest.mark.parametrize("score,biased,renormalize", [("softmax", False, True), ("softmax", False, False), ("softmax", True, True),
                                                      ("sigmoid", False, False), ("sigmoid", True, True)])
@pytest.mark.parametrize("E,groups,top_groups", [(60, 1, 1), (60, 3, 2), (60, 4, 2), (64, 2, 1), (128, 1, 1), (128, 2, 1), (128, 4, 3)])
@pytest.mark.parametrize("k", [4, 8, 16])
def test_as_few_tokens(E, groups, top_groups, k, score, biased, renormalize):
    rng = np.random.default_rng(E + groups + k)
    x = (rng.standard_normal((T, E)) + 0.5 * rng.standard_normal(E)).astype(np.float32)
    x[::3] = torch.from_numpy(x[::3]).bfloat16().float().numpy()  # ties
    x[5], x[6, ::2], x[7] = 0.25, -np.inf, 30.0 + np.arange(E) % 5
    x[8, 3], x[9, E - 1] = np.nan, np.inf
    bias = (0.05 * rng.standard_normal(E)).astype(np.float32) if biased else None
    lx = torch.from_numpy(x).to(dev)
    at = np.r_[0:24, T - 20:T, rng.integers(0, T, 20)]
    for group_score in ("top2", "max") if groups > 1 else ("max",):
        print(f"case E={E} groups={groups} of which {top_groups} k={k} {score} bias={biased} {group_score}", flush=True)
        router = moe.Router(score, None if bias is None else torch.from_numpy(bias).to(dev), groups, top_groups, group_score, renormalize, 1.5)
        idx, w = moe.route_experts(lx, k, router)
        few, fw = (torch.cat(p) for p in zip(*[moe.route_experts(lx[a:a + 1000], k, router) for a in range(0, T, 1000)]))
        torch.cuda.synchronize()
        assert torch.equal(idx, few)
        ok = torch.isfinite(fw)
        assert torch.equal(torch.isfinite(w), ok) and ((w - fw).abs()[ok] <= 16 * U * fw.abs()[ok]).all()
        with np.errstate(invalid="ignore"):
            want, ww = st.route_experts(x[at], k, score, bias, groups, top_groups, 2 if group_score == "top2" else 1, renormalize, 1.5)
        np.testing.assert_array_equal(idx.cpu().numpy()[at], want)
        got, fine = w.cpu().numpy()[at], np.isfinite(ww)
        assert (np.abs(got - ww)[fine] <= 50 * U * np.abs(ww)[fine] + 1e-38).all()
