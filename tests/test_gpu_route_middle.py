"""Routing of 2048 to 16384 tokens, between the calls of few lanes and of many: ids as in calls of few tokens bit for
bit and, for some rows, against the plain form."""
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


@pytest.mark.parametrize("T", [2047, 2048, 4095, 4096, 8191, 8192, 16383, 16384])
@pytest.mark.parametrize("E,groups,top_groups,k", [(8, 1, 1, 2), (64, 1, 1, 8), (100, 1, 1, 4), (256, 8, 4, 8), (512, 1, 1, 16),
                                                   (1000, 4, 2, 8), (1024, 64, 9, 8)])
def test_as_few_tokens(T, E, groups, top_groups, k):
    rng = np.random.default_rng(E + T)
    x = (rng.standard_normal((T, E)) + 0.5 * rng.standard_normal(E)).astype(np.float32)
    x[5], x[6, ::2] = 0.25, -np.inf
    bias = (0.05 * rng.standard_normal(E)).astype(np.float32)
    lx = torch.from_numpy(x).to(dev)
    at = np.r_[0:12, T - 12:T]
    for score, b in (("softmax", None), ("softmax", bias), ("sigmoid", bias)):
        print(f"case T={T} E={E} groups={groups} k={k} {score} bias={b is not None}", flush=True)
        router = moe.Router(score, None if b is None else torch.from_numpy(b).to(dev), groups, top_groups, "top2", True, 1.5)
        idx, w = moe.route_experts(lx, k, router)
        few, fw = (torch.cat(p) for p in zip(*[moe.route_experts(lx[a:a + 1000], k, router) for a in range(0, T, 1000)]))
        torch.cuda.synchronize()
        assert torch.equal(idx, few) and ((w - fw).abs() <= 4 * U * fw.abs()).all()
        want, _ = st.route_experts(x[at], k, score, b, groups, top_groups, 2, True, 1.5)
        np.testing.assert_array_equal(idx.cpu().numpy()[at], want)
