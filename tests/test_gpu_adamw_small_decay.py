"""Weight decay at small rates: the mean change over many elements, where single ones are rounded.

Elements in [1, 2) lie 2^-23 apart, and a step's result is rounded to the nearest. Over a step y (in
units of 2^-23) with density f the error's mean is an integral of f times a sawtooth of period 1, whose own
integral lies between 0 and 1/8: at most 1/8 of f's total variation. The step here is lr u with
u = x / (|x| + 1) of a uniform x in [-1, 1], so that u has the density 1 / (2 (1 - |u|)^2) up to |u| = 1/2: from 0 up to 2,
down to 1/2, up to 2 and down to 0, 7 in all; in units y of lr 2^23 that is 7 / (lr 2^23), and the mean is off by at
most 7/8 2^-46 / lr. The mean of 2^20 elements deviates by 2^-24 / sqrt(3) / 2^10 besides, five of which are allowed;
the step's own roundings are u 2^-24 of lr and of the decay each, a thousandth is allowed.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import token_dispatch_grouped_amd as moe  # noqa: E402

dev = torch.device("cuda:0")
N = 1 << 20


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("lr,wd", [(1e-6, 3.0), (1e-6, 0.1), (2e-7, 0.1), (1e-4, 1e-4)])
def test_mean_decay(lr, wd, master, bits):
    gen = torch.Generator(device=dev).manual_seed(1)
    w = 1.0 + torch.rand(N, generator=gen, device=dev)
    before = w.double()
    p = w.to(torch.bfloat16) if master else w
    grad = torch.rand(N, generator=gen, device=dev) * 2e-3 - 1e-3
    m, v = moe.adamw_states([p], bits)
    # the first step is lr times g / (|g| + eps): with this eps between -1/2 and 1/2 of lr
    eps = 1e-3
    moe.adamw([p], [grad], m, v, 1, lr, (0.9, 0.95), eps, wd, masters=[w] if master else None)
    torch.cuda.synchronize()
    update = lr * (grad.double() / (grad.double().abs() + eps))
    change = before - w.double() - update
    got, want = float((change / before).mean()), lr * wd
    slack = 7 / 8 * 2.0 ** -46 / lr + 5 * 2.0 ** -24 / np.sqrt(3) / np.sqrt(N) + 1e-3 * want
    print(f"  mean decay {got:.4e}, want {want:.4e}, slack {slack:.1e}", flush=True)
    assert abs(got - want) <= slack
