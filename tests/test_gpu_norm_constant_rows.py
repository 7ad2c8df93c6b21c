"""Layer norm of constant rows. With c the constant, u = 2^-24 and d elements:

bf16 rows: c has 8 significant bits and d <= 32768 = 2^15, so every partial sum is a
whole number of c's last place below 2^24 of it: exact, as is the quotient. y is the
bias, rstd the rounded 1 / sqrt(eps).

fp32 rows: a sum of d values passes through at most 32 additions in a thread, 6 among
the lanes and 15 among the waves, each off by u of its result, and the quotient rounds
once more: the mean is off by at most 54 u |c| (and second-order terms, in the 55th).
The deviation f - mean is exact (the two differ by less than a factor of two), so
with e the mean's error the variance is e^2 within 60 u of itself, and
  |y - b| <= |w| e / sqrt(e^2 + eps) (1 + 64 u) + u |b|
where e is read off the mean that the call returns.
"""
import numpy as np
import pytest

from tests import _gpu as g

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import token_dispatch_grouped_amd as moe  # noqa: E402

U, EPS = 2.0 ** -24, 1e-5
VALUES = [0.0, 0.1, -3.3, 1000.1, 5.0, 1.0 / 3.0, 65504.0, -123456.789, 1e-30]
DIMS = [8, 136, 264, 1032, 2880, 7168, 16392, 32768]


def _case(d, dt):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(d)
    x = torch.tensor(VALUES, device="cuda").to(dt)[:, None].expand(len(VALUES), d).contiguous()
    return x, torch.randn(d, generator=gen, device="cuda"), torch.randn(d, generator=gen, device="cuda")


@pytest.mark.parametrize("d", DIMS)
def test_bf16_rows_are_exact(d):
    x, w, b = _case(d, torch.bfloat16)
    y, _, mean, rstd = moe.layer_norm(x, w, b, EPS)
    torch.cuda.synchronize()
    assert torch.equal(mean, x[:, 0].float())
    assert torch.equal(y, b.bfloat16().expand_as(y))
    assert (np.abs(g.to_f64(rstd) - EPS ** -0.5) <= 4 * U * EPS ** -0.5).all()  # eps in fp32, root, quotient


@pytest.mark.parametrize("d", DIMS)
def test_fp32_rows_are_off_by_their_mean(d):
    x, w, b = _case(d, torch.float32)
    y, s, mean, rstd = moe.layer_norm(x, w, b, EPS)
    torch.cuda.synchronize()
    c, got = g.to_f64(x[:, 0]), g.to_f64(mean)
    e = np.abs(got - c)
    print(f"  d={d}: mean off by {(e[1:] / np.abs(c[1:])).max() / U:.2f} u at most", flush=True)
    assert (e <= 55 * U * np.abs(c)).all()
    bound = (e / np.sqrt(e ** 2 + EPS) * (1 + 64 * U))[:, None] * np.abs(g.to_f64(w)) + U * np.abs(g.to_f64(b)) + 1e-37
    assert (np.abs(g.to_f64(y) - g.to_f64(b)) <= bound).all()
    # the gradient takes the same mean and rstd: no row of it is far
    dy = torch.ones_like(x)
    dx, _, db = moe.layer_norm_backward(dy, s, w, mean, rstd)
    torch.cuda.synchronize()
    assert torch.isfinite(dx).all() and torch.equal(db, torch.full_like(b, float(len(VALUES))))
