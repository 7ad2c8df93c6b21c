"""Layer norm written over its own input: what the call returns has to fit what the
gradient is told to start from."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import token_dispatch_grouped_amd as moe  # noqa: E402

EPS = 1e-5


def _case(T, d, dt, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return [torch.randn(s, generator=gen, device="cuda").to(dt) for s in ((T, d), (d,), (d,), (T, d))]


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,d", [(1, 8), (33, 264), (5, 2880), (3, 16392)])
def test_without_a_residual_the_rows_are_gone(T, d, dt):
    x, w, b, dy = _case(T, d, dt, T + d)
    y, s, mean, rstd = moe.layer_norm(x, w, b, EPS)
    assert s is x
    for view in (lambda t: t, lambda t: t.view(-1).view(T, d)):  # the same memory under another tensor
        own = x.clone()
        y2, s2, mean2, rstd2 = moe.layer_norm(own, w, b, EPS, y=view(own))
        torch.cuda.synchronize()
        assert torch.equal(y2, y) and torch.equal(own, y) and torch.equal(mean2, mean) and torch.equal(rstd2, rstd)
        assert s2 is None  # x holds y now: not the rows that mean and rstd belong to
        with pytest.raises(ValueError):
            moe.layer_norm_backward(dy, s2, w, mean2, rstd2)


def test_every_place_that_keeps_the_rows():
    x, w, b, dy = _case(17, 520, torch.bfloat16, 1)
    r = _case(17, 520, torch.bfloat16, 2)[0]
    y, s, mean, rstd = moe.layer_norm(x, w, b, EPS, residual=r)
    want = moe.layer_norm_backward(dy, s, w, mean, rstd)
    for y_in, s_in in ((0, 1), (1, 0), (0, None), (1, None), (None, 0), (None, 1)):
        own = [x.clone(), r.clone()]
        pick = lambda i: None if i is None else own[i]  # noqa: E731
        y2, s2, mean2, rstd2 = moe.layer_norm(own[0], w, b, EPS, residual=own[1], y=pick(y_in), s=pick(s_in))
        assert torch.equal(y2, y) and torch.equal(s2, s), (y_in, s_in)
        assert all(torch.equal(p, q) for p, q in zip(moe.layer_norm_backward(dy, s2, w, mean2, rstd2), want))


def test_no_rows_in_place():
    x, w, b, dy = _case(0, 64, torch.bfloat16, 3)
    y, s, mean, rstd = moe.layer_norm(x, w, b, EPS, y=x)
    assert y is x and s is x  # nothing was overwritten
    dx, dw, db = moe.layer_norm_backward(dy, s, w, mean, rstd)
    torch.cuda.synchronize()
    assert dx.shape == (0, 64) and not dw.any() and not db.any()
