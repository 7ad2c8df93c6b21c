"""The forward's dict and layer_backward: what a caller keeps in it, and logits that changed meanwhile."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import token_dispatch_grouped_amd as moe  # noqa: E402

dev = torch.device("cuda:0")
T, D, D_FF, E, K = 40, 128, 64, 8, 2


def _normal(shape, std, seed, dtype=torch.bfloat16):
    gen = torch.Generator(device=dev).manual_seed(seed)
    return (torch.randn(shape, generator=gen, device=dev) * std).to(dtype)


def _inputs():
    return (_normal((T, D), 1.0, 1), _normal((T, E), 1.0, 2, torch.float32),
            _normal((E, D, 2 * D_FF), D ** -0.5, 3), _normal((E, D_FF, D), D_FF ** -0.5, 4), _normal((T, D), 1.0, 5))


def test_logits_kept_by_the_caller():
    """Without a router, a "logits" of the caller's in the dict is of no account."""
    x, logits, wgu, wdn, up = _inputs()
    fwd = moe.layer(x, logits, wgu, wdn, K, 0, E, fused=True)
    want = moe.layer_backward(x, wgu, wdn, fwd, up, K, 0, E)
    fwd["logits"] = logits
    got = moe.layer_backward(x, wgu, wdn, fwd, up, K, 0, E)
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    with pytest.raises(ValueError, match="router"):
        moe.layer_backward(x, wgu, wdn, fwd, up, K, 0, E, router=moe.Router())


def test_the_forwards_router_is_needed():
    x, logits, wgu, wdn, up = _inputs()
    router = moe.Router("sigmoid")
    fwd = moe.layer(x, logits, wgu, wdn, K, 0, E, fused=True, router=router)
    with pytest.raises(ValueError, match="router"):
        moe.layer_backward(x, wgu, wdn, fwd, up, K, 0, E)
    want = moe.layer_backward(x, wgu, wdn, fwd, up, K, 0, E, router=router)
    # a dict put together by hand, without the router
    hand = {k: v for k, v in fwd.items() if k != "router"}
    got = moe.layer_backward(x, wgu, wdn, hand, up, K, 0, E, router=router)
    torch.cuda.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
