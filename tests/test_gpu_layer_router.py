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


def test_overwritten_logits_are_refused():
    x, logits, wgu, wdn, up = _inputs()
    router = moe.Router("sigmoid", renormalize=False)
    want = moe.layer_backward(x, wgu, wdn, moe.layer(x, logits.clone(), wgu, wdn, K, 0, E, fused=True, router=router), up, K,
                              0, E, router=router)
    fwd = moe.layer(x, logits, wgu, wdn, K, 0, E, fused=True, router=router)
    for _ in range(2):
        got = moe.layer_backward(x, wgu, wdn, fwd, up, K, 0, E, router=router)
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want)
    logits.copy_(_normal((T, E), 1.0, 6, torch.float32))  # the next batch's, in the same buffer
    with pytest.raises(ValueError, match="overwritten"):
        moe.layer_backward(x, wgu, wdn, fwd, up, K, 0, E, router=router)
    fwd = moe.layer(x, logits, wgu, wdn, K, 0, E, fused=True, router=router)
    moe.layer_backward(x, wgu, wdn, fwd, up, K, 0, E, router=router)
    torch.cuda.synchronize()


def test_logits_in_a_buffer_of_several():
    """Views count the changes of each other: filling one after the other's forward is no change of it."""
    x, logits, wgu, wdn, up = _inputs()
    router = moe.Router("sigmoid")
    both = torch.empty((2, T, E), device=dev)
    both[0].copy_(logits)
    first = moe.layer(x, both[0], wgu, wdn, K, 0, E, fused=True, router=router)
    both[1].copy_(_normal((T, E), 1.0, 6, torch.float32))
    second = moe.layer(x, both[1], wgu, wdn, K, 0, E, fused=True, router=router)
    for fwd, z in ((first, both[0]), (second, both[1])):
        want = moe.layer_backward(x, wgu, wdn, moe.layer(x, z.clone(), wgu, wdn, K, 0, E, fused=True, router=router), up, K,
                                  0, E, router=router)
        got = moe.layer_backward(x, wgu, wdn, fwd, up, K, 0, E, router=router)
        torch.cuda.synchronize()
        assert torch.equal(got["d_logits"], want["d_logits"])


def test_inference_tensors_have_no_count():
    x, logits, wgu, wdn, up = _inputs()
    router = moe.Router("sigmoid")
    with torch.inference_mode():
        z = logits.clone()
        fwd = moe.layer(x, z, wgu, wdn, K, 0, E, fused=True, router=router)
        moe.layer_backward(x, wgu, wdn, fwd, up, K, 0, E, router=router)
    torch.cuda.synchronize()
