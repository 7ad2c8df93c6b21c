"""The gradient norm and clipping against fp64.

The squares of fp32 and bf16 values are exact in fp64 and are summed there: n
terms are off by at most n 2^-53 of their sum, 1e-9 for the lengths here, so the
norm is off by the rounding to fp32 (2^-24) and a relative 1e-9. The factor is
max_norm / (norm + 1e-6) in fp32: the norm's 2^-24, the sum's and the quotient's
2^-24 each; the product rounds once more, and once to the type:
relative 5 * 2^-24 + half a step (bf16 2^-8, fp32 2^-24).
"""
import numpy as np
import pytest

from oracle import around as oa
from tests import _gpu as g

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import token_dispatch_grouped_amd as moe  # noqa: E402

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
BF, F = torch.bfloat16, torch.float32


def _grads(spec, seed, std=1e-2):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return [(torch.randn(shape, generator=gen, device="cuda") * std).to(dt) for shape, dt in spec]


def _check(grads, before, max_norm, norm, outs):
    ref = oa.grad_norm([g.to_f64(t) for t in before])
    got = float(norm[0])
    print(f"  norm {got:.6g} (fp64 {ref:.9g})", flush=True)
    assert abs(got - ref) <= ref * (1.001 * U + 1e-9)
    c = oa.clip_factor(ref, max_norm)
    for b, o in zip(before, outs):
        want = g.to_f64(b) * c
        assert (np.abs(g.to_f64(o) - want) <= np.abs(want) * (5 * U + 1.001 * HALF[b.dtype]) + 1e-44).all()


SPECS = [
    [((1,), F)],
    [((7,), BF)],
    [((8, 64, 320), BF), ((8, 160, 64), BF), ((64,), F), ((5, 3), F), ((1,), BF)],
    [((n,), (BF, F)[n % 2]) for n in list(range(1, 60)) + [4095, 4096, 4097, 16383, 16384, 16385, 100003]],
    [((3, 1 << 20), F), ((1 << 22,), BF)],
    [((i % 13 + 1,), (BF, F)[i % 2]) for i in range(200)],  # more tensors than one launch takes
    [((0,), F), ((33,), F), ((0, 4), BF)],
]


@pytest.mark.parametrize("spec", SPECS, ids=[f"list{i}" for i in range(len(SPECS))])
@pytest.mark.parametrize("max_norm", [1e-3, 1e6])
def test_norm_and_clip(spec, max_norm):
    grads = _grads(spec, seed=len(spec))
    print(f"case {len(spec)} tensors, max_norm {max_norm}", flush=True)
    before = [t.clone() for t in grads]
    outs = [torch.full_like(t, 7.0) for t in grads]
    n1 = moe.grad_norm(grads)
    n2 = moe.clip_grad_norm(grads, max_norm, out=outs)
    assert all(torch.equal(a, b) for a, b in zip(grads, before))  # read only
    n3 = moe.clip_grad_norm(grads, max_norm)  # in place
    torch.cuda.synchronize()
    _check(grads, before, max_norm, n1, outs)
    assert torch.equal(n1, n2) and torch.equal(n1, n3)
    assert all(torch.equal(a, b) for a, b in zip(grads, outs))
    again = [t.clone() for t in before]
    moe.clip_grads(again, n1, max_norm)  # the two halves
    assert all(torch.equal(a, b) for a, b in zip(again, outs))
    if max_norm > 1:
        assert all(torch.equal(a, b) for a, b in zip(outs, before))


@pytest.mark.parametrize("dt", [BF, F])
def test_views_at_every_offset(dt):
    """Views of one flat buffer: every alignment of source and destination, with the
    neighbours left as they were."""
    base = _grads([((20000,), F)], seed=11)[0].to(dt)
    for off in range(9):
        for n in (1, 5, 8, 17, 9000):
            for shift in (0, 3):
                flat, dst = base.clone(), torch.full_like(base, 2.0)
                view, out = flat[off:off + n], dst[off + shift:off + shift + n]
                norm = moe.clip_grad_norm([view], 1e-4, out=[out])
                torch.cuda.synchronize()
                _check([view], [base[off:off + n]], 1e-4, norm, [out])
                assert torch.equal(flat, base)
                assert (dst[:off + shift] == 2).all() and (dst[off + shift + n:] == 2).all()
                moe.clip_grads([view], norm, 1e-4)
                assert torch.equal(view, out)
                assert torch.equal(flat[:off], base[:off]) and torch.equal(flat[off + n:], base[off + n:])


def test_extreme_gradients():
    """Squares that fp32 could not hold."""
    for v in (1e30, 1e-30, 3e38):
        t = torch.full((1000,), v, device="cuda")
        got = float(moe.grad_norm([t])[0])
        want = float(np.float32(v)) * 1000 ** 0.5
        if want < 3.4e38:
            assert abs(got - want) <= want * (2 * U)
        else:
            assert got == float("inf")


def test_non_finite_gradients():
    t = torch.ones(5000, device="cuda")
    t[4321] = float("inf")
    norm = moe.clip_grad_norm([t], 1.0)
    assert float(norm[0]) == float("inf")
    assert torch.isnan(t[4321]) and not t[:4321].any() and not t[4322:].any()
    t = torch.ones(5000, dtype=BF, device="cuda")
    t[17] = float("nan")
    norm = moe.clip_grad_norm([t], 1.0)
    assert torch.isnan(norm).all() and torch.isnan(t).all()


def test_zero_gradients():
    t = torch.zeros(4097, device="cuda")
    assert float(moe.clip_grad_norm([t], 0.0)[0]) == 0.0
    t = torch.ones(4097, device="cuda")
    moe.clip_grad_norm([t], 0.0)
    assert not t.any()


def test_same_bits_on_other_streams():
    grads = _grads([((1 << 21,), BF), ((1000003,), F)], seed=3)
    ref = moe.grad_norm(grads)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [moe.grad_norm(grads, stream=s) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(ref, n) for n in got)


def test_dense_but_transposed_gradients_are_refused():
    t = torch.ones(4, 6, device="cuda")
    with pytest.raises(ValueError):
        moe.grad_norm([t.t()])
    with pytest.raises(moe.MoeError) as e:
        moe.clip_grad_norm([t, t], 1.0)
    assert e.value.status == moe.MOE_EINVAL
    assert (t == 1).all()


def test_graph_replays():
    spec = [((3, 4099), BF), ((70001,), F), ((1,), F)]
    bufs = _grads(spec, seed=0)
    ws = torch.empty(moe.grad_norm_workspace_bytes(3), dtype=torch.uint8, device="cuda")
    norm = torch.empty(1, device="cuda")

    def step():
        moe.clip_grad_norm(bufs, 0.5, norm=norm, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(3):
        fresh = _grads(spec, seed=50 + i)
        for b, f in zip(bufs, fresh):
            b.copy_(f)
        want = moe.clip_grad_norm(fresh, 0.5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, want), i
        assert all(torch.equal(a, b) for a, b in zip(bufs, fresh)), i
