"""The clip of lists that take many launches: the same numbers as its two halves, and a
cost that does not grow faster than the list."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import token_dispatch_grouped_amd as moe  # noqa: E402

EACH = 1 << 18  # fp32 elements of a tensor: 1 MB, 32 workgroups


def _list(n, dt=torch.float32, each=EACH):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(n)
    flat = torch.empty(n * each, dtype=dt, device="cuda")
    for part in flat.split(1 << 27):
        part.copy_(torch.randn(part.numel(), generator=gen, device="cuda"))
    return flat, list(flat.split(each))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [63, 64, 65, 66, 129, 500])
def test_the_clip_is_its_two_halves(n, dt):
    """Around 64 tensors, where one launch's workgroups and partial sums end (2048)."""
    flat, grads = _list(n, dt, EACH if dt == torch.float32 else 2 * EACH)
    before = flat.clone()
    norm = moe.grad_norm(grads)
    want = (before.double() ** 2).sum().sqrt()
    # the rounding to fp32 is off by 2^-24, the fp64 sums of 2^27 squares by less than 2^27 2^-53 on each side
    assert abs(float(norm[0]) - float(want)) <= float(want) * (2.0 ** -24 + 2.0 ** -25)
    half = float(norm[0]) / 2
    outs = [torch.empty_like(t) for t in grads]
    got = moe.clip_grad_norm(grads, half, out=outs)
    assert torch.equal(got, norm) and torch.equal(flat, before)
    moe.clip_grads(grads, norm, half)
    assert all(torch.equal(a, b) for a, b in zip(grads, outs))
    flat.copy_(before)
    assert torch.equal(moe.clip_grad_norm(grads, half), norm)  # in place
    assert all(torch.equal(a, b) for a, b in zip(grads, outs))


def test_a_replayed_clip_of_many_launches():
    flat, grads = _list(130)
    fresh = flat.clone()
    ws = torch.empty(moe.grad_norm_workspace_bytes(130), dtype=torch.uint8, device="cuda")
    norm = torch.empty(1, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        moe.clip_grad_norm(grads, 2.0, norm=norm, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.clip_grad_norm(grads, 2.0, norm=norm, workspace=ws)
    for i in range(3):
        flat.copy_(fresh * (i + 1))
        other = flat.clone()
        want = moe.clip_grad_norm(list(other.split(EACH)), 2.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, want) and torch.equal(flat, other), i


def _time(call):
    """The least of five replays of the captured call, in ms: no host time in it."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    best = float("inf")
    for _ in range(6):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


def test_the_cost_of_a_long_list():
    """4096 tensors of 1 MB, none of which has to be scaled: the clip reads them once, for
    the norm, so it takes the time of the norm alone and 64 launches that find nothing to
    do (1.3 ms for the norm's 0.95). When every workgroup of every launch added all
    partial sums again, the clip took 8.3 ms."""
    _, grads = _list(4096)
    norm, ws = torch.empty(1, device="cuda"), torch.empty(moe.grad_norm_workspace_bytes(4096), dtype=torch.uint8,
                                                          device="cuda")
    alone = _time(lambda: moe.grad_norm(grads, norm=norm, workspace=ws))
    clip = _time(lambda: moe.clip_grad_norm(grads, 1e9, norm=norm, workspace=ws))
    print(f"  norm {alone:.2f} ms, norm and clip {clip:.2f} ms", flush=True)
    assert clip <= 3 * alone
