"""Calls given a stream that is not the current one: everything that a call allocates
belongs to that stream, so no other stream's work is handed memory that the call
still uses, and what a call returns may be freed while the caller's stream reads it."""
import pytest

import moe_inputs as mi
from tests import _gpu as g

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import token_dispatch_grouped_amd as moe  # noqa: E402

EPS = 1e-5


def _inputs(w):
    x, lg = g.to_dev(mi.hidden_states(w), w.dtype), g.to_dev(mi.router_logits(w), "f32")
    wgu, wdn = (g.to_dev(a, w.dtype) for a in mi.expert_weights(w))
    gen = torch.Generator(device="cuda")
    gen.manual_seed(w.seed)
    nw = torch.randn(w.d, generator=gen, device="cuda")
    d_out = torch.randn((w.T, w.d), generator=gen, device="cuda").to(x.dtype)
    return x, lg, wgu, wdn, (nw, nw, EPS), d_out


def _train(w, args, stream, fused, save=False):
    x, lg, wgu, wdn, norm, d_out = args
    fwd = moe.layer(x, lg, wgu, wdn, w.k, 0, w.E, stream=stream, fused=fused, save=save, norm=norm)
    bwd = moe.layer_backward(x, wgu, wdn, fwd, d_out, w.k, 0, w.E, stream=stream, norm=norm)
    total = moe.clip_grad_norm([bwd["d_w_gate_up"], bwd["d_w_down"], bwd["d_norm_weight"]], 0.5, stream=stream)
    return {**fwd, **bwd, "total": total}


def _serve(w, args, stream):
    x, lg, wgu, wdn, norm, _ = args
    experts = moe.quantize_experts(wgu, wdn, stream=stream)
    res = moe.layer_int8(x, lg, experts, w.k, 0, w.E, stream=stream, norm=norm)
    return {**res, "wq": experts.w_gate_up, "sq": experts.down_scale,
            "norm": moe.grad_norm([args[3]], stream=stream)}


W = mi.Workload("streams", 300, 256, 160, 8, 2, 0, 8, "bf16", 95)
FORMS = {"fused": lambda s, a: _train(W, a, s, True), "saved": lambda s, a: _train(W, a, s, True, True),
         "gathered": lambda s, a: _train(W, a, s, False), "int8": lambda s, a: _serve(W, a, s),
         "int8 few": lambda s, a: _serve(W, (a[0][:5].contiguous(), a[1][:5].contiguous(), *a[2:]), s)}


def _same(got, want):
    for k, v in want.items():
        if torch.is_tensor(v) and k not in ("h", "y", "gu", "d_y", "d_x_perm", "x_perm"):  # (rows behind the last pair)
            assert torch.equal(got[k], v), k


@pytest.mark.parametrize("form", FORMS, ids=[f.replace(" ", "_") for f in FORMS])
def test_what_a_call_allocates_belongs_to_its_stream(form, monkeypatch):
    args = _inputs(W)
    want = FORMS[form](None, args)
    torch.cuda.synchronize()
    made = []

    def recorded(make):
        def run(*a, **kw):
            made.append(make(*a, **kw))
            return made[-1]
        return run

    side = torch.cuda.Stream()
    for name in ("empty", "empty_like"):
        monkeypatch.setattr(torch, name, recorded(getattr(torch, name)))
    got = FORMS[form](side, args)
    monkeypatch.undo()
    torch.cuda.synchronize()
    _same(got, want)
    segments = [(s["address"], s["address"] + s["total_size"], s["stream"]) for s in torch.cuda.memory_snapshot()]
    assert len(made) > 10  # workspaces among them, which the results do not hold
    for t in made:
        if t.numel():
            at = t.data_ptr()
            owner = [s for lo, hi, s in segments if lo <= at < hi]
            assert owner == [side.cuda_stream], (tuple(t.shape), t.dtype)


@pytest.mark.parametrize("form", FORMS, ids=[f.replace(" ", "_") for f in FORMS])
def test_calls_on_two_streams_with_work_on_a_third(form):
    """Two calls at once from one host thread, neither on the current stream, while the
    current stream allocates, writes and frees: each gives the one-at-a-time results."""
    args = _inputs(W)
    want = FORMS[form](None, args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    here = torch.cuda.current_stream()
    for _ in range(5):
        got = []
        for s in streams:
            got.append(FORMS[form](s, args))
            for n in (1 << 10, 1 << 14, 1 << 18, 1 << 22):  # memory that a call might have given back too early
                torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda")
        for s in streams:
            here.wait_stream(s)
        for one in got:
            _same(one, want)  # (waits)


def test_results_freed_while_the_callers_stream_reads_them():
    args = _inputs(W)
    x, lg, wgu, wdn, norm, _ = args
    want = moe.layer_norm(x, norm[0], norm[1], EPS)[0]
    torch.cuda.synchronize()
    side, here = torch.cuda.Stream(), torch.cuda.current_stream()
    y, _, _, _ = moe.layer_norm(x, norm[0], norm[1], EPS, stream=side)
    at = y.data_ptr()
    here.wait_stream(side)
    a = torch.randn((4096, 4096), device="cuda")
    for _ in range(20):  # the reading below waits behind this
        a = a @ a.clamp(-1, 1) / 4096
    copy = y.clone()
    del y
    with torch.cuda.stream(side):
        taken = torch.full(x.shape, 7.0, dtype=x.dtype, device="cuda")
    reused_early = taken.data_ptr() == at
    torch.cuda.synchronize()
    assert torch.equal(copy, want) and not reused_early


def test_a_stream_that_is_current_already():
    args = _inputs(W)
    want = FORMS["fused"](None, args)
    got = FORMS["fused"](torch.cuda.current_stream(), args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = FORMS["fused"](side, args)
    torch.cuda.synchronize()
    _same(got, want)
    _same(other, want)


def test_captured_on_streams_that_fork_and_join():
    """Two layers of 8-bit experts on two side streams inside one graph, replayed on fresh inputs."""
    args = _inputs(W)
    x, lg, wgu, wdn, norm, _ = args
    experts = moe.quantize_experts(wgu, wdn)
    bufs = [(x.clone(), lg.clone()) for _ in range(2)]
    sides = [torch.cuda.Stream() for _ in range(2)]
    outs = [None, None]

    def step():
        here = torch.cuda.current_stream()
        for i, s in enumerate(sides):
            s.wait_stream(here)
            outs[i] = moe.layer_int8(*bufs[i], experts, W.k, 0, W.E, stream=s, norm=norm)["normed"]
        for s in sides:
            here.wait_stream(s)

    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        step()
    torch.cuda.current_stream().wait_stream(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    captured = list(outs)
    for i in range(4):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(200 + i)
        want = []
        for b in bufs:
            b[0].copy_(torch.randn(x.shape, generator=gen, device="cuda"))
            b[1].copy_(torch.randn(lg.shape, generator=gen, device="cuda"))
            want.append(moe.layer_int8(b[0], b[1], experts, W.k, 0, W.E, norm=norm)["normed"])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip(captured, want):
            assert torch.equal(got, w), i
