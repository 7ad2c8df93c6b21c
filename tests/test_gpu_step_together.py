"""The operators as a program uses them: a serving block (RMS norm into 8-bit rows, scored
routing, experts in 8-bit integers, RMS norm of the sum) and a training step (norm,
routing, experts, norm, their gradients, the gradient norm, AdamW), against the plain
forms and against autograd in fp64."""
import numpy as np
import pytest

from oracle import around as oa
from oracle import step as st
from tests import _gpu as g

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import token_dispatch_grouped_amd as moe  # noqa: E402

dev = torch.device("cuda:0")
EPS = 1e-6


def _normal(shape, std, seed, dtype=torch.bfloat16, mean=0.0):
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    return (torch.randn(shape, generator=gen, device=dev) * std + mean).to(dtype)


def _dequantised(rows, d):
    c = rows.codes.cpu().numpy()
    return oa.from_kblocks(c, d).astype(np.float64) * g.to_f64(rows.scale)[:, None]


# few tokens (rows quantised inside the product), a medium batch and a large one; all experts
# and a share of them; widths that do not fill a K-block
@pytest.mark.parametrize("T,d,d_ff,E,lo,hi,k", [(1, 200, 136, 8, 0, 8, 2), (6, 520, 640, 8, 0, 8, 3), (32, 1000, 264, 32, 8, 24, 4),
                                                (300, 264, 200, 8, 0, 8, 2), (700, 512, 256, 16, 0, 16, 4),
                                                (2000, 256, 512, 4, 0, 2, 2)])
def test_rows_in_8_bits_are_the_rows_the_experts_make(T, d, d_ff, E, lo, hi, k):
    """Rows that are multiples of a power of two times integers up to 127 have the same codes from
    rms_norm's layout as from the experts' own quantisation: the products agree bit for bit."""
    gen = np.random.default_rng(T + d)
    q = gen.integers(-127, 128, (T, d))
    q[:, 3] = 127
    x = torch.from_numpy((q * 2.0 ** -6).astype(np.float32)).to(dev).to(torch.bfloat16)  # exact in bf16
    experts = moe.quantize_experts(_normal((hi - lo, d, 2 * d_ff), d ** -0.5, 1), _normal((hi - lo, d_ff, d), d_ff ** -0.5, 2))
    logits = _normal((T, E), 1.0, 3, torch.float32)
    codes = torch.from_numpy(np.ascontiguousarray(oa.kblocks(q.astype(np.int8)))).to(dev)
    rows = moe.Int8Rows(codes, torch.full((T,), 2.0 ** -6, device=dev))
    want = moe.layer_int8(x, logits, experts, k, lo, hi)
    got = moe.layer_int8(rows, logits, experts, k, lo, hi)
    torch.cuda.synchronize()
    n = int(want["offsets"][hi] - want["offsets"][lo])
    assert torch.equal(got["idx"], want["idx"]) and torch.equal(got["perm"], want["perm"])
    assert torch.equal(got["y"][:n], want["y"][:n]) and torch.equal(got["out"], want["out"])


@pytest.mark.parametrize("T", [1, 19, 200])
def test_serving_block(T):
    d, d_ff, E, k = 264, 200, 16, 4
    router = moe.Router("sigmoid", _normal((E,), 0.05, 9, torch.float32), 4, 2, "top2", True, 2.5)
    x, r = _normal((T, d), 1.0, 4), _normal((T, d), 0.5, 5)
    w1, w2 = _normal((d,), 0.2, 6, mean=1.0), _normal((d,), 0.2, 7, mean=1.0)
    wr = _normal((d, E), d ** -0.5, 8, torch.float32)
    experts = moe.quantize_experts(_normal((E, d, 2 * d_ff), d ** -0.5, 1), _normal((E, d_ff, d), d_ff ** -0.5, 2))

    rows, y, s, _ = moe.rms_norm_int8(x, w1, EPS, residual=r)
    logits = y.float() @ wr
    res = moe.layer_int8(rows, logits, experts, k, 0, E, norm=moe.RmsNorm(w2, EPS), router=router, residual=s)
    torch.cuda.synchronize()

    # the same from the 8-bit rows on, in fp64
    lg = logits.cpu().numpy()
    idx, w = st.route_experts(lg, k, "sigmoid", router.bias.cpu().numpy(), 4, 2, 2, True, 2.5)
    np.testing.assert_array_equal(res["idx"].cpu().numpy(), idx)
    xq = _dequantised(rows, d)
    wgu = np.moveaxis(experts.w_gate_up.cpu().numpy(), 1, 2).reshape(E, 2 * d_ff, -1)[:, :, :d].astype(np.float64)
    wgu *= g.to_f64(experts.gate_up_scale)[:, :, None]
    wdn = np.moveaxis(experts.w_down.cpu().numpy(), 1, 2).reshape(E, d, -1)[:, :, :d_ff].astype(np.float64)
    wdn *= g.to_f64(experts.down_scale)[:, :, None]
    out = np.zeros((T, d))
    for t in range(T):
        for j in range(k):
            e = idx[t, j]
            h = oa.swiglu((xq[t] @ wgu[e].T)[None])
            out[t] += w[t, j] * (h @ wdn[e].T)[0]
    # h is quantised once more (half of 1/127 of its row's largest) and y rounded to bf16
    assert g.rel_err(g.to_f64(res["out"]), out) <= 2e-2
    total = g.to_f64(s) + g.to_f64(res["out"])
    assert np.abs(g.to_f64(res["sum"]) - total).max() <= 2.0 ** -8 * np.abs(total).max()
    ny, _, nr = st.rms_norm(g.to_f64(res["sum"]), g.to_f64(w2), EPS)
    assert (np.abs(g.to_f64(res["normed"]) - ny) <= 2.0 ** -8 * 1.01 * np.abs(ny) + 1e-37).all()
    assert res["mean"] is None and (np.abs(g.to_f64(res["rstd"]) - nr) <= 2.0 ** -23 * nr).all()


@pytest.mark.parametrize("score,renormalize", [("sigmoid", True), ("softmax", False)])
def test_training_step(score, renormalize):
    """s = a + b; y = rms(s); out = layer(y); z = rms(s + out); loss = <z, u>: every gradient, then
    the clipped update. The GPU works in bf16: its gradients may be off by 3e-2 of each tensor's
    largest (the experts' own bound is 2e-2, and two norms round on the way)."""
    T, d, d_ff, E, k = 96, 160, 96, 8, 2
    bias = _normal((E,), 0.05, 1, torch.float32)
    router = moe.Router(score, bias, 2, 1, "top2", renormalize, 1.5)
    a, b = _normal((T, d), 1.0, 2), _normal((T, d), 0.5, 3)
    w1, w2 = _normal((d,), 0.2, 4, mean=1.0), _normal((d,), 0.2, 5, mean=1.0)
    wr = _normal((d, E), d ** -0.5, 6, torch.float32)
    wgu, wdn = _normal((E, d, 2 * d_ff), d ** -0.5, 7), _normal((E, d_ff, d), d_ff ** -0.5, 8)
    up = _normal((T, d), 1.0, 9)

    y, s, rstd = moe.rms_norm(a, w1, EPS, residual=b)
    logits = y.float() @ wr
    norm = moe.RmsNorm(w2, EPS)
    fwd = moe.layer(y, logits, wgu, wdn, k, 0, E, fused=True, save=True, norm=norm, router=router, residual=s)
    bwd = moe.layer_backward(y, wgu, wdn, fwd, up, k, 0, E, norm=norm, router=router)
    d_y = (bwd["d_x"].float() + bwd["d_logits"] @ wr.t()).to(torch.bfloat16)
    d_wr = y.float().t() @ bwd["d_logits"]
    d_s, d_w1 = moe.rms_norm_backward(d_y, s, w1, rstd, d_s=bwd["d_sum"])
    torch.cuda.synchronize()

    # autograd in fp64 on the CPU, for the experts that the GPU chose
    P = {n: t.detach().cpu().double().requires_grad_() for n, t in
         dict(s=s, w1=w1, w2=w2, wr=wr, wgu=wgu, wdn=wdn).items()}
    idx = fwd["idx"].cpu().long()

    def rms(x, w):
        return x / torch.sqrt((x * x).mean(dim=1, keepdim=True) + EPS) * w

    yy = rms(P["s"], P["w1"])
    ll = yy @ P["wr"]
    sc = torch.sigmoid(ll) if score == "sigmoid" else torch.softmax(ll, dim=1)
    ww = torch.gather(sc, 1, idx)
    if renormalize:
        ww = ww / ww.sum(dim=1, keepdim=True)
    ww = ww * 1.5
    out = torch.zeros(T, d, dtype=torch.float64)
    for e in range(E):
        gate, upp = (yy @ P["wgu"][e]).split(d_ff, dim=1)
        ye = (torch.nn.functional.silu(gate) * upp) @ P["wdn"][e]
        out = out + ye * torch.where(idx == e, ww, torch.zeros_like(ww)).sum(dim=1, keepdim=True)
    (rms(P["s"] + out, P["w2"]) * up.cpu().double()).sum().backward()
    got = dict(s=d_s, w1=d_w1, w2=bwd["d_norm_weight"], wr=d_wr, wgu=bwd["d_w_gate_up"], wdn=bwd["d_w_down"])
    for n, t in got.items():
        err = g.rel_err(g.to_f64(t), P[n].grad.numpy())
        print(f"  d_{n}: {err:.2e}", flush=True)
        assert err <= 3e-2, n

    # the update: masters of the bf16 weights, the router in fp32
    params, grads = [wgu, wdn, w1, w2, wr], [got[n] for n in ("wgu", "wdn", "w1", "w2", "wr")]
    masters = [p.float() if p.dtype == torch.bfloat16 else None for p in params]
    start = [g.to_f64(p) for p in params]
    m, v = moe.adamw_states(params, 8)
    gn = moe.grad_norm(grads)
    limit = 0.5 * float(gn)
    moe.adamw(params, grads, m, v, 1, 1e-2, weight_decay=0.1, masters=masters, norm=gn, max_norm=limit)
    torch.cuda.synchronize()
    total = oa.grad_norm([g.to_f64(t) for t in grads])
    assert abs(float(gn) - total) <= 2.0 ** -22 * total
    for p, w, gr, p0 in zip(params, masters, grads, start):
        zero = np.zeros_like(p0)
        want, _, _ = st.adamw(p0, g.to_f64(gr), zero, zero, 1, 1e-2, (0.9, 0.999), 1e-8, 0.1, st.clip_factor(total, limit))
        # a step of lr, off by 24 u of itself, or a share of it where |g| is near eps; g itself is fp32 exact
        got64 = g.to_f64(p if w is None else w)
        assert np.abs(got64 - want).max() <= 2.0 ** -24 * 4 * np.abs(p0).max() + 1e-2 * 2.0 ** -18
        if w is not None:
            assert torch.equal(p, w.to(torch.bfloat16))


def test_router_in_a_layer_is_route_topk_for_plain_softmax():
    T, d, d_ff, E, k = 64, 128, 64, 16, 4
    x, logits = _normal((T, d), 1.0, 1), _normal((T, E), 1.0, 2, torch.float32)
    w = (_normal((E, d, 2 * d_ff), d ** -0.5, 3), _normal((E, d_ff, d), d_ff ** -0.5, 4))
    a = moe.layer(x, logits, *w, k, 0, E, fused=True)
    b = moe.layer(x, logits, *w, k, 0, E, fused=True, router=moe.Router())
    torch.cuda.synchronize()
    assert torch.equal(a["idx"], b["idx"]) and (a["w"] - b["w"]).abs().max() <= 2.0 ** -22
    u = _normal((T, d), 1.0, 5)
    ga = moe.layer_backward(x, *w, a, u, k, 0, E)
    gb = moe.layer_backward(x, *w, b, u, k, 0, E, router=moe.Router())
    torch.cuda.synchronize()
    assert g.rel_err(g.to_f64(gb["d_logits"]), g.to_f64(ga["d_logits"])) <= 1e-5


def test_rms_norm_adds_the_experts_input_unless_told_otherwise():
    T, d, d_ff, E, k = 40, 128, 64, 8, 2
    x, logits, other = _normal((T, d), 1.0, 1), _normal((T, E), 1.0, 2, torch.float32), _normal((T, d), 1.0, 3)
    w = (_normal((E, d, 2 * d_ff), d ** -0.5, 4), _normal((E, d_ff, d), d_ff ** -0.5, 5))
    norm = moe.RmsNorm(_normal((d,), 0.2, 6, mean=1.0), EPS)
    a = moe.layer(x, logits, *w, k, 0, E, fused=True, norm=norm)
    b = moe.layer(x, logits, *w, k, 0, E, fused=True, norm=norm, residual=x)
    c = moe.layer(x, logits, *w, k, 0, E, fused=True, norm=norm, residual=other)
    layer = moe.layer(x, logits, *w, k, 0, E, fused=True, norm=(norm.weight, None, EPS), residual=other)
    torch.cuda.synchronize()
    assert torch.equal(a["normed"], b["normed"]) and torch.equal(a["sum"], b["sum"])
    assert torch.equal(a["sum"], (x.float() + a["out"].float()).to(torch.bfloat16))
    assert torch.equal(c["sum"], (other.float() + c["out"].float()).to(torch.bfloat16))
    assert torch.equal(layer["sum"], c["sum"]) and layer["mean"] is not None


def test_serving_block_in_a_graph():
    """Captured once, replayed on other inputs, with eager work between the replays."""
    T, d, d_ff, E, k = 24, 264, 200, 16, 4
    router = moe.Router("sigmoid", torch.zeros(E, device=dev), 4, 2, "top2", True, 1.0)
    w1, w2 = _normal((d,), 0.2, 6, mean=1.0), _normal((d,), 0.2, 7, mean=1.0)
    experts = moe.quantize_experts(_normal((E, d, 2 * d_ff), d ** -0.5, 1), _normal((E, d_ff, d), d_ff ** -0.5, 2))
    x, r, logits = _normal((T, d), 1.0, 4), _normal((T, d), 0.5, 5), _normal((T, E), 1.0, 8, torch.float32)

    def block():
        rows, _, s, _ = moe.rms_norm_int8(x, w1, EPS, residual=r, keep_y=False)
        return moe.layer_int8(rows, logits, experts, k, 0, E, norm=moe.RmsNorm(w2, EPS), router=router, residual=s)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = block()
    for i in range(3):
        x.copy_(_normal((T, d), 1.0, 40 + i))
        r.copy_(_normal((T, d), 1.0, 50 + i))
        logits.copy_(_normal((T, E), 1.0, 60 + i, torch.float32))
        want = block()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for key in ("idx", "w", "out", "sum", "normed", "rstd"):
            assert torch.equal(held[key], want[key]), (i, key)
