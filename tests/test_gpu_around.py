"""What stands around the experts, run together as a training step and as serving.

Training: layer(norm=...) -> layer_backward(norm=...) -> clip_grad_norm over every
parameter's gradient. The layer's own tolerance (2e-2 of the largest value, bf16)
covers the chain; the norm's rows enter the layer's gradient through fp32 sums.
"""
import numpy as np
import pytest

import moe_inputs as mi
import oracle
from oracle import around as oa
from tests import _gpu as g

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import token_dispatch_grouped_amd as moe  # noqa: E402

TOL = g.TOL["bf16"]
EPS = 1e-5


def _norm_params(d, seed):
    rng = np.random.default_rng(seed)
    w, b = 1 + 0.2 * rng.standard_normal(d), 0.1 * rng.standard_normal(d)
    return torch.from_numpy(w).float().cuda(), torch.from_numpy(b).float().cuda()


@pytest.mark.parametrize("save", [False, True])
def test_training_step(save):
    w = mi.Workload("around_train", 300, 256, 160, 8, 2, 0, 8, "bf16", 81)
    logits, x = mi.router_logits(w), mi.hidden_states(w)
    wgu, wdn = mi.expert_weights(w)
    dx_, dl = g.to_dev(x, "bf16"), g.to_dev(logits, "f32")
    dgu, ddn = g.to_dev(wgu, "bf16"), g.to_dev(wdn, "bf16")
    nw, nb = _norm_params(w.d, 82)
    rng = np.random.default_rng(83)
    d_out = torch.from_numpy(rng.standard_normal((w.T, w.d))).bfloat16().cuda()
    d_sum = torch.from_numpy(rng.standard_normal((w.T, w.d))).bfloat16().cuda()
    norm = (nw, nb, EPS)
    fwd = moe.layer(dx_, dl, dgu, ddn, w.k, 0, w.E, fused=True, save=save, norm=norm)
    bwd = moe.layer_backward(dx_, dgu, ddn, fwd, d_out, w.k, 0, w.E, norm=norm, d_sum=d_sum)
    grads = [bwd["d_w_gate_up"], bwd["d_w_down"], bwd["d_norm_weight"], bwd["d_norm_bias"]]
    before = [t.clone() for t in grads]
    total = moe.clip_grad_norm(grads, 1.0)
    torch.cuda.synchronize()
    # the chain in fp64
    x64, wgu64, wdn64 = mi.to_f64(x, "bf16"), mi.to_f64(wgu, "bf16"), mi.to_f64(wdn, "bf16")
    ref = oracle.moe_layer(x64, logits, w.k, 0, w.E, wgu64, wdn64)
    y, s, mean, rstd = oa.layer_norm(ref["out"], g.to_f64(nw), g.to_f64(nb), EPS, residual=x64)
    assert g.rel_err(g.to_f64(fwd["normed"]), y) <= TOL
    assert g.rel_err(g.to_f64(fwd["sum"]), s) <= TOL
    ds, dnw, dnb = oa.layer_norm_backward(g.to_f64(d_out), s, g.to_f64(nw), mean, rstd, g.to_f64(d_sum))
    rb = oracle.moe_layer_backward(x64, logits, w.k, 0, w.E, list(wgu64), list(wdn64), ds)
    for name, want in (("d_sum", ds), ("d_x", rb["d_x"]), ("d_logits", rb["d_logits"])):
        assert g.rel_err(g.to_f64(bwd[name]), want) <= TOL, name
    for got, want in zip(before, (rb["d_w_gate_up"], rb["d_w_down"], dnw, dnb)):
        assert g.rel_err(g.to_f64(got), np.asarray(want)) <= TOL
    c = oa.clip_factor(oa.grad_norm([g.to_f64(t) for t in before]), 1.0)
    assert c < 1
    for got, b in zip(grads, before):
        want = g.to_f64(b) * c
        half = 2.0 ** -8 if b.dtype == torch.bfloat16 else 2.0 ** -24
        assert (np.abs(g.to_f64(got) - want) <= np.abs(want) * (half * 1.001 + 6 * 2.0 ** -24)).all()
    assert abs(float(moe.grad_norm(grads)[0]) - 1.0) <= 1e-3  # the clipped gradients have norm 1


def test_serving_step_is_its_parts():
    w = mi.Workload("around_serve", 33, 328, 264, 16, 4, 0, 16, "bf16", 84)
    logits, x = g.to_dev(mi.router_logits(w), "f32"), g.to_dev(mi.hidden_states(w), "bf16")
    wgu, wdn = (g.to_dev(a, "bf16") for a in mi.expert_weights(w))
    nw, nb = _norm_params(w.d, 85)
    experts = moe.quantize_experts(wgu, wdn)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        res = moe.layer_int8(x, logits, experts, w.k, 0, w.E, norm=(nw, nb, EPS))
    torch.cuda.current_stream().wait_stream(side)
    plain = moe.layer_int8(x, logits, experts, w.k, 0, w.E)
    normed, s, _, _ = moe.layer_norm(plain["out"], nw, nb, EPS, residual=x)
    torch.cuda.synchronize()
    assert torch.equal(res["out"], plain["out"]) and torch.equal(res["sum"], s) and torch.equal(res["normed"], normed)
    # the next block's rows: one more layer on the normalised stream
    nxt = moe.layer_int8(res["normed"], logits, experts, w.k, 0, w.E, norm=(nw, None, EPS))
    torch.cuda.synchronize()
    assert torch.isfinite(nxt["normed"].float()).all()


def test_norm_of_a_backward_without_its_forward_is_refused():
    w = mi.Workload("around_err", 16, 64, 64, 8, 2, 0, 8, "bf16", 86)
    x, lg = g.to_dev(mi.hidden_states(w), "bf16"), g.to_dev(mi.router_logits(w), "f32")
    wgu, wdn = (g.to_dev(a, "bf16") for a in mi.expert_weights(w))
    fwd = moe.layer(x, lg, wgu, wdn, w.k, 0, w.E, fused=True)
    nw, nb = _norm_params(w.d, 87)
    with pytest.raises(ValueError):
        moe.layer_backward(x, wgu, wdn, fwd, x, w.k, 0, w.E, norm=(nw, nb, EPS))
    with pytest.raises(ValueError):
        moe.layer_backward(x, wgu, wdn, fwd, x, w.k, 0, w.E, d_sum=x)
