"""The AdamW step against the fp64 form.

Tolerances, with u = 2^-24 (the fp32 constants beta, 1 - beta, lr and the clip factor are
each off by u, every operation by u):
  m      6 u (beta1 |m| + (1 - beta1) |g|)
  v      8 u (beta2 v + (1 - beta2) g^2)
  p      3 u |p| + 24 u lr / (1 - beta1^t) * (beta1 |m| + (1 - beta1) |g|) / (sqrt(v_hat) + eps) + h |p|
         with h the half step of the held type (bf16 2^-8, fp32 2^-24)
1 - beta^t is computed in fp64. 8-bit states are compared code for code: what they are
taken from is rounded operation by operation in fp32, on both sides in the same order.
"""
import math

import numpy as np
import pytest

from oracle import step as st
from tests import _gpu as g

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import token_dispatch_grouped_amd as moe  # noqa: E402

U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
BETAS, EPS = (0.9, 0.95), 1e-8
dev = torch.device("cuda:0")


def _gen(seed):
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    return gen


def _tensors(sizes, pt, gt, master, bits, seed, shapes=None):
    gen = _gen(seed)
    out = dict(params=[], grads=[], masters=[], m=[], v=[])
    for i, n in enumerate(sizes):
        r = lambda std: torch.randn(n, generator=gen, device=dev) * std  # noqa: E731
        w = r(0.02)
        out["params"].append(w.to(DT[pt]))
        out["masters"].append(w if master else None)
        out["grads"].append((r(1e-3) * torch.exp(r(1.0))).to(DT[gt]))
        m, root = r(3e-4), r(1e-3).abs() + 1e-6
        if bits == 32:
            out["m"].append(m)
            out["v"].append(root * root)
        else:
            for k, a in (("m", m), ("v", root)):
                codes, scale = st.encode_state(a.cpu().numpy(), root=k == "v")
                out[k].append(moe.Float8State(torch.from_numpy(codes).to(dev).view(torch.float8_e4m3fn),
                                              torch.from_numpy(scale).to(dev)))
    if not master:
        out["masters"] = None
    return out


def _state64(s):
    if isinstance(s, moe.Float8State):
        return st.decode_state(s.codes.view(torch.uint8).cpu().numpy(), s.scale.cpu().numpy())
    return g.to_f64(s)


def _copy(ts):
    def one(t):
        return None if t is None else moe.Float8State(t.codes.clone(), t.scale.clone()) if isinstance(t, moe.Float8State) else t.clone()
    return {k: None if v is None else [one(t) for t in v] for k, v in ts.items()}


def _step(ts, step, lr, wd=0.1, norm=None, max_norm=0.0, **kw):
    moe.adamw(ts["params"], ts["grads"], ts["m"], ts["v"], step, lr, BETAS, EPS, wd, ts["masters"], norm, max_norm, **kw)


def _check(name, got, want, bound):
    err = np.abs(got - want)
    worst = float((err / np.maximum(bound, 1e-300)).max()) if err.size else 0.0
    assert (err <= bound).all(), (name, worst)
    return worst


def _verify(before, after, pt, bits, step, lr, wd, coef):
    worst = dict(m=0.0, v=0.0, p=0.0)
    b1, b2 = BETAS
    for i in range(len(before["params"])):
        decay = wd if isinstance(wd, float) else wd[i]
        w = before["masters"][i] if before["masters"] is not None else before["params"][i]
        g64, p64 = g.to_f64(before["grads"][i]), g.to_f64(w)
        m64, v64 = _state64(before["m"][i]), _state64(before["v"][i])
        if bits == 8:
            v64 = v64 ** 2
        p, m, v = st.adamw(p64, g64, m64, v64, step, lr, BETAS, EPS, decay, coef)
        m_part = b1 * np.abs(m64) + (1 - b1) * np.abs(g64 * coef)
        rate = 1.0 / (1 - b1 ** step) / (np.sqrt(v / (1 - b2 ** step)) + EPS)
        p_bound = 3 * U * np.abs(p64) + 24 * U * abs(lr) * rate * m_part + 1e-38
        if before["masters"] is not None:
            got = g.to_f64(after["masters"][i])
            worst["p"] = max(worst["p"], _check("master", got, p, p_bound + U * np.abs(p)))
            assert torch.equal(after["params"][i], after["masters"][i].to(torch.bfloat16))
        else:
            worst["p"] = max(worst["p"], _check("p", g.to_f64(after["params"][i]), p, p_bound * 1.01 + HALF[pt] * 1.001 * np.abs(p)))
        if bits == 32:
            worst["m"] = max(worst["m"], _check("m", g.to_f64(after["m"][i]), m, 6 * U * m_part + 1e-44))
            worst["v"] = max(worst["v"], _check("v", g.to_f64(after["v"][i]), v, 8 * U * v + 1e-44))
        else:
            states = []
            for k in ("m", "v"):
                s = before[k][i]
                scale = np.repeat(s.scale.cpu().numpy(), st.BLOCK)[:g64.size]
                states.append(st.from_e4m3(s.codes.view(torch.uint8).cpu().numpy()).astype(np.float32) * scale)
            g32 = before["grads"][i].float().cpu().numpy()
            for k, a in zip(("m", "v"), st.adamw_states32(g32, *states, BETAS, np.float32(coef))):
                codes, scale = st.encode_state(a, root=k == "v")
                np.testing.assert_array_equal(after[k][i].scale.cpu().numpy(), scale)
                np.testing.assert_array_equal(after[k][i].codes.view(torch.uint8).cpu().numpy().reshape(-1), codes)
            # and half a step of the exact state (the least root: a whole one), for the formula's sake
            for k, a in (("m", m), ("v", np.sqrt(v))):
                scale = np.repeat(after[k][i].scale.cpu().numpy().astype(np.float64), st.BLOCK)[:a.size]
                _check(k, _state64(after[k][i]), a, np.maximum(np.abs(a) * 2.0 ** -4, scale * 2.0 ** (-9 if k == "v" else -10)) * (1 + 1e-4))
    print(f"  worst of its bound: {worst}", flush=True)


SIZES = [1, 7, 127, 128, 129, 4095, 4096, 4097, 8192, 20001, 300000, 0, 64]
KINDS = [("f32", "f32", False), ("f32", "bf16", False), ("bf16", "bf16", True), ("bf16", "f32", True), ("bf16", "bf16", False), ("bf16", "f32", False)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("kind", KINDS, ids=["-".join(map(str, k)) for k in KINDS])
@pytest.mark.parametrize("step,lr", [(1, 1e-3), (1000, 3e-4)])
def test_types_and_lengths(kind, bits, step, lr):
    pt, gt, master = kind
    print(f"case {kind} bits={bits} step={step}", flush=True)
    ts = _tensors(SIZES, pt, gt, master, bits, seed=step)
    before = _copy(ts)
    _step(ts, step, lr)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ts["grads"], before["grads"]))
    _verify(before, ts, pt, bits, step, lr, 0.1, 1.0)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("over", [0.25, 1.0, 3.0])
def test_clip_on_the_way(bits, over):
    ts = _tensors([5000, 333, 128], "bf16", "f32", True, bits, seed=5)
    before = _copy(ts)
    norm = moe.grad_norm(ts["grads"])
    max_norm = float(norm) * over
    _step(ts, 7, 1e-3, norm=norm, max_norm=max_norm)
    torch.cuda.synchronize()
    n32 = np.float32(float(norm)) + np.float32(1e-6)
    coef = min(np.float32(1), np.float32(max_norm) * (np.float32(1) / n32))
    assert abs(float(coef) - st.clip_factor(float(norm), max_norm)) <= 4 * U
    _verify(before, ts, "bf16", bits, 7, 1e-3, 0.1, float(coef))


def test_clip_as_clip_grad_norm_does():
    """The step after clip_grad_norm, and with the clip on the way: factors that are a unit apart."""
    a = _tensors([70000, 4000], "f32", "f32", False, 32, seed=6)
    b = _copy(a)
    norm = moe.grad_norm(a["grads"])
    limit = 0.5 * float(norm)
    _step(a, 3, 1e-2, norm=norm, max_norm=limit)
    moe.clip_grad_norm(b["grads"], limit)
    _step(b, 3, 1e-2)
    torch.cuda.synchronize()
    for x, y in zip(a["m"] + a["v"], b["m"] + b["v"]):
        assert (x - y).abs().max() <= 16 * U * y.abs().max()


@pytest.mark.parametrize("bits", [32, 8])
def test_views_at_odd_offsets(bits):
    """Consecutive views of flat buffers, and what lies around them."""
    sizes = [13, 4096, 1, 777, 128, 9001]
    for pt, gt, master in (("f32", "f32", False), ("bf16", "bf16", True)):
        ts = _tensors(sizes, pt, gt, master, bits, seed=8)
        want = _copy(ts)
        _step(want, 5, 1e-3)
        total = sum(sizes) + 6
        flat, views = [], {}
        for k, dtype in (("params", DT[pt]), ("grads", DT[gt]), ("masters", torch.float32), ("m", None), ("v", None)):
            if ts[k] is None:
                views[k] = None
                continue
            eight = bits == 8 and k in "mv"
            dtype = dtype or (torch.uint8 if eight else torch.float32)
            buf = torch.full((total,), 3, device=dev).to(dtype)
            at, out = 3, []
            for i, n in enumerate(sizes):
                v = buf[at:at + n]
                src = ts[k][i].codes.view(torch.uint8) if eight else ts[k][i]
                v.copy_(src)
                out.append(moe.Float8State(v.view(torch.float8_e4m3fn), ts[k][i].scale) if eight else v)
                at += n
            flat.append(buf)
            views[k] = out
        _step(views, 5, 1e-3)
        torch.cuda.synchronize()
        for buf in flat:
            assert (buf[:3] == 3).all() and (buf[-3:] == 3).all()
        for k in ("params", "m", "v") + (("masters",) if master else ()):
            for a, b in zip(views[k], want[k]):
                if isinstance(a, moe.Float8State):
                    assert torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8)) and torch.equal(a.scale, b.scale)
                else:
                    assert torch.equal(a, b)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors_and_own_decays(bits):
    """More tensors than one launch takes, empty ones among them, a decay for each."""
    sizes = [(i * 37) % 400 for i in range(150)]
    ts = _tensors(sizes, "f32", "f32", False, bits, seed=9)
    before = _copy(ts)
    wd = [0.0 if i % 3 else 0.01 * i for i in range(150)]
    _step(ts, 11, 1e-3, wd=wd)
    torch.cuda.synchronize()
    _verify(before, ts, "f32", bits, 11, 1e-3, wd, 1.0)


def test_only_empty_tensors():
    ts = _tensors([0, 0], "bf16", "bf16", True, 8, seed=1)
    _step(ts, 1, 1e-3)
    torch.cuda.synchronize()


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_states_and_zero_gradients(bits):
    """The first steps from adamw_states; an element whose gradient is 0 only decays."""
    params = [torch.randn(3, 70, generator=_gen(2), device=dev), torch.randn(129, generator=_gen(3), device=dev)]
    grads = [torch.randn(3, 70, generator=_gen(4), device=dev), torch.randn(129, generator=_gen(5), device=dev) * 1e-12]
    grads[0][1] = 0.0
    m, v = moe.adamw_states(params, bits)
    p64 = [p.double() for p in params]
    moe.adamw(params, grads, m, v, 1, 0.01, BETAS, 1e-20, 0.5)
    torch.cuda.synchronize()
    for p, q, gr in zip(params, p64, grads):
        want = q * (1 - 0.01 * 0.5) - 0.01 * torch.sign(gr.double())  # m_hat / sqrt(v_hat) = sign(g)
        assert (p.double() - want).abs().max() <= 32 * U * 4
    for _ in range(3):
        moe.adamw(params, grads, m, v, 2, 0.01, BETAS, 1e-20, 0.5)
    torch.cuda.synchronize()
    assert all(torch.isfinite(p).all() for p in params)


def test_small_elements_of_a_block_do_not_run_away():
    """A gradient 1e-9 of its block's largest: its root is held as the least code rather than 0,
    so that no later step is m / eps."""
    p = torch.zeros(128, device=dev)
    grad = torch.full((128,), 1e-9, device=dev)
    grad[0] = 1.0
    m, v = moe.adamw_states([p], 8)
    for t in range(1, 30):
        before = p.clone()
        moe.adamw([p], [grad], m, v, t, 1e-3, BETAS, 1e-30, 0.0)
        assert float((p - before).abs().max()) <= 1e-3 * 1.001 * math.sqrt(1 / 0.05), t
    torch.cuda.synchronize()


@pytest.mark.parametrize("bits", [32, 8])
def test_non_finite_gradients(bits):
    ts = _tensors([500], "f32", "f32", False, bits, seed=3)
    ts["grads"][0][130] = float("nan")
    ts["grads"][0][131] = float("inf")
    clean = _copy(ts)
    clean["grads"][0][130:132] = 0.0
    _step(ts, 4, 1e-3)
    _step(clean, 4, 1e-3)
    torch.cuda.synchronize()
    p, q = ts["params"][0], clean["params"][0]
    bad = torch.zeros(500, dtype=torch.bool, device=dev)
    bad[130:132] = True
    assert torch.isnan(p[bad]).all() and torch.equal(p[~bad], q[~bad])
    if bits == 8:  # the block of the two is lost, the others are as without them
        s, c = ts["m"][0], clean["m"][0]
        assert torch.isnan(s.scale[1]) and not s.codes.view(torch.uint8)[128:256].any()
        rest = [0, 2, 3]
        assert torch.equal(s.scale[rest], c.scale[rest])
    else:
        assert torch.equal(ts["m"][0][~bad], clean["m"][0][~bad])


def test_non_finite_norm():
    for norm, nan in ((float("inf"), False), (float("nan"), True)):
        ts = _tensors([300], "f32", "f32", False, 32, seed=4)
        before = _copy(ts)
        _step(ts, 4, 1e-3, norm=torch.full((1,), norm, device=dev), max_norm=1.0)
        torch.cuda.synchronize()
        if nan:
            assert torch.isnan(ts["params"][0]).all()
        else:  # the gradients count as 0
            before["grads"][0].zero_()
            _verify(before, ts, "f32", 32, 4, 1e-3, 0.1, 1.0)


def test_rate_and_step_in_device_memory_and_a_graph():
    ts = _tensors([6000, 130], "bf16", "bf16", True, 8, seed=7)
    ref = _copy(ts)
    step = torch.zeros(1, dtype=torch.int64, device=dev)
    lr = torch.zeros(1, device=dev)
    norm = torch.zeros(1, device=dev)

    def run(t):
        moe.grad_norm(t["grads"], norm=norm)
        _step(t, step, lr, norm=norm, max_norm=0.05)

    warm = _copy(ts)
    step.fill_(1)
    run(warm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        run(ts)
    step.zero_()
    for t, rate in ((1, 1e-3), (2, 5e-4), (3, 0.0), (4, 2e-3)):
        lr.fill_(rate)
        for a, b in zip(ts["grads"], ref["grads"]):
            a.mul_(1.5)
            b.copy_(a)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        n = moe.grad_norm(ref["grads"])
        # the same rate as the fp32 value holds it
        _step(ref, t, float(np.float32(rate)), norm=n, max_norm=0.05)
        torch.cuda.synchronize()
        assert int(step) == t
        for k in ("params", "masters"):
            assert all(torch.equal(a, b) for a, b in zip(ts[k], ref[k])), (t, k)
        for k in ("m", "v"):
            assert all(torch.equal(a.scale, b.scale) and torch.equal(a.codes.view(torch.uint8), b.codes.view(torch.uint8))
                       for a, b in zip(ts[k], ref[k])), (t, k)


def test_two_streams():
    a, b = (_tensors([40000, 77], "f32", "bf16", False, 32, seed=s) for s in (1, 2))
    ra, rb = _copy(a), _copy(b)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    _step(a, 3, 1e-3, stream=s1)
    _step(b, 3, 1e-3, stream=s2)
    _step(ra, 3, 1e-3)
    _step(rb, 3, 1e-3)
    torch.cuda.synchronize()
    for x, y in ((a, ra), (b, rb)):
        assert all(torch.equal(p, q) for k in ("params", "m", "v") for p, q in zip(x[k], y[k]))


@pytest.mark.parametrize("bits", [32, 8])
def test_a_tensor_past_32_bit_offsets(bits):
    """More than 2^32 bytes of one parameter (and, in 8 bits, 2^30 codes), streamed past the caches."""
    n = (1 << 30) + 300
    p = torch.full((n,), 0.5, device=dev)
    grad = torch.full((n,), 0.25, dtype=torch.bfloat16, device=dev)
    m, v = moe.adamw_states([p], bits)
    at = torch.tensor([0, (1 << 29) + 1, (1 << 30) - 1, (1 << 30), n - 1], device=dev)
    grad[at] = torch.tensor([1.0, -1.0, 2.0, -0.5, 4.0], device=dev, dtype=torch.bfloat16)
    few = [p[at].clone()], [grad[at].clone()], *moe.adamw_states([p[at]], 32)
    moe.adamw([p], [grad], m, v, 1, 0.125, BETAS, EPS, 0.5)
    moe.adamw(*few, 1, 0.125, BETAS, EPS, 0.5)
    torch.cuda.synchronize()
    assert torch.equal(p[at], few[0][0])
    assert torch.equal(p[1:1000], p[1].expand(999)) and torch.equal(p[-200:-1], p[1].expand(199))
    if bits == 32:
        assert torch.equal(m[0][at], few[2][0]) and torch.equal(v[0][at], few[3][0])
    else:
        held = m[0].codes[at].float() * m[0].scale[at // 128]
        assert ((held - few[2][0]).abs() <= 2.0 ** -4 * few[2][0].abs() * 1.0001).all()
