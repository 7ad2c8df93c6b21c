"""8-bit AdamW states with dithered codes: codes bit for bit against the plain form, and runs
of many steps against the averages that they stand for, in fp64."""
import numpy as np
import pytest

from oracle import step as st
from tests import _gpu as g

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import token_dispatch_grouped_amd as moe  # noqa: E402

dev = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed):
    return torch.Generator(device=dev).manual_seed(seed)


def _state(a, root, rounding="dither"):
    codes, scale = st.encode_state(a.cpu().numpy(), root=root)
    return moe.Float8State(torch.from_numpy(codes).to(dev).view(torch.float8_e4m3fn), torch.from_numpy(scale).to(dev), rounding)


def _tensors(sizes, pt, gt, master, seed):
    gen = _gen(seed)
    out = dict(p=[], g=[], w=[] if master else None, m=[], v=[])
    for n in sizes:
        r = lambda std: torch.randn(n, generator=gen, device=dev) * std  # noqa: E731
        w = r(0.02)
        out["p"].append(w.to(DT[pt]))
        if master:
            out["w"].append(w)
        out["g"].append((r(1e-3) * torch.exp(r(1.0))).to(DT[gt]))
        out["m"].append(_state(r(3e-4), False))
        out["v"].append(_state(r(1e-3).abs() + 1e-6, True))
    return out


def _copy(ts):
    one = lambda t: moe.Float8State(t.codes.clone(), t.scale.clone(), t.rounding) if isinstance(t, moe.Float8State) else t.clone()  # noqa: E731
    return {k: None if v is None else [one(t) for t in v] for k, v in ts.items()}


def _step(ts, step, lr=1e-3, betas=(0.9, 0.999), **kw):
    moe.adamw(ts["p"], ts["g"], ts["m"], ts["v"], step, lr, betas, masters=ts["w"], **kw)


def _codes(s):
    return s.codes.view(torch.uint8).reshape(-1)


def _values32(s):
    codes = _codes(s).cpu().numpy()
    return st.from_e4m3(codes).astype(np.float32) * np.repeat(s.scale.cpu().numpy(), st.BLOCK)[:codes.size]


SIZES = [1, 7, 127, 128, 129, 4095, 4096, 4097, 20001, 300000, 0, 64]


@pytest.mark.parametrize("pt,gt,master", [("f32", "f32", False), ("f32", "bf16", False), ("bf16", "bf16", True), ("bf16", "f32", True),
                                          ("bf16", "bf16", False), ("bf16", "f32", False)])
@pytest.mark.parametrize("step", [1, 1000, (1 << 32) + 7])
def test_codes(pt, gt, master, step):
    ts = _tensors(SIZES, pt, gt, master, seed=step % 1000)
    before = _copy(ts)
    _step(ts, step)
    near = _copy(before)
    for s in near["m"] + near["v"]:
        s.rounding = "nearest"
    _step(near, step)
    torch.cuda.synchronize()
    for i, n in enumerate(SIZES):
        # the step itself goes by the states before their rounding
        assert torch.equal(ts["p"][i], near["p"][i])
        grad = before["g"][i].float().cpu().numpy()
        states = st.adamw_states32(grad, _values32(before["m"][i]), _values32(before["v"][i]), (0.9, 0.999))
        bits = st.dither_bits(np.arange(n), step)
        for k, a in zip("mv", states):
            codes, scale = st.encode_state(a, root=k == "v", bits=bits)
            np.testing.assert_array_equal(ts[k][i].scale.cpu().numpy(), scale)
            np.testing.assert_array_equal(_codes(ts[k][i]).cpu().numpy(), codes)


def test_codes_do_not_hang_on_the_list():
    """A tensor's codes are the same alone, in a list of many and as a view at an odd offset; another step's differ."""
    sizes = [5000, 1, 4096 * 3 + 5, 128]
    ts = _tensors(sizes, "f32", "f32", False, seed=3)
    alone, other = _copy(ts), _copy(ts)
    _step(ts, 9)
    for i in range(len(sizes)):
        one = {k: None if v is None else [v[i]] for k, v in alone.items()}
        for k in "mv":
            flat = torch.zeros(sizes[i] + 8, dtype=torch.uint8, device=dev)
            view = flat[3:3 + sizes[i]]
            view.copy_(_codes(one[k][0]))
            one[k] = [moe.Float8State(view.view(torch.float8_e4m3fn), one[k][0].scale, "dither")]
        _step(one, 9)
        torch.cuda.synchronize()
        for k in "mv":
            assert torch.equal(_codes(one[k][0]), _codes(ts[k][i])) and torch.equal(one[k][0].scale, ts[k][i].scale)
    _step(other, 10)
    torch.cuda.synchronize()
    assert not torch.equal(_codes(other["v"][0]), _codes(ts["v"][0]))


def _held(s):
    return st.decode_state(_codes(s).cpu().numpy(), s.scale.cpu().numpy())


@pytest.mark.parametrize("betas,steps,fades_at", [((0.9, 0.95), 600, 200), ((0.9, 0.999), 5000, 2000)])
def test_states_follow_their_averages(betas, steps, fades_at):
    """States of adamw_states over a run in which the gradients fade to a tenth next to each block's
    largest. A step moves a root by a share whose mean size is at most (1 - beta2) / 2; codes are at most an eighth apart, so
    that a step adds a relative variance of at most (1 - beta2) / 16: in balance 1 / 32, and a fall to a tenth at
    most ln 10 / 16 more, a logarithm's deviation of 0.42, three of which are a factor of 3.6; the median within 1.2."""
    n = 128 * 40 + 64
    gen = _gen(11)
    p = [torch.zeros(n, device=dev)]
    m, v = moe.adamw_states(p, 8)
    v64 = torch.zeros(n, dtype=torch.float64, device=dev)
    grad = [torch.empty(n, device=dev)]
    for t in range(1, steps + 1):
        grad[0].copy_(torch.randn(n, generator=gen, device=dev)).mul_(1e-3 if t <= fades_at else 1e-4)
        grad[0][::128] = 1e-2
        moe.adamw(p, grad, m, v, t, 1e-4, betas)
        v64.mul_(betas[1]).addcmul_(grad[0].double(), grad[0].double(), value=1 - betas[1])
    torch.cuda.synchronize()
    small = np.arange(n) % 128 != 0
    ratio = _held(v[0])[small] / np.sqrt(v64.cpu().numpy()[small])
    print(f"  held / true: {np.percentile(ratio, [1, 10, 50, 90, 99]).round(3)}", flush=True)
    assert 1 / 1.2 <= np.median(ratio) <= 1.2
    assert np.percentile(ratio, 1) >= 1 / 3.6 and np.percentile(ratio, 99) <= 3.6


def test_an_element_without_gradients_stops():
    """After 0.9^300 nothing is left of its first state, and it no longer moves."""
    n = 128 * 8
    p = [torch.zeros(n, device=dev)]
    m, v = moe.adamw_states(p, 8)
    gen = _gen(12)
    grad = [torch.empty(n, device=dev)]
    for t in range(1, 801):
        grad[0].copy_(torch.randn(n, generator=gen, device=dev)).mul_(1e-3 if t <= 400 else 0.0)
        grad[0][::128] = 1e-2
        if t == 701:
            at = p[0].clone()
        moe.adamw(p, grad, m, v, t, 1e-3)
    torch.cuda.synchronize()
    small = torch.arange(n, device=dev) % 128 != 0
    assert not (_codes(m[0])[small] & 0x7F).any() and torch.equal(p[0][small], at[small])


def test_replays_take_the_step_from_device_memory():
    ts = _tensors([6000, 130], "bf16", "bf16", True, seed=7)
    ref = _copy(ts)
    step = torch.zeros(1, dtype=torch.int64, device=dev)
    warm = _copy(ts)
    step.fill_(1)
    _step(warm, step)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.add_(1)
        _step(ts, step)
    step.zero_()
    for t in range(1, 5):
        for a, b in zip(ts["g"], ref["g"]):
            a.mul_(1.5)
            b.copy_(a)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        _step(ref, t)
        torch.cuda.synchronize()
        for k in "pw":
            assert all(torch.equal(a, b) for a, b in zip(ts[k], ref[k])), (t, k)
        for k in "mv":
            assert all(torch.equal(a.scale, b.scale) and torch.equal(_codes(a), _codes(b)) for a, b in zip(ts[k], ref[k])), (t, k)


def test_non_finite_gradients():
    ts = _tensors([500], "f32", "f32", False, seed=3)
    clean = _copy(ts)
    ts["g"][0][130] = float("nan")
    ts["g"][0][131] = float("inf")
    _step(ts, 4)
    _step(clean, 4)
    torch.cuda.synchronize()
    for k in "mv":
        assert torch.isnan(ts[k][0].scale[1]) and not _codes(ts[k][0])[128:256].any()
        rest = torch.tensor([0, 2, 3], device=dev)
        assert torch.equal(ts[k][0].scale[rest], clean[k][0].scale[rest])
        keep = (torch.arange(500, device=dev) // 128) != 1
        assert torch.equal(_codes(ts[k][0])[keep], _codes(clean[k][0])[keep])


def test_indices_past_32_bits():
    """The hash takes all bits of an element's index."""
    n = (1 << 32) + 256
    p = torch.zeros(n, dtype=torch.bfloat16, device=dev)
    grad = torch.full((n,), 0.25, dtype=torch.bfloat16, device=dev)
    edge = torch.cat([torch.arange(0, 256), torch.arange((1 << 32) - 128, n)])
    grad[edge.to(dev)] = torch.randn(edge.numel(), generator=_gen(5), device=dev).to(torch.bfloat16)
    m, v = moe.adamw_states([p], 8)
    moe.adamw([p], [grad], m, v, 3, 1e-3, (0.9, 0.95))
    torch.cuda.synchronize()
    g32 = grad[edge.to(dev)].float().cpu().numpy()
    zero = np.zeros_like(g32)
    bits = st.dither_bits(edge.numpy(), 3)
    for s, a, root in zip((m[0], v[0]), st.adamw_states32(g32, zero, zero, (0.9, 0.95)), (False, True)):
        codes, scale = st.encode_state(a, root, bits)
        np.testing.assert_array_equal(_codes(s)[edge.to(dev)].cpu().numpy(), codes)
        blocks = (edge[::128] // 128).to(dev)
        np.testing.assert_array_equal(s.scale[blocks].cpu().numpy(), scale)
