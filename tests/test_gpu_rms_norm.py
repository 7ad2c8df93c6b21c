"""Residual add and RMS norm, its 8-bit rows and its gradient, against the fp64 forms.

Tolerances, with u = 2^-24 and h the half step of the output type (bf16 2^-8, fp32
2^-24). The squares are summed in fp64, so
  rstd   2 u relative (its rounding to fp32)
  y      two products and what rstd is off: 4 u |y|, then h |y|
  codes  |code * scale - y| <= scale * (1/2 + 127 * 8 u): half a step, and the roundings of
         y (4 u), of 1 / scale, the product and the scale
A row's terms of the gradient's dot product pass through at most D = 60 additions (32 in
a thread, 6 + 16 in the joins), with 4 roundings of a term:
  dx     (D + 16) u rstd (|g| + |hat| mean|g hat|) + u |ds| + h |dx|
and a column sum over T rows passes through at most D2 = ceil(T / 256) + 60 additions:
(D2 + 4) u sum|terms| + h |sum|.
"""
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

U, D = 2.0 ** -24, 60
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
EPS = 1e-6


def _make(T, d, dt, wdt, seed, std=1.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(shape, std, off, t):
        return (torch.randn(shape, generator=gen, device="cuda") * std + off).to(DT[t])

    return dict(x=normal((T, d), std, 0.1 * std, dt), r=normal((T, d), 0.5 * std, 0.0, dt), w=normal((d,), 0.2, 1.0, wdt),
                dy=normal((T, d), 1.0, 0.0, dt), ds=normal((T, d), 1.0, 0.0, dt))


def _hold(dt):
    def f(a):  # the fp32 sum of two held values, rounded to the type
        return a.astype(np.float32).astype(np.float64) if dt == "f32" else g.to_f64(torch.from_numpy(
            a.astype(np.float32)).to(torch.bfloat16))
    return f


def _check(name, got, want, bound):
    err = np.abs(got - want)
    worst = float((err / np.maximum(bound, 1e-300)).max()) if err.size else 0.0
    print(f"  {name}: worst error {worst:.3f} of its bound", flush=True)
    assert (err <= bound).all(), (name, worst)


def _codes(rows, d):
    """[T, d] int codes, after a look at the padding."""
    c = rows.codes.cpu().numpy()
    flat = oa.from_kblocks(c, c.shape[0] * 64)
    assert not flat[:, d:].any()
    return flat[:, :d].astype(np.float64)


def _forward(case, dt, residual, int8=False, eps=EPS, **kw):
    x, r, w = case["x"], case["r"] if residual else None, case["w"]
    rows = None
    if int8:
        rows, y, s, rstd = moe.rms_norm_int8(x, w, eps, residual=r, **kw)
    else:
        y, s, rstd = moe.rms_norm(x, w, eps, residual=r, **kw)
    torch.cuda.synchronize()
    ry, rs, rrstd = st.rms_norm(g.to_f64(x), g.to_f64(w), eps, g.to_f64(r) if residual else None, _hold(dt))
    np.testing.assert_array_equal(g.to_f64(s), rs)
    _check("rstd", g.to_f64(rstd), rrstd, 2 * U * rrstd)
    if y is not None:
        _check("y", g.to_f64(y), ry, (4 * U + HALF[dt] * 1.001) * np.abs(ry) + 1e-37)
    if rows is not None:
        scale = g.to_f64(rows.scale)
        top = np.abs(ry).max(axis=1)
        _check("scale", scale, np.maximum(top / 127, 2.0 ** -126), 8 * U * top / 127 + 1e-44)
        q = _codes(rows, x.shape[1])
        assert np.abs(q).max(initial=0) <= 127
        _check("codes", q * scale[:, None], ry, (scale * (0.5 + 127 * 8 * U))[:, None] + 0 * ry)
    return y, s, rstd, rows


def _backward(case, dt, wdt, s, rstd, ds, **kw):
    dx, dw = moe.rms_norm_backward(case["dy"], s, case["w"], rstd, d_s=case["ds"] if ds else None, **kw)
    torch.cuda.synchronize()
    T = s.shape[0]
    dy64, s64, w64, r64 = g.to_f64(case["dy"]), g.to_f64(s), g.to_f64(case["w"]), g.to_f64(rstd)
    ds64 = g.to_f64(case["ds"]) if ds else None
    rdx, rdw = st.rms_norm_backward(dy64, s64, w64, r64, ds64)
    hat, gw = s64 * r64[:, None], dy64 * w64
    part = r64[:, None] * (np.abs(gw) + np.abs(hat) * np.abs(gw * hat).mean(axis=1, keepdims=True))
    _check("dx", g.to_f64(dx), rdx, (D + 16) * U * part + (0 if ds64 is None else U * np.abs(ds64))
           + HALF[dt] * 1.001 * np.abs(rdx) + 1e-37)
    D2 = -(-T // 256) + 60
    _check("dw", g.to_f64(dw), rdw, (D2 + 4) * U * np.abs(dy64 * hat).sum(axis=0) + HALF[wdt] * 1.001 * np.abs(rdw))
    return dx, dw


TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]
# full and ragged last vectors of every group of threads, and the widest rows
DIMS = [8, 16, 56, 64, 72, 128, 136, 256, 264, 512, 520, 768, 1024, 1032, 1544, 2048, 2056, 2880, 4096, 4104, 5128, 6152, 7168, 8200,
        12296, 16384, 16392, 24584, 32768]


@pytest.mark.parametrize("dt,wdt", TYPES, ids=["-".join(t) for t in TYPES])
@pytest.mark.parametrize("d", DIMS)
def test_every_row_shape(d, dt, wdt):
    T = 37 if d <= 8200 else 9
    case = _make(T, d, dt, wdt, seed=d)
    print(f"case T={T} d={d} {dt} {wdt}", flush=True)
    _, s, rstd, _ = _forward(case, dt, residual=True)
    _backward(case, dt, wdt, s, rstd, ds=True)
    y, s, rstd, _ = _forward(case, dt, residual=False)
    assert s.data_ptr() == case["x"].data_ptr()
    _backward(case, dt, wdt, s, rstd, ds=False)
    if dt == "bf16":
        plain, ps, prstd, _ = _forward(case, dt, residual=True)
        y, s, rstd, _ = _forward(case, dt, residual=True, int8=True)
        assert torch.equal(y, plain) and torch.equal(s, ps) and torch.equal(rstd, prstd)
        rows, y, _, _ = moe.rms_norm_int8(case["x"], case["w"], EPS, keep_y=False)
        both, _, _, _ = moe.rms_norm_int8(case["x"], case["w"], EPS)
        assert y is None and torch.equal(rows.codes, both.codes) and torch.equal(rows.scale, both.scale)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 127, 255, 300, 511, 512, 513, 1500, 2047, 2048, 4099])
@pytest.mark.parametrize("d", [64, 136, 640, 2880])
def test_row_counts(T, d):
    case = _make(T, d, "bf16", "f32", seed=T + d)
    print(f"case T={T} d={d}", flush=True)
    _, s, rstd, _ = _forward(case, "bf16", residual=True, int8=True)
    _backward(case, "bf16", "f32", s, rstd, ds=False)


@pytest.mark.parametrize("T,d", [(6000, 7168), (40000, 1032)])
def test_rows_past_the_caches(T, d):
    """Sizes whose rows are streamed past the caches."""
    case = _make(T, d, "bf16", "bf16", seed=T)
    print(f"case T={T} d={d}", flush=True)
    _, s, rstd, _ = _forward(case, "bf16", residual=True, int8=True)
    _backward(case, "bf16", "bf16", s, rstd, ds=True)


def test_rows_past_32_bit_offsets():
    """Rows, sums, codes and gradients whose elements lie past 2^31 and 2^32, as in a call of a few rows."""
    T, d = (1 << 20) + 3, 4096
    few = _make(40, d, "bf16", "bf16", seed=21)
    at = torch.randint(0, T, (40,), generator=torch.Generator().manual_seed(2)).cuda()
    at[0], at[1], at[2], at[3] = T - 1, (1 << 31) // d + 1, (1 << 32) // d - 1, (1 << 31) // (2 * d) + 1
    x = few["x"][:1].expand(T, d).contiguous()
    x[at] = few["x"]
    rows, y, s, rstd = moe.rms_norm_int8(x, few["w"], EPS, residual=x)
    few_rows, fy, fs, frstd = moe.rms_norm_int8(x[at].contiguous(), few["w"], EPS, residual=x[at].contiguous())
    assert torch.equal(y[at], fy) and torch.equal(s[at], fs) and torch.equal(rstd[at], frstd)
    assert torch.equal(rows.codes[:, at], few_rows.codes) and torch.equal(rows.scale[at], few_rows.scale)
    del rows, y
    dx, _ = moe.rms_norm_backward(x, s, few["w"], rstd, d_s=s)
    fdx, _ = moe.rms_norm_backward(x[at].contiguous(), fs, few["w"], frstd, d_s=fs)
    assert torch.equal(dx[at], fdx)


def test_no_rows():
    case = _make(0, 64, "bf16", "bf16", seed=1)
    rows, y, s, rstd = moe.rms_norm_int8(case["x"], case["w"], EPS, residual=case["r"])
    assert y.shape == (0, 64) and s.shape == (0, 64) and rstd.shape == (0,) and rows.codes.shape == (1, 0, 64)
    dw = torch.full_like(case["w"], 3.0)
    moe.rms_norm_backward(case["dy"], s, case["w"], rstd, d_weight=dw)
    torch.cuda.synchronize()
    assert not dw.any()


@pytest.mark.parametrize("std", [1e-25, 1e18, 1e30])
def test_far_values(std):
    """Rows whose squares lie outside fp32."""
    for dt in ("bf16", "f32"):
        case = _make(20, 264, dt, dt, seed=9, std=std)
        _forward(case, dt, residual=True, eps=0.0)


def test_zero_and_non_finite_rows():
    case = _make(7, 264, "bf16", "bf16", seed=3)
    x = case["x"]
    x[1] = 0.0
    x[2, 7] = float("inf")
    x[4, 263] = float("nan")
    rows, y, _, rstd = moe.rms_norm_int8(x, case["w"], EPS)
    torch.cuda.synchronize()
    assert not y[1].any() and abs(float(rstd[1]) - 1000) < 1e-3 and not rows.codes[:, 1].any()
    assert float(rows.scale[1]) == 2.0 ** -126
    assert torch.isnan(y[2, 7]) and not y[2, :7].any() and not y[2, 8:].any() and float(rstd[2]) == 0
    assert torch.isnan(y[4]).all()
    for t in (2, 4):
        assert torch.isnan(rows.scale[t]) and not rows.codes[:, t].any()
    rest = [0, 3, 5, 6]
    alone, want, _, _ = moe.rms_norm_int8(x[rest].contiguous(), case["w"], EPS)
    assert torch.equal(y[rest], want) and torch.equal(rows.codes[:, rest], alone.codes)


def test_in_place_is_the_same():
    case = _make(33, 2880, "bf16", "bf16", seed=4)
    rows, y, s, rstd = moe.rms_norm_int8(case["x"], case["w"], EPS, residual=case["r"])
    x2, r2 = case["x"].clone(), case["r"].clone()
    y2, s2, _ = moe.rms_norm(x2, case["w"], EPS, residual=r2, y=x2, s=r2)
    assert torch.equal(y2, y) and torch.equal(s2, s) and s2.data_ptr() == r2.data_ptr()
    x3, r3 = case["x"].clone(), case["r"].clone()
    rows3, y3, s3, _ = moe.rms_norm_int8(x3, case["w"], EPS, residual=r3, y=r3, s=x3)
    assert torch.equal(y3, y) and torch.equal(s3, s) and torch.equal(rows3.codes, rows.codes)
    x4 = case["x"].clone()
    y4, s4, _ = moe.rms_norm(x4, case["w"], EPS, y=x4)
    assert s4 is None and torch.equal(y4, moe.rms_norm(case["x"], case["w"], EPS)[0])
    dx, dw = moe.rms_norm_backward(case["dy"], s, case["w"], rstd, d_s=case["ds"])
    for own in ("dy", "ds"):
        c = {k: v.clone() for k, v in case.items()}
        dx2, dw2 = moe.rms_norm_backward(c["dy"], s, c["w"], rstd, d_s=c["ds"], d_x=c[own])
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_gradient_against_differences_of_the_forward():
    """fp32 rows; with h = 2^-5, y is off by 5 u |y| on each side, and h^2 / 6 of a third
    derivative (of rstd, |y| below 4: under 30) stays."""
    case = _make(5, 24, "f32", "f32", seed=11)
    x, w, dy = case["x"], case["w"], case["dy"]
    _, s, rstd = moe.rms_norm(x, w, EPS)
    dx, dw = moe.rms_norm_backward(dy, s, w, rstd)
    h = 2.0 ** -5
    size = float(dy.abs().sum(dim=1).max())
    for t, j in [(0, 0), (1, 7), (2, 23), (4, 12), (3, 3)]:
        e = torch.zeros_like(x)
        e[t, j] = h
        hi, lo = (float((dy.double() * moe.rms_norm(x + k * e, w, EPS)[0].double()).sum()) for k in (1, -1))
        assert abs((hi - lo) / (2 * h) - float(dx[t, j])) <= size * (20 * U / h + 5 * h * h * 0.1)
    for j in (0, 11, 23):
        e = torch.zeros_like(w)
        e[j] = 1.0
        hi, lo = (float((dy.double() * moe.rms_norm(x, w + k * e, EPS)[0].double()).sum()) for k in (1, -1))
        assert abs((hi - lo) / 2 - float(dw[j])) <= 1e-4 * float(dy[:, j].abs().sum()) * 4  # linear in w


def test_other_streams_and_repeated_calls():
    case = _make(700, 1032, "bf16", "f32", seed=5)
    ref = moe.rms_norm_int8(case["x"], case["w"], EPS, residual=case["r"])
    gref = moe.rms_norm_backward(case["dy"], ref[2], case["w"], ref[3], d_s=case["ds"])
    torch.cuda.synchronize()
    outs = []
    for s in [torch.cuda.Stream() for _ in range(2)]:  # two calls at once, each with its own workspace
        f = moe.rms_norm_int8(case["x"], case["w"], EPS, residual=case["r"], stream=s)
        outs.append((f, moe.rms_norm_backward(case["dy"], f[2], case["w"], f[3], d_s=case["ds"], stream=s)))
    torch.cuda.synchronize()
    for f, b in outs:
        assert torch.equal(f[0].codes, ref[0].codes) and torch.equal(f[0].scale, ref[0].scale)
        assert all(torch.equal(p, q) for p, q in zip(f[1:], ref[1:]))
        assert all(torch.equal(p, q) for p, q in zip(b, gref))


def test_misaligned_and_foreign_tensors_are_refused():
    flat = torch.zeros(4 * 64 + 1, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        moe.rms_norm(flat[1:].view(4, 64), w)
    with pytest.raises(ValueError):
        moe.rms_norm(flat[:256].view(4, 64), w.cpu())
    with pytest.raises(ValueError):
        moe.rms_norm(flat[:256].view(64, 4).t(), w)  # not dense


def test_graph_replays():
    case = _make(130, 2880, "bf16", "bf16", seed=6)
    buf = {k: v.clone() for k, v in case.items()}
    out = {}

    def step():
        out["f"] = moe.rms_norm_int8(buf["x"], buf["w"], EPS, residual=buf["r"])
        out["g"] = moe.rms_norm_backward(buf["dy"], out["f"][2], buf["w"], out["f"][3], d_s=buf["ds"])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    captured = dict(out)
    for i in range(3):
        fresh = _make(130, 2880, "bf16", "bf16", seed=100 + i)
        for k in buf:
            buf[k].copy_(fresh[k])
        f = moe.rms_norm_int8(fresh["x"], fresh["w"], EPS, residual=fresh["r"])
        b = moe.rms_norm_backward(fresh["dy"], f[2], fresh["w"], f[3], d_s=fresh["ds"])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured["f"][0].codes, f[0].codes) and torch.equal(captured["f"][0].scale, f[0].scale)
        assert all(torch.equal(p, q) for p, q in zip(captured["f"][1:], f[1:])), i
        assert all(torch.equal(p, q) for p, q in zip(captured["g"], b)), i
