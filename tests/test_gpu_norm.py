"""Residual add and layer norm, and its gradient, against the fp64 forms.

Tolerances, with u = 2^-24 and h the half step of the output type (bf16 2^-8,
fp32 2^-24). A sum of n terms that passes through D additions is off by at most
D u sum|terms|. A row's terms pass through at most D = 90 additions (64 in a
thread, 6 + 16 in the joins, a few roundings of the terms). Hence
  mean   (D + 2) u mean|s|
  rstd   relative (D + 8) u, plus what the mean's error adds to the variance
         (its square: below u^2 D^2 mean|s|^2 rstd^2, under 1e-9 here)
  y      |w| rstd (D + 2) u mean|s| + (D + 12) u |y - b| + 2 u |y| + h |y|
  dx     (D + 16) u rstd (|g| + mean|g| + |hat| mean|g hat|) + u |ds| + h |dx|
and a column sum over T rows passes through at most D2 = ceil(T / 512) + 60
additions (rows of a workgroup, its row groups, the partial rows of a wave, the
waves): (D2 + 4) u sum|terms| + h |sum|.
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

U, D = 2.0 ** -24, 90
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
EPS = 1e-5


def _make(T, d, dt, wdt, seed, mean=0.25):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(shape, std, off, t):
        return (torch.randn(shape, generator=gen, device="cuda") * std + off).to(DT[t])

    return dict(x=normal((T, d), 1.0, mean, dt), r=normal((T, d), 0.5, 0.0, dt), w=normal((d,), 0.2, 1.0, wdt),
                b=normal((d,), 0.1, 0.0, wdt), dy=normal((T, d), 1.0, 0.0, dt), ds=normal((T, d), 1.0, 0.0, dt))


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


def _forward(case, dt, bias, residual, **kw):
    x, r, w, b = case["x"], case["r"] if residual else None, case["w"], case["b"] if bias else None
    y, s, mean, rstd = moe.layer_norm(x, w, b, EPS, residual=r, **kw)
    torch.cuda.synchronize()
    ry, rs, rmean, rrstd = oa.layer_norm(g.to_f64(x), g.to_f64(w), g.to_f64(b) if bias else None, EPS,
                                         g.to_f64(r) if residual else None, _hold(dt))
    got = g.to_f64(s)
    np.testing.assert_array_equal(got, rs)
    ms = np.abs(rs).mean(axis=1)
    _check("mean", g.to_f64(mean), rmean, (D + 2) * U * ms + 1e-300)
    _check("rstd", g.to_f64(rstd), rrstd, rrstd * ((D + 8) * U + (D * U * ms * rrstd) ** 2))
    w64 = np.abs(g.to_f64(w))
    nob = np.abs(ry - (g.to_f64(b) if bias else 0))
    _check("y", g.to_f64(y), ry, w64 * (rrstd * (D + 2) * U * ms)[:, None] + (D + 12) * U * nob
           + (2 * U + HALF[dt] * 1.001) * np.abs(ry) + 1e-37)
    return y, s, mean, rstd


def _backward(case, dt, wdt, s, mean, rstd, bias, ds, **kw):
    dx, dw, db = moe.layer_norm_backward(case["dy"], s, case["w"], mean, rstd, d_s=case["ds"] if ds else None,
                                         bias=bias, **kw)
    torch.cuda.synchronize()
    T = s.shape[0]
    dy64, s64, w64 = g.to_f64(case["dy"]), g.to_f64(s), g.to_f64(case["w"])
    m64, r64 = g.to_f64(mean), g.to_f64(rstd)
    ds64 = g.to_f64(case["ds"]) if ds else None
    rdx, rdw, rdb = oa.layer_norm_backward(dy64, s64, w64, m64, r64, ds64)
    hat, gw = (s64 - m64[:, None]) * r64[:, None], dy64 * w64
    part = r64[:, None] * (np.abs(gw) + np.abs(gw).mean(axis=1, keepdims=True)
                           + np.abs(hat) * np.abs(gw * hat).mean(axis=1, keepdims=True))
    _check("dx", g.to_f64(dx), rdx, (D + 16) * U * part + (0 if ds64 is None else U * np.abs(ds64))
           + HALF[dt] * 1.001 * np.abs(rdx) + 1e-37)
    D2 = -(-T // 512) + 60
    _check("dw", g.to_f64(dw), rdw, (D2 + 4) * U * np.abs(dy64 * hat).sum(axis=0) + HALF[wdt] * 1.001 * np.abs(rdw))
    if bias:
        _check("db", g.to_f64(db), rdb, (D2 + 4) * U * np.abs(dy64).sum(axis=0) + HALF[wdt] * 1.001 * np.abs(rdb))
    else:
        assert db is None
    return dx, dw, db


TYPES = [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")]
# every row shape: groups of 16, 32, 64 threads with full and ragged last vectors,
# workgroups of 256 and 1024, and the widest rows
DIMS = [8, 72, 128, 136, 256, 264, 512, 520, 1024, 1032, 1544, 2048, 2056, 2880, 4096, 4104, 6152, 7168, 8200, 12296, 16384,
        16392, 32768]


@pytest.mark.parametrize("dt,wdt", TYPES, ids=["-".join(t) for t in TYPES])
@pytest.mark.parametrize("d", DIMS)
def test_every_row_shape(d, dt, wdt):
    T = 37 if d <= 8200 else 9
    case = _make(T, d, dt, wdt, seed=d)
    print(f"case T={T} d={d} {dt} {wdt}", flush=True)
    _, s, mean, rstd = _forward(case, dt, bias=True, residual=True)
    _backward(case, dt, wdt, s, mean, rstd, bias=True, ds=True)
    y, s, mean, rstd = _forward(case, dt, bias=False, residual=False)
    assert s.data_ptr() == case["x"].data_ptr()
    _backward(case, dt, wdt, s, mean, rstd, bias=False, ds=False)


@pytest.mark.parametrize("T", [1, 2, 15, 16, 17, 127, 255, 300, 511, 512, 513, 1500, 2047, 2048, 4099])
@pytest.mark.parametrize("d", [64, 136, 640, 2880])
def test_row_counts(T, d):
    case = _make(T, d, "bf16", "f32", seed=T + d)
    print(f"case T={T} d={d}", flush=True)
    _, s, mean, rstd = _forward(case, "bf16", bias=True, residual=True)
    _backward(case, "bf16", "f32", s, mean, rstd, bias=True, ds=False)


def test_no_rows():
    case = _make(0, 64, "bf16", "bf16", seed=1)
    y, s, mean, rstd = moe.layer_norm(case["x"], case["w"], case["b"], EPS, residual=case["r"])
    assert y.shape == (0, 64) and s.shape == (0, 64) and mean.shape == (0,)
    dw, db = torch.full_like(case["w"], 3.0), torch.full_like(case["b"], 3.0)
    moe.layer_norm_backward(case["dy"], s, case["w"], mean, rstd, d_weight=dw, d_bias=db)
    torch.cuda.synchronize()
    assert not dw.any() and not db.any()


def test_far_mean_keeps_its_digits():
    """Rows around 1000 with deviations of 1: the variance is taken around the mean."""
    case = _make(64, 2880, "f32", "f32", seed=9, mean=1000.0)
    _forward(case, "f32", bias=True, residual=True)


def test_constant_and_non_finite_rows():
    case = _make(6, 264, "bf16", "bf16", seed=3)
    x = case["x"]
    x[1] = 5.0
    x[2, 7] = float("inf")
    x[4, 263] = float("nan")
    y, _, mean, rstd = moe.layer_norm(x, case["w"], case["b"], EPS)
    torch.cuda.synchronize()
    assert torch.equal(y[1].float(), case["b"].float())  # no deviation: the bias
    assert abs(float(rstd[1]) - EPS ** -0.5) <= 1e-4 * EPS ** -0.5
    assert torch.isnan(y[2]).all() and torch.isnan(y[4]).all()
    rest = [0, 3, 5]
    want, _, _, _ = moe.layer_norm(x[rest].contiguous(), case["w"], case["b"], EPS)
    assert torch.equal(y[rest], want)  # other rows as without them


def test_in_place_is_the_same():
    case = _make(33, 2880, "bf16", "bf16", seed=4)
    y, s, mean, rstd = moe.layer_norm(case["x"], case["w"], case["b"], EPS, residual=case["r"])
    x2, r2 = case["x"].clone(), case["r"].clone()
    y2, s2, _, _ = moe.layer_norm(x2, case["w"], case["b"], EPS, residual=r2, y=x2, s=r2)
    assert torch.equal(y2, y) and torch.equal(s2, s) and s2.data_ptr() == r2.data_ptr()
    dx, dw, db = moe.layer_norm_backward(case["dy"], s, case["w"], mean, rstd, d_s=case["ds"])
    for own in ("dy", "ds"):
        c = {k: v.clone() for k, v in case.items()}
        dx2, dw2, db2 = moe.layer_norm_backward(c["dy"], s, c["w"], mean, rstd, d_s=c["ds"], d_x=c[own])
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)


def test_other_streams_and_repeated_calls():
    case = _make(700, 1032, "bf16", "f32", seed=5)
    ref = moe.layer_norm(case["x"], case["w"], case["b"], EPS, residual=case["r"])
    gref = moe.layer_norm_backward(case["dy"], ref[1], case["w"], ref[2], ref[3], d_s=case["ds"])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for st in streams:  # two calls at once, each with its own workspace
        f = moe.layer_norm(case["x"], case["w"], case["b"], EPS, residual=case["r"], stream=st)
        outs.append((f, moe.layer_norm_backward(case["dy"], f[1], case["w"], f[2], f[3], d_s=case["ds"], stream=st)))
    torch.cuda.synchronize()
    for f, b in outs:
        assert all(torch.equal(p, q) for p, q in zip(f, ref))
        assert all(torch.equal(p, q) for p, q in zip(b, gref))


def test_misaligned_and_foreign_tensors_are_refused():
    flat = torch.zeros(4 * 64 + 1, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        moe.layer_norm(flat[1:].view(4, 64), w)
    with pytest.raises(ValueError):
        moe.layer_norm(flat[:256].view(4, 64), w.cpu())
    with pytest.raises(ValueError):
        moe.layer_norm(flat[:256].view(64, 4).t(), w)  # not dense


def test_graph_replays():
    case = _make(130, 2880, "bf16", "bf16", seed=6)
    buf = {k: v.clone() for k, v in case.items()}
    ws = torch.empty(moe.layer_norm_backward_workspace_bytes(130, 2880), dtype=torch.uint8, device="cuda")
    out = {}

    def step():
        out["f"] = moe.layer_norm(buf["x"], buf["w"], buf["b"], EPS, residual=buf["r"])
        out["g"] = moe.layer_norm_backward(buf["dy"], out["f"][1], buf["w"], out["f"][2], out["f"][3], d_s=buf["ds"],
                                           workspace=ws)

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
        f = moe.layer_norm(fresh["x"], fresh["w"], fresh["b"], EPS, residual=fresh["r"])
        b = moe.layer_norm_backward(fresh["dy"], f[1], fresh["w"], f[2], f[3], d_s=fresh["ds"])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(captured["f"], f)), i
        assert all(torch.equal(p, q) for p, q in zip(captured["g"], b)), i
