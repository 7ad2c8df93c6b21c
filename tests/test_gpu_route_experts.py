"""Routing by scores and its gradient against the fp64 forms.

The ids are compared bit for bit: choice values are held in fp32 on both sides, from
fp64 scores that differ in their last bits, so they disagree only where a score lies
within 2^-52 of the middle between two fp32 numbers.

Weights, with u = 2^-24: an fp32 score is off by at most 4 u (the exponential, the sum
with one, the division), the one of a far logit by u |x - max| e^(x - max) <= 0.4 u of the
largest more, a sum of up to 1024 of them passes through at most 40 additions, two more
roundings follow: 50 u of the weight. The gradient's terms go through the same, twice:
with part = |ds/dx| (|u_j| + sum |u s| / S) / S it is off by at most 110 u part.
"""
import numpy as np
import pytest

from oracle import step as st

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import token_dispatch_grouped_amd as moe  # noqa: E402

U = 2.0 ** -24
dev = torch.device("cuda:0")


def _inputs(T, E, seed, held="f32", spread=1.0):
    rng = np.random.default_rng(seed)
    x = (spread * rng.standard_normal((T, E)) + 0.5 * rng.standard_normal(E)).astype(np.float32)
    if held == "bf16":  # as a product in bf16 leaves them: many ties
        x = torch.from_numpy(x).bfloat16().float().numpy()
    return x, (0.05 * rng.standard_normal(E)).astype(np.float32)


def _gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dev)


def _check(x, k, score, bias, groups, top_groups, group_score, renormalize, scale):
    router = moe.Router(score, None if bias is None else _gpu(bias), groups, top_groups, group_score, renormalize, scale)
    lx = _gpu(x)
    idx, w = moe.route_experts(lx, k, router)
    torch.cuda.synchronize()
    want, ww = st.route_experts(x, k, score, bias, groups, top_groups, 2 if group_score == "top2" else 1, renormalize, scale)
    np.testing.assert_array_equal(idx.cpu().numpy(), want)
    err = np.abs(w.cpu().numpy() - ww) / np.maximum(np.abs(ww), 1e-38)
    print(f"  weights: worst {err.max(initial=0) / U:.1f} u", flush=True)
    assert (err <= 50 * U).all()
    return lx, idx, router


def _check_backward(x, lx, idx, router, seed):
    T, E = x.shape
    k = idx.shape[1]
    d_w = np.random.default_rng(seed).standard_normal((T, k)).astype(np.float32)
    got = moe.route_experts_backward(lx, idx, _gpu(d_w), router)
    torch.cuda.synchronize()
    ids = idx.cpu().numpy()
    want = st.route_experts_backward(x, ids, d_w, router.score, router.renormalize, router.scale)
    # |ds/dx| (|u_j| + sum |u s| / S) / S, for every expert
    u = np.abs(router.scale * d_w.astype(np.float64))
    up = np.zeros((T, E))
    np.put_along_axis(up, ids, u, 1)
    if router.score == "sigmoid":
        s = np.take_along_axis(st.sigmoid(x), ids, 1)
        slope = np.zeros((T, E))
        np.put_along_axis(slope, ids, s * np.take_along_axis(st.sigmoid(-x.astype(np.float64)), ids, 1), 1)
        S = s.sum(axis=1, keepdims=True) if router.renormalize else np.ones((T, 1))
        part = slope / S * (up + (u * s).sum(axis=1, keepdims=True) / S)
    else:
        x64 = x.astype(np.float64)
        p = st.softmax(x64)
        if router.renormalize:
            q = np.zeros((T, E))
            np.put_along_axis(q, ids, st.softmax(np.take_along_axis(x64, ids, 1)), 1)
            p = q
        part = p * (up + (np.take_along_axis(p, ids, 1) * u).sum(axis=1, keepdims=True))
    err = np.abs(got.cpu().numpy() - want)
    print(f"  gradient: worst {(err / np.maximum(part, 1e-300)).max(initial=0) / U:.1f} u", flush=True)
    assert (err <= 110 * U * part + 1e-38).all()
    if not (router.score == "softmax" and not router.renormalize):
        chosen = np.zeros((T, E), bool)
        np.put_along_axis(chosen, ids, True, 1)
        assert not got.cpu().numpy()[~chosen].any()


KINDS = [("softmax", False, True), ("softmax", False, False), ("softmax", True, True), ("softmax", True, False),
         ("sigmoid", False, True), ("sigmoid", False, False), ("sigmoid", True, True), ("sigmoid", True, False)]


@pytest.mark.parametrize("kind", KINDS, ids=["-".join(map(str, c)) for c in KINDS])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (3, 1), (7, 5), (8, 2), (16, 4), (17, 6), (33, 8), (60, 4), (64, 6), (65, 9),
                                 (128, 4), (129, 16), (160, 6), (250, 8), (256, 8), (257, 17), (500, 8), (512, 10),
                                 (1000, 24), (1024, 8), (1024, 16)])
def test_without_groups(E, k, kind):
    score, biased, renormalize = kind
    x, bias = _inputs(203, E, seed=E + k)
    print(f"case E={E} k={k} {kind}", flush=True)
    lx, idx, router = _check(x, k, score, bias if biased else None, 1, 1, "max", renormalize, 1.0)
    _check_backward(x, lx, idx, router, E)


@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("E,groups,top_groups,k", [
    (8, 2, 1, 4), (8, 8, 3, 3), (12, 4, 2, 5), (16, 2, 2, 8), (64, 8, 3, 6), (72, 9, 4, 8), (160, 8, 3, 6), (160, 5, 2, 8),
    (256, 8, 4, 8), (256, 16, 1, 16), (256, 64, 7, 8), (320, 16, 4, 8), (384, 12, 5, 12), (512, 8, 4, 8), (768, 3, 2, 8), (990, 33, 2, 9),
    (1024, 32, 4, 8), (1024, 128, 9, 8), (1020, 1020, 30, 20), (1024, 64, 64, 31)])
def test_groups(E, groups, top_groups, k, biased, group_score):
    for score in ("softmax", "sigmoid"):
        x, bias = _inputs(120, E, seed=E + groups + k)
        print(f"case E={E} groups={groups} of which {top_groups} k={k} bias={biased} {group_score} {score}", flush=True)
        _check(x, k, score, bias if biased else None, groups, top_groups, group_score, True, 2.5)


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 15, 16, 17, 63, 64, 65, 255, 257, 1000, 4099])
@pytest.mark.parametrize("E,k,groups,top_groups", [(8, 2, 1, 1), (60, 4, 1, 1), (128, 4, 1, 1), (256, 8, 8, 4), (512, 8, 1, 1)])
def test_row_counts(T, E, k, groups, top_groups):
    x, bias = _inputs(T, E, seed=T + E)
    print(f"case T={T} E={E}", flush=True)
    lx, idx, router = _check(x, k, "sigmoid", bias, groups, top_groups, "top2", True, 2.5)
    _check_backward(x, lx, idx, router, T)
    lx, idx, router = _check(x, k, "softmax", None, 1, 1, "top2", False, 1.0)
    _check_backward(x, lx, idx, router, T + 1)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_ties(score):
    """Logits held in bf16 (ties everywhere), all equal, and a zero bias."""
    for E, groups, top_groups, k in [(64, 1, 1, 8), (256, 8, 4, 8), (96, 3, 2, 6)]:
        x, _ = _inputs(300, E, seed=E, held="bf16", spread=0.25)
        x[7] = 0.5
        x[8] = -0.0
        x[9, ::2] = 0.0
        for bias in (None, np.zeros(E, dtype=np.float32)):
            print(f"case E={E} {score} bias={bias is not None}", flush=True)
            for group_score in ("max", "top2"):
                _check(x, k, score, bias, groups, top_groups, group_score, True, 1.0)


def test_far_logits():
    """Sigmoids that round to 0 or 1 in fp32, softmaxes with one expert alone."""
    x, bias = _inputs(100, 64, seed=4, spread=40.0)
    for score in ("softmax", "sigmoid"):
        for biased in (False, True):
            lx, idx, router = _check(x, 4, score, bias if biased else None, 1, 1, "max", True, 1.0)
            _check_backward(x, lx, idx, router, 3)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,top_groups,group_score", [(1, 1, "max"), (4, 2, "top2"), (4, 2, "max")])
@pytest.mark.parametrize("biased", [False, True])
def test_infinities_and_nan(score, groups, top_groups, group_score, biased):
    """Any values give distinct ids of groups that stay; rows without them are not touched by them."""
    x, bias = _inputs(64, 32, seed=8)
    clean = x.copy()
    x[1, 3] = -np.inf  # an expert out
    x[2, :30] = -np.inf
    x[3] = -np.inf
    x[4, 5] = np.nan
    x[5] = np.nan
    x[6, 9] = np.inf
    x[7, 9:12] = np.inf
    if biased:
        bias[13] = -np.inf
        bias[14] = np.nan
    router = moe.Router(score, _gpu(bias) if biased else None, groups, top_groups, group_score, True, 1.0)
    idx, w = moe.route_experts(_gpu(x), 6, router)
    torch.cuda.synchronize()
    ids = idx.cpu().numpy()
    with np.errstate(invalid="ignore"):
        want, ww = st.route_experts(x, 6, score, bias if biased else None, groups, top_groups,
                                    2 if group_score == "top2" else 1)
    np.testing.assert_array_equal(ids, want)
    got = w.cpu().numpy()
    finite = np.isfinite(ww)
    np.testing.assert_array_equal(np.isfinite(got), finite)
    assert (np.abs(got - ww)[finite] <= 50 * U * np.abs(ww)[finite] + 1e-38).all()
    for t in range(64):
        assert len(set(ids[t])) == 6 and ids[t].min() >= 0 and ids[t].max() < 32
    other, _ = moe.route_experts(_gpu(clean), 6, router)
    assert torch.equal(other[8:], idx[8:])


def test_masked_experts_pass_no_gradient():
    x, _ = _inputs(40, 24, seed=2)
    x[:, 5] = -np.inf
    x[:, 20] = -np.inf
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            router = moe.Router(score, renormalize=renormalize)
            lx = _gpu(x)
            idx, w = moe.route_experts(lx, 22, router)
            g = moe.route_experts_backward(lx, idx, torch.randn(40, 22, device=dev), router)
            torch.cuda.synchronize()
            assert torch.isfinite(w).all() and torch.isfinite(g).all() and not g[:, [5, 20]].any()


def test_ids_outside_are_left_out():
    x, _ = _inputs(50, 16, seed=3)
    idx = np.tile(np.array([3, -1, 7, 16, 2 ** 31 - 1, 9], dtype=np.int32), (50, 1))
    d_w = np.random.default_rng(1).standard_normal((50, 6)).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            got = moe.route_experts_backward(_gpu(x), _gpu(idx), _gpu(d_w), moe.Router(score, renormalize=renormalize))
            want = st.route_experts_backward(x, idx, d_w, score, renormalize)
            torch.cuda.synchronize()
            assert np.abs(got.cpu().numpy() - want).max() <= 110 * U * 6  # |u| < 3, |ds/dx| <= 1 / 4


def test_gradient_against_differences_of_the_forward():
    """(w(x + h) - w(x - h)) / 2h of the GPU's own forward, whose weights are off by 50 u: with
    h = 2^-6 the quotient is off by 50 u / h and by h^2 / 6 of a third derivative (below 6)."""
    rng = np.random.default_rng(12)
    T, E, k, h = 4, 12, 4, 2.0 ** -6
    x = (2.0 * rng.standard_normal((T, E))).astype(np.float32)
    u = rng.standard_normal((T, k)).astype(np.float32)
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            router = moe.Router(score, renormalize=renormalize)
            idx, _ = moe.route_experts(_gpu(x), k, router)
            got = moe.route_experts_backward(_gpu(x), idx, _gpu(u), router).cpu().numpy()
            ids = idx.cpu().numpy()

            def value(z, t):  # the forward's weights of the same ids (its choice may be another order or set)
                i, w = (a.cpu().numpy() for a in moe.route_experts(_gpu(z), k, router))
                at = {e: j for j, e in enumerate(i[t])}
                return None if set(at) != set(ids[t]) else sum(u[t, j] * float(w[t, at[e]]) for j, e in enumerate(ids[t]))

            checked = 0
            for t in range(T):
                for e in range(E):
                    d = np.zeros((T, E), dtype=np.float32)
                    d[t, e] = h
                    hi, lo = value(x + d, t), value(x - d, t)
                    if hi is None or lo is None:
                        continue
                    checked += 1
                    slack = np.abs(u[t]).sum() * (50 * U / h + h * h) + 1e-6
                    assert abs((hi - lo) / (2 * h) - got[t, e]) <= slack, (score, renormalize, t, e)
            assert checked > T * E // 2


def test_no_tokens_and_unaligned_views():
    idx, w = moe.route_experts(torch.empty((0, 8), device=dev), 2, moe.Router("sigmoid"))
    assert idx.shape == (0, 2) and w.shape == (0, 2)
    x, bias = _inputs(37, 64, seed=6)
    want = moe.route_experts(_gpu(x), 6, moe.Router("sigmoid", _gpu(bias)))
    for off in (1, 2, 3):
        flat = torch.empty(37 * 64 + off, device=dev)
        flat[off:] = _gpu(x).reshape(-1)
        fb = torch.empty(64 + off, device=dev)
        fb[off:] = _gpu(bias)
        lx, router = flat[off:].view(37, 64), moe.Router("sigmoid", fb[off:])
        buf = torch.full((37 * 6 + off,), -1.0, device=dev)
        ids = torch.full((37 * 6 + off,), -1, dtype=torch.int32, device=dev)
        got = moe.route_experts(lx, 6, router, topk_idx=ids[off:].view(37, 6), topk_w=buf[off:].view(37, 6))
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert (buf[:off] == -1).all() and (ids[:off] == -1).all()
        d_w = torch.randn(37, 6, device=dev)
        ref = moe.route_experts_backward(_gpu(x), want[0], d_w, router)
        dflat = torch.full((37 * 64 + off + 3,), 7.0, device=dev)
        moe.route_experts_backward(lx, want[0], d_w, router, d_logits=dflat[off:off + 37 * 64].view(37, 64))
        assert torch.equal(dflat[off:off + 37 * 64].view(37, 64), ref)
        assert (dflat[:off] == 7).all() and (dflat[off + 37 * 64:] == 7).all()


def test_streams_and_graph():
    x, bias = _inputs(900, 256, seed=10)
    lx, b = _gpu(x), _gpu(bias)
    router = moe.Router("sigmoid", b, 8, 4, "top2", True, 2.5)
    d_w = torch.randn(900, 8, device=dev)
    ref = (*moe.route_experts(lx, 8, router), None)
    ref = (ref[0], ref[1], moe.route_experts_backward(lx, ref[0], d_w, router))
    torch.cuda.synchronize()
    outs = []
    for s in [torch.cuda.Stream() for _ in range(2)]:
        f = moe.route_experts(lx, 8, router, stream=s)
        outs.append((*f, moe.route_experts_backward(lx, f[0], d_w, router, stream=s)))
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(p, q) for p, q in zip(o, ref))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = moe.route_experts(lx, 8, router)
        g = moe.route_experts_backward(lx, f[0], d_w, router)
    for i in range(3):
        y, bias2 = _inputs(900, 256, seed=20 + i)
        lx.copy_(_gpu(y))
        b.copy_(_gpu(bias2))
        want = moe.route_experts(lx, 8, router)
        gw = moe.route_experts_backward(lx, want[0], d_w, router)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(f[0], want[0]) and torch.equal(f[1], want[1]) and torch.equal(g, gw), i


def _in_few(lx, k, router, rows=1000):
    """The same tokens in calls of a few, which compare every score in fp64."""
    parts = [moe.route_experts(lx[at:at + rows], k, router) for at in range(0, lx.shape[0], rows)]
    return tuple(torch.cat(p) for p in zip(*parts))


BIASES = {"small": lambda r, E: 0.05 * r.standard_normal(E), "zero": lambda r, E: np.zeros(E),
          "far apart": lambda r, E: r.choice([-1000.0, 1000.0, 3.0], E) + 0.01 * r.standard_normal(E),
          "large": lambda r, E: 1e6 + r.integers(0, 4, E)}


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", sorted(BIASES))
@pytest.mark.parametrize("E,groups,top_groups,k", [(128, 1, 1, 4), (100, 1, 1, 8), (200, 8, 3, 6), (256, 8, 4, 8), (256, 8, 4, 16), (256, 16, 5, 3),
                                                   (264, 1, 1, 8), (384, 3, 2, 12), (512, 8, 4, 8), (512, 32, 8, 16), (1000, 4, 2, 8),
                                                   (1024, 1, 1, 2)])
def test_many_tokens_choose_as_few_do(E, groups, top_groups, k, bias, score):
    """Sizes at which candidates are found on fp32 values: ids as in calls of a few tokens bit for
    bit, weights to a rounding, and 60 rows against the plain form."""
    T = 16391 if E <= 256 else 8209
    rng = np.random.default_rng(E + groups + k)
    x, _ = _inputs(T, E, seed=E + k)
    x[::3] = torch.from_numpy(x[::3]).bfloat16().float().numpy()  # ties
    x[5] = 0.25  # all equal
    x[6, : E // 2] = x[6, E // 2: 2 * (E // 2)]
    x[7] = -30.0 - np.arange(E) % 7  # sigmoids near 0
    x[8] = 30.0 + np.arange(E) % 5  # that round to 1
    x[9, ::2] = -np.inf
    x[10, 3], x[11, E - 1], x[12, 1] = np.nan, np.inf, -np.nan
    b = BIASES[bias](rng, E).astype(np.float32)
    print(f"case E={E} groups={groups} of which {top_groups} k={k} bias {bias} {score}", flush=True)
    lx = _gpu(x)
    at = np.r_[0:20, T - 20:T, rng.integers(0, T, 20)]
    for group_score in ("top2", "max"):
        router = moe.Router(score, _gpu(b), groups, top_groups, group_score, True, 1.5)
        idx, w = moe.route_experts(lx, k, router)
        few, fw = _in_few(lx, k, router)
        torch.cuda.synchronize()
        assert torch.equal(idx, few)
        ok = torch.isfinite(fw)
        assert torch.equal(torch.isfinite(w), ok) and ((w - fw).abs()[ok] <= 4 * U * fw.abs()[ok]).all()
        with np.errstate(invalid="ignore"):
            want, _ = st.route_experts(x[at], k, score, b, groups, top_groups, 2 if group_score == "top2" else 1, True, 1.5)
        np.testing.assert_array_equal(idx.cpu().numpy()[at], want)


@pytest.mark.parametrize("score,renormalize", [("softmax", True), ("softmax", False), ("sigmoid", False)])
@pytest.mark.parametrize("E,k", [(128, 4), (250, 8), (256, 16), (512, 8), (1024, 8)])
def test_many_tokens_by_their_logits(E, k, score, renormalize):
    T = 16391 if E <= 256 else 8209
    x, bias = _inputs(T, E, seed=E, held="bf16")
    x[3] = 1.0
    lx = _gpu(x)
    for b in (None, bias):
        router = moe.Router(score, None if b is None else _gpu(b), renormalize=renormalize)
        idx, w = moe.route_experts(lx, k, router)
        few, fw = _in_few(lx, k, router)
        torch.cuda.synchronize()
        assert torch.equal(idx, few) and ((w - fw).abs() <= 16 * U * fw.abs()).all()
        want, _ = st.route_experts(x[:30], k, score, b, 1, 1, 1, renormalize)
        np.testing.assert_array_equal(idx.cpu().numpy()[:30], want)
        d_w = torch.randn(T, k, device=dev, generator=torch.Generator(device=dev).manual_seed(1))
        g = moe.route_experts_backward(lx, idx, d_w, router)
        gf = torch.cat([moe.route_experts_backward(lx[a:a + 1000], idx[a:a + 1000], d_w[a:a + 1000], router) for a in range(0, T, 1000)])
        torch.cuda.synchronize()
        assert torch.equal(g, gf)


def test_many_tokens_past_32_bit_offsets():
    """Rows whose elements lie past 2^31 and 2^32 bytes; one expert a token and a whole row."""
    T, E = (1 << 23) + 5, 264
    row, bias = _inputs(64, E, seed=30)
    lx = torch.empty((T, E), device=dev)
    lx[:] = _gpu(row[0])
    at = torch.randint(0, T, (63,), generator=torch.Generator().manual_seed(1))
    at[0], at[1], at[2] = T - 1, (1 << 31) // (4 * E) + 1, (1 << 32) // (4 * E) + 1
    lx[at.to(dev)] = _gpu(row[1:])
    router = moe.Router("sigmoid", _gpu(bias), 8, 4, "top2", True, 2.5)
    idx, w = moe.route_experts(lx, 8, router)
    few = moe.route_experts(lx[at.to(dev)].contiguous(), 8, router)
    assert torch.equal(idx[at.to(dev)], few[0]) and torch.equal(w[at.to(dev)], few[1])
    d_w = torch.randn(T, 8, device=dev)
    g = moe.route_experts_backward(lx, idx, d_w, router)
    gf = moe.route_experts_backward(lx[at.to(dev)].contiguous(), few[0], d_w[at.to(dev)].contiguous(), router)
    assert torch.equal(g[at.to(dev)], gf)
