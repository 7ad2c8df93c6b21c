"""The experts in 8-bit integers, step by step against the definition.

The codes and scales of a row are fixed by fp32 operations that round correctly
on both sides, so they have to be equal bit for bit. The integer sums are exact.
What rounds (u = 2^-24):
  h   G and U: the sum to fp32, two products: 3 u each. silu(G) U: exp2 and the
      reciprocal of the hardware are good to 1 ulp (2 u) each, the exponent's
      argument G log2(e) to 2 u |G|, which the sigmoid passes on by at most its own
      size; two products. Relative (4 |G| + 24) u, and 3 u |G| of G's own error
      through silu (whose logarithmic derivative is at most 1 + |G|): bounded by
      (8 |G| + 32) u; then half a step of bf16, 2^-8.
  y   the sum to fp32 and two products: 4 u; then half a step of bf16.
The workspace holds, each at a multiple of 256 bytes, the codes and scales of x's
rows, h, and h's codes and scales, in this order: that is where h is read from.
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

U = 2.0 ** -24


def _np(t):
    return t.cpu().numpy()


def _parts(ws, n, d, f):
    """The workspace's parts for n rows: x codes [kb, n, 64], x scales, h [n, f], h codes, h scales."""
    kb = lambda v: (v + 63) // 64  # noqa: E731
    at, out = 0, []
    for size, view in ((n * kb(d) * 64, lambda b: b.view(torch.int8).view(kb(d), n, 64)),
                       (n * 4, lambda b: b.view(torch.float32)),
                       (n * f * 2, lambda b: b.view(torch.bfloat16).view(n, f)),
                       (n * kb(f) * 64, lambda b: b.view(torch.int8).view(kb(f), n, 64)),
                       (n * 4, lambda b: b.view(torch.float32))):
        out.append(view(ws[at:at + size]))
        at += -(-size // 256) * 256
    return out  # the list of row tiles follows


def _equal_scales(got, want):
    np.testing.assert_array_equal(got.view(np.uint32)[~np.isnan(want)], want.view(np.uint32)[~np.isnan(want)])
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))


def _inputs(w, logits=None):
    logits = mi.router_logits(w) if logits is None else logits
    x = mi.hidden_states(w)
    wgu, wdn = mi.expert_weights(w)
    return g.to_dev(x, "bf16"), g.to_dev(logits, "f32"), g.to_dev(wgu, "bf16"), g.to_dev(wdn, "bf16")


def _run(w, x, logits, experts, y=None, idx=None):
    if idx is None:
        idx, _ = moe.route_topk(logits, w.k)
    disp = moe.dispatch(x, idx, w.E, w.e_begin, w.e_end, gather=False)
    ws = torch.full((moe.grouped_gemm_int8_workspace_bytes(w.T, w.d, w.d_ff, w.E, w.k, w.e_begin, w.e_end),), 0x5A,
                    dtype=torch.uint8, device="cuda")
    if y is None:
        y = torch.full((w.n_max, w.d), 9.0, dtype=torch.bfloat16, device="cuda")
    moe.grouped_gemm_int8(x, disp.perm, disp.offsets, experts, w.k, w.E, w.e_begin, w.e_end, y=y, workspace=ws)
    torch.cuda.synchronize()
    return disp, ws, y


def _check(w, x, logits, experts, idx=None):
    print(f"case {w}", flush=True)
    disp, ws, y = _run(w, x, logits, experts, idx=idx)
    offs, perm = _np(disp.offsets), _np(disp.perm)
    lo = offs[w.e_begin]
    n_loc = min(int(offs[w.e_end] - lo), w.n_max)  # ids that a token repeats may give more: rows past n_max are dropped
    tok = perm[lo:lo + n_loc] // w.k
    xq, xs, h, hq, hs = _parts(ws, w.n_max, w.d, w.d_ff)
    x32 = x.float().cpu().numpy()[tok]
    want_q, want_s = oa.quantize(x32)
    h_got = g.to_f64(h)[:n_loc]
    hq_want, hs_want = oa.quantize(h_got.astype(np.float32))
    if not bool((ws[:xq.numel()] == 0x5A).all()):  # (the codes of few rows stay on the chip)
        np.testing.assert_array_equal(_np(xq)[:, :n_loc], oa.kblocks(want_q))
        _equal_scales(_np(xs)[:n_loc], want_s)
        np.testing.assert_array_equal(_np(hq)[:, :n_loc], oa.kblocks(hq_want))
        _equal_scales(_np(hs)[:n_loc], hs_want)
    wgu, sgu = oa.from_kblocks(_np(experts.w_gate_up), w.d), _np(experts.gate_up_scale)
    wdn, sdn = oa.from_kblocks(_np(experts.w_down), w.d_ff), _np(experts.down_scale)
    y_got = g.to_f64(y)
    worst = [0.0, 0.0]
    for e in range(w.E_loc):
        r0, r1 = (min(int(offs[w.e_begin + e + i] - lo), w.n_max) for i in (0, 1))
        if r0 == r1:
            continue
        gu = oa.int8_product(want_q[r0:r1], want_s[r0:r1], wgu[e], sgu[e])
        want = oa.swiglu(gu)
        bound = np.abs(want) * (2.0 ** -8 * 1.001 + (8 * np.abs(gu[:, :w.d_ff]) + 32) * U) + 1e-30
        err = np.abs(h_got[r0:r1] - want)
        worst[0] = max(worst[0], float((err / bound).max()))
        assert (err <= bound).all(), ("h", e, worst[0])
        want = oa.int8_product(hq_want[r0:r1], hs_want[r0:r1], wdn[e], sdn[e])
        bound = np.abs(want) * (2.0 ** -8 * 1.001 + 4 * U) + 1e-30
        err = np.abs(y_got[r0:r1] - want)
        worst[1] = max(worst[1], float((err / bound).max()))
        assert (err <= bound).all(), ("y", e, worst[1])
    print(f"  worst error of its bound: h {worst[0]:.3f}, y {worst[1]:.3f}", flush=True)
    assert (y_got[n_loc:] == 9.0).all()  # rows behind the last pair stay as they were
    return disp, y


def _case(w, logits=None):
    x, lg, wgu, wdn = _inputs(w, logits)
    return _check(w, x, lg, moe.quantize_experts(wgu, wdn))


W = mi.Workload
CASES = [
    W("i8_small", 600, 256, 160, 8, 2, 0, 8, "bf16", 61),
    W("i8_share", 900, 192, 128, 32, 4, 8, 16, "bf16", 62),
    W("i8_skew", 1000, 320, 128, 64, 8, 0, 16, "bf16", 63, 1.5),
    W("i8_decode", 5, 256, 192, 128, 4, 0, 128, "bf16", 64),
    W("i8_one_token", 1, 1000, 1480, 32, 4, 0, 32, "bf16", 65),
    W("i8_ragged", 300, 72, 136, 4, 2, 0, 4, "bf16", 66),       # K tails of 8, channels past whole tiles
    W("i8_tiny", 3, 8, 8, 2, 1, 0, 2, "bf16", 67),
    W("i8_one_expert", 700, 328, 264, 1, 1, 0, 1, "bf16", 68),
    W("i8_all_of_k", 40, 64, 520, 8, 8, 0, 8, "bf16", 69),
    W("i8_wide_k", 20, 2056, 4104, 4, 2, 0, 2, "bf16", 70),     # rows of 256-thread groups
    W("i8_wider_k", 6, 64, 8712, 2, 1, 0, 2, "bf16", 71),       # rows of 1024-thread groups
    W("i8_few", 16, 200, 328, 32, 4, 8, 16, "bf16", 77),        # a few tokens, two rows per expert
    W("i8_few_many_rows", 64, 136, 72, 64, 1, 0, 64, "bf16", 78, 3.0),  # skewed: several row tiles of one expert
    W("i8_few_wide", 8, 512, 2056, 64, 4, 0, 64, "bf16", 79),   # enough channels for the wide workgroups
    W("i8_few_long_k", 1, 64, 8712, 2, 1, 0, 2, "bf16", 80),    # more of a row than its threads hold
    W("i8_few_twelve", 96, 200, 136, 8, 1, 0, 8, "bf16", 85),   # twelve rows per expert, four at a time
    W("i8_few_share", 128, 136, 264, 64, 1, 8, 24, "bf16", 86, 2.0),  # skewed: some experts take several turns
    W("i8_few_full", 16, 64, 3008, 4, 1, 0, 4, "bf16", 87),     # sixteen rows, all of the LDS
    W("i8_few_longest", 1, 64, 48904, 2, 1, 0, 2, "bf16", 88),  # one row, all of the LDS
    W("i8_few_wide_rows", 2, 2056, 8200, 8, 8, 0, 8, "bf16", 89),  # two long rows, one after the other
    W("i8_long_rows", 9273, 2824, 784, 2, 1, 1, 2, "bf16", 83),  # one expert of thousands, several rounds
    W("i8_stages", 260, 448, 192, 2, 1, 0, 2, "bf16", 72),      # 7 and 3 K stages
]


@pytest.mark.parametrize("w", CASES, ids=[w.name for w in CASES])
def test_experts_match_the_definition(w):
    _case(w)


def test_every_row_count():
    """Expert row counts at the edges of the row tiles, empty experts among them."""
    counts = [0, 1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 289, 0, 513]
    E, T = len(counts), sum(counts)
    logits = _routed(counts, 73)
    disp, _ = _case(W("i8_rows", T, 256, 160, E, 1, 0, E, "bf16", 73), logits)
    np.testing.assert_array_equal(_np(disp.counts), counts)


@pytest.mark.parametrize("T,k,E,lo,hi", [(4, 4, 8, 0, 8), (20, 4, 64, 0, 64), (20, 4, 64, 7, 8), (64, 2, 64, 3, 9),
                                         (300, 4, 8, 0, 8), (300, 4, 8, 3, 4)])
def test_ids_that_a_token_repeats(T, k, E, lo, hi):
    """Ids from elsewhere that name an expert several times: it gets more rows than there are tokens."""
    w = W("i8_again", T, 200, 328, E, k, lo, hi, "bf16", 84)
    x, lg, wgu, wdn = _inputs(w)
    idx = torch.full((T, k), min(7, E - 1) if E > 8 else 3, dtype=torch.int32, device="cuda")
    idx[::5, 0] = 5  # and a few elsewhere
    _check(w, x, lg, moe.quantize_experts(wgu, wdn), idx=idx)


def _routed(counts, seed):
    """Logits that send counts[e] tokens to expert e, in random order."""
    rng = np.random.default_rng(seed)
    T, E = sum(counts), len(counts)
    owner = np.repeat(np.arange(E), counts)
    rng.shuffle(owner)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    logits[np.arange(T), owner] += 50.0
    return logits


@pytest.mark.parametrize("d,f", [(256, 160), (264, 1352), (1480, 72), (136, 520), (520, 136), (64, 1032)])
def test_every_row_count_of_many_rows(d, f):
    """Many rows per expert at the edges of the row tiles, empty and light experts among them."""
    counts = [256, 0, 257, 288, 289, 300, 512, 544, 545, 1, 384, 600, 40]
    disp, _ = _case(W("i8_many", sum(counts), d, f, 13, 1, 0, 13, "bf16", 74), _routed(counts, 74))
    np.testing.assert_array_equal(_np(disp.counts), counts)


# the last two pairs of sizes, with 272 rows per expert on average, go to the tallest tiles
@pytest.mark.parametrize("d,f", [(200, 520), (200, 3320), (712, 2184), (1160, 2360), (1288, 2472)])
@pytest.mark.parametrize("counts", [(545, 1, 257, 300, 257), (544, 255, 129, 0, 432), (288, 272, 264, 280, 256)])
def test_every_row_count_of_tall_tiles(counts, d, f):
    """Tiles of 256 rows, remainders that ride along (up to 288 rows) or get a tile of their
    own, whole and halved."""
    disp, _ = _case(W("i8_tall", sum(counts), d, f, 5, 1, 0, 5, "bf16", 82), _routed(counts, 82))
    np.testing.assert_array_equal(_np(disp.counts), counts)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("e,d,f", [(3, 72, 136), (1, 8, 8), (2, 256, 64), (2, 200, 520)])
def test_quantized_weights(e, d, f, dt):
    rng = np.random.default_rng(e + d)
    gu, dn = rng.standard_normal((e, d, 2 * f)).astype(np.float32), rng.standard_normal((e, f, d)).astype(np.float32)
    gu[0, :, 1] = 0.0          # a channel of zeros
    gu[-1, 3, 2] = np.inf      # channels without a finite scale
    dn[0, 5, 3] = np.nan
    dn[0, :, 0] *= 1e-39       # below the smallest scale
    a, b = torch.from_numpy(gu).cuda(), torch.from_numpy(dn).cuda()
    if dt == "bf16":
        a, b = a.bfloat16(), b.bfloat16()
    got = moe.quantize_experts(a, b)
    torch.cuda.synchronize()
    for w, q, s in ((a, got.w_gate_up, got.gate_up_scale), (b, got.w_down, got.down_scale)):
        want_q, want_s = oa.quantize(np.swapaxes(w.float().cpu().numpy(), 1, 2))
        np.testing.assert_array_equal(_np(q), oa.kblocks(want_q))
        _equal_scales(_np(s), want_s)


def test_non_finite_rows_stay_in_their_rows():
    w = CASES[0]
    x, lg, wgu, wdn = _inputs(w)
    experts = moe.quantize_experts(wgu, wdn)
    disp, _, clean = _run(w, x, lg, experts)
    bad = x.clone()
    bad[7, 3], bad[100, 255] = float("nan"), float("-inf")
    bad[200] = 0.0
    _, _, y = _run(w, bad, lg, experts)
    pos = _np(disp.pair_pos).reshape(w.T, w.k)
    nan = torch.isnan(y).all(dim=1).cpu().numpy()
    rows = np.zeros(w.n_max, dtype=bool)
    rows[pos[7]] = rows[pos[100]] = True
    np.testing.assert_array_equal(nan, rows)
    assert not y[torch.from_numpy(pos[200]).cuda().long()].any()  # a row of zeros gives zeros
    same = ~rows
    same[pos[200]] = False
    assert torch.equal(y[torch.from_numpy(same).cuda()], clean[torch.from_numpy(same).cuda()])


def test_no_local_rows_and_no_tokens():
    w = W("i8_none", 20, 64, 64, 8, 1, 4, 8, "bf16", 74)
    logits = np.zeros((20, 8), np.float32)
    logits[:, 1] = 9.0  # every token goes to an expert of another rank
    disp, y = _case(w, logits)
    assert (g.to_f64(y) == 9.0).all()
    w0 = w.with_(T=0)
    experts = moe.quantize_experts(*(torch.zeros(s, dtype=torch.bfloat16, device="cuda")
                                     for s in ((4, 64, 128), (4, 64, 64))))
    y = moe.grouped_gemm_int8(torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"),
                              torch.empty(0, dtype=torch.int32, device="cuda"),
                              torch.zeros(9, dtype=torch.int32, device="cuda"), experts, 1, 8, 4, 8)
    assert y.shape == (w0.n_max, 64)


@pytest.mark.parametrize("d,f", [(1160, 2360), (200, 520)])
def test_a_row_has_the_same_bits_in_any_batch(d, f):
    """The same tokens for one expert: one at a time, in a few, and among many (other workgroups each time)."""
    x = g.to_dev(mi.hidden_states(W("i8_bits", 1360, d, f, 1, 1, 0, 1, "bf16", 90)), "bf16")
    wgu, wdn = (g.to_dev(a, "bf16") for a in mi.expert_weights(W("i8_bits", 8, d, f, 1, 1, 0, 1, "bf16", 90)))
    experts = moe.quantize_experts(wgu, wdn)

    def run(n):
        perm = torch.arange(n, dtype=torch.int32, device="cuda")
        return moe.grouped_gemm_int8(x[:n], perm, torch.tensor([0, n], dtype=torch.int32, device="cuda"), experts, 1, 1,
                                     0, 1)

    most = run(1360)
    for n in (1, 2, 5, 16, 40, 100, 272, 700):
        assert torch.equal(run(n), most[:n]), n


def test_a_row_has_the_same_bits_in_the_tallest_tiles():
    E, rows, d, f = 5, 272, 1160, 2360
    T = E * rows
    x = g.to_dev(mi.hidden_states(W("i8_bits", T, d, f, E, 1, 0, E, "bf16", 91)), "bf16")
    wgu, wdn = (g.to_dev(a, "bf16") for a in mi.expert_weights(W("i8_bits", 8, d, f, E, 1, 0, E, "bf16", 91)))
    perm = torch.arange(T, dtype=torch.int32, device="cuda")
    offsets = torch.arange(0, T + 1, rows, dtype=torch.int32, device="cuda")
    every = moe.grouped_gemm_int8(x, perm, offsets, moe.quantize_experts(wgu, wdn), 1, E, 0, E)
    ends = torch.tensor([0, 16], dtype=torch.int32, device="cuda")
    for e in range(E):
        one = moe.quantize_experts(wgu[e:e + 1].contiguous(), wdn[e:e + 1].contiguous())
        for r in (e * rows, e * rows + 100, (e + 1) * rows - 16):
            few = moe.grouped_gemm_int8(x[r:r + 16].contiguous(), perm[:16], ends, one, 1, 1, 0, 1)
            assert torch.equal(few, every[r:r + 16]), (e, r)


def test_streams_repeats_and_shared_inputs():
    w = CASES[2]
    x, lg, wgu, wdn = _inputs(w)
    experts = moe.quantize_experts(wgu, wdn)
    disp, _, ref = _run(w, x, lg, experts)
    n = int((disp.offsets[w.e_end] - disp.offsets[w.e_begin]).item())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ys = [moe.grouped_gemm_int8(x, disp.perm, disp.offsets, experts, w.k, w.E, w.e_begin, w.e_end, stream=s)
          for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(v[:n], ref[:n]) for v in ys)


def test_layer_int8_follows_the_bf16_layer():
    """The whole int8 layer: its steps one by one, bit for bit, and near the fp64
    layer on the unquantised weights. Each operand of a product is off by at most
    half a step of its row, a relative 2^-8 of the row's largest value; with normal
    rows (largest about 3.5 standard deviations) that is 0.0079 of the standard
    deviation in the root mean square (step / sqrt(12)), so a product of two such
    operands is off by 0.011 of its own root mean square, three products in a row
    (gate and up enter together) by less than 0.03, next to bf16's roundings."""
    w = W("i8_layer", 512, 512, 384, 16, 4, 0, 16, "bf16", 75)
    x, lg, wgu, wdn = _inputs(w)
    experts = moe.quantize_experts(wgu, wdn)
    res = moe.layer_int8(x, lg, experts, w.k, 0, w.E)
    y = moe.grouped_gemm_int8(x, res["perm"], res["offsets"], experts, w.k, w.E, 0, w.E)
    out = moe.combine(y, res["pair_pos"], res["w"], w.T, w.k, w.E, 0, w.E)
    torch.cuda.synchronize()
    assert torch.equal(y, res["y"]) and torch.equal(out, res["out"])
    ref = oracle.moe_layer(g.to_f64(x), _np(lg), w.k, 0, w.E, g.to_f64(wgu), g.to_f64(wdn))["out"]
    err = np.sqrt(((g.to_f64(out) - ref) ** 2).mean() / (ref ** 2).mean())
    print(f"  root mean square error {err:.4f} of the output's", flush=True)
    assert err <= 0.03


def test_graph_replays_and_two_graphs_on_one_workspace():
    w = W("i8_graph", 48, 256, 192, 64, 4, 0, 64, "bf16", 76)
    x, lg, wgu, wdn = _inputs(w)
    experts = moe.quantize_experts(wgu, wdn)
    ws = torch.empty(moe.grouped_gemm_int8_workspace_bytes(w.T, w.d, w.d_ff, w.E, w.k, 0, w.E), dtype=torch.uint8,
                     device="cuda")
    bx, blg = x.clone(), lg.clone()
    disp = moe.dispatch_alloc(bx, w.k, w.E, 0, w.E, gather=False)
    idx = torch.empty((w.T, w.k), dtype=torch.int32, device="cuda")
    wt = torch.empty((w.T, w.k), dtype=torch.float32, device="cuda")

    def step(y):
        moe.route_topk(blg, w.k, idx, wt)
        moe.dispatch(bx, idx, w.E, 0, w.E, out=disp, gather=False)
        moe.grouped_gemm_int8(bx, disp.perm, disp.offsets, experts, w.k, w.E, 0, w.E, y=y, workspace=ws)

    ys = [torch.empty((w.n_max, w.d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(ys[0])
    torch.cuda.current_stream().wait_stream(side)
    graphs = []
    for y in ys:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step(y)
        graphs.append(gr)
    for i in range(3):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(i)
        fx = torch.randn((w.T, w.d), generator=gen, device="cuda").bfloat16()
        fl = torch.randn((w.T, w.E), generator=gen, device="cuda")
        bx.copy_(fx)
        blg.copy_(fl)
        want = moe.layer_int8(fx, fl, experts, w.k, 0, w.E)["y"]
        torch.cuda.synchronize()
        for gr, y in zip(graphs, ys):  # in turn on one stream
            y.zero_()
            gr.replay()
        torch.cuda.synchronize()
        for y in ys:
            assert torch.equal(y, want), i
