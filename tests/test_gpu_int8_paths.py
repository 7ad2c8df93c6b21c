"""The experts in 8-bit integers, one kind of workgroup after the other: each test says
which kind it means and sees from the workspace that this kind ran.

The list of row tiles is the workspace's last part: two ints (how many entries, and how
many are of experts with more than 128 rows), then from byte 256 on 16 bytes a tile: row0,
row_end (int32), expert, index (int16), tiles, last, alone (int8) of the tile's group.
An expert's rows are cut every 32 (thin), every 128 (short) or every 256 rows, where up
to 32 rows behind the last whole tile ride along on it (tall). A call of few rows lists
none and writes no codes. Bounds are derived in test_gpu_int8.py.
"""
import numpy as np
import pytest

import moe_inputs as mi
from tests import _gpu as g

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import token_dispatch_grouped_amd as moe  # noqa: E402
from oracle import around as oa  # noqa: E402
from tests import test_gpu_int8 as base  # noqa: E402

W = mi.Workload
ENTRY = np.dtype([("row0", "<i4"), ("row_end", "<i4"), ("expert", "<i2"), ("index", "<i2"), ("tiles", "i1"),
                  ("last", "i1"), ("alone", "i1"), ("pad", "i1")])


def _tiles(kind, rows):
    full, rest = divmod(rows, {"thin": 32, "short": 128, "tall": 256}[kind])
    if kind == "tall" and full and rest <= 32:
        return full
    return full + (rest > 0)


def _kind(ws, w, offsets):
    """The kind of workgroup that a call on this workspace (filled with 0x5A before) used; kinds, where the
    experts' rows are too few to tell them apart by their tiles."""
    n, up = w.n_max, lambda v: -(-v // 256) * 256  # noqa: E731
    kb = lambda v: -(-v // 64)  # noqa: E731
    at = up(n * kb(w.d) * 64) + 2 * up(n * 4) + up(n * w.d_ff * 2) + up(n * kb(w.d_ff) * 64)
    plan = ws[at:].cpu().numpy()
    if (plan[:8] == 0x5A).all():
        assert bool((ws[:min(up(n * kb(w.d) * 64), 4096)] == 0x5A).all())  # no codes either
        return "few"
    count, over_128 = (int(v) for v in plan[:8].view("<i4"))
    entries = plan[256:256 + 16 * count].view(ENTRY)
    offs = offsets.cpu().numpy()
    lo = offs[w.e_begin]
    rows = [int(min(offs[w.e_begin + e + 1] - lo, n) - min(offs[w.e_begin + e] - lo, n)) for e in range(w.E_loc)]
    got = np.bincount(entries["expert"], minlength=w.E_loc).tolist()
    fits = [k for k in ("thin", "short", "tall") if [_tiles(k, r) for r in rows] == got]
    assert fits, (rows, got)
    big = [e for e, r in enumerate(rows) if r > 128]
    assert over_128 == sum(got[e] for e in big) and sorted(set(entries["expert"][:over_128])) == big
    return " or ".join(fits)


def _ran(w, kind, idx=None, logits=None):
    """The whole check of one call, after seeing that it was of this kind."""
    x, lg, wgu, wdn = base._inputs(w, logits)
    experts = moe.quantize_experts(wgu, wdn)
    disp, ws, _ = base._run(w, x, lg, experts, idx=idx)
    assert _kind(ws, w, disp.offsets) == kind
    base._check(w, x, lg, experts, idx=idx)
    return x, lg, experts, disp, ws


KINDS = [
    ("few", W("few_decode", 32, 256, 192, 64, 4, 0, 64, "bf16", 101)),
    ("few", W("few_share", 100, 136, 264, 64, 1, 8, 24, "bf16", 102)),
    ("thin or short or tall", W("light_batch", 300, 1176, 344, 64, 4, 0, 64, "bf16", 103)),  # 19 rows an expert
    ("thin", W("thin_deep", 348, 64, 7536, 4, 2, 0, 4, "bf16", 109)),
    ("thin", W("thin_share", 520, 264, 136, 32, 4, 8, 16, "bf16", 104)),
    ("short", W("short_batch", 1000, 1032, 2056, 4, 2, 0, 4, "bf16", 105)),
    ("short", W("short_deep", 700, 2824, 4104, 8, 2, 0, 4, "bf16", 106)),
    ("tall", W("tall_one", 9273, 2824, 784, 2, 1, 1, 2, "bf16", 107)),
    ("short", W("short_share", 8192, 2824, 2824, 32, 4, 0, 4, "bf16", 113)),
    ("tall", W("tall_share", 2048, 2824, 2824, 32, 4, 8, 24, "bf16", 114)),  # sixteen experts of 256 rows
    ("short", W("short_many", 8192, 1288, 2472, 16, 2, 0, 16, "bf16", 108)),
]


@pytest.mark.parametrize("kind,w", KINDS, ids=[f"{k}-{w.name}" for k, w in KINDS])
def test_each_kind(kind, w):
    _ran(w, kind)


# K of 128 x 64 .. 1024 x 64: rows of 64, 256 and 1024 threads, as the quantiser cuts them
LONG = [(64, 4160), (64, 8712), (64, 16392), (64, 20040), (64, 32768), (64, 32776), (64, 65536), (16392, 64),
        (32776, 64), (65536, 64)]


@pytest.mark.parametrize("d,f", LONG, ids=[f"{d}x{f}" for d, f in LONG])
def test_long_rows_codes(d, f):
    """Rows past 16384 elements are quantised by 1024 threads, of x (through perm) and of h; their codes and
    scales are in the workspace, and compared bit for bit."""
    w = W("long_rows", 200, d, f, 2, 1, 0, 2, "bf16", 110)
    x, lg, wgu, wdn = base._inputs(w)
    x[3] = 0
    x[5, -1], x[9, 0] = float("inf"), float("nan")
    x[11] *= 1e-30
    experts = moe.quantize_experts(wgu, wdn)
    disp, ws, _ = base._run(w, x, lg, experts)
    assert _kind(ws, w, disp.offsets) in ("thin", "short")
    tok = disp.perm.cpu().numpy()
    xq, xs, h, hq, hs = base._parts(ws, w.n_max, d, f)
    want_q, want_s = oa.quantize(x.float().cpu().numpy()[tok])
    np.testing.assert_array_equal(xq.cpu().numpy(), oa.kblocks(want_q))
    base._equal_scales(xs.cpu().numpy(), want_s)
    want_q, want_s = oa.quantize(h.float().cpu().numpy())
    np.testing.assert_array_equal(hq.cpu().numpy(), oa.kblocks(want_q))
    base._equal_scales(hs.cpu().numpy(), want_s)
    assert np.isnan(want_s).sum() == 2  # the two rows without a finite scale


@pytest.mark.parametrize("d,f", [(64, 20040), (64, 65536), (65536, 64)])
def test_long_rows(d, f):
    w = W("long_rows", 200, d, f, 2, 1, 0, 2, "bf16", 111)
    x, lg, wgu, wdn = base._inputs(w)
    experts = moe.quantize_experts(wgu, wdn)
    base._check(w, x, lg, experts)


def _equal_rows(rows, E, d, f, seed):
    """E experts of `rows` rows each, token t with expert t / rows."""
    T = E * rows
    w = W("equal", T, d, f, E, 1, 0, E, "bf16", seed)
    x = g.to_dev(mi.hidden_states(w), "bf16")
    wgu, wdn = (g.to_dev(a, "bf16") for a in mi.expert_weights(w))
    perm = torch.arange(T, dtype=torch.int32, device="cuda")
    offsets = torch.arange(0, T + 1, rows, dtype=torch.int32, device="cuda")
    return w, x, wgu, wdn, perm, offsets


def _call(w, x, perm, offsets, experts):
    ws = torch.full((moe.grouped_gemm_int8_workspace_bytes(w.T, w.d, w.d_ff, w.E, w.k, w.e_begin, w.e_end),), 0x5A,
                    dtype=torch.uint8, device="cuda")
    y = moe.grouped_gemm_int8(x, perm, offsets, experts, w.k, w.E, w.e_begin, w.e_end, workspace=ws)
    torch.cuda.synchronize()
    return y, _kind(ws, w, offsets)


@pytest.mark.parametrize("kind,rows,E,d,f", [("thin", 65, 8, 264, 136), ("short", 272, 4, 1032, 2056),
                                             ("short", 200, 4, 2824, 4104), ("tall", 272, 5, 1288, 2472),
                                             ("tall", 288, 16, 1288, 2472)])
def test_a_row_has_the_bits_of_the_few_kind(kind, rows, E, d, f):
    w, x, wgu, wdn, perm, offsets = _equal_rows(rows, E, d, f, 112)
    every, ran = _call(w, x, perm, offsets, moe.quantize_experts(wgu, wdn))
    assert ran == kind
    ends = torch.tensor([0, 8], dtype=torch.int32, device="cuda")
    for e in range(0, E, max(1, E // 4)):
        one = moe.quantize_experts(wgu[e:e + 1].contiguous(), wdn[e:e + 1].contiguous())
        for r in (e * rows, e * rows + rows // 2, (e + 1) * rows - 8):
            few, ran = _call(w.with_(T=8, E=1, e_end=1), x[r:r + 8].contiguous(), perm[:8], ends, one)
            assert ran == "few" and torch.equal(few, every[r:r + 8]), (e, r)


@pytest.mark.parametrize("kind,w", [KINDS[0], KINDS[2], KINDS[3], KINDS[5]],
                         ids=["few", "light", "thin", "short"])
def test_non_finite_rows_stay_in_their_rows_in_each_kind(kind, w):
    x, lg, wgu, wdn = base._inputs(w)
    experts = moe.quantize_experts(wgu, wdn)
    disp, _, clean = base._run(w, x, lg, experts)
    bad = x.clone()
    bad[3, 5], bad[7, 0], bad[11] = float("nan"), float("-inf"), 0.0
    disp, ws, y = base._run(w, bad, lg, experts)
    assert _kind(ws, w, disp.offsets) == kind
    pos = disp.pair_pos.cpu().numpy().reshape(w.T, w.k)
    rows, zero = np.zeros(w.n_max, dtype=bool), np.zeros(w.n_max, dtype=bool)
    rows[np.r_[pos[3], pos[7]]] = True
    zero[pos[11]] = True
    np.testing.assert_array_equal(torch.isnan(y).all(dim=1).cpu().numpy(), rows)
    assert not y[torch.from_numpy(zero).cuda()].any()
    same = torch.from_numpy(~rows & ~zero).cuda()
    assert torch.equal(y[same], clean[same])
