"""The gradients of layer norm's weight and bias, with the number of additions that the
kernels really make.

A workgroup takes every B-th turn of the rows, B workgroups in all, and a turn is
256 / G rows side by side where a row has G <= 64 threads, else one. B is 512 where
there are at least 2048 turns and a row has at most 768 16-byte vectors; else half the
turns, at least 128 and at most 256 (and no more than the turns). A column's sum then
passes through ceil(turns / B) additions in a workgroup, the join of its row groups,
ceil(B / 16) in a wave of the second launch and 16 in the join of its waves: D in all.
With u = 2^-24 each is off by u of its result at most, the terms dy * h by 3 u (f - m,
its product with rstd, the product in the sum, which does not round by itself), so
  |error| <= (D + 4) u sum|terms| + half a step of the type * |sum|.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import token_dispatch_grouped_amd as moe  # noqa: E402

U, EPS = 2.0 ** -24, 1e-5
BF, F = torch.bfloat16, torch.float32
HALF = {BF: 2.0 ** -8, F: 2.0 ** -24}


def _additions(T, d, dt):
    vec = d // (8 if dt == BF else 4)
    group = next((g for g in (16, 32) if vec <= g), 64)
    side = 256 // group if vec <= 192 else 1
    turns = -(-T // side)
    blocks = 512 if turns >= 2048 and vec <= 768 else min(turns, max(128, min(256, turns // 2)))
    return -(-turns // blocks) + side + -(-blocks // 16) + 16


def _normal(shape, seed, dt, mean=0.0):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    out = torch.empty(shape, dtype=dt, device="cuda")
    rows = max(1, (1 << 27) // shape[1])
    for at in range(0, shape[0], rows):
        part = out[at:at + rows]
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda") + mean)
    return out


def _check(T, d, dt, wdt):
    print(f"case T={T} d={d} {dt} {wdt}", flush=True)
    s, dy, w = _normal((T, d), T, dt, 0.25), _normal((T, d), d, dt), _normal((1, d), 1, wdt)[0]
    _, _, mean, rstd = moe.layer_norm(s, w, None, EPS)
    _, dw, db = moe.layer_norm_backward(dy, s, w, mean, rstd)
    torch.cuda.synchronize()
    sums = torch.zeros((4, d), dtype=torch.float64, device="cuda")  # of dy h, |dy h|, dy, |dy|
    rows = max(1, (1 << 25) // d)
    for at in range(0, T, rows):
        g = dy[at:at + rows].double()
        p = g * ((s[at:at + rows].double() - mean[at:at + rows].double()[:, None]) * rstd[at:at + rows].double()[:, None])
        for i, v in enumerate((p, p.abs(), g, g.abs())):
            sums[i] += v.sum(dim=0)
    n = _additions(T, d, dt)
    for name, got, want, size in (("dw", dw, sums[0], sums[1]), ("db", db, sums[2], sums[3])):
        bound = (n + 4) * U * size + 1.001 * HALF[wdt] * want.abs()
        worst = float(((got.double() - want).abs() / bound).max())
        print(f"  {name}: worst error {worst:.3f} of its bound ({n} additions)", flush=True)
        assert worst <= 1, name


@pytest.mark.parametrize("dt,wdt", [(BF, BF), (BF, F), (F, F)])
@pytest.mark.parametrize("T,d", [(1, 8), (37, 136), (300, 264), (777, 2880), (2047, 1032), (2048, 6144), (2100, 6152),
                                 (16384, 72), (16385, 520), (33000, 8), (70001, 136), (5000, 16392), (4100, 32768)])
def test_column_sums(T, d, dt, wdt):
    _check(T, d, dt, wdt)


def test_column_sums_past_32_bit_offsets():
    d = 8192
    _check((1 << 31) // d + 37, d, BF, BF)
