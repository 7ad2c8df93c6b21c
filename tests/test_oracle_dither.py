"""The plain form of dithered 8-bit states. No GPU."""
import numpy as np
import pytest

from oracle import step as st


def test_hash_worked():
    # the finaliser's published values, and an element past 2^32
    assert [int(st.mix(np.uint32(h))) for h in (0, 1)] == [0, 0x514E28B7]
    key = st.mix(np.uint32(5) ^ st.mix(np.uint32(0)))
    with np.errstate(over="ignore"):
        want = st.mix(np.uint32(3) ^ st.mix(np.uint32(1) + key))
    assert int(st.dither_bits(np.array([(1 << 32) + 3]), 5)[0]) == int(want)
    assert int(st.dither_bits(np.array([3]), 5)[0]) != int(want)


def test_codes_around_a_value_with_its_mean():
    """N steps of a value between two codes d apart: their mean is off by at most five times
    d / (2 sqrt(N)), the largest deviation of such a mean, and 2^-17 d of the bits' own step."""
    N = 4000
    a = np.concatenate([np.geomspace(1e-4, 447.9, 300), [0.0, 2.0 ** -9, 2.0 ** -6, 2.0 ** -6 * 0.999, 448.0, 448.00006]]).astype(np.float32)
    a[::2] *= -1
    hi = np.searchsorted(st.E4M3, np.minimum(np.abs(a).astype(np.float64), 448.0))
    lo = np.where(st.E4M3[hi] == np.abs(a), hi, np.maximum(hi - 1, 0))
    d = st.E4M3[hi] - st.E4M3[lo]
    for shift in (0, 16):
        total = np.zeros(a.size)
        for t in range(1, N + 1):
            codes = st.to_e4m3_dithered(a, st.dither_bits(np.arange(a.size), t) >> np.uint32(shift) & np.uint32(0xFFFF))
            assert (((codes & 0x7F) == lo) | ((codes & 0x7F) == hi)).all() and ((codes >> 7 == 1) == np.signbit(a)).all()
            total += st.from_e4m3(codes)
        assert (np.abs(total / N - np.clip(a, -448, 448)) <= 5 * d / (2 * np.sqrt(N)) + 2.0 ** -17 * d).all()


def _run(beta2, rounded, steps, fades_at, to, n=128 * 8, beta1=0.9):
    """(held root / true root at the end, exp_avg codes) of the elements that are not their block's largest, whose
    gradients fade to `to` of themselves after fades_at steps; the largest stays."""
    rng, f = np.random.default_rng(1), np.float32
    mc, vc, ms, vs, v = np.zeros(n, np.uint8), np.zeros(n, np.uint8), np.zeros(n // 128, f), np.zeros(n // 128, f), np.zeros(n)
    for t in range(1, steps + 1):
        g = rng.standard_normal(n).astype(f) * f(1e-3 if t <= fades_at else 1e-3 * to)
        g[::128] = f(1e-2)
        m, root = (st.from_e4m3(c).astype(f) * np.repeat(s, 128) for c, s in ((mc, ms), (vc, vs)))
        m, root = st.adamw_states32(g, m, root, (beta1, beta2))
        v = beta2 * v + (1 - beta2) * g.astype(np.float64) ** 2
        bits = st.dither_bits(np.arange(n), t) if rounded == "dither" else None
        mc, ms = st.encode_state(m, False, bits)
        vc, vs = st.encode_state(root, True, bits)
    small = np.arange(n) % 128 != 0
    return (st.decode_state(vc, vs) / np.sqrt(v))[small], mc[small]


@pytest.mark.parametrize("beta2,steps,fades_at", [(0.95, 600, 200), (0.999, 5000, 2000)])
def test_a_dithered_root_follows_its_average(beta2, steps, fades_at):
    """A step moves a root by a share whose mean size is at most (1 - beta2) / 2; codes are at most
    an eighth apart, so that a step adds a relative variance of at most (1 - beta2) / 16. In balance, where
    deviations of v fade by 1 - beta2 a step, that is 1 / 32, and a fall to a tenth, ln 10, adds at most ln 10 / 8 / 2
    more: a logarithm's deviation of 0.42, three of which are a factor of 3.6. The median's
    half variance down and a code's half step: 1.2."""
    ratio, _ = _run(beta2, "dither", steps, fades_at, 0.1)
    assert 1 / 1.2 <= np.median(ratio) <= 1.2
    assert np.percentile(ratio, 1) >= 1 / 3.6 and np.percentile(ratio, 99) <= 3.6


def test_a_root_of_nearest_codes_stays():
    """What the nearest code cannot do, and why it is not the default of a run."""
    ratio, _ = _run(0.95, "nearest", 600, 200, 0.1)
    assert np.median(ratio) > 5


def test_a_first_state_without_gradients_ends():
    """An element without gradients loses its average by 0.9 a step: as nearest codes it stops at four times the
    least one, as dithered ones it is gone after 300 steps (0.9^300 of 2^15 least codes)."""
    _, codes = _run(0.999, "dither", 700, 400, 0.0)
    assert not (codes & 0x7F).any()
    _, codes = _run(0.999, "nearest", 700, 400, 0.0)
    assert (codes & 0x7F).all()
