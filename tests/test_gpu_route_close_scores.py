"""Choice values next to the middle between two fp32 numbers.

Pairs of experts: A with a far logit x and a bias that brings s(x) + bias within 4 to 5.5 * 2^-52 s of the
middle between two fp32 numbers f < g, and B, of the lower id, whose value is f itself. If A's rounds up, A
comes first, else B. The score in fp64 is off by at most 3.5 * 2^-52 of itself: its exponential by 0.25 for the
two steps of the argument's reduction (half a unit of a number below 0.35 each), 0.75 for the series' first term left
out, 0.75 for the last steps of its sum, then half for the sum with one, three quarters for the inverse's two
steps, half for the sum with the bias. An argument reduced by ln 2 as one double is off by 8 to 10 more here."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import token_dispatch_grouped_amd as moe  # noqa: E402

dev = torch.device("cuda:0")
L = np.longdouble  # 64 bits of significand


def _pairs(count, seed):
    """(x, bias of A, the value f, whether A's value rounds up) of `count` pairs, as many of either kind."""
    rng = np.random.default_rng(seed)
    out = {True: [], False: []}
    while min(map(len, out.values())) < count // 2:
        x = np.float32(-rng.uniform(55, 66))
        s = 1 / (1 + np.exp(-L(x)))
        f = np.float32(s)
        f = f if L(f) <= s else np.nextafter(f, np.float32(0))
        g = np.nextafter(f, np.float32(1))
        middle = (L(f) + L(g)) / 2
        bias = np.float32(middle - s)
        gap = (s + L(bias) - middle) / s * 2.0 ** 52
        if 4 <= abs(gap) <= 5.5 and len(out[bool(gap > 0)]) < count // 2:
            out[bool(gap > 0)].append((x, bias, f, gap > 0))
    return [p for both in zip(out[True], out[False]) for p in both]


@pytest.mark.skipif(np.finfo(np.longdouble).nmant < 63, reason="needs 64 bits of significand on the host")
@pytest.mark.parametrize("seed", [1, 2, 3])
def test_values_next_to_the_middle(seed):
    n = 32
    pairs = _pairs(n, seed)
    logits = np.full((1, 2 * n), -300.0, dtype=np.float32)  # B's score is below every bias' last bit
    bias = np.zeros(2 * n, dtype=np.float32)
    value = np.zeros(2 * n)
    for i, (x, b, f, up) in enumerate(pairs):
        logits[0, 2 * i + 1], bias[2 * i + 1], bias[2 * i] = x, b, f
        value[2 * i], value[2 * i + 1] = f, np.nextafter(f, np.float32(1)) if up else f
    want = sorted(range(2 * n), key=lambda e: (-value[e], e))
    router = moe.Router("sigmoid", torch.from_numpy(bias).to(dev))
    # all in order by one wave a token; the first sixteen by sorted lists, of few and of many tokens
    for T, k in ((1, 2 * n), (3, 16), (40000, 16)):
        idx, _ = moe.route_experts(torch.from_numpy(logits).to(dev).expand(T, -1).contiguous(), k, router)
        torch.cuda.synchronize()
        got = idx.cpu().numpy()
        np.testing.assert_array_equal(got, np.tile(np.array(want[:k], dtype=np.int32), (T, 1)))
