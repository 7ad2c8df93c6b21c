"""Calls whose offsets pass 32 bits: buffers of more than 2^31 elements or bytes. Only rows
near both ends and around the 2^31 marks are compared, each with a small call on the
same row (bit for bit) or with a closed form."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import token_dispatch_grouped_amd as moe  # noqa: E402

EPS = 1e-5
BF = torch.bfloat16


def _normal(shape, seed, dtype=BF):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    out = torch.empty(shape, dtype=dtype, device="cuda")
    rows = max(1, (1 << 27) // shape[1])
    for at in range(0, shape[0], rows):
        out[at:at + rows] = torch.randn((min(rows, shape[0] - at), shape[1]), generator=gen, device="cuda").to(dtype)
    return out


def test_layer_norm_and_its_gradient():
    d = 8192
    T = (1 << 31) // d + 37  # more than 2^31 elements
    x, dy = _normal((T, d), 1), _normal((T, d), 2)
    w = _normal((1, d), 3)[0]
    y, s, mean, rstd = moe.layer_norm(x, w, w, EPS)
    dx, dw, db = moe.layer_norm_backward(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    for r in (0, 1, T // 2, (1 << 31) // d - 1, (1 << 31) // d, T - 1):
        yr, _, mr, sr = moe.layer_norm(x[r:r + 1], w, w, EPS)
        dr, _, _ = moe.layer_norm_backward(dy[r:r + 1], x[r:r + 1], w, mr, sr)
        assert torch.equal(y[r:r + 1], yr) and torch.equal(mean[r:r + 1], mr) and torch.equal(rstd[r:r + 1], sr), r
        assert torch.equal(dx[r:r + 1], dr), r
    # db: T values near N(0, 1) are summed; (T / 512 + 60 + 4) 2^-24 of the sum of their sizes, half a step of bf16
    want = torch.zeros(d, dtype=torch.float64, device="cuda")
    size = torch.zeros(d, dtype=torch.float64, device="cuda")
    for at in range(0, T, 16384):
        part = dy[at:at + 16384].double()
        want += part.sum(dim=0)
        size += part.abs().sum(dim=0)
    bound = (T / 512 + 64) * 2.0 ** -24 * size + 2.0 ** -8 * 1.001 * want.abs()
    assert bool(((db.double() - want).abs() <= bound).all())


def test_layer_norm_of_more_rows_than_a_launch_has_threads_for():
    d, T = 8, (1 << 28) + 21  # 16 threads a row: 2^32 and more
    x = _normal((1 << 20, d), 6).repeat(T // (1 << 20) + 1, 1)[:T]
    w = _normal((1, d), 7)[0]
    y, _, mean, rstd = moe.layer_norm(x, w, None, EPS)
    torch.cuda.synchronize()
    part = T % (1 << 20)
    yr, _, mr, sr = moe.layer_norm(x[:1 << 20], w, None, EPS)
    torch.cuda.synchronize()
    for at in (0, T // (1 << 21) << 20, T - part):
        n = min(1 << 20, T - at)
        assert torch.equal(y[at:at + n], yr[:n]) and torch.equal(mean[at:at + n], mr[:n]), at
        assert torch.equal(rstd[at:at + n], sr[:n]), at


def test_gradient_norm_and_clip():
    n = (1 << 32) + 5  # elements, past 32 bits
    g = torch.full((n,), 0.5, dtype=BF, device="cuda")
    g[0], g[1 << 31], g[-1] = 3.0, 2.0, 1.0
    small = torch.ones(7, device="cuda")
    want = (0.25 * (n - 3) + 9 + 4 + 1 + 7) ** 0.5
    norm = moe.clip_grad_norm([small, g], want / 2)
    torch.cuda.synchronize()
    assert abs(float(norm[0]) - want) <= want * 2.0 ** -23
    # the factor is 0.5 to within 4 roundings of fp32, far less than half a step of bf16: exact halves
    assert [float(g[i]) for i in (0, 1, (1 << 31) - 1, 1 << 31, (1 << 31) + 1, n - 2, n - 1)] == \
        [1.5, 0.25, 0.25, 1.0, 0.25, 0.25, 0.5]
    assert bool((g[1:1 << 20] == 0.25).all()) and bool((g[-(1 << 20):-1] == 0.25).all())


@pytest.mark.parametrize("T,d,f,E", [(1 << 20, 64, 2056, 4), (40, 64, 32768, 600), (1 << 19, 2056, 64, 2)])
def test_int8_experts(T, d, f, E):
    """Codes, h and weights of more than 2^31 bytes, in turn."""
    x = _normal((T, d), 4)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(5)

    def weight(K, N):
        kb = (K + 63) // 64
        q = torch.randint(-127, 128, (E, kb, N, 64), generator=gen, device="cuda", dtype=torch.int8)
        return q, torch.rand((E, N), generator=gen, device="cuda") * (2.0 / (127 * K ** 0.5))

    experts = moe.Int8Experts(*weight(d, 2 * f), *weight(f, d))
    owner = torch.arange(T, device="cuda") * E // T  # token t goes to expert t E / T: rows in token order
    perm = torch.arange(T, device="cuda", dtype=torch.int32)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = torch.cumsum(torch.bincount(owner, minlength=E), 0).to(torch.int32)
    y = moe.grouped_gemm_int8(x, perm, offsets, experts, 1, E, 0, E)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(y.view(-1)[::4099].float()).all())
    for t in (0, 1, T // 3, T // 2, T - 2, T - 1):
        e = int(owner[t])
        one = moe.Int8Experts(*(v[e:e + 1].contiguous() for v in (experts.w_gate_up, experts.gate_up_scale,
                                                                  experts.w_down, experts.down_scale)))
        want = moe.grouped_gemm_int8(x[t:t + 1], perm[:1], torch.tensor([0, 1], dtype=torch.int32, device="cuda"), one,
                                     1, 1, 0, 1)
        torch.cuda.synchronize()
        assert torch.equal(y[t:t + 1], want), t
