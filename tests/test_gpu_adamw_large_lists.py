"""The step's other launches: lists of more than 1024 pieces that fit the memory-side cache, and those that do
not, in every type, at odd offsets of flat buffers. The bits are those of the same tensors in short lists, which the
plain form pins."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no GPU", allow_module_level=True)

import token_dispatch_grouped_amd as moe  # noqa: E402

dev = torch.device("cuda:0")
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
# pieces of 4096 elements: more than 1024 of them (cached), and bytes past 256 MB (streamed) in every type and state
SIZES = {"cached": [1 << 20, 3, 2000001, 4097, 1500000, 0, 129, 1777777], "streamed": [14000001, 7, 20000130, 4095, 12000000, 1, 300003]}
KINDS = [("f32", "f32", False), ("f32", "bf16", False), ("bf16", "bf16", True), ("bf16", "f32", True), ("bf16", "bf16", False), ("bf16", "f32", False)]


def _lists(sizes, pt, gt, master, bits, rounding, first):
    """Consecutive views of flat buffers from element `first` on, and the buffers."""
    gen = torch.Generator(device=dev).manual_seed(len(sizes))
    total = sum(sizes) + 16
    r = lambda std: torch.randn(total, generator=gen, device=dev).mul_(std)  # noqa: E731
    w = r(0.02)
    flat = dict(p=w.to(DT[pt]) if master else w.to(DT[pt]).clone(), g=r(1e-3).to(DT[gt]))
    if master:
        flat["w"] = w
    if bits == 32:
        flat["m"], flat["v"] = r(3e-4), r(1e-3).square_()
    else:  # codes of any value: NaN has none
        codes = lambda: torch.randint(0, 255, (total,), generator=gen, device=dev).to(torch.uint8)  # noqa: E731
        m, v = codes(), codes()
        flat["m"], flat["v"] = torch.where(m & 127 == 127, 0, m), torch.where(v & 127 == 127, 0, v) & 127
        blocks = sum(-(-n // 128) for n in sizes)
        flat["ms"], flat["vs"] = (torch.rand(blocks, generator=gen, device=dev) * s for s in (1e-6, 3e-6))
    at = [first]
    block = [0]
    for n in sizes:
        at.append(at[-1] + n)
        block.append(block[-1] + -(-n // 128))
    view = lambda k: [flat[k][a:a + n] for a, n in zip(at, sizes)]  # noqa: E731
    out = dict(p=view("p"), g=view("g"), w=view("w") if master else None, m=view("m"), v=view("v"))
    if bits == 8:
        for k, s in (("m", "ms"), ("v", "vs")):
            out[k] = [moe.Float8State(c.view(torch.float8_e4m3fn), flat[s][b:e], rounding) for c, b, e in zip(out[k], block, block[1:])]
    return out, flat


def _step(ts, lo=0, hi=None, wd=0.1):
    part = lambda v: None if v is None else v[lo:hi]  # noqa: E731
    moe.adamw(part(ts["p"]), part(ts["g"]), part(ts["m"]), part(ts["v"]), 5, 1e-3, (0.9, 0.95), 1e-8, wd, part(ts["w"]))


@pytest.mark.parametrize("bits,rounding", [(32, None), (8, "nearest"), (8, "dither")])
@pytest.mark.parametrize("kind", KINDS, ids=["-".join(map(str, k)) for k in KINDS])
@pytest.mark.parametrize("size", sorted(SIZES))
def test_same_bits_as_short_lists(size, kind, bits, rounding):
    pt, gt, master = kind
    sizes = SIZES[size]
    per = (6 if master else 2 if pt == "bf16" else 4) + (2 if gt == "bf16" else 4) + (2 if bits == 8 else 8)
    bytes_ = sum(sizes) * per
    assert (bytes_ > 1 << 28) == (size == "streamed") and sum(-(-n // 4096) for n in sizes) > 1024
    print(f"case {size} {kind} {bits} {rounding}: {bytes_ >> 20} MB", flush=True)
    first = 3
    ts, flat = _lists(sizes, pt, gt, master, bits, rounding, first)
    ref, ref_flat = _lists(sizes, pt, gt, master, bits, rounding, first)
    _step(ts)
    # the same in lists of at most 2^22 elements of one tensor (cut at whole blocks, and so other pieces): the small
    # pieces' launch. Dithered codes go by the index in the tensor, so those tensors stay whole there
    for i, n in enumerate(sizes):
        cut = 1 << 21
        if n <= cut or rounding == "dither":
            _step(ref, i, i + 1)
            continue
        for a in range(0, n, cut):
            b = min(n, a + cut)
            piece = lambda v: None if v is None else [v[i][a:b]]  # noqa: E731, B023
            if bits == 8:
                states = [[moe.Float8State(s.codes[a:b], s.scale[a // 128:-(-b // 128)], rounding)] for s in (ref["m"][i], ref["v"][i])]
            else:
                states = [piece(ref["m"]), piece(ref["v"])]
            moe.adamw(piece(ref["p"]), piece(ref["g"]), *states, 5, 1e-3, (0.9, 0.95), 1e-8, 0.1, piece(ref["w"]))
    torch.cuda.synchronize()
    for k in flat:
        same = flat[k].view(torch.uint8) if flat[k].dtype != torch.uint8 else flat[k]
        want = ref_flat[k].view(torch.uint8) if ref_flat[k].dtype != torch.uint8 else ref_flat[k]
        assert torch.equal(same, want), k
    start, start_flat = _lists(sizes, pt, gt, master, bits, rounding, first)
    for k in ("p", "g", "m", "v"):  # what lies around the views, and the gradients
        assert torch.equal(flat[k][:first].view(torch.uint8), start_flat[k][:first].view(torch.uint8)), k
        end = first + sum(sizes)
        assert torch.equal(flat[k][end:].view(torch.uint8), start_flat[k][end:].view(torch.uint8)), k
    assert torch.equal(flat["g"].view(torch.uint8), start_flat["g"].view(torch.uint8))
    assert not torch.equal(flat["p"].view(torch.uint8), start_flat["p"].view(torch.uint8))


def test_the_least_code_of_a_root():
    """Roots far below their block's largest (scaled values down to 2^-130) have the least code, not 0."""
    grad = torch.full((256,), 1e-21, device=dev)
    grad[0], grad[128] = 1e18, 1.0
    p = torch.zeros(256, device=dev)
    for rounding in ("nearest", "dither"):
        m, v = moe.adamw_states([p], 8)
        for s in m + v:
            s.rounding = rounding
        moe.adamw([p], [grad], m, v, 1, 1e-3, (0.9, 0.95))
        torch.cuda.synchronize()
        codes = v[0].codes.view(torch.uint8).cpu().numpy()
        want = np.ones(256, dtype=np.uint8)
        want[[0, 128]] = 126
        np.testing.assert_array_equal(codes, want)
