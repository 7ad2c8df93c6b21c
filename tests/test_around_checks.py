"""Layer norm, the experts in 8-bit integers and the gradient norm refuse wrong
arguments on the host: the C ABI with MOE_EINVAL / MOE_EUNSUPPORTED before
anything is enqueued, the binding with TypeError (dtype) and ValueError (shape)
ahead of the device check. No GPU needed."""
import ctypes
import os

import pytest

import token_dispatch_grouped_amd as moe

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(not os.path.exists(moe.lib_path), reason="libmoe.so not built")

NULL, FAKE, OFF = ctypes.c_void_p(0), ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008)
FAKE2 = ctypes.c_void_p(0x2000)
BF, F = moe.MOE_BF16, moe.MOE_F32
bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
EINVAL, EUNSUP = moe.MOE_EINVAL, moe.MOE_EUNSUPPORTED


def t(shape, dtype):
    return torch.zeros(shape, dtype=dtype)


def _norm(T=16, d=64, dt=BF, wdt=BF, eps=1e-5, **kw):
    a = dict(x=FAKE, r=FAKE, w=FAKE, b=FAKE, y=FAKE, s=FAKE2, mean=FAKE, rstd=FAKE)
    a.update(kw)
    sh = moe.shape(T, d, 8, 1, 1, 0, 1)
    return moe.lib().moe_layer_norm(ctypes.byref(sh), dt, a["x"], a["r"], wdt, a["w"], a["b"], eps, a["y"], a["s"],
                                    a["mean"], a["rstd"], NULL)


def test_layer_norm_refusals():
    for name in ("x", "w", "y", "s", "mean", "rstd"):
        assert _norm(**{name: NULL}) == EINVAL, name
    for name in ("x", "r", "w", "b", "y", "s"):
        assert _norm(**{name: OFF}) == EINVAL, name
    assert _norm(s=FAKE, y=FAKE) == EINVAL  # both outputs in one buffer
    for kw in (dict(T=-1), dict(d=0), dict(d=12), dict(dt=7), dict(wdt=7), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf"))):
        assert _norm(**kw) == EINVAL, kw
    assert _norm(d=32776) == EUNSUP
    assert _norm(dt=F, wdt=BF) == EUNSUP
    assert _norm(T=0, x=NULL, y=NULL, s=NULL, mean=NULL, rstd=NULL) == moe.MOE_OK
    assert moe.lib().moe_layer_norm(None, BF, *[FAKE] * 2, BF, *[FAKE] * 2, 1e-5, *[FAKE] * 4, NULL) == EINVAL


def _norm_bwd(T=16, d=64, dt=BF, wdt=BF, **kw):
    a = dict(dy=FAKE, s=FAKE, w=FAKE, mean=FAKE, rstd=FAKE, ds=FAKE, dx=FAKE, dw=FAKE, db=FAKE2, ws=FAKE)
    a.update(kw)
    sh = moe.shape(T, d, 8, 1, 1, 0, 1)
    return moe.lib().moe_layer_norm_backward(ctypes.byref(sh), dt, a["dy"], a["s"], wdt, a["w"], a["mean"], a["rstd"],
                                             a["ds"], a["dx"], a["dw"], a["db"], a["ws"], NULL)


def test_layer_norm_backward_refusals():
    for name in ("dy", "s", "w", "mean", "rstd", "dx", "dw", "ws"):
        assert _norm_bwd(**{name: NULL}) == EINVAL, name
    for name in ("dy", "s", "w", "ds", "dx", "dw", "db", "ws"):
        assert _norm_bwd(**{name: OFF}) == EINVAL, name
    assert _norm_bwd(dw=FAKE, db=FAKE) == EINVAL
    assert _norm_bwd(d=20) == EINVAL and _norm_bwd(d=32776) == EUNSUP and _norm_bwd(dt=F, wdt=BF) == EUNSUP
    ws = moe.layer_norm_backward_workspace_bytes
    assert ws(0, 64) == 0 and ws(3, 64) == 3 * 2 * 64 * 4 and ws(10 ** 6, 64) == ws(512, 64)


def _int8(dt=BF, **kw):
    a = dict(x=FAKE, perm=FAKE, offsets=FAKE, qg=FAKE, sg=FAKE, qd=FAKE, sd=FAKE, y=FAKE, ws=FAKE)
    sh = dict(T=16, d=64, d_ff=64, E=8, k=2, e_begin=0, e_end=8)
    for k, v in kw.items():
        (sh if k in sh else a)[k] = v
    s = moe.shape(**sh)
    return moe.lib().moe_grouped_gemm_int8(ctypes.byref(s), dt, *a.values(), NULL)


def test_int8_refusals():
    names = ("x", "perm", "offsets", "qg", "sg", "qd", "sd", "y", "ws")
    for name in names:
        assert _int8(**{name: NULL}) == EINVAL, name
    for name in ("x", "qg", "qd", "y", "ws"):
        assert _int8(**{name: OFF}) == EINVAL, name
    for kw in (dict(T=-1), dict(d=12), dict(d_ff=0), dict(k=0), dict(k=9), dict(e_begin=4, e_end=4), dict(e_end=9),
               dict(T=2 ** 30, k=4), dict(dt=7)):
        assert _int8(**kw) == EINVAL, kw
    for kw in (dict(dt=F), dict(d=65544), dict(d_ff=65544), dict(E=1025, e_end=1025)):
        assert _int8(**kw) == EUNSUP, kw
    assert _int8(T=0, **{n: NULL for n in names}) == moe.MOE_OK
    # codes of x, its scales, h, its codes and its scales, each rounded up to 256 bytes, and the list of
    # row tiles: a 256-byte header and 16 bytes a tile
    n = 16 * 2
    assert moe.grouped_gemm_int8_workspace_bytes(16, 72, 136, 8, 2, 0, 8) == \
        n * 128 + 256 + n * 136 * 2 + n * 192 + 256 + 512
    assert moe.grouped_gemm_int8_workspace_bytes(0, 72, 136, 8, 2, 0, 8) == 0


def test_quantize_experts_refusals():
    s = moe.shape(0, 64, 32, 4, 1, 0, 4)
    fn = moe.lib().moe_quantize_experts
    for i in range(6):
        p = [FAKE] * 6
        p[i] = NULL
        assert fn(ctypes.byref(s), BF, *p, NULL) == EINVAL, i
    for i in (0, 1, 2, 4):
        p = [FAKE] * 6
        p[i] = OFF
        assert fn(ctypes.byref(s), BF, *p, NULL) == EINVAL, i
    assert fn(ctypes.byref(s), 7, *[FAKE] * 6, NULL) == EINVAL
    big = moe.shape(0, 65544, 32, 4, 1, 0, 4)
    assert fn(ctypes.byref(big), BF, *[FAKE] * 6, NULL) == EUNSUP


def _list(*entries):
    arr = (moe.moe_tensor * len(entries))()
    for i, e in enumerate(entries):
        arr[i] = moe.moe_tensor(*e)
    return arr


def test_gradient_list_refusals():
    lib = moe.lib()
    good = _list((0x1000, 8, F), (0x2002, 9, BF))
    for bad in (_list((0, 8, F)), _list((0x1002, 8, F)), _list((0x1001, 8, BF)), _list((0x1000, -1, F)),
                _list((0x1000, 8, 7))):
        assert lib.moe_grad_norm(bad, 1, FAKE, FAKE, NULL) == EINVAL
        assert lib.moe_clip_grads(bad, None, 1, FAKE, 1.0, NULL) == EINVAL
        assert lib.moe_clip_grad_norm(bad, None, 1, 1.0, FAKE, FAKE, NULL) == EINVAL
        assert lib.moe_clip_grads(good, bad, 1, FAKE, 1.0, NULL) == EINVAL
    assert lib.moe_grad_norm(good, -1, FAKE, FAKE, NULL) == EINVAL
    assert lib.moe_grad_norm(None, 1, FAKE, FAKE, NULL) == EINVAL
    assert lib.moe_grad_norm(good, 2, NULL, FAKE, NULL) == EINVAL
    assert lib.moe_grad_norm(good, 2, FAKE, NULL, NULL) == EINVAL
    assert lib.moe_grad_norm(good, 2, FAKE, ctypes.c_void_p(0x1004), NULL) == EINVAL
    assert lib.moe_clip_grads(good, None, 2, NULL, 1.0, NULL) == EINVAL
    for m in (-1.0, float("nan"), float("inf")):
        assert lib.moe_clip_grads(good, None, 2, FAKE, m, NULL) == EINVAL
        assert lib.moe_clip_grad_norm(good, None, 2, m, FAKE, FAKE, NULL) == EINVAL
    assert lib.moe_clip_grads(None, None, 0, FAKE, 1.0, NULL) == moe.MOE_OK
    # the sizes of a pair have to agree
    assert lib.moe_clip_grads(good, _list((0x3000, 7, F), (0x4000, 9, BF)), 2, FAKE, 1.0, NULL) == EINVAL
    assert lib.moe_clip_grads(good, _list((0x3000, 8, F), (0x4000, 9, F)), 2, FAKE, 1.0, NULL) == EINVAL
    assert moe.grad_norm_workspace_bytes(-1) == 0 and moe.grad_norm_workspace_bytes(1) > 0
    assert moe.grad_norm_workspace_bytes(65) == 2 * moe.grad_norm_workspace_bytes(64)


def test_clip_refuses_overlaps():
    lib = moe.lib()

    def clip(g, o=None):
        return lib.moe_clip_grads(_list(*g), None if o is None else _list(*o), len(g), FAKE, 1.0, NULL)

    a, b = (0x1000, 16, F), (0x1020, 4, F)  # b lies inside a's 64 bytes
    assert clip([a, b]) == EINVAL
    assert clip([b, a]) == EINVAL
    assert clip([a, a]) == EINVAL  # the same tensor twice would be scaled twice
    c = (0x2000, 16, F)
    assert clip([a, c], [(0x3000, 16, F), (0x3000, 16, F)]) == EINVAL  # two results in one place
    assert clip([a, c], [c, a]) == EINVAL  # a result over another gradient
    assert clip([a], [(0x1004, 16, F)]) == EINVAL  # a result over its own gradient, shifted


def test_clip_refuses_a_norm_or_workspace_among_the_tensors():
    lib = moe.lib()
    g, o = _list((0x1000, 16, F)), _list((0x8000, 16, F))
    far, ws = ctypes.c_void_p(0x100000), ctypes.c_void_p(0x200000)
    for at in (0x1000, 0x103C):
        inside = ctypes.c_void_p(at)
        assert lib.moe_clip_grads(g, None, 1, inside, 1.0, NULL) == EINVAL  # scaled while others read it
        assert lib.moe_clip_grad_norm(g, o, 1, 1.0, inside, ws, NULL) == EINVAL  # written while others read the gradient
    assert lib.moe_clip_grads(g, o, 1, ctypes.c_void_p(0x8004), 1.0, NULL) == EINVAL
    assert lib.moe_clip_grad_norm(g, o, 1, 1.0, ctypes.c_void_p(0x8004), ws, NULL) == EINVAL
    for at in (0x1000, 0x8000, 0x1000 - 8):
        assert lib.moe_clip_grad_norm(g, o, 1, 1.0, far, ctypes.c_void_p(at), NULL) == EINVAL
    assert lib.moe_clip_grad_norm(g, o, 1, 1.0, ws, ws, NULL) == EINVAL


def test_layer_norm_binding_checks():
    x, w = t((4, 64), bf16), t((64,), bf16)
    with pytest.raises(TypeError):
        moe.layer_norm(t((4, 64), torch.float16), w)
    with pytest.raises(ValueError):
        moe.layer_norm(t((64,), bf16), w)
    with pytest.raises(TypeError):
        moe.layer_norm(t((4, 64), f32), w)  # bf16 weights with fp32 rows
    with pytest.raises(ValueError):
        moe.layer_norm(x, t((63,), bf16))
    with pytest.raises(TypeError):
        moe.layer_norm(x, w, t((64,), f32))  # weight and bias differ
    with pytest.raises(ValueError):
        moe.layer_norm(x, w, residual=t((3, 64), bf16))
    with pytest.raises(ValueError):
        moe.layer_norm(x, w, s=t((4, 64), bf16))
    with pytest.raises(TypeError):
        moe.layer_norm(x, w, mean=t((4,), bf16))
    with pytest.raises(ValueError):
        moe.layer_norm(x, w)  # not on a GPU
    m = t((4,), f32)
    with pytest.raises(TypeError):
        moe.layer_norm_backward(x, t((4, 64), f32), w, m, m)
    with pytest.raises(ValueError):
        moe.layer_norm_backward(x, x, w, t((5,), f32), m)
    with pytest.raises(ValueError):
        moe.layer_norm_backward(x, x, w, m, m, workspace=t((1,), torch.uint8))
    with pytest.raises(ValueError):
        moe.layer_norm_backward(x, x, w, m, m, bias=False, d_bias=w)


def _experts(e=8, d=64, f=32, **kw):
    kb = lambda v: (v + 63) // 64  # noqa: E731
    a = dict(w_gate_up=t((e, kb(d), 2 * f, 64), torch.int8), gate_up_scale=t((e, 2 * f), f32),
             w_down=t((e, kb(f), d, 64), torch.int8), down_scale=t((e, d), f32))
    a.update(kw)
    return moe.Int8Experts(**a)


def test_int8_binding_checks():
    x, perm, offs = t((16, 64), bf16), t((32,), i32), t((9,), i32)
    with pytest.raises(TypeError):
        moe.grouped_gemm_int8(t((16, 64), f32), perm, offs, _experts(), 2, 8, 0, 8)
    for kw, exc in ((dict(w_gate_up=t((8, 1, 64, 64), torch.uint8)), TypeError),
                    (dict(w_gate_up=t((8, 64, 64), torch.int8)), ValueError),
                    (dict(gate_up_scale=t((8, 63), f32)), ValueError),
                    (dict(gate_up_scale=t((8, 64), bf16)), TypeError),
                    (dict(w_down=t((8, 1, 72, 64), torch.int8)), ValueError),
                    (dict(down_scale=t((7, 64), f32)), ValueError)):
        with pytest.raises(exc):
            moe.grouped_gemm_int8(x, perm, offs, _experts(**kw), 2, 8, 0, 8)
    with pytest.raises(ValueError):
        moe.grouped_gemm_int8(x, perm, offs, _experts(e=7), 2, 8, 0, 8)
    with pytest.raises(ValueError):
        moe.grouped_gemm_int8(x, perm, offs, _experts(), 2, 8, 0, 8, y=t((31, 64), bf16))
    with pytest.raises(ValueError):
        moe.grouped_gemm_int8(x, perm, offs, _experts(), 2, 8, 0, 8, workspace=t((1,), torch.uint8))
    with pytest.raises(TypeError):
        moe.quantize_experts(t((2, 64, 64), f32), t((2, 32, 64), bf16))
    with pytest.raises(ValueError):
        moe.quantize_experts(t((2, 64, 63), bf16), t((2, 32, 64), bf16))


def test_gradient_binding_checks():
    g = t((5,), f32)
    with pytest.raises(TypeError):
        moe.grad_norm(g)  # a tensor, not a list
    with pytest.raises(ValueError):
        moe.grad_norm([])
    with pytest.raises(TypeError):
        moe.grad_norm([t((5,), torch.float16)])
    with pytest.raises(TypeError):
        moe.clip_grads([g], t((1,), torch.float64), 1.0)
    with pytest.raises(ValueError):
        moe.clip_grad_norm([g], 1.0, out=[g, g])
    with pytest.raises(TypeError):
        moe.clip_grad_norm([g], 1.0, out=[t((5,), bf16)])
    with pytest.raises(ValueError):
        moe.clip_grad_norm([g], 1.0, workspace=t((8,), torch.uint8))


def test_layer_norm_of_a_partial_output_is_refused():
    x, lg = t((4, 64), bf16), t((4, 8), f32)
    with pytest.raises(ValueError):
        moe.layer(x, lg, t((4, 64, 64), bf16), t((4, 32, 64), bf16), 2, 0, 4, norm=(t((64,), bf16), None, 1e-5))
    with pytest.raises(ValueError):
        moe.layer_int8(x, lg, _experts(e=4), 2, 0, 4, norm=(t((64,), bf16), None, 1e-5))
