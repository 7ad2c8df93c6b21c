"""Routing by scores, RMS norm, the experts on 8-bit rows and AdamW refuse wrong
arguments on the host: the C ABI with MOE_EINVAL / MOE_EUNSUPPORTED before anything is
enqueued, the binding with TypeError (dtype) and ValueError (shape) ahead of the device
check. No GPU needed."""
import ctypes
import os

import pytest

import token_dispatch_grouped_amd as moe

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(not os.path.exists(moe.lib_path), reason="libmoe.so not built")

NULL, FAKE, OFF, ODD = ctypes.c_void_p(0), ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008), ctypes.c_void_p(0x1002)
FAKE2 = ctypes.c_void_p(0x2000)
BF, F = moe.MOE_BF16, moe.MOE_F32
bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
EINVAL, EUNSUP = moe.MOE_EINVAL, moe.MOE_EUNSUPPORTED


def t(shape, dtype):
    return torch.zeros(shape, dtype=dtype)


def _shape(**kw):
    base = dict(T=16, d=64, d_ff=64, E=8, k=2, e_begin=0, e_end=8)
    base.update(kw)
    return moe.shape(**base)


# ------------------------------------------------------------------------ routing

def _route(shape=None, ptrs=None, **kw):
    r = dict(score=0, groups=2, top_groups=1, group_top=2, renormalize=1, scale=1.0, bias=0x1000)
    r.update(kw)
    p = dict(logits=FAKE, idx=FAKE2, w=FAKE)
    p.update(ptrs or {})
    s = _shape(**(shape or {}))
    return moe.lib().moe_route_experts(ctypes.byref(s), ctypes.byref(moe.moe_router(**r)), *p.values(), NULL)


def test_route_refusals():
    for name in ("logits", "idx", "w"):
        assert _route(ptrs={name: NULL}) == EINVAL, name
        assert _route(ptrs={name: ODD}) == EINVAL, name
    for kw in (dict(score=2), dict(score=-1), dict(groups=0), dict(groups=3), dict(groups=16), dict(top_groups=0),
               dict(top_groups=3), dict(group_top=0), dict(group_top=3), dict(renormalize=2), dict(bias=0x1002),
               dict(scale=float("nan")), dict(scale=float("inf"))):
        assert _route(**kw) == EINVAL, kw
    for sh in (dict(T=-1), dict(k=0), dict(k=9), dict(k=5), dict(T=2 ** 31), dict(T=2 ** 30, k=4)):
        assert _route(shape=sh) == EINVAL, sh  # 5 of the 4 experts of a group
    assert _route(shape=dict(E=1026)) == EUNSUP
    assert _route(shape=dict(T=0), ptrs=dict(logits=NULL, idx=NULL, w=NULL)) == moe.MOE_OK
    s = _shape()
    assert moe.lib().moe_route_experts(ctypes.byref(s), None, FAKE, FAKE, FAKE, NULL) == EINVAL
    assert moe.lib().moe_route_experts(None, ctypes.byref(moe.moe_router()), FAKE, FAKE, FAKE, NULL) == EINVAL


def test_route_backward_refusals():
    def call(shape=None, ptrs=None, **kw):
        # the choice's fields are not looked at
        r = dict(score=1, groups=0, top_groups=-1, group_top=9, renormalize=0, scale=1.0, bias=0x1001)
        r.update(kw)
        p = dict(logits=FAKE, idx=FAKE, dw=FAKE, dl=FAKE2)
        p.update(ptrs or {})
        s = _shape(**(shape or {}))
        return moe.lib().moe_route_experts_backward(ctypes.byref(s), ctypes.byref(moe.moe_router(**r)), *p.values(), NULL)

    for name in ("logits", "idx", "dw", "dl"):
        assert call(ptrs={name: NULL}) == EINVAL and call(ptrs={name: ODD}) == EINVAL, name
    for kw in (dict(score=7), dict(renormalize=-1), dict(scale=float("inf"))):
        assert call(**kw) == EINVAL, kw
    assert call(shape=dict(k=9)) == EINVAL and call(shape=dict(E=1025)) == EUNSUP
    assert call(shape=dict(T=0)) == moe.MOE_OK


def test_binding_route():
    x = t((4, 8), f32)
    R = moe.Router
    for router in (R(groups=3), R(groups=0), R(groups=2, top_groups=3), R(groups=2, top_groups=0), R(score="tanh"),
                   R(group_score="top3"), R(scale=float("nan")), R(bias=t((7,), f32))):
        with pytest.raises(ValueError):
            moe.route_experts(x, 2, router)
    with pytest.raises(ValueError):
        moe.route_experts(x, 5, R(groups=2, top_groups=1))
    with pytest.raises(TypeError):
        moe.route_experts(x.double(), 2, R())
    with pytest.raises(TypeError):
        moe.route_experts(x, 2, R(bias=t((8,), bf16)))
    with pytest.raises(TypeError):
        moe.route_experts(x, 2, R(), topk_idx=t((4, 2), torch.int64))
    with pytest.raises(ValueError):
        moe.route_experts(x, 2, R(), topk_w=t((4, 3), f32))
    with pytest.raises(ValueError, match="GPU"):
        moe.route_experts(x, 2, R())
    with pytest.raises(ValueError):
        moe.route_experts_backward(x, t((3, 2), i32), t((3, 2), f32), R())
    with pytest.raises(ValueError):
        moe.route_experts_backward(x, t((4, 9), i32), t((4, 9), f32), R())
    with pytest.raises(TypeError):
        moe.route_experts_backward(x, t((4, 2), i32), t((4, 2), bf16), R())
    with pytest.raises(ValueError, match="GPU"):
        moe.route_experts_backward(x, t((4, 2), i32), t((4, 2), f32), R())


# ----------------------------------------------------------------------- RMS norm

def _rms(T=16, d=64, dt=BF, wdt=BF, eps=1e-6, **kw):
    a = dict(x=FAKE, r=FAKE, w=FAKE, y=FAKE, s=FAKE2, rstd=FAKE, q=FAKE, qs=FAKE)
    a.update(kw)
    sh = moe.shape(T, d, 8, 1, 1, 0, 1)
    return moe.lib().moe_rms_norm(ctypes.byref(sh), dt, a["x"], a["r"], wdt, a["w"], eps, a["y"], a["s"], a["rstd"],
                                  a["q"], a["qs"], NULL)


def test_rms_norm_refusals():
    for name in ("x", "w", "s", "rstd", "q", "qs"):
        assert _rms(**{name: NULL}) == EINVAL, name
    for name in ("x", "r", "w", "y", "s", "q"):
        assert _rms(**{name: OFF}) == EINVAL, name
    for name in ("rstd", "qs"):
        assert _rms(**{name: ODD}) == EINVAL, name
    assert _rms(s=FAKE, y=FAKE) == EINVAL
    assert _rms(y=NULL, q=NULL, qs=NULL) == EINVAL  # nothing to write
    for kw in (dict(T=-1), dict(d=0), dict(d=12), dict(dt=7), dict(wdt=7), dict(eps=-1.0), dict(eps=float("nan")),
               dict(eps=float("inf"))):
        assert _rms(**kw) == EINVAL, kw
    assert _rms(d=32776) == EUNSUP and _rms(dt=F, wdt=BF) == EUNSUP
    assert _rms(dt=F, wdt=F) == EUNSUP  # 8-bit rows of fp32 rows
    assert _rms(T=0, x=NULL, y=NULL, s=NULL, rstd=NULL, q=NULL, qs=NULL) == moe.MOE_OK


def test_rms_norm_backward_refusals():
    def call(T=16, d=64, dt=BF, wdt=BF, **kw):
        a = dict(dy=FAKE, s=FAKE, w=FAKE, rstd=FAKE, ds=FAKE, dx=FAKE, dw=FAKE, ws=FAKE)
        a.update(kw)
        sh = moe.shape(T, d, 8, 1, 1, 0, 1)
        return moe.lib().moe_rms_norm_backward(ctypes.byref(sh), dt, a["dy"], a["s"], wdt, a["w"], a["rstd"], a["ds"],
                                               a["dx"], a["dw"], a["ws"], NULL)

    for name in ("dy", "s", "w", "rstd", "dx", "dw", "ws"):
        assert call(**{name: NULL}) == EINVAL, name
    for name in ("dy", "s", "w", "ds", "dx", "dw", "ws"):
        assert call(**{name: OFF}) == EINVAL, name
    assert call(rstd=ODD) == EINVAL and call(d=20) == EINVAL and call(d=32776) == EUNSUP
    assert call(dt=F, wdt=BF) == EUNSUP
    ws = moe.rms_norm_backward_workspace_bytes
    assert ws(0, 64) == 0 and ws(3, 64) == 3 * 64 * 4 and ws(10 ** 6, 64) == ws(10 ** 7, 64)


def test_binding_rms_norm():
    x, w = t((4, 64), bf16), t((64,), bf16)
    with pytest.raises(ValueError):
        moe.rms_norm(x, t((72,), bf16))
    with pytest.raises(TypeError):
        moe.rms_norm(x, t((64,), torch.float16))
    with pytest.raises(TypeError):
        moe.rms_norm(t((4, 64), f32), w)
    with pytest.raises(ValueError):
        moe.rms_norm(x, w, s=t((4, 64), bf16))  # without a residual
    with pytest.raises(ValueError):
        moe.rms_norm(x, w, residual=t((4, 72), bf16))
    with pytest.raises(TypeError):
        moe.rms_norm(x, w, rstd=t((4,), bf16))
    with pytest.raises(ValueError, match="GPU"):
        moe.rms_norm(x, w)
    with pytest.raises(TypeError):
        moe.rms_norm_int8(t((4, 64), f32), t((64,), f32))
    with pytest.raises(ValueError):
        moe.rms_norm_int8(x, w, rows=moe.Int8Rows(t((1, 5, 64), torch.int8), t((4,), f32)))
    with pytest.raises(TypeError):
        moe.rms_norm_int8(x, w, rows=moe.Int8Rows(t((1, 4, 64), torch.uint8), t((4,), f32)))
    with pytest.raises(ValueError):
        moe.rms_norm_int8(x, w, rows=moe.Int8Rows(None, t((4,), f32)))
    with pytest.raises(ValueError):
        moe.rms_norm_int8(x, w, y=t((4, 64), bf16), keep_y=False)
    with pytest.raises(ValueError):
        moe.rms_norm_backward(x, None, w, t((4,), f32))
    with pytest.raises(ValueError):
        moe.rms_norm_backward(x, x, w, t((5,), f32))
    with pytest.raises(ValueError):
        moe.rms_norm_backward(x, x, w, t((4,), f32), workspace=t((10,), torch.uint8))


# ------------------------------------------------------------------- 8-bit rows

def test_int8_rows_refusals():
    def call(**kw):
        a = dict(x=FAKE, sx=FAKE, perm=FAKE, offsets=FAKE, qg=FAKE, sg=FAKE, qd=FAKE, sd=FAKE, y=FAKE, ws=FAKE)
        sh = dict(T=16, d=64, d_ff=64, E=8, k=2, e_begin=0, e_end=8)
        for key, v in kw.items():
            (sh if key in sh else a)[key] = v
        s = moe.shape(**sh)
        return moe.lib().moe_grouped_gemm_int8_rows(ctypes.byref(s), *a.values(), NULL)

    for name in ("x", "sx", "perm", "offsets", "qg", "sg", "qd", "sd", "y", "ws"):
        assert call(**{name: NULL}) == EINVAL, name
    for name in ("x", "qg", "qd", "y", "ws"):
        assert call(**{name: OFF}) == EINVAL, name
    assert call(sx=ODD) == EINVAL and call(d=20) == EINVAL and call(k=9) == EINVAL and call(E=2000, e_end=2000) == EUNSUP
    assert call(T=0, x=NULL, sx=NULL, y=NULL, ws=NULL) == moe.MOE_OK


def test_binding_int8_rows():
    experts = moe.Int8Experts(t((2, 2, 16, 64), torch.int8), t((2, 16), f32), t((2, 1, 72, 64), torch.int8), t((2, 72), f32))
    perm, offsets = t((8,), i32), t((3,), i32)
    with pytest.raises(ValueError):  # codes of 64 columns, experts of 72
        moe.grouped_gemm_int8(moe.Int8Rows(t((1, 4, 64), torch.int8), t((4,), f32)), perm, offsets, experts, 2, 2, 0, 2)
    with pytest.raises(TypeError):
        moe.grouped_gemm_int8(moe.Int8Rows(t((2, 4, 64), torch.uint8), t((4,), f32)), perm, offsets, experts, 2, 2, 0, 2)
    rows = moe.Int8Rows(t((2, 4, 64), torch.int8), t((4,), f32))
    with pytest.raises(ValueError, match="GPU"):
        moe.grouped_gemm_int8(rows, perm, offsets, experts, 2, 2, 0, 2)
    with pytest.raises(ValueError, match="residual"):
        moe.layer_int8(rows, t((4, 2), f32), experts, 2, 0, 2, norm=moe.RmsNorm(t((72,), bf16)))
    with pytest.raises(ValueError, match="norm"):
        moe.layer_int8(rows, t((4, 2), f32), experts, 2, 0, 2, residual=t((4, 72), bf16))
    with pytest.raises(ValueError):
        moe.layer_int8(rows, t((5, 2), f32), experts, 2, 0, 2)


# -------------------------------------------------------------------------- AdamW

def _adamw(n=1, tensors=None, entry=None, **kw):
    e = dict(param=0x10000, grad=0x20000, master=0, exp_avg=0x30000, exp_avg_sq=0x40000, exp_avg_scale=0x50000,
             exp_avg_sq_scale=0x60000, numel=100, param_dt=F, grad_dt=BF)
    e.update(entry or {})
    a = dict(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1, step=1, state=moe.MOE_STATE_F32)
    a.update(kw)
    host = (moe.moe_adamw_tensor * 2)(*[moe.moe_adamw_tensor(**x) for x in (tensors or [e, e])])
    return moe.lib().moe_adamw(host, n, ctypes.byref(moe.moe_adamw_args(**a)), NULL)


def test_adamw_refusals():
    for name in ("param", "grad", "exp_avg", "exp_avg_sq"):
        assert _adamw(entry={name: 0}) == EINVAL, name
        assert _adamw(entry={name: 0x90001}) == EINVAL, name
    for name in ("exp_avg_scale", "exp_avg_sq_scale"):
        assert _adamw(entry={name: 0}, state=1) == EINVAL and _adamw(entry={name: 0x90002}, state=1) == EINVAL, name
    nan, inf = float("nan"), float("inf")
    for kw in (dict(lr=nan), dict(lr=inf), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=nan),
               dict(eps=0.0), dict(eps=-1e-8), dict(eps=nan), dict(eps=inf), dict(eps=1e-40), dict(eps=1e39),
               dict(weight_decay=nan), dict(step=0), dict(step=-3), dict(state=2), dict(norm=0x70002),
               dict(norm=0x70000, max_norm=-1.0), dict(norm=0x70000, max_norm=inf), dict(norm=0x70000, max_norm=nan),
               dict(d_lr=0x70001), dict(d_step=0x70004)):
        assert _adamw(**kw) == EINVAL, kw
    decays = (ctypes.c_double * 2)(0.1, nan)
    host = dict(weight_decays=ctypes.cast(decays, ctypes.c_void_p).value)
    far = dict(param=0x110000, grad=0x120000, exp_avg=0x130000, exp_avg_sq=0x140000, numel=7, param_dt=F, grad_dt=F)
    near = dict(far, param=0x210000, grad=0x220000, exp_avg=0x230000, exp_avg_sq=0x240000)
    assert _adamw(2, [far, near], **host) == EINVAL
    assert _adamw(entry=dict(numel=-1)) == EINVAL and _adamw(entry=dict(numel=2 ** 41)) == EUNSUP
    assert _adamw(entry=dict(param_dt=5)) == EINVAL and _adamw(entry=dict(grad_dt=5)) == EINVAL
    assert _adamw(entry=dict(master=0x80000)) == EINVAL  # of an fp32 param
    assert _adamw(-1) == EINVAL
    assert moe.lib().moe_adamw(None, 1, ctypes.byref(moe.moe_adamw_args()), NULL) == EINVAL
    assert moe.lib().moe_adamw(None, 0, None, NULL) == EINVAL
    assert _adamw(0) == moe.MOE_OK
    assert _adamw(entry=dict(numel=0, param=0, grad=0, exp_avg=0, exp_avg_sq=0)) == moe.MOE_OK


def test_adamw_overlaps_are_refused():
    base = dict(param=0x10000, grad=0x20000, exp_avg=0x30000, exp_avg_sq=0x40000, numel=1024, param_dt=F, grad_dt=F)
    for name, at in (("grad", 0x10FFC), ("exp_avg", 0x10004), ("exp_avg_sq", 0x2FFFC), ("param", 0x1F004),
                     ("exp_avg", 0x20000)):
        assert _adamw(entry=dict(base, **{name: at})) == EINVAL, (name, hex(at))
    other = dict(base, param=0x110000, grad=0x120000, exp_avg=0x130000, exp_avg_sq=0x140000)
    assert _adamw(2, [base, dict(other, param=0x10000)]) == EINVAL  # the same parameter twice
    assert _adamw(2, [base, dict(other, exp_avg_sq=0x2F010)]) == EINVAL
    for name in ("norm", "d_lr", "d_step"):  # among the written tensors
        assert _adamw(entry=base, **{name: 0x40008}) == EINVAL, name
    e8 = dict(base, exp_avg_scale=0x50000, exp_avg_sq_scale=0x5001C)  # eight blocks of 32 bytes
    assert _adamw(entry=e8, state=1) == EINVAL


def test_binding_adamw():
    p, g, m = [t((4, 8), f32)], [t((4, 8), f32)], [t((4, 8), f32)]
    f8 = lambda n=1, dt=f32: moe.Float8State(t((4, 8), torch.float8_e4m3fn), t((n,), dt))  # noqa: E731
    call = lambda p=p, g=g, m=m, v=m, step=1, lr=1e-3, **kw: moe.adamw(p, g, m, v, step, lr, **kw)  # noqa: E731
    for kw in (dict(p=[]), dict(g=[]), dict(g=[t((4, 9), f32)]), dict(m=[t((32,), f32)]), dict(v=[]), dict(step=0),
               dict(m=[f8(2)], v=[f8()]), dict(masters=[t((4, 8), f32)]), dict(masters=[]), dict(max_norm=1.0),
               dict(weight_decay=[0.1, 0.2]), dict(norm=t((2,), f32))):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(p=p[0]), dict(p=[t((4, 8), torch.float16)]), dict(g=[t((4, 8), torch.float16)]), dict(m=[t((4, 8), bf16)]),
               dict(m=[f8()]), dict(m=[f8(), m[0]], p=p * 2, g=g * 2, v=m * 2), dict(m=[f8(dt=bf16)], v=[f8()]),
               dict(step=t((1,), i32)), dict(lr=t((1,), torch.float64)), dict(norm=t((1,), torch.float64)),
               dict(p=[t((4, 8), bf16)], masters=[t((4, 8), bf16)])):
        with pytest.raises(TypeError):
            call(**kw)
    with pytest.raises(ValueError, match="GPU"):
        call()
    with pytest.raises(ValueError):
        moe.adamw_states(p, bits=16)
    with pytest.raises((TypeError, ValueError)):
        call(weight_decay=["much"])
    first, second = moe.adamw_states([t((3, 50), bf16), t((0,), f32)], bits=8)
    assert first[0].codes.dtype is torch.float8_e4m3fn and first[0].codes.shape == (3, 50) and second[0].scale.shape == (2,)
    assert first[1].scale.shape == (0,) and not second[0].scale.any()
    first, _ = moe.adamw_states(p)
    assert first[0].dtype is f32 and not first[0].any()


def test_layer_refuses_what_does_not_go_together():
    x, logits = t((4, 64), bf16), t((4, 8), f32)
    w = (t((8, 64, 32), bf16), t((8, 16, 64), bf16))
    with pytest.raises(ValueError, match="residual"):
        moe.layer(x, logits, *w, 2, 0, 8, residual=x)
    with pytest.raises(ValueError, match="partial"):
        moe.layer(x, logits, t((4, 64, 32), bf16), t((4, 16, 64), bf16), 2, 0, 4, norm=moe.RmsNorm(t((64,), bf16)))
    fwd = dict(counts=t((8,), i32), sum=x, rstd=t((4,), f32), mean=t((4,), f32))
    with pytest.raises(ValueError, match="router"):
        moe.layer_backward(x, *w, fwd, x, 2, 0, 8, router=moe.Router())
    with pytest.raises(ValueError, match="router"):
        moe.layer_backward(x, *w, dict(fwd, logits=logits), x, 2, 0, 8)
    with pytest.raises(ValueError, match="norm"):
        moe.layer_backward(x, *w, fwd, x, 2, 0, 8, norm=moe.RmsNorm(t((64,), bf16)))
    with pytest.raises(ValueError, match="norm"):
        moe.layer_backward(x, *w, dict(fwd, mean=None), x, 2, 0, 8, norm=(t((64,), bf16), None, 1e-5))


def test_sizes_past_32_bits_are_refused():
    """Not taken modulo 2^32; tensors without memory stand for the long rows."""
    wide = (1 << 32) + 8
    meta = lambda shape, dtype=bf16: torch.empty(shape, dtype=dtype, device="meta")  # noqa: E731
    rows, w, stats = meta((0, wide)), meta(wide), meta(0, f32)
    with pytest.raises(ValueError, match="32 bits"):
        moe.rms_norm(rows, w)
    with pytest.raises(ValueError, match="32 bits"):
        moe.rms_norm_int8(rows, w)
    with pytest.raises(ValueError, match="32 bits"):
        moe.rms_norm_backward(rows, rows, w, stats)
    with pytest.raises(ValueError, match="32 bits"):
        moe.rms_norm_backward_workspace_bytes(1, wide)
    with pytest.raises(ValueError):
        moe.route_experts(meta((0, wide), f32), 2, moe.Router(groups=wide, top_groups=wide))
    with pytest.raises(ValueError):
        moe.route_experts_backward(meta((0, wide), f32), meta((0, 2), i32), meta((0, 2), f32), moe.Router())
    experts = moe.Int8Experts(meta((1, wide // 64 + 1, 16, 64), torch.int8), meta((1, 16), f32),
                              meta((1, 1, wide, 64), torch.int8), meta((1, wide), f32))
    with pytest.raises(ValueError, match="32 bits"):
        moe.grouped_gemm_int8(moe.Int8Rows(meta((wide // 64 + 1, 0, 64), torch.int8), meta(0, f32)), meta(0, i32), meta(2, i32),
                              experts, 1, 1, 0, 1)
