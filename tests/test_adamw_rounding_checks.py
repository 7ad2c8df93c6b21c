"""Which rounding a step of 8-bit states takes, and what it refuses. No GPU."""
import ctypes

import pytest

import token_dispatch_grouped_amd as moe

torch = pytest.importorskip("torch")
NULL = ctypes.c_void_p(0)


def _state(rounding=None):
    return moe.Float8State(torch.zeros(4, 8, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.zeros(1), *([rounding] if rounding else []))


def _rounding(m, v, betas):
    return moe._rounding({s.rounding for s in m + v}, betas)


def test_roundings():
    plain, near, dither = _state(), _state("nearest"), _state("dither")
    assert plain.rounding is None
    for betas in ((0.9, 0.999), (0.9, 0.951), (0.99, 0.9)):
        assert _rounding([plain], [plain], betas) == moe.MOE_DITHER
        assert _rounding([plain, dither], [dither, plain], betas) == moe.MOE_DITHER
        assert _rounding([near], [near], betas) == moe.MOE_NEAREST
    assert _rounding([plain], [plain], (0.9, 0.95)) == moe.MOE_NEAREST
    assert _rounding([dither], [dither], (0.9, 0.95)) == moe.MOE_DITHER
    for bits_states in moe.adamw_states([torch.zeros(3)], bits=8):
        assert bits_states[0].rounding == "dither"


@pytest.mark.parametrize("m,v,betas", [("nearest", "dither", (0.9, 0.95)), (None, "dither", (0.9, 0.95)), (None, "nearest", (0.9, 0.999)),
                                       ("up", "up", (0.9, 0.95)), ("up", None, (0.9, 0.95))])
def test_states_of_two_roundings_are_refused(m, v, betas):
    p = [torch.zeros(4, 8)]
    with pytest.raises(ValueError, match="rounding"):
        moe.adamw(p, [torch.zeros(4, 8)], [_state(m)], [_state(v)], 1, 1e-3, betas)


def test_binding_refusals_of_the_library():
    entry = moe.moe_adamw_tensor(param=0x10000, grad=0x20000, exp_avg=0x30000, exp_avg_sq=0x40000, exp_avg_scale=0x50000,
                                 exp_avg_sq_scale=0x60000, numel=0)
    def call(**kw):  # noqa: E306
        args = moe.moe_adamw_args(lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1, **kw)
        return moe.lib().moe_adamw(ctypes.byref(entry), 1, ctypes.byref(args), NULL)
    for rounding in (0, 1):
        assert call(state=1, rounding=rounding) == moe.MOE_OK
    for rounding in (-1, 2):
        assert call(state=1, rounding=rounding) == moe.MOE_EINVAL
        assert call(state=0, rounding=rounding) == moe.MOE_OK
