"""Sizes that the library's 32-bit fields cannot hold are refused, not taken modulo 2^32.
No GPU needed: tensors without memory stand for the long rows."""
import os

import pytest

import token_dispatch_grouped_amd as moe

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(not os.path.exists(moe.lib_path), reason="libmoe.so not built")

WIDE = (1 << 32) + 8  # 8, modulo 2^32


@pytest.mark.parametrize("i,name", enumerate(["d", "d_ff", "E", "k", "e_begin", "e_end"]))
@pytest.mark.parametrize("value", [WIDE, 1 << 31, -(1 << 31) - 1, (1 << 64) + 1])
def test_a_shape_holds_what_it_is_given(i, name, value):
    good = [8, 8, 8, 2, 0, 8]
    s = moe.shape(1, *good)
    assert [s.d, s.d_ff, s.E, s.k, s.e_begin, s.e_end] == good
    good[i] = value
    with pytest.raises(ValueError, match="32 bits"):
        moe.shape(1, *good)


def test_the_largest_shape():
    top = (1 << 31) - 1
    s = moe.shape((1 << 63) - 1, top, top, top, top, top, top)
    assert (s.T, s.d, s.d_ff, s.E, s.k, s.e_begin, s.e_end) == ((1 << 63) - 1, top, top, top, top, top, top)
    with pytest.raises(ValueError):
        moe.shape(1 << 63, 8, 8, 8, 2, 0, 8)


def _meta(shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def test_layer_norm_of_wide_rows():
    rows, w, stats = _meta((0, WIDE)), _meta(WIDE), _meta(0, torch.float32)
    with pytest.raises(ValueError, match="32 bits"):
        moe.layer_norm(rows, w)
    with pytest.raises(ValueError, match="32 bits"):
        moe.layer_norm_backward(rows, rows, w, stats, stats)
    with pytest.raises(ValueError, match="32 bits"):
        moe.layer_norm_backward_workspace_bytes(1, WIDE)


def test_experts_of_wide_rows():
    e = moe.Int8Experts(_meta((1, WIDE // 64 + 1, 16, 64), torch.int8), _meta((1, 16), torch.float32),
                        _meta((1, 1, WIDE, 64), torch.int8), _meta((1, WIDE), torch.float32))
    with pytest.raises(ValueError, match="32 bits"):
        moe.grouped_gemm_int8(_meta((0, WIDE)), _meta(0, torch.int32), _meta(2, torch.int32), e, 1, 1, 0, 1)
    with pytest.raises(ValueError, match="32 bits"):
        moe.grouped_gemm_int8_workspace_bytes(1, WIDE, 8, 1, 1, 0, 1)
    with pytest.raises(ValueError, match="32 bits"):
        moe.quantize_experts(_meta((1, WIDE, 16)), _meta((1, 8, WIDE)))
