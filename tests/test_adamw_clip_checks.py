"""adamw's norm and max_norm go together. No GPU."""
import pytest

import token_dispatch_grouped_amd as moe

torch = pytest.importorskip("torch")


def _call(**kw):
    ts = [[torch.zeros(4, 8)] for _ in range(4)]
    moe.adamw(*ts, 1, 1e-3, **kw)


def test_one_needs_the_other():
    norm = torch.ones(1)
    with pytest.raises(ValueError, match="max_norm, what to clip to"):
        _call(norm=norm)
    with pytest.raises(ValueError, match="max_norm needs norm"):
        _call(max_norm=1.0)
    # both, neither, and a limit of 0 that the caller gives: refused for the CPU tensors only
    for kw in (dict(norm=norm, max_norm=1.0), dict(norm=norm, max_norm=0.0), {}, dict(max_norm=0.0)):
        with pytest.raises(ValueError, match="GPU"):
            _call(**kw)
