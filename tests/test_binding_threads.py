"""The binding's first call, made by two threads at once. No GPU needed: the calls get
as far as the refusal of host tensors."""
import os
import threading

import pytest

import token_dispatch_grouped_amd as moe

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.skipif(not os.path.exists(moe.lib_path), reason="libmoe.so not built")


def test_a_second_thread_during_the_first_call(monkeypatch):
    """Another thread's call comes in while the first fills the table of types."""
    seen = []

    def other():
        try:
            moe.grad_norm([torch.zeros(4)])
        except Exception as e:  # noqa: BLE001
            seen.append(e)

    class Table(dict):
        def update(self, *args):
            if not seen:
                seen.append(None)
                t = threading.Thread(target=other)
                t.start()
                t.join(60)
            super().update(*args)

    monkeypatch.setattr(moe, "_TORCH", None)
    monkeypatch.setattr(moe, "_CODES", Table())
    with pytest.raises(ValueError, match="on the GPU"):
        moe.layer_norm(torch.zeros(4, 8), torch.ones(8))
    assert len(seen) == 2 and isinstance(seen[1], ValueError) and "on the GPU" in str(seen[1]), seen
