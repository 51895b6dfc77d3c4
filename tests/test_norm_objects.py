"""What a layer norm's object keeps between calls, with stand-ins for tensors (CPU only: no call here reaches a kernel)."""
import pytest

torch = pytest.importorskip("torch")

from allreduce_ddp_assign_gb300 import lm
from test_lm_objects import BF16, F32, OnGpu, two_gpus   # noqa: F401

T, DIM = 4, 8


def test_the_workspace_is_that_of_the_gpu_at_hand(two_gpus, monkeypatch):   # noqa: F811
    """Its size follows from a GPU's multiprocessors, and one object may be used on several GPUs."""
    current, asked = [0], []
    monkeypatch.setattr(lm, "_current_device", lambda: current[0])
    monkeypatch.setattr(lm, "ddp_layer_norm_workspace", lambda n, dim: (1000, 2000)[current[0]])
    monkeypatch.setattr(lm, "_empty", lambda size, **kw: asked.append(size) or torch.empty(1))
    f = lm.LayerNorm(DIM, BF16)
    for device in (0, 1, 0, 1):
        current[0] = device
        m, c, stats = (lambda: OnGpu((T, DIM), BF16, device)), (lambda: OnGpu((DIM,), F32, device)), OnGpu((2, T), F32, device)
        f.backward(m(), m(), c(), stats, grad_x=m(), grad_weight=c(), grad_bias=c())
    assert asked == [1000, 2000, 1000, 2000]


def test_a_width_below_one_is_refused():
    for dim in (0, -8):
        with pytest.raises(ValueError, match="dim"):
            lm.LayerNorm(dim, BF16)
