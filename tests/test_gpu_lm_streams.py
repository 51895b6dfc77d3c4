"""Objects made on a stream that their tensors do not come from: memory stays in use until the work there is done."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no CUDA device", allow_module_level=True)

from allreduce_ddp_assign_gb300 import lm
from test_gpu_adamw import Problem
from test_gpu_lm import BF16, F32


def dropped_while_queued(tensors, make, use):
    """make() and use(object) on a side stream that is busy; the caller's `tensors` are then dropped with the object, and
    others of their sizes made on their own stream."""
    places = {t.data_ptr() for t in tensors}
    sizes = [(t.shape, t.dtype, t.device) for t in tensors]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o = make()
        torch.cuda._sleep(1_000_000_000)
        use(o)
    del o
    tensors.clear()
    new = [torch.empty(shape, dtype=dtype, device=device) for shape, dtype, device in sizes for _ in range(3)]
    waiting = not s.query()
    assert waiting   # else the check says nothing
    assert not places & {t.data_ptr() for t in new}
    s.synchronize()


@pytest.mark.parametrize("bits", [32, 8])
def test_an_optimizer_made_on_another_stream(bits):
    warm = Problem(11, [3001, 70, 5000], F32, F32, BF16, 0)
    warm.optimizer(state_bits=bits).step()   # (a kernel's first launch waits for the whole GPU)
    torch.cuda._sleep(1)
    torch.cuda.synchronize()
    q = [Problem(11, [3001, 70, 5000], F32, F32, BF16, 0)]
    q[0].before.clear()
    tensors = list(q[0].flat.values())
    dropped_while_queued(tensors, lambda: q.pop().optimizer(state_bits=bits), lambda opt: opt.step())


@pytest.mark.parametrize("out", [False, True])
def test_a_clipper_made_on_another_stream(out):
    warm = [torch.ones(100, device="cuda") for _ in range(2)]
    lm.GradClipper(warm[:1], out=warm[1:] if out else None).clip(1.0)
    torch.cuda._sleep(1)
    torch.cuda.synchronize()
    tensors = list(Problem(12, [3001, 70, 5000], F32, F32, BF16, 0).flat.values())
    g, o = [tensors[0], tensors[1], tensors[2]], [torch.empty_like(t) for t in tensors] if out else None
    tensors += o or []

    def make():
        c = lm.GradClipper(g, out=o)
        g.clear()
        if o:
            o.clear()
        return c

    dropped_while_queued(tensors, make, lambda c: c.clip(1.0))
