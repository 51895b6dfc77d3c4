"""Which streams the allocator is told of by the objects that keep a program's tensors, with stand-ins for tensors
(CPU only: no call here reaches a kernel)."""
import pytest

torch = pytest.importorskip("torch")

from allreduce_ddp_assign_gb300 import lm
from test_lm_objects import BF16, F32, OnGpu, two_gpus   # noqa: F401


class Kept(OnGpu):
    """A tensor of device 0 with memory of its own, beside which tables may be made without a GPU."""

    made = 0

    def __init__(self, shape, dtype):
        super().__init__(shape, dtype, 0)
        self.device = torch.device("cpu", 0)
        Kept.made += 1
        self.at = 0x10000 * Kept.made

    def get_device(self):
        return 0

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return self.at


@pytest.fixture
def lent(two_gpus, monkeypatch):   # noqa: F811
    """What the allocator is told: (stream, tensor), of a current stream that `lent.current` names."""

    class Lent(list):
        current = 7

        def to(self, stream):
            return {id(t) for s, t in self if s == stream}

    told = Lent()
    monkeypatch.setattr(lm, "_raw_stream", lambda index: told.current)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: told.current)
    monkeypatch.setattr(lm, "_lend", lambda stream, *ts: told.extend((stream, t) for t in ts if t is not None))
    told.calls = two_gpus.calls
    return told


def optimizer(bits):
    p, g, c = [Kept((5,), F32), Kept((300,), F32)], [Kept((5,), BF16), None], [None, Kept((300,), BF16)]
    opt = lm.AdamW(p, g, copies=c, state_bits=bits)
    own = [t for t in (opt._tables, opt.exp_avg, opt.exp_avg_sq, opt.exp_avg_scale, opt.exp_avg_sq_scale) if t is not None]
    return opt, {id(t) for t in p + own + [g[0], c[1]]}


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_on_the_stream_the_optimizer_was_made_on_lends_it_everything(lent, bits):
    """The parameters, gradients and copies may come from any other stream."""
    opt, everything = optimizer(bits)
    opt.step()
    assert lent.to(7) == everything and lent.calls == ["ddp_adamw_step"]
    told = len(lent)
    opt.step()
    assert len(lent) == told   # once
    lent.current = 8
    opt.step()
    assert lent.to(8) == everything


@pytest.mark.parametrize("bits", [32, 8])
def test_a_state_loaded_or_copied_on_another_stream_lends_it_the_moments(lent, bits):
    opt, everything = optimizer(bits)
    for k, use in enumerate((lambda: opt.load_state_dict(state), lambda: opt.moments(1), opt.state_dict)):
        state = {"step": 3, "exp_avg": opt.exp_avg.clone(), "exp_avg_sq": opt.exp_avg_sq.clone()}
        if bits == 8:
            state.update(exp_avg_scale=opt.exp_avg_scale.clone(), exp_avg_sq_scale=opt.exp_avg_sq_scale.clone())
        lent.current = 20 + k
        use()
        assert lent.to(20 + k) >= {id(t) for t in (opt.exp_avg, opt.exp_avg_sq, opt._tables)}


@pytest.mark.parametrize("call", [lambda c: c.norm(), lambda c: c.clip(1.0)])
@pytest.mark.parametrize("out", [False, True])
def test_a_call_on_the_stream_the_clipper_was_made_on_lends_it_everything(lent, monkeypatch, call, out):
    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: empty(*a, **kw))
    g = [Kept((5,), F32), None, Kept((300,), BF16)]
    o = [Kept((5,), F32), None, None] if out else None
    c = lm.GradClipper(g, out=o)
    call(c)
    assert lent.to(7) == {id(t) for t in (c._tables, g[0], g[2], *(o or ())) if t is not None}
    told = len(lent)
    call(c)
    assert len(lent) == told   # once
