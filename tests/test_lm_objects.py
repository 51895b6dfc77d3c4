"""What the language-model objects refuse about where tensors lie and whose they are, with
stand-ins for tensors on two GPUs (CPU only: no call here reaches a kernel)."""
import pytest

torch = pytest.importorskip("torch")

import allreduce_ddp_assign_gb300 as D
from allreduce_ddp_assign_gb300 import lm

BF16, F32, I64 = torch.bfloat16, torch.float32, torch.int64


class OnGpu:
    """The attributes of a contiguous tensor on cuda:`index`."""

    def __init__(self, shape, dtype, index):
        self.shape, self.dtype, self.is_cuda = torch.Size(shape), dtype, True
        self.device = torch.device("cuda", index)

    def get_device(self):
        return self.device.index

    def dim(self):
        return len(self.shape)

    def stride(self):
        return (self.shape[-1], 1) if len(self.shape) == 2 else (1,)

    def numel(self):
        return self.shape.numel()

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 0x1000 * (1 + self.device.index)


class Library:
    """Takes every call and counts them."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append(name) or 0


@pytest.fixture
def two_gpus(monkeypatch):
    """Device 0 is current; nothing is launched."""
    library = Library()
    monkeypatch.setattr(lm, "_current_device", lambda: 0)
    monkeypatch.setattr(lm, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(lm, "lib", lambda: library)
    monkeypatch.setattr(lm, "ddp_vocab_loss_workspace", lambda *a: (256, 256))
    monkeypatch.setattr(lm, "ddp_embedding_workspace", lambda *a: 256)
    return library


V, DIM, T = 10, 8, 4
SHAPES = dict(weight=((V, DIM), BF16), hidden=((T, DIM), BF16), ids=((T,), I64), out=((T, DIM), BF16),
              lse=((T,), F32), grad_loss=((T,), F32), grad_hidden=((T, DIM), BF16), grad_weight=((V, DIM), F32))


def tensors(names, away):
    return [OnGpu(*SHAPES[n], int(n in away)) for n in names]


CALLS = {
    "lookup": (lambda a: lm.TokenEmbedding(V, DIM, BF16).forward(*a), ["weight", "ids", "out"]),
    "embedding gradient": (lambda a: lm.TokenEmbedding(V, DIM, BF16).backward(*a), ["hidden", "ids", "grad_weight"]),
    "loss": (lambda a: lm.VocabLoss(V, DIM, BF16).forward(*a), ["hidden", "weight", "ids"]),
    "loss gradient": (lambda a: lm.VocabLoss(V, DIM, BF16).backward(*a),
                      ["hidden", "weight", "ids", "lse", "grad_loss", "grad_hidden", "grad_weight"]),
}


@pytest.mark.parametrize("call,away", [(c, [n]) for c, (_, names) in CALLS.items() for n in names] +
                         [(c, names) for c, (_, names) in CALLS.items()])
def test_tensors_of_another_gpu_are_refused(two_gpus, call, away):
    """One of them elsewhere, and all of them on a GPU that is not the current one."""
    run, names = CALLS[call]
    with pytest.raises(ValueError, match="is on cuda:1, the current device is cuda:0"):
        run(tensors(names, away))
    assert not two_gpus.calls


def test_tensors_of_the_current_gpu_are_taken(two_gpus):
    run, names = CALLS["lookup"]
    run(tensors(names, []))
    assert two_gpus.calls == ["ddp_embedding_forward"]


@pytest.mark.parametrize("where", ["first", "second", "output", "all"])
def test_gradients_of_another_gpu_are_refused(two_gpus, where):
    g = [OnGpu((5,), F32, int(where in ("first", "all"))), OnGpu((7,), BF16, int(where in ("second", "all")))]
    out = [OnGpu((5,), F32, int(where == "all")), OnGpu((7,), BF16, int(where in ("output", "all")))]
    with pytest.raises(ValueError, match="is on cuda:1, the current device is cuda:0"):
        lm.GradClipper(g, out=out)


@pytest.mark.parametrize("call", [lambda c: c.norm(), lambda c: c.clip(1.0)])
def test_a_clipper_is_refused_where_another_gpu_is_current(two_gpus, call):
    c = object.__new__(lm.GradClipper)
    c.device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="gradients are on cuda:1, the current device is cuda:0"):
        call(c)
    assert not two_gpus.calls


class Reducer:
    """Two parameters' views of a main_grad."""

    def __init__(self, mode, main_grad=()):
        self.mode, self.main_grad = mode, main_grad
        self.plan = type("Plan", (), {"nparams": 2})

    def view(self, p, w):
        return OnGpu((5 + p,), F32, 0)


def test_clipping_after_a_reduce_scatter_is_refused(two_gpus):
    """A replica's main_grad holds reduced values in its own shard only."""
    with pytest.raises(ValueError, match="its own shard"):
        lm.GradClipper.of_reducer(Reducer(D.DDP_REDUCE_SCATTER))
    with pytest.raises(ValueError, match="no main_grad"):
        lm.GradClipper.of_reducer(Reducer(D.DDP_ALLREDUCE, None))
