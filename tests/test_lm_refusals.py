"""What the clipping, embedding and vocabulary-loss calls refuse, on the host,
before anything is launched (CPU only: no call here reaches a kernel)."""
import math

import pytest

import allreduce_ddp_assign_gb300 as D

BIG = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def built():
    from allreduce_ddp_assign_gb300 import _build

    _build.build()


def refused(match, fn, args, **change):
    a = dict(args)
    a.update(change)
    with pytest.raises(D.DdpError, match=match) as e:
        fn(**a, stream=0)
    assert e.value.status == D.DDP_E_INVAL


CLIP = dict(grads=0x1000, out=None, offset=0x2000, dtypes=0x3000, ntensors=3, total=100, norm_type=D.DDP_NORM_L2,
            max_norm=1.0, norm=0x4000, workspace=0x10000, workspace_bytes=D.DDP_CLIP_WORKSPACE_BYTES)


@pytest.mark.parametrize("match,change", [
    ("ntensors", dict(ntensors=-1)), ("total", dict(total=-1)), ("without tensors", dict(ntensors=0)),
    ("norm_type", dict(norm_type=7)), ("norm is NULL", dict(norm=None)), ("table", dict(grads=None)),
    ("table", dict(offset=None)), ("table", dict(dtypes=None)), ("workspace is NULL", dict(workspace=None)),
    ("workspace of", dict(workspace_bytes=100)), ("aligned", dict(workspace=0x10004)),
    ("max_norm", dict(max_norm=-1.0)), ("max_norm", dict(max_norm=math.nan))])
def test_clip(match, change):
    refused(match, D.ddp_clip_grads, CLIP, **change)
    if "max_norm" not in change:
        norm = {k: v for k, v in CLIP.items() if k not in ("out", "max_norm")}
        refused(match, D.ddp_grad_norm, norm, **change)


FWD = dict(weight=0x1000, weight_stride=64, dtype=D.DDP_F32, vocab=100, dim=64, ids=0x2000, id_bytes=8, ntokens=10,
           scale=1.0, out=0x3000, out_stride=64)
BWD = dict(grad_out=0x1000, grad_stride=64, dtype=D.DDP_BF16, ids=0x2000, id_bytes=8, ntokens=10, scale=1.0,
           padding_idx=-1, vocab=100, dim=64, grad_weight=0x3000, gw_stride=64, gw_dtype=D.DDP_BF16, accumulate=0,
           workspace=0x10000, workspace_bytes=BIG)


@pytest.mark.parametrize("match,change", [
    ("ntokens", dict(ntokens=-1)), ("ntokens", dict(ntokens=1 << 31)), ("vocab", dict(vocab=0)),
    ("vocab", dict(vocab=1 << 31)), ("dim", dict(dim=0)), ("dtype", dict(dtype=5)), ("id_bytes", dict(id_bytes=2)),
    ("ids is NULL", dict(ids=None))])
def test_embedding(match, change):
    refused(match, D.ddp_embedding_forward, FWD, **change)
    refused(match, D.ddp_embedding_backward, BWD, **change)


def test_embedding_each_side():
    refused("weight is NULL", D.ddp_embedding_forward, FWD, weight=None)
    refused("out is NULL", D.ddp_embedding_forward, FWD, out=None)
    refused("weight's stride", D.ddp_embedding_forward, FWD, weight_stride=63)
    refused("out's stride", D.ddp_embedding_forward, FWD, out_stride=63)
    refused("grad_out is NULL", D.ddp_embedding_backward, BWD, grad_out=None)
    refused("grad_weight is NULL", D.ddp_embedding_backward, BWD, grad_weight=None)
    refused("grad_out's stride", D.ddp_embedding_backward, BWD, grad_stride=63)
    refused("grad_weight's stride", D.ddp_embedding_backward, BWD, gw_stride=63)
    refused("gw_dtype", D.ddp_embedding_backward, BWD, gw_dtype=D.DDP_F16)
    refused("workspace", D.ddp_embedding_backward, BWD, workspace=None)
    refused("workspace", D.ddp_embedding_backward, BWD, workspace=0x10004)
    need = D.ddp_embedding_workspace(10, 100, 64)
    refused("workspace", D.ddp_embedding_backward, BWD, workspace_bytes=need - 1)
    D.ddp_embedding_forward(**{**FWD, "ntokens": 0, "ids": None, "weight": None, "out": None}, stream=0)
    D.ddp_embedding_backward(**{**BWD, "ntokens": 0, "ids": None, "grad_out": None, "accumulate": 1}, stream=0)
    with pytest.raises(D.DdpError):
        D.ddp_embedding_workspace(-1, 10, 10)


LOSS = dict(hidden=0x1000, hidden_stride=64, weight=0x2000, weight_stride=64, dtype=D.DDP_BF16, ntokens=10, vocab=100,
            dim=64, targets=0x3000, id_bytes=8, ignore_index=-100, loss=0x4000, lse=0x5000, workspace=0x10000,
            workspace_bytes=BIG)
GRAD = dict(hidden=0x1000, hidden_stride=64, weight=0x2000, weight_stride=64, dtype=D.DDP_BF16, ntokens=10, vocab=100,
            dim=64, targets=0x3000, id_bytes=8, ignore_index=-100, lse=0x5000, grad_loss=0x6000, grad_loss_stride=1,
            grad_hidden=0x7000, gh_stride=64, grad_weight=0x8000, gw_stride=64, gw_dtype=D.DDP_F32, accumulate=0,
            piece=0, workspace=0x10000, workspace_bytes=BIG)


@pytest.mark.parametrize("match,change", [
    ("ntokens", dict(ntokens=-1)), ("ntokens", dict(ntokens=1 << 31)), ("vocab", dict(vocab=0)),
    ("vocab", dict(vocab=1 << 31)), ("dim", dict(dim=0)), ("dim", dict(dim=1 << 24)), ("dtype", dict(dtype=D.DDP_F32)),
    ("id_bytes", dict(id_bytes=3)), ("hidden's stride", dict(hidden_stride=63)),
    ("weight's stride", dict(weight_stride=63)), ("weight is NULL", dict(weight=None)), ("hidden", dict(hidden=None)),
    ("targets", dict(targets=None)), ("lse", dict(lse=None)), ("workspace", dict(workspace=None)),
    ("workspace", dict(workspace=0x10008)), ("workspace", dict(workspace_bytes=1000))])
def test_vocab_loss(match, change):
    refused(match, D.ddp_vocab_loss_forward, LOSS, **change)
    refused(match, D.ddp_vocab_loss_backward, GRAD, **change)


def test_vocab_loss_each_side():
    refused("loss", D.ddp_vocab_loss_forward, LOSS, loss=None)
    refused("both outputs", D.ddp_vocab_loss_backward, GRAD, grad_hidden=None, grad_weight=None)
    refused("grad_hidden's stride", D.ddp_vocab_loss_backward, GRAD, gh_stride=63)
    refused("grad_weight's stride", D.ddp_vocab_loss_backward, GRAD, gw_stride=63)
    refused("gw_dtype", D.ddp_vocab_loss_backward, GRAD, gw_dtype=D.DDP_F16)
    refused("grad_loss_stride", D.ddp_vocab_loss_backward, GRAD, grad_loss_stride=2)
    refused("grad_loss is NULL", D.ddp_vocab_loss_backward, GRAD, grad_loss=None)
    refused("piece", D.ddp_vocab_loss_backward, GRAD, piece=-1)
    f, b = D.ddp_vocab_loss_workspace(10, 100, 64)
    refused("workspace", D.ddp_vocab_loss_forward, LOSS, workspace_bytes=f - 1)
    refused("workspace", D.ddp_vocab_loss_backward, GRAD, workspace_bytes=b - 1)
    # a weight off its 16-byte boundary needs room for a copy
    f2, b2 = D.ddp_vocab_loss_workspace(10, 100, 64, weight_aligned=0)
    assert f2 > f and b2 > b
    refused("workspace", D.ddp_vocab_loss_forward, LOSS, weight=0x2002, workspace_bytes=f)
    D.ddp_vocab_loss_forward(**{**LOSS, "ntokens": 0, "hidden": None, "targets": None}, stream=0)
    for bad in (dict(ntokens=-1), dict(vocab=0), dict(dim=0), dict(piece=-1)):
        with pytest.raises(D.DdpError):
            D.ddp_vocab_loss_workspace(**{**dict(ntokens=10, vocab=100, dim=64, piece=0), **bad})


def test_workspace_follows_the_piece():
    """The backward pass's memory is bounded by the piece, not by the vocabulary."""
    small = D.ddp_vocab_loss_workspace(8192, 50257, 768, piece=1024)[1]
    large = D.ddp_vocab_loss_workspace(8192, 50257, 768, piece=16384)[1]
    assert large - small == 2 * 8192 * (16384 - 1024)
    assert D.ddp_vocab_loss_workspace(8192, 50257, 768, piece=1000)[1] == small   # rounded up to 256 words


def test_objects_refuse_on_the_host():
    torch = pytest.importorskip("torch")
    from allreduce_ddp_assign_gb300 import lm

    cpu = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="norm_type"):
        lm.GradClipper([], norm_type=1)
    with pytest.raises(ValueError, match="on the GPU"):
        lm.GradClipper([cpu])
    with pytest.raises(ValueError, match="float64"):
        lm.GradClipper([cpu.double()])
    with pytest.raises(ValueError, match="outputs for"):
        lm.GradClipper([None], out=[])
    with pytest.raises(ValueError, match="has an output"):
        lm.GradClipper([None], out=[cpu])
    with pytest.raises(ValueError, match="float64"):
        lm.TokenEmbedding(10, 8, torch.float64)
    e = lm.TokenEmbedding(4, 8, torch.float32)
    with pytest.raises(ValueError, match="ids must be"):
        e.forward(cpu, torch.zeros(3))
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        lm.VocabLoss(10, 8, torch.float32)


def test_token_counts_whose_loops_would_leave_32_bits():
    """The kernels step through the tokens in 32 bits, beyond the last one by up to a step."""
    for n in ((1 << 31) - 4096, (1 << 31) - 2048, (1 << 31) - 600, (1 << 31) - 1):
        refused("ntokens", D.ddp_embedding_backward, BWD, ntokens=n)
        refused("ntokens", D.ddp_vocab_loss_forward, LOSS, ntokens=n)
        refused("ntokens", D.ddp_vocab_loss_backward, GRAD, ntokens=n)
        for sizes in (D.ddp_embedding_workspace, D.ddp_vocab_loss_workspace):
            with pytest.raises(D.DdpError, match="ntokens"):
                sizes(n, 100, 64)
    assert D.ddp_embedding_workspace((1 << 31) - 4097, 100, 64) > 8 << 31
    assert D.ddp_vocab_loss_workspace((1 << 31) - 4097, 100, 64)[0] > 2 * 64 << 31
