"""What the layer-norm and AdamW calls refuse, on the host, before anything is launched (CPU only: no call here
reaches a kernel)."""
import math

import pytest

import allreduce_ddp_assign_gb300 as D
from test_lm_refusals import refused


@pytest.fixture(scope="module", autouse=True)
def built():
    from allreduce_ddp_assign_gb300 import _build

    _build.build()


FWD = dict(x=0x1000, x_stride=64, residual=0x2000, residual_stride=64, dtype=D.DDP_BF16, ntokens=10, dim=64, weight=0x3000,
           bias=0x4000, w_dtype=D.DDP_F32, eps=1e-5, out=0x5000, out_stride=64, sum=0x6000, sum_stride=64, mean=0x7000,
           rstd=0x8000)
BWD = dict(grad_out=0x1000, grad_stride=64, x=0x2000, x_stride=64, mean=0x3000, rstd=0x4000, grad_sum=0x5000,
           grad_sum_stride=64, dtype=D.DDP_F16, ntokens=10, dim=64, weight=0x6000, w_dtype=D.DDP_F16, grad_x=0x7000,
           grad_x_stride=64, grad_weight=0x8000, grad_bias=0x9000, gw_dtype=D.DDP_F32, accumulate=0, workspace=0x10000,
           workspace_bytes=1 << 40)


@pytest.mark.parametrize("match,change", [
    ("ntokens", dict(ntokens=-1)), ("ntokens", dict(ntokens=1 << 31)), ("ntokens", dict(ntokens=(1 << 31) - 4096)),
    ("dim", dict(dim=0)), ("dim", dict(dim=(1 << 24) + 1)), ("unknown dtype", dict(dtype=3)), ("w_dtype", dict(w_dtype=D.DDP_F16, dtype=D.DDP_BF16)),
    ("x is NULL", dict(x=None)), ("x's stride", dict(x_stride=63)), ("weight is NULL", dict(weight=None)),
    ("mean or rstd", dict(mean=None)), ("mean or rstd", dict(rstd=None))])
def test_both_passes(match, change):
    refused(match, D.ddp_layer_norm_forward, FWD, **change)
    refused(match, D.ddp_layer_norm_backward, BWD, **change)


def test_each_pass():
    refused("out is NULL", D.ddp_layer_norm_forward, FWD, out=None)
    refused("out's stride", D.ddp_layer_norm_forward, FWD, out_stride=63)
    refused("residual's stride", D.ddp_layer_norm_forward, FWD, residual_stride=63)
    refused("sum's stride", D.ddp_layer_norm_forward, FWD, sum_stride=63)
    refused("come together", D.ddp_layer_norm_forward, FWD, residual=None)
    refused("come together", D.ddp_layer_norm_forward, FWD, sum=None)
    for eps in (-1e-5, math.inf, math.nan):
        refused("eps", D.ddp_layer_norm_forward, FWD, eps=eps)
    refused("grad_out is NULL", D.ddp_layer_norm_backward, BWD, grad_out=None)
    refused("grad_x is NULL", D.ddp_layer_norm_backward, BWD, grad_x=None)
    refused("grad_out's stride", D.ddp_layer_norm_backward, BWD, grad_stride=63)
    refused("grad_sum's stride", D.ddp_layer_norm_backward, BWD, grad_sum_stride=63)
    refused("grad_x's stride", D.ddp_layer_norm_backward, BWD, grad_x_stride=63)
    refused("gw_dtype", D.ddp_layer_norm_backward, BWD, gw_dtype=D.DDP_BF16)
    refused("workspace is NULL", D.ddp_layer_norm_backward, BWD, workspace=None)
    refused("aligned", D.ddp_layer_norm_backward, BWD, workspace=0x10010)
    refused("workspace of", D.ddp_layer_norm_backward, BWD, workspace_bytes=100)
    refused("out is sum", D.ddp_layer_norm_forward, FWD, out=0x6000)
    refused("grad_weight is grad_bias", D.ddp_layer_norm_backward, BWD, grad_weight=0x9000)
    # no tokens: nothing is read
    D.ddp_layer_norm_forward(**{**FWD, "ntokens": 0, "x": None, "weight": None, "mean": None}, stream=0)
    D.ddp_layer_norm_backward(**{**BWD, "ntokens": 0, "x": None, "weight": None, "accumulate": 1}, stream=0)
    D.ddp_layer_norm_backward(**{**BWD, "ntokens": 0, "grad_weight": None, "grad_bias": None, "workspace": None}, stream=0)
    for bad in ((-1, 10), (10, 0), (1 << 31, 10), (10, (1 << 24) + 1)):
        with pytest.raises(D.DdpError):
            D.ddp_layer_norm_workspace(*bad)


def test_workspace_is_bounded():
    assert D.ddp_layer_norm_workspace(1, 768) >= 8 * 768
    assert D.ddp_layer_norm_workspace(1 << 20, 768) < 4 << 20
    assert D.ddp_layer_norm_workspace(1 << 20, 16384) < 64 << 20
    # rows that no team of warps holds
    assert D.ddp_layer_norm_workspace(1 << 20, 1 << 20) <= (64 << 20) + 256
    assert D.ddp_layer_norm_workspace(1 << 20, 1 << 24) <= (128 << 20) + 256


STEP = dict(tensors=0x1000, first_block=0x2000, ntensors=3, nblocks=10, exp_avg=0x3000, exp_avg_sq=0x4000,
            exp_avg_scale=0x5000, exp_avg_sq_scale=0x6000, state_bits=8, state=0x7000, lr=1e-3, lr_at=None, beta1=0.9,
            beta2=0.999, eps=1e-8, seed=0, grad_scale=1.0, norm=0x8000, max_norm=1.0)


@pytest.mark.parametrize("match,change", [
    ("ntensors", dict(ntensors=-1)), ("nblocks", dict(nblocks=-1)), ("without tensors", dict(ntensors=0)),
    ("state_bits", dict(state_bits=16)), ("state is NULL", dict(state=None)), ("table", dict(tensors=None)),
    ("table", dict(first_block=None)), ("moment is NULL", dict(exp_avg=None)), ("moment is NULL", dict(exp_avg_sq=None)),
    ("aligned", dict(exp_avg=0x3008)), ("aligned", dict(exp_avg_sq=0x4004)), ("scale is NULL", dict(exp_avg_scale=None)),
    ("scale is NULL", dict(exp_avg_sq_scale=None)), ("lr", dict(lr=-1.0)), ("lr", dict(lr=math.nan)), ("lr", dict(lr=math.inf)),
    ("beta1", dict(beta1=1.0)), ("beta1", dict(beta1=-0.1)), ("beta2", dict(beta2=1.0)), ("beta2", dict(beta2=math.nan)),
    ("eps", dict(eps=-1e-8)), ("eps", dict(eps=math.nan)), ("grad_scale", dict(grad_scale=0.0)),
    ("grad_scale", dict(grad_scale=-2.0)), ("grad_scale", dict(grad_scale=math.nan)), ("max_norm", dict(max_norm=-1.0)),
    ("max_norm", dict(max_norm=math.nan))])
def test_adamw(match, change):
    refused(match, D.ddp_adamw_step, STEP, **change)


@pytest.mark.parametrize("match,change", [
    # its reciprocal, which the gradients are multiplied by, would be infinite
    ("grad_scale", dict(grad_scale=1e-39)), ("grad_scale", dict(grad_scale=5e-324)),
    # the step's quotient takes a divisor below 2^-126 for 0, and 0 / 0 is not 0
    ("eps", dict(eps=1e-60)), ("eps", dict(eps=2.0 ** -127))])
def test_adamw_numbers_that_fp32_does_not_hold(match, change):
    refused(match, D.ddp_adamw_step, STEP, **change)


def test_objects_refuse_on_the_host():
    torch = pytest.importorskip("torch")
    from allreduce_ddp_assign_gb300 import lm

    cpu = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="float64"):
        lm.LayerNorm(8, torch.float64)
    f = lm.LayerNorm(8, torch.float32)
    with pytest.raises(ValueError, match="x is not on the GPU"):
        f.forward(cpu, cpu[0])
    with pytest.raises(ValueError, match="x has dtype"):
        f.forward(cpu.half(), cpu[0])
    with pytest.raises(ValueError, match="s is not on the GPU"):
        f.backward(cpu, cpu, cpu[0], cpu)
    for bad, match in ((dict(state_bits=16), "state_bits"), (dict(weight_decay=[0.1, 0.2]), "weight decays"),
                       (dict(weight_decay=-1.0), "negative"), (dict(copies=[]), "copies")):
        with pytest.raises(ValueError, match=match):
            lm.AdamW([cpu], [cpu], **bad)
    with pytest.raises(ValueError, match="gradients and"):
        lm.AdamW([cpu], [])
    with pytest.raises(ValueError, match="parameter 0 is None"):
        lm.AdamW([None], [cpu])
    with pytest.raises(ValueError, match="on the GPU"):
        lm.AdamW([cpu], [cpu])
    with pytest.raises(ValueError, match="float64"):
        lm.AdamW([cpu.double()], [cpu])


# ---------------------------------------------------------------------------
# where tensors lie, with stand-ins for tensors on two GPUs
# ---------------------------------------------------------------------------
from test_lm_objects import BF16, F32, OnGpu, Reducer, two_gpus   # noqa: E402,F401

T, DIM = 4, 8
MATRIX, COLUMN, STATS = ((T, DIM), BF16), ((DIM,), F32), ((2, T), F32)
CALLS = {
    "forward": (lambda f, a: f.forward(a[0], a[1], a[2], residual=a[3], out=a[4], sum_out=a[5]),
                [MATRIX, COLUMN, COLUMN, MATRIX, MATRIX, MATRIX]),
    "backward": (lambda f, a: f.backward(a[0], a[1], a[2], a[3], grad_sum=a[4], grad_x=a[5], grad_weight=a[6], grad_bias=a[7]),
                 [MATRIX, MATRIX, COLUMN, STATS, MATRIX, MATRIX, COLUMN, COLUMN]),
}


@pytest.mark.parametrize("call,away", [(c, [i]) for c, (_, kinds) in CALLS.items() for i in range(len(kinds))] +
                         [(c, list(range(len(kinds)))) for c, (_, kinds) in CALLS.items()])
def test_tensors_of_another_gpu_are_refused(two_gpus, call, away):
    from allreduce_ddp_assign_gb300 import lm

    run, kinds = CALLS[call]
    with pytest.raises(ValueError, match="is on cuda:1, the current device is cuda:0"):
        run(lm.LayerNorm(DIM, BF16), [OnGpu(*k, int(i in away)) for i, k in enumerate(kinds)])
    assert not two_gpus.calls


@pytest.mark.parametrize("where", ["parameter", "gradient", "copy"])
def test_an_optimizer_over_another_gpu_is_refused(two_gpus, where):
    from allreduce_ddp_assign_gb300 import lm

    p, g, c = (OnGpu((5,), F32, int(where == n)) for n in ("parameter", "gradient", "copy"))
    with pytest.raises(ValueError, match="is on cuda:1, the current device is cuda:0"):
        lm.AdamW([p], [g], copies=[c])


def test_a_step_is_refused_where_another_gpu_is_current(two_gpus):
    import torch

    from allreduce_ddp_assign_gb300 import lm

    o = object.__new__(lm.AdamW)
    o.device = torch.device("cuda", 1)
    with pytest.raises(ValueError, match="parameters are on cuda:1, the current device is cuda:0"):
        o.step()
    assert not two_gpus.calls


def test_an_optimizer_after_a_reduce_scatter_is_refused(two_gpus):
    from allreduce_ddp_assign_gb300 import lm

    with pytest.raises(ValueError, match="its own shard"):
        lm.AdamW.of_reducer(Reducer(D.DDP_REDUCE_SCATTER), [])
    with pytest.raises(ValueError, match="no main_grad"):
        lm.AdamW.of_reducer(Reducer(D.DDP_ALLREDUCE, None), [])


def test_tensors_that_share_memory_are_refused():
    import torch

    from allreduce_ddp_assign_gb300 import lm

    names = ("parameter", "copy", "gradient")
    x = torch.zeros(100)
    a, b, c = x[:30], x[30:60], x[60:]
    lm._apart(names, ([a, b], [None, c], [torch.zeros(3), None]))
    same = torch.zeros(5)
    lm._apart(names, ([a, b], [], [same, same]))   # (gradients are only read)
    for lists in (([a, a], [], []), ([x, b], [], []), ([a, b], [None, x[50:61]], []), ([a], [], [a]), ([b], [], [x]),
                  ([a, b], [], [x[29:31]]), ([], [a], [x[10:12]])):
        with pytest.raises(ValueError, match="shares memory"):
            lm._apart(names, lists)
