"""The scales and codes of 8-bit moments, every one of them: equal to those of the formulas in fp32, rounded after each
operation (an operation of torch on fp32 tensors rounds once, roots and quotients among them)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no CUDA device", allow_module_level=True)

from test_gpu_adamw import BLOCK, SIZES, Problem, chances, steps_of
from test_gpu_lm import BF16, DEV, F16, F32


def f32(x):
    """x, rounded to fp32 from 64 bits."""
    return torch.tensor(x, dtype=torch.float64).float().to(DEV)


def held(x, chance, root):
    """Blocks of values as multiples of their scales, by chance, and the scales."""
    scale = x.abs().amax(dim=1) * f32(1 / 448)
    scale = torch.where(scale < 2.0 ** -126, torch.zeros_like(scale), scale)
    q = x.abs() / torch.where(scale > 0, scale, torch.ones_like(scale))[:, None]
    q = torch.where(scale[:, None] > 0, q, torch.zeros_like(q))
    # (the multiples of a step and their fractions are exact from here on)
    low = q < 2.0 ** -6
    a = torch.where(low, (q * 2.0 ** 29).round() * 2.0 ** -29, q).double()
    step = steps_of(a)
    a = (a / step + (chance.double() + 0.5) / 2 ** 16).floor() * step
    if root:
        a = torch.where(x > 0, a.clamp(min=2.0 ** -9), a)
    return torch.where(x < 0, -a, a), scale


def in_blocks(tensors, opt):
    out = torch.zeros(opt.nblocks * BLOCK, device=DEV)
    for k, t in enumerate(tensors):
        a = int(opt.first_block[k]) * BLOCK
        out[a:a + t.numel()] = t.float()
    return out.view(-1, BLOCK)


def factor(norm, max_norm, scale):
    """What a gradient is multiplied by: 1 / grad_scale from 64 bits, then fp32."""
    inverse = f32(1 / scale)
    if norm is None:
        return inverse
    ratio = f32(max_norm) / (norm * inverse + f32(1e-6))
    return inverse * ratio.clamp(max=1.0)


@pytest.mark.parametrize("name", ["edges", "many", "long"])
@pytest.mark.parametrize("gdt", [F32, BF16, F16])
@pytest.mark.parametrize("shift", [0, 3])
@pytest.mark.parametrize("betas,clip", [((0.9, 0.999), None), ((0.8, 0.95), (3.7, 0.31, 1.0)), ((0.9, 0.99), (90.0, 1.0, 24.0))])
def test_every_scale_and_code(name, gdt, shift, betas, clip):
    q = Problem(21, SIZES[name], BF16 if gdt != F32 else F32, gdt, None, shift)
    # a block's values over many binades, so that codes of every size are there
    spread = torch.linspace(-12, 0, 977, device=DEV).exp2()
    flat = q.flat["g"]
    wide = flat.float() * spread[torch.arange(flat.numel(), device=DEV) % 977]
    # (none between 0 and 2^-26: times a factor above 2^-7, squared, times 0.001 that is above 2^-76, and a root is held
    # as half of itself at least)
    flat.copy_(torch.where(wide.abs() < 2.0 ** -26, 0.0, wide))
    q.before["g"] = flat.clone()
    seed = 0xC0FFEE1234567
    opt = q.optimizer(lr=1e-3, betas=betas, state_bits=8, seed=seed)
    b1, b2, o1, o2 = (f32(x) for x in (*betas, 1 - betas[0], 1 - betas[1]))
    norm = None if clip is None else f32([clip[0]])
    c = factor(norm, *clip[1:]) if clip else factor(None, None, 1.0)
    g = in_blocks(q.g, opt)
    for t in (1, 2, 3, 4):
        m = opt.exp_avg.float() * opt.exp_avg_scale[:, None]
        r = opt.exp_avg_sq.float() * opt.exp_avg_sq_scale[:, None]
        opt.step(norm=norm, max_norm=clip[1] if clip else None, grad_scale=clip[2] if clip else 1.0)
        x = g * c
        m = m * b1 + x * o1
        v = (r * r) * b2 + (x * x) * o2
        # where the header promises it: no v between 0 and 2^-102, every largest m that is not 0 from 2^-62 on
        assert bool(((v == 0) | (v >= 2.0 ** -102)).all())
        top = m.abs().amax(dim=1)
        assert bool(((top == 0) | (top >= 2.0 ** -62)).all())
        chance = chances(seed, t, opt.nblocks)
        for what, y, codes, scale, k in (("m", m, opt.exp_avg, opt.exp_avg_scale, chance.view(-1, 2).flip(1).reshape(-1, BLOCK)),
                                         ("root", v.sqrt(), opt.exp_avg_sq, opt.exp_avg_sq_scale, chance)):
            want, s = held(y, k, what == "root")
            assert torch.equal(scale, s), what
            assert torch.equal(codes.double(), want), what
    q.guards()
