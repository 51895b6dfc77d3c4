"""The example that runs the embedding, the vocabulary loss, the bucket reduction and
the clipping together, and one of its steps against the formulas."""
import math
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("no CUDA device", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import tied_lm as X


def test_training_lowers_the_loss_and_replicas_agree():
    losses, norms, master = X.train(steps=60)
    assert all(math.isfinite(v) for v in losses + norms)
    # it starts at random weights (about log V) and learns the mapping
    assert abs(losses[0] - math.log(X.VOCAB)) < 1.0
    assert losses[-1] < 0.5 * losses[0]
    for a, b in zip(*master):
        assert torch.equal(a, b)


def test_one_step_moves_the_weights_by_the_clipped_gradient():
    """After one step the weights have moved by lr times a gradient whose norm is at most max_norm."""
    lr, most = 0.25, 0.01
    before = X.train(steps=0, lr=lr, max_norm=most)[2][0]
    _, norms, after = X.train(steps=1, lr=lr, max_norm=most)
    assert norms[0] > most
    moved = math.sqrt(sum(float((a - b).double().square().sum()) for a, b in zip(after[0], before)))
    # the factor is off by fp32 roundings; each weight's step is rounded at the weight's size (below 1): 2^-24
    # an element, sqrt(elements) in the norm
    n = sum(b.numel() for b in before)
    assert abs(moved - lr * most) <= 1e-4 * lr * most + math.sqrt(n) * 2.0 ** -24
