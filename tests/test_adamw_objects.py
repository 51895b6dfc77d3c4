"""What an optimizer's object takes and refuses, with stand-ins for tensors (CPU only: no call here reaches a kernel)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from allreduce_ddp_assign_gb300 import lm
from test_lm_objects import F32, two_gpus   # noqa: F401
from test_lm_streams import Kept


def decays(**kw):
    p = [Kept((5,), F32), Kept((7,), F32)]
    opt = lm.AdamW(p, [None, None], **kw)
    words = opt._tables.numpy()[2 + 3:]
    return words.view(lm._RECORD)["weight_decay"].tolist()


def test_one_weight_decay_is_any_number(two_gpus):   # noqa: F811
    for d in (0.5, 0, np.float32(0.5), np.float64(0.5), np.int64(1)):
        assert decays(weight_decay=d) == [float(d)] * 2
    assert decays(weight_decay=np.array([0.25, 0.5])) == [0.25, 0.5]
    assert decays(weight_decay=(0.25, np.float32(0.5))) == [0.25, 0.5]


def test_a_weight_decay_that_fp32_does_not_hold_is_refused(two_gpus):   # noqa: F811
    for bad in (1e39, [0.1, 1e39], float("inf"), float("nan"), -0.1):
        with pytest.raises(ValueError, match="weight decay"):
            decays(weight_decay=bad)
