"""GPU tests of the experts' calls at their edges: what lies around the
operands, far tails, sizes past one launch, overlapping tensors, replayed
steps.  Against the binary64 oracle, with the bounds of
tests/test_gpu_experts.py (its docstring derives them)."""

import numpy as np
import pytest
import torch

from tests import test_gpu_experts as T
from tests.gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


class Fenced:
    """Puts CPU tensors on the GPU with 64 KiB of NaN bit patterns before and
    behind them (any element there that reached a sum would show)."""

    def __init__(self, shift=0):
        self.shift = shift

    def __call__(self, t):
        if t is None:
            return None
        side = 65536 // t.element_size()
        buf = torch.full((t.numel() + 2 * side + 8,), float("nan"), dtype=t.dtype, device=DEV)
        out = buf[side + self.shift:side + self.shift + t.numel()].reshape(t.shape)
        out.copy_(t)
        return out


@pytest.mark.parametrize("i", [8, 64, 72, 128, 200])
@pytest.mark.parametrize("sizes,o", [([2500, 0, 130, 1], 4104), ([64] * 16, 1032), ([1, 0, 3], 264)])
def test_short_reductions(sizes, o, i, monkeypatch):
    """Reductions of one to four steps, where the steps loaded ahead lie past
    the end: nothing from around the operands reaches a result."""
    require_gpu()
    monkeypatch.setattr(T, "Shifted", Fenced)
    T._say(f"short reductions {len(sizes)} groups {i} {o}")
    T._forward_linear(T.Problem(60, sizes, i, o), "none", True, True, True)
    T._forward_gated(T.Problem(61, sizes, i, o // 2), "silu", True)
    T._backward_linear(T.Problem(62, sizes, o, i), "relu")
    T._backward_gated(T.Problem(63, sizes, o, i), "silu")


def test_gelu_far_tail():
    """x Phi(x) and its slope relative to themselves, for every bf16 from -12.5
    to -1/16.  Phi within 1.1e-6 of the formula and z^2, z = |x| / sqrt 2 <= 8.9,
    rounded to fp32 three times before e^(-z^2): 79 * 2^-22 and the
    exponential's own argument, 114 * 2^-24, together below 2^-14; the slope's
    two terms likewise, and one rounding to bf16 each."""
    require_gpu()
    bits = torch.arange(0xBD80, 0xC149, dtype=torch.int32).to(torch.int16)
    x = bits.view(BF).reshape(-1, 1).to(DEV)
    one = torch.ones(1, 1, 1, dtype=BF, device=DEV)
    y, d_x = torch.empty_like(x), torch.empty_like(x)
    T.rrb.expert_linear(x, None, one, y, activation="gelu")
    T.rrb.expert_linear_backward(torch.ones_like(x), x, None, one, pre=x, activation="gelu", d_x=d_x)
    nx = T._np(x)
    assert nx.min() == -12.5 and nx.max() == -0.0625
    want, slope = T.OE.act("gelu", nx), T.OE.act_grad("gelu", nx)
    T._check("act", y, want, 2.0 ** -14 * np.abs(want))
    phi = want / nx
    T._check("slope", d_x, slope, 2.0 ** -14 * (phi + np.abs(slope - phi)))
