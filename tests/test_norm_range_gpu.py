"""fa_qk_norm_rope and its gradient over the whole range of bf16: heads whose
squares, and gradients whose products with them, leave fp32.

Tolerances as in test_norm_rope_gpu.py: what is taken at another scale is taken
at a power of two, which rounds nothing; a root times that scale below 2^-126
keeps 21 bits, which the gradient's 2^-18 counts.
"""
import numpy as np
import pytest
import torch

from exact_attention_94_gb300 import ops
from tests.test_norm_rope_gpu import check_bwd, check_fwd, weights
from tests.test_rope_gpu import bf, plan_lists

pytestmark = pytest.mark.gpu


def setting(d, kind="one"):
    axis, freq = plan_lists(d, kind)
    plan = ops.RopePlan(d, axis, freq)
    pos = np.random.default_rng(d).integers(0, 5000, (plan.n_axes, 6))
    return axis, freq, plan, pos, torch.tensor(pos, dtype=torch.int32).cuda()


def both(x, dy, d, eps, kind="one"):
    axis, freq, plan, pos, p = setting(d, kind)
    w = weights(d, 3, True)
    check_fwd(ops.qk_norm_rope(x, None, w, None, p, plan, eps)[0], x, w, pos, axis, freq, False, eps)
    dx, _, dw, _ = ops.qk_norm_rope_bwd(dy, None, x, None, w, None, p, plan, eps)
    check_bwd(dx, dw, dy, x, w, pos, axis, freq, False, 0, eps)


def scaled(t, log2):
    return (t.double() * 2.0 ** log2).to(torch.bfloat16)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", ["one", "any"])
@pytest.mark.parametrize("log2,eps", [(57, 1e-6), (60, 0.0), (62, 1e-6), (64, 3e38), (110, 1e-6), (124, 1e-6), (125, 0.0), (125, 3e38)])
def test_large_heads(d, kind, log2, eps):
    both(scaled(bf((6, 3, d), 1), log2), scaled(bf((6, 3, d), 2), 40), d, eps, kind)


@pytest.mark.parametrize("d", [64, 128])
def test_the_largest_values(d):
    """Heads of nothing but the largest number, of one, of two and of one beside small ones."""
    top = torch.finfo(torch.bfloat16).max
    x = bf((6, 3, d), 1)
    x[0, 0] = top
    x[1, 1] = torch.where(x[1, 1] > 0, top, -top)
    x[2, 2] = 0
    x[2, 2, 5] = top
    x[3, 0] = 0
    x[3, 0, 7] = x[3, 0, d - 1] = -top
    x[4, 1, 9] = top
    x[5, 2] = 2.0 ** 127
    both(x, scaled(bf((6, 3, d), 2), 40), d, 1e-6)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("x_log2,dy_log2,eps", [(59, 70, 1e-6), (40, 100, 0.0), (20, 120, 1e-6), (100, 90, 1e-6),
                                                (-40, -110, 0.0), (-30, -115, 1e-20), (-8, -115, 1e-6), (-100, -20, 0.0)])
def test_gradients_whose_products_leave_fp32(d, x_log2, dy_log2, eps):
    both(scaled(bf((6, 3, d), 1), x_log2), scaled(bf((6, 3, d), 2), dy_log2), d, eps)
