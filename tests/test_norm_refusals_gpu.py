"""What the norms' gradient refuses it calls by the argument's name."""
import pytest
import torch

from exact_attention_94_gb300 import ops
from tests.test_norm_rope_gpu import weights
from tests.test_rope_gpu import bf

pytestmark = pytest.mark.gpu


def test_names_in_refusals():
    plan = ops.rope_plan(64, [32])
    x, w, p = bf((4, 2, 64), 6), weights(64, 1, False), torch.zeros((1, 4), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="^dyq has shape"):
        ops.qk_norm_rope_bwd(x[:3], None, x, None, w, None, p, plan)
    with pytest.raises(TypeError, match="^dyk must be"):
        ops.qk_norm_rope_bwd(None, x.float(), None, x, None, w, p, plan)
    with pytest.raises(ValueError, match="^dyk must live"):
        ops.qk_norm_rope_bwd(x, x.cpu(), x, x, w, w, p, plan)
