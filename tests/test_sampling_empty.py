"""The gradient of the head norms for no tokens at all: its sizes are divided by
what is at least 1.  Run in a process of its own, without a GPU: a division by
zero would end it."""
import os
import subprocess
import sys

from exact_attention_94_gb300 import build

CALL = """
import ctypes
from exact_attention_94_gb300 import _lib
from tests.test_serving_abi import A, NUL, rope_plan
lib = _lib.load()
for Hq, Hkv, d in ((2, 1, 64), (1, 0, 128), (0, 3, 64), (65000, 535, 128)):
    st = lib.fa_qk_norm_rope_bwd(*(A,) * 11, ctypes.byref(rope_plan()), 0, Hq, Hkv, d, *(Hq * d, Hkv * d) * 3, 0, 1e-6, A, NUL)
    assert st == _lib.FA_ERR_LAUNCH, st  # (there is no GPU to launch on)
"""


def test_gradient_of_no_tokens():
    build.build()
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", CALL], cwd=root, env={**os.environ, "CUDA_VISIBLE_DEVICES": ""},
                       capture_output=True, text=True)
    assert r.returncode == 0, (r.returncode, r.stderr[-500:])
