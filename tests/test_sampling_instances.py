"""The main kernel over shared prefixes is built for what calls can ask for, and
nothing else: no row by warps, 8 or 16, the last not over 8-bit pages of d = 128."""
import re
import shutil
import subprocess

import pytest

from exact_attention_94_gb300 import build


@pytest.mark.skipif(shutil.which("nm") is None, reason="no nm")
def test_instances_of_the_main_kernel():
    build.build()
    names = subprocess.run(["nm", "-C", build.LIB], capture_output=True, text=True, check=True).stdout
    built = set(re.findall(r"fa_decode_shared_kernel<(\d+), (\d+), (true|false)>", names))
    wanted = {(d, few, kv8) for d in ("64", "128") for few in ("0", "1", "2") for kv8 in ("true", "false")}
    assert built == wanted - {("128", "2", "true")}
