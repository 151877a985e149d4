"""The library holds no kernels that no launch names. No GPU is needed."""
import re
import shutil
import subprocess

import pytest

from block_scaled_fp4_histogram_amd import build as B


@pytest.mark.skipif(shutil.which("nm") is None, reason="needs nm")
def test_last_rounds_are_joined_in_the_shapes_that_the_plan_splits():
    r = subprocess.run(["nm", "-C", B.LIB], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    joins = set(re.findall(r" moe::k_tail_join<(\d+), (\d+), (\d+), (\d+), \d+>", r.stdout))
    # operation and type: gated block of 16 bits and by either sum of 8-bit floats, its gradient, 8-bit products
    kinds = {("4", "1"), ("4", "2"), ("4", "5"), ("4", "6"), ("5", "1"), ("5", "2"), ("1", "5"), ("1", "6")}
    assert joins == {(*k, *s) for k in kinds for s in (("256", "128"), ("128", "256"))}
