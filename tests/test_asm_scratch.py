"""Static check that the tile kernels keep their accumulators in registers.

Their loops over accumulators are unrolled, so that every index is a constant. Where a loop's body grows past
what the compiler unrolls, the array goes to scratch memory without a word (a gradient's epilogue did so: 271 ->
321 us). An accumulator array is 256 bytes a lane or more; the few registers that the compiler spills take less.
No GPU is needed."""
import os
import re
import subprocess

import pytest

from block_scaled_fp4_histogram_amd import build as B


@pytest.mark.parametrize("source", ["moe_mm.hip", "moe_glu.hip", "moe_fp8.hip"])
def test_no_accumulators_in_scratch_memory(source):
    flags = [f for f in B.FLAGS if f not in ("-shared", "-Wl,--no-undefined")]
    r = subprocess.run([B.HIPCC, *flags, "--cuda-device-only", "-S", "-Rpass-analysis=kernel-resource-usage",
                        os.path.join(B.CSRC, source), "-o", os.devnull], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    used = re.findall(r"Function Name: (\S+).*?ScratchSize \[bytes/lane\]: (\d+)", r.stderr, re.S)
    tiles = [(n, int(b)) for n, b in used if "k_mm_tile" in n]
    assert len(tiles) >= 16
    assert not [t for t in tiles if t[1] >= 256]
