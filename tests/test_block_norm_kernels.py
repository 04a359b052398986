"""The norm kernels that are built are those that a call can reach: rows have at
most 8192 values, so eight waves of four chunks a thread (more than 1024 chunks of
16 bytes) are for float32 alone."""
import re
import shutil
import subprocess

import pytest

from _libutil import ensure_built


@pytest.mark.skipif(shutil.which("nm") is None, reason="needs nm")
def test_every_built_norm_kernel_is_reached():
    ensure_built()
    from bit_block_quantized_nvfp4_amd import _lib

    names = subprocess.run(["nm", "-C", _lib.LIB_PATH], capture_output=True, text=True, check=True).stdout
    fwd = {tuple(map(int, m)) for m in re.findall(r"stub__k_block_norm<(\d), (\d), (\d)>", names)}
    bwd = {tuple(map(int, m)) for m in re.findall(r"stub__k_block_norm_grad<(\d), (\d), (\d), \d>", names)}
    assert fwd and bwd

    def reached(grad):
        out = set()
        for dt, size in ((0, 2), (1, 2), (2, 4)):
            for H in range(8, 8193, 8):
                for T in (1, 1000):
                    c = H * size // 16
                    waves = 8 if c > 1024 else 4 if c > 256 or (c > 64 and (grad or T <= 512)) else 1
                    out.add((dt, -(-c // (64 * waves)) > 1 and 4 or 1, waves))
        return out

    assert fwd == reached(False) and bwd == reached(True)
