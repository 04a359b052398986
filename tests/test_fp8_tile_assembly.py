"""The e4m3 tiles' loads to LDS in the code that is built: each one's m0 is written
in its own asm block, two instructions before, and nothing else touches m0."""
import os
import re
import subprocess

import pytest

from bit_block_quantized_nvfp4_amd import build as b


@pytest.mark.slow
def test_m0_belongs_to_the_loads(tmp_path):
    try:
        cc = b.hipcc()
    except RuntimeError:
        pytest.skip("needs hipcc")
    out = tmp_path / "tile.s"
    subprocess.run([cc, *b.HIP_FLAGS, "-w", "--cuda-device-only", "-S", os.path.join(b.CSRC, "moe_fp8_tile.hip"),
                    "-o", str(out)], check=True, capture_output=True)
    code = [ln.split(";")[0].strip() for ln in out.read_text().splitlines()]
    code = [ln for ln in code if ln and not ln.startswith(".") and not ln.endswith(":")]
    writes = [i for i, ln in enumerate(code) if re.search(r"\bm0\b", ln)]
    loads = [i for i, ln in enumerate(code) if ln.startswith("buffer_load") and ln.endswith(" lds")]
    assert len(loads) > 100 and [i + 2 for i in writes] == loads
    assert all(code[i].startswith("s_mov_b32 m0, s") and code[i + 1] == "s_nop 0" for i in writes)
    # the scalar offset was written five states before at least, or by a scalar instruction
    for i in loads:
        off = code[i].split(",")[-1].split()[0]
        late = code[max(0, i - 6):i - 2]
        assert not any(re.match(rf"v_readfirstlane_b32 {off},", ln) for ln in late), code[i - 8:i + 1]
