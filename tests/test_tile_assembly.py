"""The 16-bit and 8-bit integer tiles' loads to LDS in the code that is built: each one's
m0 is written in its own asm block, two instructions before, and nothing else touches m0; a
scalar register that such a load reads was not written by a vector instruction within the
five states before it; nothing is spilled to memory."""
import os
import re
import subprocess

import pytest

from bit_block_quantized_nvfp4_amd import build as b


def _scalars(operand):
    m = re.fullmatch(r"s\[(\d+):(\d+)\]", operand)
    if m:
        return set(range(int(m[1]), int(m[2]) + 1))
    m = re.fullmatch(r"s(\d+)", operand)
    return {int(m[1])} if m else set()


@pytest.mark.slow
@pytest.mark.parametrize("source", ["moe_dense.hip", "moe_dense_grad.hip", "moe_int8.hip"])
def test_loads_to_lds(tmp_path, source):
    try:
        cc = b.hipcc()
    except RuntimeError:
        pytest.skip("needs hipcc")
    out = tmp_path / "tile.s"
    subprocess.run([cc, *b.HIP_FLAGS, "-w", "--cuda-device-only", "-S", os.path.join(b.CSRC, source), "-o", str(out)],
                   check=True, capture_output=True)
    text = out.read_text()
    assert not re.search(r"vgpr_spill_count:\s*[1-9]|private_segment_fixed_size:\s*[1-9]", text)
    code = [ln.split(";")[0].strip() for ln in text.splitlines()]
    code = [ln for ln in code if ln and not ln.startswith(".") and not ln.endswith(":")]
    writes = [i for i, ln in enumerate(code) if re.search(r"\bm0\b", ln)]
    loads = [i for i, ln in enumerate(code) if ln.startswith("buffer_load") and ln.endswith(" lds")]
    assert len(loads) > 100 and [i + 2 for i in writes] == loads
    assert all(code[i].startswith("s_mov_b32 m0, s") and code[i + 1] == "s_nop 0" for i in writes)
    for i in loads:
        ops = [o.strip() for o in code[i].split(None, 1)[1].split(",")]
        read = _scalars(ops[1]) | _scalars(ops[2].split()[0])
        states, j = 0, i - 1
        while states < 5:
            name, _, rest = code[j].partition(" ")
            if name.startswith("v_") and _scalars(rest.split(",")[0].strip()) & read:
                pytest.fail("\n".join(code[j:i + 1]))
            states += int(rest) + 1 if name == "s_nop" else 1
            j -= 1
