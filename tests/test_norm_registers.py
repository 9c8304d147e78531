"""The norm's backward has an SM to itself and is compiled for that: no instance is squeezed into the
registers that two blocks an SM would leave."""

import re
import subprocess
from pathlib import Path

from int4_quantised_moe_b200 import build as b

SOURCE = """
#include "{csrc}/norm_kernels.cuh"
namespace r4 {{
cudaError_t instances(const NormArgs& a, cudaStream_t st) {{
  launch_bwd<__nv_bfloat16, 4, true, 1 + RAWINT4_CKPT_E4M3, true, true>(a, RAWINT4_TYPE_BF16, st);
  launch_bwd<__nv_bfloat16, 4, true, 1 + RAWINT4_CKPT_INT8, true, true>(a, RAWINT4_TYPE_BF16, st);
  return launch_bwd<__nv_bfloat16, 4, true, 0, true, true>(a, RAWINT4_TYPE_BF16, st);
}}
}}
"""


def test_four_chunks_have_the_registers_of_one_block(tmp_path):
    source = tmp_path / "instances.cu"
    source.write_text(SOURCE.format(csrc=Path(b.CSRC)))
    run = subprocess.run([b._nvcc(), *b.NVCC_FLAGS, "-Xptxas", "-v", "-c", str(source), "-o", str(tmp_path / "o")],
                         capture_output=True, text=True, check=True)
    registers = [int(n) for n in re.findall(r"Used (\d+) registers", run.stderr)]
    spills = [int(n) for n in re.findall(r"(\d+) bytes spill stores", run.stderr)]
    assert len(registers) == 3 and min(registers) > 64, registers  # 512 threads leave 128 each
    assert max(spills) < 512, spills
