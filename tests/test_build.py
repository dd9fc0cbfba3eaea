"""What the compiler makes of the kernels that move registers between warps (no GPU is needed)."""
import os
import re
import subprocess

import pytest

from mixture_experts_layer_index_gb300 import build as b


def test_registers_of_the_split(tmp_path):
    """Products with block scales launch with as many registers per thread as their split of them adds up to; with
    others they would refuse every launch.  A compiler that chooses otherwise shows here."""
    source = os.path.join(b.CSRC, "linear_fp8.cu")
    with open(source) as f:
        text = f.read()
    launch = int(re.search(r"constexpr int LAUNCH_REGS = (\d+)", text).group(1))
    try:
        nvcc = b._nvcc()
    except RuntimeError:
        pytest.skip("no nvcc")
    r = subprocess.run([nvcc, *b.ARCH, *b.FLAGS, "-Xptxas", "-v", "-c", source, "-o", str(tmp_path / "o.o")], capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    used = re.findall(r"Compiling entry function '(\S*linear_fp8_kernel\S*)'.*?Used (\d+) registers", r.stderr, re.S)
    assert len({name for name, _ in used}) == len(re.findall(r"launch_shape<\d, \d+, (?:true|false)>\(a,", text))
    assert all(int(n) == launch for _, n in used), used
