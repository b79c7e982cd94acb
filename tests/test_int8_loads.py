"""The decode form of the 8-bit layer leaves pieces past a row of W, and rows past W, to
the range check of its buffer loads, which covers a load's lane offset and not its
scalar one: in the machine code no such load may have a scalar offset."""

import os
import re
import subprocess

from dequant_gemm_nf4_amd import build


def test_decode_loads_have_no_scalar_offset(tmp_path):
    out = str(tmp_path / "few.s")
    subprocess.run([build.HIPCC, *build.FLAGS, "-S", "--offload-device-only",
                    os.path.join(build.CSRC, "bnbx_int8_few.hip"), "-o", out], check=True,
                   capture_output=True)
    loads = re.findall(r"buffer_load_dwordx4\s+\S+ \S+ s\[\S+\], (\S+)", open(out).read())
    assert len(loads) >= 4 * 16          # four a batch, in each of 16 kernels
    assert set(loads) == {"0"}, sorted(set(loads))
