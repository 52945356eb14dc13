"""Build properties of the MXFP4 and few-token kernels' device code (no GPU
needed): no kernel keeps registers in scratch memory, whose loads would queue
behind the operand loads in flight, and the matrix kernels leave room for two
waves per SIMD, as their eight-wave workgroups need."""

import os
import re
import shutil
import subprocess

import pytest

from mxfp8_block_scaled_06_amd import build as b


def _resources(src, out):
    try:
        cc = b.hipcc()
    except RuntimeError:
        pytest.skip("hipcc not available")
    if shutil.which(cc) is None and not os.path.exists(cc):
        pytest.skip("hipcc not available")
    proc = subprocess.run([cc, *b.HIP_FLAGS, "-I", b.INCLUDE, "-I", b.CSRC, "-x", "hip", "--cuda-device-only", "-S",
                           os.path.join(b.CSRC, src), "-o", str(out)],
                          stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    assert proc.returncode == 0, proc.stdout[-4000:]
    res, name = {}, None
    for line in out.read_text().splitlines():
        m = re.match(r"^(_ZN3mxk\S*kernel\S*):", line)
        name = m.group(1) if m else name
        m = re.match(r"^; (NumVgprs|NumAgprs|ScratchSize|Occupancy): (\d+)", line)
        if m and name:
            res.setdefault(name, {})[m.group(1)] = int(m.group(2))
    return res


@pytest.mark.parametrize("src,kernels,matrix", [("mx_fp4.hip", 8, False), ("mx_fp4_gemm.hip", 10, True),
                                                ("mx_moe.hip", 14, True)])
def test_no_scratch_and_two_waves_per_simd(tmp_path, src, kernels, matrix):
    res = _resources(src, tmp_path / "k.s")
    assert len(res) == kernels, sorted(res)
    for name, r in res.items():
        assert r["ScratchSize"] == 0, (name, r)
        assert not matrix or (r["NumVgprs"] + r["NumAgprs"] <= 256 and r["Occupancy"] >= 2), (name, r)
