"""Build properties of the gated activation's device code (no GPU needed): nothing in
scratch memory, and no conversion to E4M3 before the wave has set them to saturate."""

import re

from mxfp8_block_scaled_06_amd import build as b
from test_build_fp4_asm import _resources

SETS = "s_setreg_imm32_b32 hwreg(HW_REG_MODE, 23, 1), 1"


def test_conversions_come_after_the_mode_that_saturates_them(tmp_path):
    res = _resources("mx_swiglu.hip", tmp_path / "k.s")
    assert all(r["ScratchSize"] == 0 for r in res.values())
    bodies = re.split(r"^(_ZN3mxk\S*kernel\S*):", (tmp_path / "k.s").read_text(), flags=re.M)
    converting = 0
    for name, body in zip(bodies[1::2], bodies[2::2]):
        body = body.split(".Lfunc_end")[0]
        first = re.search(r"v_cvt_scalef32_pk_fp8_", body)
        if first is None:
            continue
        converting += 1
        assert 0 <= body.find(SETS) < first.start(), name
        # set once, and before the first load
        assert body.count("s_setreg") == 1 and body.find(SETS) < re.search(r"global_load_dwordx4", body).start(), name
    assert converting == 4, converting          # the dense forward with a checkpoint, the routed forms
