"""Checks on the generated gfx950 code of the gated block's and the 4-bit
format's kernels: m0 is written by the direct-to-LDS copies only, nothing
spills and nothing lives in scratch memory."""
import os
import re

import pytest

from test_codegen import HIPCC, device_build         # one compilation serves both modules

COPYING = ["k_gated_forward.hip", "k_gated_dx.hip", "k_gated_dw.hip", "k_gated_pair.hip", "k_mx4.hip"]
ALL = COPYING + ["k_gated_util.hip", "k_mx4_quant.hip", "k_mx4_skinny.hip"]

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")


@pytest.mark.parametrize("name", COPYING)
def test_m0_only_written_by_our_copies(name, tmp_path):
    body = [l.strip() for l in device_build(name, tmp_path)[0].splitlines()]
    seen = 0
    for i, l in enumerate(body):
        if re.search(r"\bm0\b", l) and not l.startswith(";"):
            seen += 1
            assert l.startswith("s_mov_b32 m0,"), "unexpected m0 use: " + l
            assert body[i + 1] == "s_nop 0" and body[i + 2].startswith("global_load_lds_dwordx4"), l
    assert seen


@pytest.mark.parametrize("name", ALL)
def test_no_register_spills(name, tmp_path):
    remarks = device_build(name, tmp_path)[1]
    spills = [int(x) for x in re.findall(r"VGPRs Spill: (\d+)", remarks)]
    scratch = [int(x) for x in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", remarks)]
    assert spills and max(spills) == 0 and max(scratch) == 0, remarks[-2000:]
