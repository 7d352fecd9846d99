"""Checks on the generated gfx950 code of the gated block's and the 4-bit
format's kernels: m0 is written by the direct-to-LDS copies only, nothing
spills and nothing lives in scratch memory."""
import os
import re

import pytest

from tests.test_codegen import CSRC, HIPCC, _compile

COPYING = ["k_gated_forward.hip", "k_gated_dx.hip", "k_gated_dw.hip", "k_mx4.hip"]
ALL = COPYING + ["k_gated_util.hip", "k_mx4_quant.hip", "k_mx4_skinny.hip"]

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")


@pytest.fixture(scope="module")
def built(tmp_path_factory):
    from concurrent.futures import ThreadPoolExecutor
    out = str(tmp_path_factory.mktemp("asm"))
    with ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        return dict(zip(ALL, ex.map(lambda n: _compile(n, out), ALL)))


@pytest.mark.parametrize("name", COPYING)
def test_m0_only_written_by_our_copies(built, name):
    assert os.path.exists(os.path.join(CSRC, name))
    body = [l.strip() for l in built[name][0].splitlines()]
    seen = 0
    for i, l in enumerate(body):
        if re.search(r"\bm0\b", l) and not l.startswith(";"):
            seen += 1
            assert l.startswith("s_mov_b32 m0,"), "unexpected m0 use: " + l
            assert body[i + 1] == "s_nop 0" and body[i + 2].startswith("global_load_lds_dwordx4"), l
    assert seen


@pytest.mark.parametrize("name", ALL)
def test_no_register_spills(built, name):
    remarks = built[name][1]
    spills = [int(x) for x in re.findall(r"VGPRs Spill: (\d+)", remarks)]
    scratch = [int(x) for x in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", remarks)]
    assert spills and max(spills) == 0 and max(scratch) == 0, remarks[-2000:]
