"""No packed FP32 arithmetic in the generated gfx950 code of any kernel: the
instructions are switched off in the build, and none is written by hand."""
import os
import re

import pytest

from test_codegen import CSRC, HIPCC, device_build

pytestmark = pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith(".hip")))
def test_no_packed_fp32(name, tmp_path):
    text = device_build(name, tmp_path)[0]
    assert "s_endpgm" in text and not re.search(r"^\s*v_pk_(add|mul|fma)_f32", text, re.M)
