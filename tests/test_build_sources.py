"""Properties of the kernels' sources that no run shows."""
import glob
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCES = sorted(glob.glob(os.path.join(ROOT, "sparse_moe_router_amd", "**", "*.hip"), recursive=True))


@pytest.mark.parametrize("path", SOURCES, ids=os.path.basename)
def test_asm_statements_declare_m0(path):
    """An asm statement that writes m0 lists it as clobbered: the compiler may keep a value there."""
    src = re.sub(r"//[^\n]*", "", open(path).read())
    for m in re.finditer(r"\basm\s+volatile\s*\((.*?)\);", src, flags=re.S):
        if re.search(r"\bs_\w+ m0\b", m.group(1)):
            assert '"m0"' in m.group(1).rsplit(":", 1)[1], m.group(0)
