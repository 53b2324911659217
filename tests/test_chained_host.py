"""What kernels that are launched while their predecessors run may read, and how: checks of their sources."""
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "quantized_kv_cache_kv8_gb300", "csrc")
CHAINED = ["beam.cu", "fork.cu", "gqa_append.cu", "gqa_attn.cu", "gqa_common.cuh", "gqa_tc.cu"]


@pytest.mark.parametrize("name", CHAINED)
def test_what_a_predecessor_writes_is_not_read_as_constant(name):
    """Non-coherent loads are for what no kernel writes while theirs lives, and the compiler may move them past the
    wait for the predecessor, which may have written the operand (queries, tables, rows)."""
    with open(os.path.join(CSRC, name)) as f:
        code = re.sub(r"//.*", "", f.read())
    assert "launch_chained" in code or name.endswith(".cuh")
    assert not re.search(r"__ldg\s*\(|ld\.global\.nc|__restrict__", code)
