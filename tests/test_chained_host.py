"""What kernels that are launched while their predecessors run may read, and how: checks of their sources."""
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "quantized_kv_cache_kv8_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//.*", "", f.read())


CHAINED = sorted(n for n in os.listdir(CSRC) if n.endswith(".cu") and "launch_chained" in source(n))


@pytest.mark.parametrize("name", CHAINED + ["gqa_common.cuh", "paged_common.cuh"])
def test_what_a_predecessor_writes_is_not_read_as_constant(name):
    """Non-coherent loads are for what no kernel writes while theirs lives, and the compiler may move them past the
    wait for the predecessor, which may have written the operand (queries, tables, rows)."""
    assert not re.search(r"__ldg\s*\(|ld\.global\.nc|__restrict__", source(name))
