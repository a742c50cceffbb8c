"""Kernels that start while the one before them ends do not read what it may
have written by the read-only path (no GPU: the sources are looked through)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_moe_expert_02_gb300", "csrc")


@pytest.mark.parametrize("name", ["act.cu", "few_rows.cuh", "groups.cuh", "int4.cu", "int4.cuh", "product_f32.cu", "product_few.cu",
                                  "product_few_bulk.cu", "product_tc.cu"])
def test_no_read_only_loads_in_dependent_kernels(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    assert not re.findall(r"__ldg\b|\.nc\b|__restrict__", text)
