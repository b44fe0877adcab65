"""Grids follow the device's number of SMs, not that of one part."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_expert_ffn_router_b200", "csrc")


@pytest.mark.parametrize("name", ["quantize.cu", "gemm_i8.cu", "gemv_i8.cu", "few_tokens.cu", "int_api.cu"])
def test_no_launch_counts_on_148_sms(name):
    code = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    assert not re.search(r"\b148\b", code)
