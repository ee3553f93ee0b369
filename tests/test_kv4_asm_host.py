"""Inline assembly says what it changes: the loads to LDS take their address
from m0, which the compiler may use too."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "quantized_weight_streaming_q8_amd", "csrc")


def test_assembly_that_writes_m0_says_so():
    found = 0
    for name in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, name)).read()
        for stmt in re.findall(r"\basm\s+volatile\s*\(.*?\);", text, flags=re.S):
            if re.search(r"s_mov_b32 m0\b", stmt):
                found += 1
                assert '"m0"' in stmt and '"memory"' in stmt, (name, stmt)
    assert found == 2
