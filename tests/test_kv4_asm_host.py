"""Inline assembly leaves m0 to the compiler: the loads to LDS take their
address from it, as an operand that the compiler puts there."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "quantized_weight_streaming_q8_amd", "csrc")


def test_assembly_takes_m0_as_an_operand():
    found = 0
    for name in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, name)).read()
        for stmt in re.findall(r"\basm\s+volatile\s*\(.*?\);", text, flags=re.S):
            assert not re.search(r"s_\w+ m0\b", stmt), (name, stmt)
            if "load_lds" in stmt:
                found += 1
                assert '"{m0}"' in stmt and '"memory"' in stmt, (name, stmt)
    assert found == 2
