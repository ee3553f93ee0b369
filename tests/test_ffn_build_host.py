"""What the compiler makes of the feed-forward side's kernels, with the product's flags."""

import os
import re
import subprocess

import pytest

from quantized_weight_streaming_q8_amd import build


def compile_source(name, *flags):
    if not os.path.exists(build.HIPCC):
        pytest.skip("no hipcc")
    out = subprocess.run([build.HIPCC, *build.FLAGS, *flags, os.path.join(build.CSRC, name)], capture_output=True, text=True)
    assert out.returncode == 0, out.stderr
    return out


def test_products_of_up_to_16_tokens_keep_their_registers(tmp_path):
    """No kernel of that way spills: its loop has its weights on their way and its tokens in registers."""
    asm = str(tmp_path / "k.s")
    compile_source("q8_mx_matmul.hip", "--cuda-device-only", "-S", "-o", asm)
    text = open(asm).read()
    scratch = dict(re.findall(r"\.name:\s+(\S*mx_narrow_kernel\S*)\s+\.private_segment_fixed_size: (\d+)", text))
    assert len(scratch) == 18 and set(scratch.values()) == {"0"}, scratch


@pytest.mark.parametrize("name", [s for s in build.SOURCES if s.startswith(("q8_mx_", "q8_norm", "q8_ffn_"))])
def test_sources_have_no_unused_names(name):
    assert not re.findall(r"warning: unused .*", compile_source(name, "-fsyntax-only", "-Wall", "-Wno-unused-function").stderr)
