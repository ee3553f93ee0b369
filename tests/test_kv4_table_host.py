"""The block table is read in one place, which no slot or position leaves: the
device function itself, compiled for the host and run on every kind of value
that batch_index, pos and a wave's lanes can give."""

import os
import re
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "quantized_weight_streaming_q8_amd", "csrc")


def test_table_reads_stay_in_the_table(tmp_path):
    exe = str(tmp_path / "kv4_table")
    subprocess.run(["g++", "-std=c++17", "-O1", "-w", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I" + os.path.join(ROOT, "include"), "-I" + CSRC, "-o", exe,
                    os.path.join(ROOT, "tests", "kv4_table_host.cpp")], check=True)
    assert subprocess.run([exe], timeout=60).returncode == 0


def test_table_is_read_in_one_place():
    reads = []
    for name in sorted(os.listdir(CSRC)):
        if name.startswith("q8_kv4"):
            text = open(os.path.join(CSRC, name)).read()
            reads += [name] * len(re.findall(r"\.table\s*[\[+]", text))
    assert reads == ["q8_kv4_internal.h"]
