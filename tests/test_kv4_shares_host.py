"""How the attention's steps are cut into shares: the arithmetic of the kernel,
compiled for the host."""

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_shares_cover_the_room_and_searches_end(tmp_path):
    exe = str(tmp_path / "kv4_shares")
    subprocess.run(["g++", "-std=c++17", "-O2", "-w", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I" + os.path.join(ROOT, "include"),
                    "-I" + os.path.join(ROOT, "quantized_weight_streaming_q8_amd", "csrc"), "-o", exe,
                    os.path.join(ROOT, "tests", "kv4_shares_host.cpp")], check=True)
    assert subprocess.run([exe], timeout=60).returncode == 0
