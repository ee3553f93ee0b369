"""Which kernel and tile a product takes: the library's arithmetic, compiled for the host.  The GPU tests' shapes
take those that they are there for, and no tile is left without one."""

import os
import subprocess

import pytest

import ffn_shapes as shapes

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FORMS = (1, 2, 3)  # q8_acts_format


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "mx_plan")
    subprocess.run(["g++", "-std=c++17", "-O2", "-w", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    "-I" + os.path.join(ROOT, "include"),
                    "-I" + os.path.join(ROOT, "quantized_weight_streaming_q8_amd", "csrc"), "-o", exe,
                    os.path.join(ROOT, "tests", "mx_plan_host.cpp")], check=True)

    def ask(calls):
        """[(format, rows, projections, quantised, tokens)] -> [("columns 4", tiles)]"""
        text = "\n".join(" ".join(str(int(v)) for v in c) for c in calls)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, check=True, timeout=60).stdout.split()
        return [(" ".join(out[i:i + 2]), int(out[i + 2])) for i in range(0, len(out), 3)]
    return ask


@pytest.mark.parametrize("name,projections,quantised", [("PRODUCTS", 1, 0), ("GATED", 2, 0), ("QUANTISED", 2, 1)])
def test_shapes_take_the_tiles_they_are_for(plan, name, projections, quantised):
    cases = getattr(shapes, name)
    for form in FORMS:
        got = plan([(form, n, projections, quantised, live) for (n, _, live), _, _ in cases])
        for (shape, want, several), (tile, tiles) in zip(cases, got):
            assert (tile, tiles > 256 and tile.startswith("columns")) == (want, several), (shape, form, tile, tiles)


def test_every_tile_has_a_shape():
    heights = {"columns 1", "columns 2", "columns 4", "columns 5", "wide 2", "wide 4"}
    for cases, need in ((shapes.PRODUCTS, heights), (shapes.GATED, heights),
                        (shapes.QUANTISED, {h for h in heights if h not in ("columns 1", "columns 5")})):
        assert {want for _, want, _ in cases} == need
        assert {(live + 15) // 16 for (_, _, live), want, _ in cases if live <= 64} >= {2, 3, 4}
        assert {want for _, want, several in cases if several} >= {"columns 4"}


def test_the_plan_holds_its_own_rules(plan):
    """Up to 16 tokens the narrow kernel; no large tiles up to 64; an even number of row groups for quantised rows."""
    calls = [(f, n, p, q, live) for f in FORMS for n in (1, 31, 32, 768, 7168, 17408, 151936, 1 << 24) for p in (1, 2)
             for q in ((0, 1) if p == 2 and n % 32 == 0 else (0,)) for live in (1, 16, 17, 64, 65, 128, 1024, 4099, 1 << 20)]
    for c, (tile, tiles) in zip(calls, plan(calls)):
        live, quantised = c[4], c[3]
        assert (tile == "narrow 0") == (live <= 16), c
        if 16 < live <= 64:
            assert tile.startswith("columns"), c
        if quantised and tile.startswith("columns"):
            assert tile in ("columns 2", "columns 4"), c
        assert tile == "narrow 0" or tiles >= 1
