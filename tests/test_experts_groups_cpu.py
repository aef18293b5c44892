"""The search for experts and row tiles of the grouped products, run on the CPU for offsets that
decrease, lie outside the rows or are anything at all (tests/host_groups_check.cpp): the header
promises that no value of offsets leads outside the arrays."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
EXPERTS = os.path.join(ROOT, "tiled_dense_gemm_bias_amd", "csrc", "experts")


def build(tmp_path, header_dir):
    if not shutil.which("g++"):
        pytest.skip("no host compiler")
    exe = str(tmp_path / "groups")
    # (An undefined shift, overflow or cast ends the program.)
    r = subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I" + header_dir,
                        os.path.join(ROOT, "tests", "host_groups_check.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-3000:]
    return subprocess.run([exe], capture_output=True, text=True, timeout=600)


def test_every_tile_lies_in_its_experts_rows(tmp_path):
    r = build(tmp_path, EXPERTS)
    assert r.returncode == 0 and "groups check ok" in r.stdout, (r.stdout + r.stderr)[-2000:]


@pytest.mark.parametrize("right,wrong", [
    ("return min(max(v, 0), T);", "return max(v, 0);"),                                  # no clamp at the end
    ("rows = max(clamp_row(hi, T) - start, 0);", "rows = clamp_row(hi, T) - start;"),    # negative groups
    ("n += t;", "n = (int)n + t;"),                                                      # a total of 32 bits
    ("const int total = min(__builtin_amdgcn_readlane(upto, 63), g.row_bound);",
     "const int total = __builtin_amdgcn_readlane(upto, 63);"),                          # more tiles than the grid
    ("return T / bm + (E < T ? E : T);", "return T / bm + 1;"),                          # a grid too small
    ("before + upto > t", "before + upto >= t"),
])
def test_a_planted_mistake_is_found(tmp_path, right, wrong):
    with open(os.path.join(EXPERTS, "gx_groups.hpp")) as f:
        src = f.read()
    assert right in src
    with open(tmp_path / "gx_groups.hpp", "w") as f:
        f.write(src.replace(right, wrong))
    assert build(tmp_path, str(tmp_path)).returncode != 0
