"""The partial results that the join of shared prompts reads, by the index arithmetic that its kernel uses, on the host:
whatever a record says is shared, a row's own partial results are not left; for sound records they are those written."""
import os
import re
import shutil
import subprocess

import pytest

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(os.path.dirname(HERE), "fp8_precision_rl_amd", "csrc")


def walk(tmp_path, *flags):
    exe = tmp_path / "walk"
    subprocess.run(["g++", "-std=c++17", "-O2", "-Wall", "-Werror", *flags, "-I", CSRC, "-o", str(exe),
                    os.path.join(HERE, "join_indices_driver.cpp")], check=True)
    return subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)


@pytest.mark.skipif(shutil.which("g++") is None, reason="needs g++")
def test_parts_of_a_row(tmp_path):
    r = walk(tmp_path)
    assert r.returncode == 0 and " 0 wrong" in r.stdout, r.stdout
    planted = walk(tmp_path, "-DUNBOUNDED")
    assert planted.returncode == 1 and "513 blocks, 576 recorded: part 71 of 66" in planted.stdout, planted.stdout


def test_the_kernels_take_records_through_the_bound():
    """A unit's record is read in three places: counted (and checked) by the shared part, bounded by the other two."""
    with open(os.path.join(CSRC, "jetfp8_attention.hip")) as f:
        uses = re.findall(r".*a\.prefix\[.*", f.read())
    assert len(uses) == 3
    assert sum("join_shared(u.block, a.prefix[unit].z)" in u for u in uses) == 2
