"""The rings between the row-parameter warp and the softmax of the tensor-memory cache
attention, against every order of tiles that short and long items give (tests/cache_rings.cc)."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "attention_score_reduction_b200", "csrc")


@pytest.fixture(scope="module")
def lines(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    exe = str(tmp_path_factory.mktemp("rings") / "cache_rings")
    subprocess.run([cxx, "-std=c++17", "-O2", "-I" + CSRC,
                    os.path.join(ROOT, "tests", "cache_rings.cc"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    got = {}
    for line in r.stdout.splitlines():
        m = re.fullmatch(r"(fp8|int4) (128|256) lead (\d+) of (\d+), V (-?\d+) of ring (\d+), "
                         r"K (-?\d+) of ring (\d+)", line)
        got[m.group(1), int(m.group(2))] = [int(x) for x in m.groups()[2:]]
    return r.returncode, got


@pytest.mark.parametrize("d", [128, 256])
@pytest.mark.parametrize("fmt", ["fp8", "int4"])
def test_no_entry_is_overwritten_while_it_is_read(lines, fmt, d):
    rc, got = lines
    lead, lead_bound, v, v_ring, k, k_ring = got[fmt, d]
    assert lead <= lead_bound and v < v_ring and k < k_ring
    assert rc == 0


def test_the_walk_reaches_the_ends_of_items(lines):
    """4 bits, d = 256: an item's last two V tiles come together, so that V gets six tiles
    on, not five, and a ring of six entries is one short."""
    assert lines[1]["int4", 256][0] == 11
    assert lines[1]["int4", 256][2] == 6
