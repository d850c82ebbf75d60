"""The message of ssd_scan_status names every kind of launch that gave up a
wait: a reset clears them all.  (Its host code, compiled by itself.)"""
import pathlib
import shutil
import subprocess

import pytest

CSRC = pathlib.Path(__file__).resolve().parent.parent / "selective_state_space_05_gb300" / "csrc"

PROGRAM = r"""
#include "ssd_status.h"
#include <stdlib.h>
int main(int argc, char** argv) {
  char m[512];
  const bool any = ssd::status_message(atoi(argv[1]), atoi(argv[2]), m, atoi(argv[3]));
  printf("%d %s", any, m);
}
"""


@pytest.fixture(scope="module")
def message(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    d = tmp_path_factory.mktemp("status")
    (d / "m.cpp").write_text(PROGRAM)
    subprocess.run([cxx, "-std=c++17", "-I", str(CSRC), str(d / "m.cpp"), "-o", str(d / "m")],
                   check=True)

    def call(scan, linear, size=512):
        out = subprocess.run([str(d / "m"), str(scan), str(linear), str(size)], check=True,
                             capture_output=True, text=True).stdout
        return out[0] == "1", out[2:]
    return call


def test_both_are_named(message):
    assert message(0, 0) == (False, "")
    scan, linear = message(10, 0), message(0, 3)
    assert scan[0] and "scan launch" in scan[1] and "0xa" in scan[1] and "proj" not in scan[1]
    assert linear[0] and "projection" in linear[1] and "0x3" in linear[1]
    assert "scan" not in linear[1]
    any_, both = message(10, 3)
    assert any_ and both == scan[1] + "; " + linear[1] and len(both) < 512


def test_a_short_buffer_is_kept_to(message):
    for size in (1, 40, 200):
        any_, m = message(10, 3, size)
        assert any_ and len(m) == size - 1
