"""The ring of copies that a CTA of the row-walking norm drains before it leaves
(csrc/ring.h), on the host: tests/ring_walk.cpp issues copies as the kernel does.

A barrier's wait for a parity passes when the phase that is under way has the
other one.  The last copy of a stage is its phase m - 1 (m copies went there), so
a wait that is worth anything names that phase's parity: any other passes while
the copy is still arriving, or waits for a phase that never comes."""
import os
import re
import shutil
import subprocess

import pytest

from _hbutil import ROOT

CSRC = os.path.join(ROOT, "chunked_prefill_decode_gb300", "csrc")


def test_a_cta_that_gives_up_waits_for_the_copies_it_issued(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("g++ not found")
    exe = str(tmp_path / "ring_walk")
    r = subprocess.run([gxx, "-std=c++17", "-Wall", "-Wextra", "-Werror", "-I", CSRC,
                        os.path.join(ROOT, "tests", "ring_walk.cpp"), "-o", exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    lines = subprocess.run([exe], capture_output=True, text=True, timeout=60).stdout.splitlines()
    assert len(lines) == sum(5 * (rows + 1) for rows in range(1, 25))
    for line in lines:
        head, parities = line.split(":")
        rows, stages, k, issued = map(int, head.split())
        # one copy more for each row that was read, as long as there are rows
        assert issued == min(rows, stages + k)
        copies = [0] * stages
        for i in range(issued):
            copies[i % stages] += 1
        assert [int(p) for p in parities.split()] == [(m - 1) & 1 for m in copies if m], line


def test_the_kernel_drains_by_that_count():
    with open(os.path.join(CSRC, "norm.cu")) as f:
        walk = f.read().split("norm_rows_kernel(", 1)[1].split("\n}\n", 1)[0]
    (drain,) = re.findall(r"for \(([^)]*(?:\(\))?[^)]*)\) drain_wait\(([^;]*)\);", walk)
    assert "ring.used()" in drain[0] and "ring.last_parity(s)" in drain[1]
    assert "RowRing ring(cfg.stages, n, k)" in walk
