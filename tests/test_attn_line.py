"""The cut of attention's line of tiles into one part per CTA, checked on the
host (no GPU): a C++ program built from the plan kernel's own header
(moe_expert_cache_gb300/csrc/attn_line.cuh) checks, up to the longest plans
that the entry points accept, that every tile is in one CTA and that the join
looks for a row's pieces where they are.  See the program's header for the
list."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_tile_has_one_cta(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = tmp_path / "attn_line_check"
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-I", os.path.join(ROOT, "moe_expert_cache_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "csrc", "attn_line_check.cpp"), "-o", str(exe)],
                   check=True, capture_output=True, text=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
