"""The pieces of a row that the norms read element by element (row_piece.h), compiled
with the host compiler and its sanitizers: what they hold, and that nothing beside the
row is read and no word from where it may not lie. No GPU is needed."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_pieces_hold_the_row_and_nothing_else(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "row_piece_check")
    build = [cxx, "-std=c++17", "-O1", "-g", "-Wall", "-Wno-unknown-pragmas", "-Werror",
             "-I", os.path.join(ROOT, "paged_expert_cache_gb300", "csrc"),
             os.path.join(ROOT, "tests", "native", "row_piece_check.cpp"), "-o", exe]
    if "-Wcast-align=strict" in subprocess.run([cxx, "--help=warnings"], capture_output=True, text=True).stdout:
        build.insert(1, "-Wcast-align=strict")  # no word from an array of elements
    checks = ["-fsanitize=address,undefined", "-fno-sanitize-recover=all"]
    if subprocess.run(build + checks, capture_output=True).returncode != 0:  # a compiler without them
        subprocess.run(build, check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
    # rows of 1 .. 40, from two pieces before them to two pieces behind
    assert r.stdout.split() == [str(sum(n + 4 * per for n in range(1, 41))) for per in (8, 4)]
