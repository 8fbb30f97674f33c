"""How the warps of an attention kernel hand pieces of work on (piece_ring.h), with
host threads for warps: no GPU is needed.

  * without a stall all takers have every piece, and votes are the same to all;
  * where a wait gives up, no warp works on a piece that was not put, none is written
    over while it is in use, and all of them end.
"""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ring(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path_factory.mktemp("ring") / "piece_ring_check")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-pthread",
                    "-I", os.path.join(ROOT, "paged_expert_cache_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "native", "piece_ring_check.cpp"), "-o", exe], check=True)

    def run(pieces, who=-1, piece=0, ms=0):
        r = subprocess.run([exe], input=f"{pieces} {who} {piece} {ms}\n", capture_output=True, text=True, check=True, timeout=30)
        return tuple(int(v) for v in r.stdout.split())
    return run


@pytest.mark.parametrize("pieces", [0, 1, 2, 3, 40])
def test_all_pieces_are_taken_by_all(ring, pieces):
    taken, gave_up, faults = ring(pieces)
    assert faults == 0 and (gave_up or taken == pieces)


@pytest.mark.parametrize("who", [0, 1, 7, 12, 15])  # the putter, takers, voters
@pytest.mark.parametrize("piece", [0, 1, 2, 5])
def test_a_wait_that_gives_up_ends_all(ring, who, piece):
    taken, gave_up, faults = ring(9, who, piece, 300)
    assert gave_up == 1 and faults == 0
    assert taken <= piece + 2
