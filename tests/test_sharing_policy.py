"""The rules by which attention over common positions chooses its form
(device_policy.h), compiled with the host compiler: no GPU is needed. They are held to
what was measured where the sides differ by a tenth or more, and to their ends."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def policy(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path_factory.mktemp("policy") / "sharing_policy_check")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror", "-fsanitize=signed-integer-overflow", "-fno-sanitize-recover=all",
                    "-I", os.path.join(ROOT, "paged_expert_cache_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "native", "sharing_policy_check.cpp"), "-o", exe], check=True)

    def run(lines):
        r = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True)
        return r.stdout.split()
    return run


# (sequences, query heads, key heads, head_dim, positions): us with the common positions read once, and each sequence by itself
MEASURED = {
    (16, 32, 4, 128, 2451): (23.4, 15.2), (16, 32, 4, 128, 20000): (30.8, 42.2), (8, 32, 4, 128, 10000): (23.1, 19.5),
    (48, 32, 4, 128, 2451): (30.7, 25.9), (48, 32, 4, 128, 5000): (32.9, 37.2), (4, 16, 16, 64, 20000): (33.6, 26.5),
    (16, 16, 16, 64, 5000): (21.9, 29.0),
}


def test_sharing_is_taken_where_it_was_faster(policy):
    lines = [f"pays {n * hq // hkv} {n} {positions} {hkv} {d}" for n, hq, hkv, d, positions in MEASURED]
    assert policy(lines) == [str(int(shared < alone)) for shared, alone in MEASURED.values()]


def test_sharing_at_the_ends(policy):
    cases = {
        "pays 0 1 1000000 4 128": "0",  # no rows
        "pays 1 1 0 1 64": "0", "pays 1 1 16 1 64": "0",
        f"pays 1 1 {2 ** 22 - 1} 1 64": "0", f"pays 1 1 {2 ** 22} 1 64": "1",   # one row: 4 * 65536 cells
        "pays 1 100000 100 1 64": "0",   # more sequences than rows
        # as many units as a call may have (2^30 of 128 positions and 8 rows), by rows and by positions
        f"pays {2 ** 30 - 8} 1 100 1 128": "1", f"pays 8 1 {2 ** 37 - 256} 1 128": "1", f"pays 8 1 {2 ** 37 // 1024 - 256} 1024 128": "1",
    }
    assert policy(list(cases)) == list(cases.values())
    for heads in (1, 4):  # more rows, positions or heads never turn it off
        got = policy([f"pays {rows} {max(rows // 8, 1)} {positions} {heads} 128" for positions in (500, 5000, 50000, 500000)
                      for rows in (1, 8, 64, 512, 4096)])
        table = [got[i:i + 5] for i in range(0, 20, 5)]
        assert all(row == sorted(row) for row in table) and all(list(c) == sorted(c) for c in zip(*table))


def test_single_tiles(policy):
    cases = {
        "single 32 1 128": "1", "single 128 1 128": "1", "single 320 1 128": "1", "single 384 1 128": "1",  # one tile, or three
        "single 160 1 128": "0", "single 256 1 128": "0", "single 385 1 128": "0", "single 512 1 128": "0",
        "single 512 4 128": "1", "single 513 4 128": "0", "single 1536 4 128": "1",  # of a group on average
        "single 1 1 128": "1", f"single 7 {2 ** 31 - 1} 128": "1", f"single {2 ** 30} 1 128": "0",
    }
    assert policy(list(cases)) == list(cases.values())
