"""What the attention entry points keep of a device (device_policy.h), compiled
with the host compiler and fed cases: no GPU is needed.

  * a kernel's settings are made once on every device that it runs on, not once
    in a process, and a setting that failed is tried again;
  * calls that make a cache's device current leave the caller's current again;
  * the append and prompt kernels choose their forms by the device's SMs.
"""
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
    exe = str(tmp_path_factory.mktemp("policy") / "device_policy_check")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-Werror",
                    "-I", os.path.join(ROOT, "paged_expert_cache_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "native", "device_policy_check.cpp"), "-o", exe], check=True)

    def run(lines):
        r = subprocess.run([exe], input="\n".join(lines) + "\n", capture_output=True, text=True, check=True)
        return r.stdout.split("\n")[:len(lines)]
    return run


def test_settings_are_made_on_every_device(policy):
    lines = ["once 0 0", "once 0 0", "once 1 0", "once 0 0", "once 1 0", "once 63 0", "once 63 0"]
    assert policy(lines) == ["1 0", "1 0", "2 0", "2 0", "2 0", "3 0", "3 0"]


def test_a_failed_setting_is_tried_again(policy):
    assert policy(["once 0 7", "once 0 7", "once 0 0", "once 0 7"]) == ["1 7", "2 7", "3 0", "3 0"]


def test_devices_past_the_table_are_set_each_time(policy):
    assert policy(["once 64 0", "once 64 0", "once -1 0"]) == ["1 0", "2 0", "3 0"]


def test_a_scope_gives_the_callers_device_back(policy):
    # current, the scope's, the one that cannot be set -> status, inside, after
    lines = ["scope 0 1 9", "scope 1 0 9", "scope 2 2 9", "scope 0 5 5", "scope -1 1 9"]
    assert policy(lines) == ["0 1 0", "0 0 1", "0 2 2", "101 0 0", "3 -1 -1"]


@pytest.mark.parametrize("sms", [152, 148, 76])
def test_forms_follow_the_sms(policy, sms):
    cases = {
        f"heads {16 * sms} {sms}": "1", f"heads {16 * sms - 1} {sms}": "0", f"heads {2 ** 40} {sms}": "1",
        f"halves {sms // 2} 64 5000 {sms}": "1", f"halves {sms // 2 + 1} 64 5000 {sms}": "0",
        f"halves {sms // 2} 128 10 {sms}": "1", f"halves {sms // 2 + 1} 128 999 {sms}": "0",
        f"halves {5 * sms // 2} 128 1000 {sms}": "1", f"halves {5 * sms // 2 + 1} 128 1000 {sms}": "0",
    }
    assert policy(list(cases)) == list(cases.values())
