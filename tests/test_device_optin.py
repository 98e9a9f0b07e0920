"""The shared-memory limit of kernels above 48 KB is set on each device that
launches them (gated_group_rmsnorm_gb300/csrc/ggrn_optin.h): the rule, built
into a small C++ program and run on the CPU, and that no kernel goes round it."""
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "gated_group_rmsnorm_gb300", "csrc")


def test_rule(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no host C++ compiler")
    exe = str(tmp_path / "optin_test")
    r = subprocess.run([cxx, "-O1", "-std=c++17", "-Wall", "-Werror", "-I", CSRC,
                        os.path.join(ROOT, "tests", "c", "ggrn_optin_test.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "failures 0" in r.stdout


def test_no_limit_is_set_once_per_process():
    """cudaFuncSetAttribute acts on the current device: it stands behind a word
    with a bit for each device, never behind a once_flag."""
    seen = 0
    for name in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, name)) as fh:
            text = fh.read()
        for m in re.finditer(r"cudaFuncSetAttribute\(", text):
            seen += 1
            before = text[max(0, m.start() - 1200):m.start()]
            assert "call_once" not in before, name
            assert "once_per_device" in before or "opted_in" in before, name
    assert seen >= 2
