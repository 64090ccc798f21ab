"""The gated forms' work plan (csrc/plan.h) for any SM count, checked on the CPU
by a host program built from the plan header alone."""

import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "kernelized_linear_attention_phi_b200", "csrc")
BUILD = os.path.join(ROOT, "tests", "_build")


def test_gated_plans_cover_every_token_for_any_sm_count():
    os.makedirs(BUILD, exist_ok=True)
    exe = os.path.join(BUILD, "gated_plan_check")
    cmd = ["g++", "-std=c++17", "-O1", "-Wall", f"-I{CSRC}", f"-I{os.path.join(ROOT, 'include')}", "-I/usr/local/cuda/include",
           os.path.join(ROOT, "tests", "cuda", "gated_plan_check.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout[-4000:]
    assert r.stdout.strip().splitlines()[-1].startswith("checked ")
