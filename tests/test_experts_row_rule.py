"""The layer of experts' second product for one token has a workgroup for every choice and 128 columns: the rule
that takes it, on the host."""
import os
import subprocess

import pytest


def test_never_more_workgroups_than_a_dispatch_counts(tmp_path):
    hipcc = "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    here = os.path.dirname(os.path.abspath(__file__))
    exe = str(tmp_path / "experts_row_rule")
    subprocess.run([hipcc, "-x", "hip", "--offload-host-only", "-std=c++17", "-O1",
                    os.path.join(here, "native", "experts_row_rule.cpp"), "-o", exe], check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout
