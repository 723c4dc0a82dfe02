"""The append's walk over pages on the host (tests/native/kv8_append_walk.cpp): runs longer than
the launch's bound must not make a workgroup take more tokens than it holds."""
import os
import subprocess

import pytest

HIPCC = "/opt/rocm/bin/hipcc"
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.mark.skipif(not os.path.exists(HIPCC), reason="hipcc not available")
def test_walk(tmp_path):
    exe = str(tmp_path / "walk")
    subprocess.run([HIPCC, "-x", "hip", "--offload-host-only", "-std=c++17", "-O1",
                    os.path.join(HERE, "native", "kv8_append_walk.cpp"), "-o", exe], check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout
