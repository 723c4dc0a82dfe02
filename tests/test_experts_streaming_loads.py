"""The weighted sum reads rows that no cache holds past the caches: the compiled kernels for them load y so, the
others do not, from the device assembly that hipcc writes for the source."""
import os
import re
import subprocess

import pytest

from rotated_bit_linear_amd import build as B


@pytest.mark.skipif(not os.path.exists(B.HIPCC), reason="hipcc not available")
def test_loads_of_the_two_forms(tmp_path):
    out = str(tmp_path / "experts.s")
    flags = [f for f in B.FLAGS if f != "-fPIC"]
    subprocess.run([B.HIPCC, *flags, "-x", "hip", "--cuda-device-only", "-S", os.path.join(B.CSRC, "experts.hip"), "-o", out],
                   check=True, capture_output=True)
    forms = {}
    for m in re.finditer(r"^(_ZN\w*combine_kernelILi(\d)ELb([01])E\w*):.*?^\.Lfunc_end", open(out).read(), re.S | re.M):
        loads = re.findall(r"global_load_dwordx4 .*", m.group(0))
        forms[int(m.group(2)), m.group(3) == "1"] = len(loads), sum(" nt" in x for x in loads)
    assert sorted(forms) == [(t, past) for t in (0, 1, 2) for past in (False, True)]
    for (_, past), (loads, streaming) in forms.items():
        assert loads == 9                              # eight rows of y and the residual
        assert streaming == (8 if past else 0)
