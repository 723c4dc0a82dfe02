"""The weighted sum over more rows than a cache holds (256 MiB), which it reads in another way: the bits of calls
over a part of the tokens each, which it reads in the usual one."""
import pytest
import torch

import experts_ref as ref
import rotated_bit_linear_amd as rbl
from helpers import dev, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,N,dtype", [(2200, 8, 8192, torch.bfloat16), (2100, 9, 8191, torch.float16),
                                         (3001, 32, 1027, torch.float32), (300007, 3, 200, torch.bfloat16)])
def test_same_bits_as_in_parts(T, k, N, dtype):
    ids, w = ref.random_choices(T, k, 40, 1, dev(), none=0.1)
    g = torch.Generator(dev()).manual_seed(2)
    y = torch.randn(T * k, N, generator=g, device=dev()).to(dtype)
    r = torch.randn(T, N, generator=g, device=dev()).to(dtype)
    assert y.nbytes > 256 << 20
    say(f"combine T={T} k={k} N={N} {dtype}, {y.nbytes >> 20} MiB")
    got = rbl.experts_combine(y, w, ids, 30, first=5, residual=r)
    step = T // 4 + 1
    for t in range(0, T, step):
        at = slice(t, min(T, t + step))
        part = rbl.experts_combine(y[t * k:at.stop * k], w[at], ids[at], 30, first=5, residual=r[at])
        assert torch.equal(got[at], part)
