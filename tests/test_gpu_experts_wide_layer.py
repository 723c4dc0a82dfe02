"""One token whose choices are all one expert, so wide that the choices' workgroups of the second product's own
form are more than a dispatch counts: the layer takes the other form.  Codes and sums are whole numbers and the
roundings the same, so the bits are those of a layer of a few of the columns, which takes the first."""
import pytest
import torch

import rotated_bit_linear_amd as rbl
from helpers import dev, say

pytestmark = pytest.mark.gpu


def test_one_token_of_very_many_columns():
    k, K, F, N = 32, 256, 130, 1 << 26
    g = torch.Generator(dev()).manual_seed(3)
    say(f"layer, one token, {k} times one expert, {N} columns")
    codes = lambda *shape: torch.randint(0, 256, shape, generator=g, dtype=torch.uint8, device=dev()) & 0x77  # noqa: E731
    a = torch.randint(-127, 128, (1, K), generator=g, dtype=torch.int8, device=dev())
    ids = torch.zeros(1, k, dtype=torch.int32, device=dev())
    weights, sa = torch.rand(1, k, generator=g, device=dev()), torch.full((1,), 1e-3, device=dev())
    w1, s1 = codes(1, 2 * F, K // 2), torch.rand(1, 2 * F, generator=g, device=dev()) / 64
    w2, s2 = codes(1, N, 128), torch.rand(1, N, generator=g, device=dev()) / 64
    got = rbl.mlp_experts_w4a8(a, sa, ids, weights, w1, s1, w2, s2)
    few = torch.cat([torch.arange(100), N // 2 + torch.arange(-50, 50), N + torch.arange(-100, 0)]).to(dev())
    want = rbl.mlp_experts_w4a8(a, sa, ids, weights, w1, s1, w2[:, few].contiguous(), s2[:, few].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(got[:, few], want) and want.abs().max() > 0
