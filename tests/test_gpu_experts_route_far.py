"""The router's sigmoid scores far below one.  1 / (1 + exp(-x)) is a number of float64 down to x of about -709.78,
where its exponential passes float64's range: experts with such logits have their order, and their shares of a
token's weight.

Tolerance: half a step of FP32 (2^-24 of the value, 2^-150 below its normal range) for the one rounding of a weight.
Before it, in float64: exponential, addition and division of each side 2^-51 in all, and 2^-51 once more where the
score lies below float64's normal range (from 5.5e-309 on it has 50 bits); sum, product and division 2^-49: within
2^-44 together.  Whole numbers have to be equal: the logits lie at least 2^-6 apart, or are equal."""
import pytest
import torch

import experts_ref as ref
import rotated_bit_linear_amd as rbl
from helpers import dev, say

pytestmark = pytest.mark.gpu


def check(x, k, bias=None, G=1, top_groups=1, group_sum=2, renorm=True):
    say(f"route {tuple(x.shape)} {x.dtype}, far sigmoids, k={k} G={G} bias={bias is not None} renorm={renorm}")
    ids, w = rbl.route_experts(x.to(dev()), k, bias=None if bias is None else bias.to(dev()), n_groups=G,
                               top_groups=top_groups, group_sum=group_sum, sigmoid=True, renorm=renorm)
    torch.cuda.synchronize()
    want_ids, want = ref.route(x, k, bias=bias, G=G, top_groups=top_groups, group_sum=group_sum, sigmoid=True, renorm=renorm)
    assert torch.equal(ids.cpu(), torch.from_numpy(want_ids))
    want = torch.from_numpy(want)
    assert ((w.cpu().double() - want).abs() <= want.abs() * (2.0 ** -24 + 2.0 ** -44) + 2.0 ** -150).all()
    return want


def rows(T, E, lo, hi, seed):
    """Logits of whole 64ths from lo to hi, in any order."""
    g = torch.Generator().manual_seed(seed)
    return torch.randint(round(lo * 64), round(hi * 64) + 1, (T, E), generator=g).float() / 64


@pytest.mark.parametrize("lo,hi", [(-709.0, -694.0), (-709.75, -708.5), (-700.0, -686.0), (-720.0, -700.0)])
@pytest.mark.parametrize("E,k", [(64, 8), (5, 5), (300, 32)])
def test_shares_of_tiny_scores(lo, hi, E, k):
    x = rows(40, E, lo, hi, E)
    want = check(x, k)
    assert (want.sum(1) > 0.999).any()
    check(x, k, renorm=False)
    x[:, 1] = 1.0                                       # beside one that is not tiny
    check(x, k)


@pytest.mark.parametrize("lo,hi", [(-709.0, -694.0), (-709.75, -708.5), (-720.0, -700.0)])
def test_order_of_tiny_keys(lo, hi):
    """A bias of zero for all: the keys are the scores, which FP32 holds as zeros."""
    x = rows(40, 64, lo, hi, 3)
    check(x, 8, bias=torch.zeros(64))
    check(x, 8, bias=torch.zeros(64), G=8, top_groups=3)
    check(x, 8, G=8, top_groups=3)
    check(x, 8, G=8, top_groups=3, group_sum=1)


def test_16_bit_logits():
    for dt in (torch.bfloat16, torch.float16):
        x = rows(20, 64, -709.0, -690.0, 5).to(dt)
        check(x, 8)
        check(x, 8, bias=torch.zeros(64))
