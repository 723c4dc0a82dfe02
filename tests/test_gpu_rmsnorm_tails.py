"""cr_quant_act_rmsnorm at every length of a last segment, with rows after it and without: codes
and sums bit for bit, and nothing written past K."""
import pytest
import torch

import rotated_bit_linear_amd as rbl
from helpers import dev
from test_gpu_rmsnorm import DT, TP, check, rows

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("flags", [0, TP])
@pytest.mark.parametrize("tail", range(1, 17))
def test_tails(dtype, flags, tail):
    K = 512 + tail
    for M in (1, 5):
        x, r = rows(M, K, DT[dtype], tail), rows(M, K, DT[dtype], tail + 20, pad=1)
        w = (1 + 0.3 * torch.randn(K, generator=torch.Generator().manual_seed(3))).to(dev())
        check(x, r, w, 1e-6, flags=flags)
        check(x, None, w, 1e-6, flags=flags)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("K", [1, 7, 263, 509, 511])
def test_nothing_past_the_row(dtype, K):
    x, r = rows(4, K, DT[dtype], 1), rows(4, K, DT[dtype], 2)
    h = torch.full((4, K + 32 - K % 16), 5.0, dtype=DT[dtype], device=dev())
    check(x, r, None, 1e-6, sum_to=h[:, :K])
    assert (h[:, K:] == 5.0).all().item()
    w = torch.full((K + 16,), float("inf"), device=dev())        # past the weights: infinities
    w[:K] = 1.5
    check(x, r, w[:K], 1e-6)


@pytest.mark.parametrize("K", [200, 4111, 4600, 5000])
def test_many_rows_a_workgroup(K):
    """Every packing of rows, several rounds of each workgroup."""
    check(rows(3000, K, torch.bfloat16, 1), rows(3000, K, torch.bfloat16, 2), None, 1e-6)
