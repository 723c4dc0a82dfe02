"""cr_attn_kv8 where numbers approach the ends of FP32: a result that is an average of values near
the top of the range, and scores that all lie far below zero."""
import pytest
import torch

import rotated_bit_linear_amd as rbl
from helpers import dev, say
from kv8_ref import F8, PAGE, Batch

pytestmark = pytest.mark.gpu


def make(kv, D, key=1.0, value=64.0, k_scale=1.0, v_scale=1.0):
    batch = Batch([1], [kv], seed=50)
    code = lambda x: torch.tensor(x).to(F8).view(torch.uint8).item()  # noqa: E731
    cache = rbl.Kv8Cache.empty(batch.n_pages, 1, D)
    cache.k.fill_(code(key))
    cache.v.fill_(code(value))
    cache.k_scale.fill_(k_scale)
    cache.v_scale.fill_(v_scale)
    return batch, cache


def run(batch, cache, new, q, Hq, sm, causal=False):
    cu = torch.tensor([0, new], dtype=torch.int32, device=dev())
    out = rbl.attn_kv8(q, cache, cu, batch.kv_lens, batch.table, new, batch.kv[0], Hq, sm_scale=sm, causal=causal)
    torch.cuda.synchronize()
    return out.double().cpu()


@pytest.mark.parametrize("new,kv", [(1, 50), (1, 300), (1, 6000), (40, 50), (40, 300), (70, 6000)])
@pytest.mark.parametrize("D", [64, 128])
def test_values_near_the_top_of_the_range(new, kv, D):
    """Every value is 2^126 (and 2^-126): so is every average, whatever number of keys it is over."""
    for scale in (2.0 ** 120, 2.0 ** -132):
        batch, cache = make(kv, D, v_scale=scale)
        q = torch.zeros(new, 2 * D, dtype=torch.bfloat16, device=dev())
        say(f"values of {64 * scale} new={new} kv={kv} D={D}")
        assert (run(batch, cache, new, q, 2, 1.0) == 64 * scale).all().item()
