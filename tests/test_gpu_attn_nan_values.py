"""A NaN code in a value reaches one element (its dim) of the rows that see its token, and nothing
else: every other element is, bit for bit, what it is with a zero in that place."""
import pytest
import torch

import rotated_bit_linear_amd as rbl
from helpers import dev, say
from kv8_ref import PAGE, Batch, random_cache
from test_gpu_attn_kv8 import queries

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("new,past,Hq,Hkv", [(1, 129, 4, 2), (4, 700, 4, 1), (6, 90, 2, 2), (40, 100, 2, 1), (150, 2300, 2, 2),
                                             (130, 0, 8, 2)])
def test_nan_value_reaches_one_element(dtype, D, causal, new, past, Hq, Hkv):
    kv, G = past + new, Hq // Hkv
    batch = Batch([new], [kv], seed=30)
    cache = random_cache(batch.n_pages, Hkv, D, 31)
    q = queries(new, Hq, D, dtype, 32)
    # (token, head, dim): the last page, pages that some rows see in part, one that all see whole
    places = {(kv - 1, 0, D - 1), (kv - 1, Hkv - 1, 0), (max(0, kv - 1 - new // 2), 0, 7), (kv - 1 - new // 3, 0, 40),
              (0, Hkv - 1, 33), (kv // PAGE * PAGE - 1 if kv >= PAGE else 0, 0, 18)}
    def run():
        say(f"NaN values new={new} kv={kv} Hq={Hq} Hkv={Hkv} D={D} {dtype} causal={causal}")
        out = rbl.attn_kv8(q, cache, batch.cu, batch.kv_lens, batch.table, new, kv, Hq, causal=causal)
        torch.cuda.synchronize()
        return out.cpu().view(new, Hq, D)
    for t, h, d in places:
        cache.v[batch.page(0, t // PAGE), h, d, t % PAGE] = 0
    if kv % PAGE:                                         # beyond the cache: seen by nobody
        cache.v[batch.page(0, kv // PAGE), :, :, kv % PAGE:] = 0x7F
    clean = run()
    nan = torch.zeros(new, Hq, D, dtype=torch.bool)
    for t, h, d in places:
        cache.v[batch.page(0, t // PAGE), h, d, t % PAGE] = 0xFF if d % 2 else 0x7F
        first = max(0, t - past) if causal else 0
        nan[first:, h * G:(h + 1) * G, d] = True
    got = run()
    assert torch.isfinite(clean).all().item()
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], clean[~nan])
