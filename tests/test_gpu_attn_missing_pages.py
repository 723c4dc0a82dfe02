"""cr_attn_kv8 where the table names no page: nothing of the page that is read in its place (page 0,
which may be another sequence's or nobody's) reaches a row.  The result is, bit for bit, what it is
with ordinary scales and codes in page 0."""
import math

import pytest
import torch

import rotated_bit_linear_amd as rbl
from helpers import dev, say
from kv8_ref import Batch, attention, random_cache
from test_gpu_attn_kv8 import queries, tolerance

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new", [1, 5, 70, 300])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("missing", [(0,), (3,), (0, 1, 4)])
def test_page_zero_is_not_seen(new, D, causal, missing):
    kv, Hq, Hkv = 300 + new, 4, 2
    batch = Batch([new], [kv], seed=20, spare=3)
    swap = int(batch.unused[0])                           # page 0 becomes nobody's
    t = batch.table_cpu
    t[t == 0] = swap
    for p in missing:
        t[0, p] = -1
    batch.table = t.to(dev())
    cache = random_cache(batch.n_pages, Hkv, D, 21)
    q = queries(new, Hq, D, torch.bfloat16, 22)
    outs = {}
    for s in (1.0, 2.0 ** 60, math.inf, math.nan):
        cache.k_scale[0] = s
        cache.v_scale[0] = s
        if s != 1.0:
            cache.k[0], cache.v[0] = 0x7F, 0xFF
        say(f"missing pages {missing} new={new} D={D} causal={causal}, page 0 scaled by {s}")
        outs[s] = rbl.attn_kv8(q, cache, batch.cu, batch.kv_lens, batch.table, new, kv, Hq, causal=causal)
        torch.cuda.synchronize()
    ref, mag, top = attention(q, cache, batch, Hq, D ** -0.5, causal)
    tol = tolerance(torch.bfloat16, ref, mag, top, batch.kv)
    assert ((outs[1.0].double().cpu().view_as(ref) - ref).abs() <= tol).all().item()
    for s, out in outs.items():
        assert torch.equal(out, outs[1.0]), s
