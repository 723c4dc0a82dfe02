"""cr_attn_kv8 where scores, or the factors that make them, lie near the ends of FP32.

Tolerance: 2^-11 for P in fp16, 2^-12 for FP32's sums and scores (at most 128 keys), both of the
mean of |v| under p, and the output's half step."""
import pytest
import torch

import rotated_bit_linear_amd as rbl
from helpers import dev, say
from kv8_ref import F8, PAGE, Batch, random_cache

pytestmark = pytest.mark.gpu

NEW = [1, 40]                                             # one row block of either kernel


def check(batch, cache, q, p):
    """q the same for every row; p the weights of the keys, in FP64."""
    new, kv, D = q.shape[0], batch.kv[0], cache.D
    cu = torch.tensor([0, new], dtype=torch.int32, device=dev())
    got = rbl.attn_kv8(q, cache, cu, batch.kv_lens, batch.table, new, kv, q.shape[1] // D, sm_scale=1.0, causal=False)
    torch.cuda.synchronize()
    v = torch.cat([cache.v[i, 0].view(F8).double().cpu().t() * cache.v_scale[i, 0].double().cpu()
                   for i in (batch.page(0, n) for n in range(-(-kv // PAGE)))])[:kv]
    p = (p / p.sum())[:, None]
    ref, mag = (p * v).sum(0), (p * v.abs()).sum(0)
    tol = (2.0 ** -11 + 2.0 ** -12) * (1 + 2.0 ** -7) * mag + 2.0 ** -8 * ref.abs()
    err = (got.double().cpu().view(-1, D) - ref).abs()
    assert (err <= tol).all().item(), (err / tol).max().item()


@pytest.mark.parametrize("new", NEW)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("size", [2.0 ** 60, 2.0 ** 100, 2.0 ** 118])
def test_all_scores_far_below_zero(new, D, size):
    """Every score is -size * D: the keys share the row; with twice that on the second page, the first has it."""
    batch = Batch([1], [100], seed=70)
    cache = random_cache(batch.n_pages, 1, D, 71, spread=0)
    cache.k.fill_(torch.tensor(1.0).to(F8).view(torch.uint8).item())
    cache.k_scale.fill_(1.0)
    q = torch.full((new, D), -size, dtype=torch.bfloat16, device=dev())
    say(f"scores of {-size * D} new={new} D={D}")
    check(batch, cache, q, torch.ones(100, dtype=torch.float64))
    cache.k_scale[batch.page(0, 1)] = 2.0
    check(batch, cache, q, (torch.arange(100) < PAGE).double())


@pytest.mark.parametrize("new", NEW)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale", [2.0 ** -110, 2.0 ** -124, 2.0 ** -126, 2.0 ** -127])
def test_small_key_scales(new, D, scale):
    """Scores of 0 and 2 (of 1 for the last scale) from large queries on keys with the smallest scales."""
    batch = Batch([1], [PAGE], seed=72)
    cache = random_cache(batch.n_pages, 1, D, 73, spread=0)
    i = batch.page(0, 0)
    cache.k.zero_()
    cache.k[i, 0, ::3, 5] = torch.tensor(256.0).to(F8).view(torch.uint8).item()
    cache.k_scale.fill_(scale)
    top = min(2.0 ** 119, 2.0 ** -7 / scale)
    q = torch.zeros(new, D, dtype=torch.bfloat16, device=dev())
    q[:, 5] = top
    say(f"key scale {scale} new={new} D={D}")
    p = torch.ones(PAGE, dtype=torch.float64)
    p[::3] = torch.tensor(top * 256 * scale, dtype=torch.float64).exp()
    check(batch, cache, q, p)
