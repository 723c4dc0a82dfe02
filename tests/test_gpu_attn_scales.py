"""cr_attn_kv8 with value scales of a sequence far apart, and rows whose weight lies on one page.

Every page's keys point along a dim of their own (the page's number), so a row with a large entry
there weighs that page alone.  Tolerance of one output, summed over the keys j that the row
sees (p_j relative to the largest, l their sum, half steps of fp16 2^-11 and, below 2^-14, 2^-25):
  sum_j max(2^-11 p_j, min(p_j, 2^-25)) |V_j| / l   P in fp16, at least as large as p_j;
  2^-12 A                     FP32: sums over up to 2560 keys (2^-12.7), scores (arguments up to 2^9:
                              2^-15 of p), A = sum p_j |V_j| / l;
  u |o| + the type's smallest step   the output's rounding."""
import pytest
import torch

import rotated_bit_linear_amd as rbl
from helpers import dev, say
from kv8_ref import F8, PAGE, Batch, dense, random_cache

pytestmark = pytest.mark.gpu


def setup(scales, D, Hkv, seed, tail=0):
    """One sequence of a page per scale (the last one short by `tail` tokens): value codes of normal
    data, keys 1 along the page's dim."""
    n = len(scales)
    kv = n * PAGE - tail
    batch = Batch([1], [kv], seed=seed)
    cache = random_cache(batch.n_pages, Hkv, D, seed + 1, spread=0)
    cache.k.zero_()
    cache.k_scale.fill_(1.0)
    one = torch.ones((), dtype=torch.float32).to(F8).view(torch.uint8).item()
    for p, s in enumerate(scales):
        i = batch.page(0, p)
        cache.k[i, :, :, p] = one
        if s == 0:                                        # a page of zeros, as the append writes it
            cache.v[i], cache.v_scale[i] = 0, 2.0 ** -126
        else:
            cache.v_scale[i] = s
    return batch, cache, kv


def reference(q, cache, batch, Hq, sm, causal, n):
    """(out, tolerance but for the output's rounding) [n, Hq, D]"""
    D, G, kv = cache.D, Hq // cache.Hkv, batch.kv[0]
    qd = q.double().cpu().view(n, Hq, D)
    out, tol = torch.zeros_like(qd), torch.zeros_like(qd)
    for r in range(Hq):
        k, v = dense(cache, batch, 0, r // G)
        s = (qd[:, r] @ k.T) * sm
        if causal:
            s = s.masked_fill(torch.ones(n, kv, dtype=torch.bool).triu(kv - n + 1), -float("inf"))
        p = torch.exp(s - s.amax(-1, keepdim=True))
        l = p.sum(-1, keepdim=True)
        lost = torch.maximum(2.0 ** -11 * p, p.clamp(max=2.0 ** -25))
        out[:, r], tol[:, r] = p @ v / l, (lost + 2.0 ** -12 * p) @ v.abs() / l
    return out, tol


def check(scales, D, few, causal, dtype=torch.bfloat16, strength=300.0, tail=0, Hkv=1):
    """Each row weighs one page (every page is some row's); few: one token, else enough for the other kernel."""
    n = len(scales)
    batch, cache, kv = setup(scales, D, Hkv, 40, tail)
    G = 4
    new = 3 if few else 40
    batch.new, batch.T = [new], new
    batch.cu = torch.tensor([0, new], dtype=torch.int32, device=dev())
    q = torch.zeros(new, Hkv * G, D)
    for i in range(new * Hkv * G):
        q.view(-1, D)[i, i % n] = strength
    q = q.to(dtype).view(new, -1).to(dev())
    say(f"scales {scales} D={D} few={few} causal={causal} {dtype}")
    got = rbl.attn_kv8(q, cache, batch.cu, batch.kv_lens, batch.table, new, kv, Hkv * G, sm_scale=1.0, causal=causal)
    torch.cuda.synchronize()
    ref, tol = reference(q, cache, batch, Hkv * G, 1.0, causal, new)
    f = torch.finfo(dtype)
    tol = tol * (1 + f.eps) + f.eps / 2 * ref.abs() + f.smallest_normal * f.eps
    err = (got.double().cpu().view_as(ref) - ref).abs()
    assert (err <= tol).all().item(), (err / tol).max().item()


SCALES = {
    "small after large": [1.0, 2.0 ** -26],
    "large after small": [2.0 ** -26, 1.0],
    "up and down": [1.0, 2.0 ** -20, 2.0 ** 10, 2.0 ** -40, 1.0, 2.0 ** -9],
    "zeros between": [2.0 ** -8, 0, 2.0 ** -8, 2.0 ** -30, 0, 2.0 ** 12],
    "no powers of two": [0.3, 3e-9, 7e5, 0.3, 1.7e-12],
    "very far": [2.0 ** 50, 2.0 ** -40, 2.0 ** 50, 2.0 ** -40],
    "all of the range": [2.0 ** -90, 1.0, 2.0 ** 90, 1.0, 2.0 ** -90],
}


@pytest.mark.parametrize("scales", list(SCALES))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_weigh_one_page(scales, D, few, causal):
    check(SCALES[scales], D, few, causal, tail=5 if causal else 0)


@pytest.mark.parametrize("few", [True, False])
@pytest.mark.parametrize("strength", [20.0, 12.0, 6.0])
def test_rows_that_weigh_other_pages_a_little(few, strength):
    """Weights of e^-20 to e^-6 beside scales 2^26 apart: both sides of what counts."""
    for scales in ("small after large", "large after small", "up and down", "no powers of two"):
        check(SCALES[scales], 64, few, False, strength=strength)


@pytest.mark.parametrize("few", [True, False])
def test_fp16_outputs(few):
    check([1.0, 2.0 ** -12, 2.0 ** 3, 2.0 ** -16], 128, few, False, dtype=torch.float16)


def test_scales_far_apart_over_split_caches():
    """The same with the cache split into runs: single tokens, and a few row blocks, over 40 pages."""
    for few in (True, False):
        scales = [2.0 ** ((-26, 0, 7, -40)[i % 4]) for i in range(40)]
        new = 1 if few else 40
        assert rbl.cr_attn_kv8_workspace_bytes(new, 1, new, 40 * PAGE, 4, 1, 64) > 0
        check(scales, 64, few, False)
