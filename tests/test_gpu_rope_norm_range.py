"""The per-head RMS norm of cr_rope_append_kv8 for heads whose squares FP32 does not hold, against
64 bits; tolerances as derived in test_gpu_rope_cache.py (the move by a power of two rounds nothing)."""
import pytest
import torch

import rotated_bit_linear_amd as rbl
from helpers import dev, say
from kv8_ref import F8, Batch, random_cache, scale_for
from test_gpu_rope_cache import E32, check_codes, inputs, reference

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("power", [-115, -80, -60, -40, 40, 62, 64, 100, 120])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("il", [False, True])
def test_heads_far_from_one(power, D, il):
    Hq, Hkv, eps, dtype = 3, 2, 0.0, torch.bfloat16
    batch = Batch([5, 1], [5, 9], seed=80)
    x, pos, w, freq, axis = inputs(batch, Hq, Hkv, D, dtype, 1, 81)
    x = x.clone()
    x[:, : (Hq + Hkv) * D] = x[:, : (Hq + Hkv) * D] / 32 * 2.0 ** power   # |x| below 2^5 before
    cache = random_cache(batch.n_pages, Hkv, D, 82)
    cache.k_scale.fill_(2.0 ** -30)
    cache.v_scale.fill_(2.0 ** -30)
    say(f"rope norm of heads around 2^{power} D={D} il={il}")
    got = rbl.rope_append_kv8(x, cache, batch.cu, batch.kv_lens, batch.table, 5, Hq, pos, freq.to(dev()), axis.to(dev()),
                              q_weight=w[0], k_weight=w[1], eps=eps, interleaved=il)
    torch.cuda.synchronize()
    q, ql, k, kl, _ = reference(x, pos, w, freq, axis, Hq, Hkv, D, eps, il)
    u = torch.finfo(dtype).eps / 2
    err = (got.double().cpu().view_as(q) - q).abs()
    assert (err <= u * q.abs() + 32 * E32 * ql * (1 + 2 * u)).all().item()
    i = batch.page(0, 0)
    want = scale_for(k[:5].abs().amax((0, 2)))
    assert torch.equal(cache.k_scale[i].double().cpu(), want)
    codes = cache.k[i, :, :5].cpu().view(F8).double().transpose(0, 1)
    check_codes(codes, want[None, :, None], k[:5], 32 * E32 * kl[:5], "keys")
