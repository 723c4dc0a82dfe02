"""cr_rope_append_kv8 where a run is longer than max_new: the first max_new tokens are processed as
if the run ended there, and no other row of q_out and no other byte of the cache changes."""
import pytest
import torch

import rotated_bit_linear_amd as rbl
from helpers import dev, say
from kv8_ref import Batch, random_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_new,new,kv,Hkv", [(1, 64, 64, 1), (1, 64, 64, 8), (32, 64, 64, 3), (1, 130, 150, 5),
                                                (3, 64, 128, 3), (64, 200, 200, 2), (16, 17, 80, 3)])
@pytest.mark.parametrize("D", [64, 128])
def test_run_longer_than_max_new(max_new, new, kv, Hkv, D):
    Hq, other = 2, 1                                      # a second sequence with one new token
    batch = Batch([new, other], [kv, 70], seed=max_new + new, spare=8)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(batch.T, (Hq + 2 * Hkv) * D, generator=g).to(torch.bfloat16).to(dev())
    pos = torch.randint(0, 5000, (batch.T, 1), generator=g).int().to(dev())
    freq, axis = rbl.rope_table(D)
    start = random_cache(batch.n_pages, Hkv, D, 4)
    names = ("k", "v", "k_scale", "v_scale")
    cut, ref = (rbl.Kv8Cache(*(getattr(start, n).clone() for n in names)) for _ in range(2))
    say(f"append max_new={max_new} new={new} kv={kv} Hkv={Hkv} D={D}")
    out = torch.full((batch.T, Hq * D), 77.0, dtype=torch.bfloat16, device=dev())
    rbl.rope_append_kv8(x, cut, batch.cu, batch.kv_lens, batch.table, max_new, Hq, pos, freq, axis, out=out)
    torch.cuda.synchronize()
    # the same rows as a batch whose runs end there
    n = min(new, max_new)
    rows = torch.tensor(list(range(n)) + [new], device=dev())
    cu = torch.tensor([0, n, n + other], dtype=torch.int32, device=dev())
    lens = torch.tensor([kv - new + n, 70], dtype=torch.int32, device=dev())
    want = rbl.rope_append_kv8(x[rows], ref, cu, lens, batch.table, max(n, other), Hq, pos[rows], freq, axis)
    torch.cuda.synchronize()
    assert torch.equal(out[rows], want)
    rest = torch.ones(batch.T, dtype=torch.bool, device=dev())
    rest[rows] = False
    assert (out[rest] == 77.0).all().item()
    for name in names:
        assert torch.equal(getattr(cut, name), getattr(ref, name)), name
