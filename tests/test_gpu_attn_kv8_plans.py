"""cr_attn_kv8 under each way of sharing out its work: whole blocks next to blocks split over the
cache, and both forms of the join.  Against attention in 64 bits, a head at a time on the device.

Tolerance of one output (A = mean of |v| under p; u = finfo(dtype).eps / 2; scales of a cache
with spread 0 lie within a factor of 2 of one another):
  2^-11 * A          P in fp16, half a step;
  u * |o|            the output's rounding;
  kv * 2^-24 * A     FP32 accumulation over the keys, P V and the sum alike: twice;
  2^-13 * A          the scores: 128 FP32 terms, sum of |q k| up to 2^7, times log2(e) / sqrt(D);
  kv * 2^-24 * top   what p below 2^-14 loses (half of 2^-24, times the scales' factor of 2)."""
import pytest
import torch

import rotated_bit_linear_amd as rbl
from helpers import dev, say
from kv8_ref import F8, PAGE, Batch, random_cache

pytestmark = pytest.mark.gpu


def check(batch, cache, Hq, dtype, causal, seed=1):
    D, G = cache.D, Hq // cache.Hkv
    q = torch.randn(batch.T, Hq * D, generator=torch.Generator().manual_seed(seed)).to(dtype).to(dev())
    say(f"attn new={batch.new} kv={batch.kv} Hq={Hq} Hkv={cache.Hkv} D={D} {dtype} causal={causal}")
    out = torch.full_like(q, 77.0)
    rbl.attn_kv8(q, cache, batch.cu, batch.kv_lens, batch.table, batch.max_q, batch.max_kv, Hq, causal=causal, out=out)
    torch.cuda.synchronize()
    u = torch.finfo(dtype).eps / 2
    for b in range(batch.B):
        n, kv, at = batch.new[b], batch.kv[b], batch.start[b]
        pages = batch.table[b, : -(-kv // PAGE)].long()
        hidden = torch.ones(n, kv, dtype=torch.bool, device=dev()).triu(kv - n + 1) if causal else None
        for r in range(Hq):
            h = r // G
            k = (cache.k[pages, h].view(F8).double() * cache.k_scale[pages, h].double()[:, None, None]).reshape(-1, D)[:kv]
            v = cache.v[pages, h].view(F8).double() * cache.v_scale[pages, h].double()[:, None, None]
            v = v.transpose(1, 2).reshape(-1, D)[:kv]
            s = q[at:at + n, r * D:(r + 1) * D].double() @ k.t().contiguous() * D ** -0.5
            p = torch.softmax(s if hidden is None else s.masked_fill(hidden, -float("inf")), -1)
            ref, mag = p @ v, p @ v.abs()
            tol = (2.0 ** -11 + 2.0 ** -13 + 2 * kv * 2.0 ** -24) * mag + u * ref.abs() + kv * 2.0 ** -24 * v.abs().max()
            err = (out[at:at + n, r * D:(r + 1) * D].double() - ref).abs()
            assert (err <= tol).all().item(), (b, r, (err / tol).max().item())


def cus():
    return torch.cuda.get_device_properties(0).multi_processor_count


def part_rows(batch, Hq, Hkv, D):
    """Rows of FP32 partial results in the workspace, (D + 2) * 4 bytes each."""
    need = rbl.cr_attn_kv8_workspace_bytes(batch.T, batch.B, batch.max_q, batch.max_kv, Hq, Hkv, D)
    assert need % ((D + 2) * 4) == 0
    return need // ((D + 2) * 4)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("D", [64, 128])
def test_whole_blocks_and_split_ones(D, causal):
    """A few blocks more than fill the device: those alone are split."""
    Hkv, slots = 4, (3 if D == 64 else 2) * cus()
    n = (slots // Hkv + 7) * 128 - 5
    batch = Batch([n], [2049], seed=1) if not causal else Batch([n], [n + 100], seed=1)
    rows = part_rows(batch, Hkv, Hkv, D)
    if not causal:
        tail = -(-n // 128) * Hkv - slots
        assert rows % (tail * 128) == 0 and 2 <= rows // (tail * 128) <= 4
    check(batch, random_cache(batch.n_pages, Hkv, D, 2, spread=0), Hkv, torch.bfloat16, causal)


def test_whole_blocks_and_split_ones_ragged():
    """The same with two sequences, one much shorter: blocks of either kind without rows or pages."""
    n = (cus() // 2 + 7) * 128
    batch = Batch([n, 700], [2049, 900], seed=3)
    assert part_rows(batch, 4, 2, 128) > 0
    check(batch, random_cache(batch.n_pages, 2, 128, 4, spread=0), 4, torch.float16, False)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,kv,per", [(1, 16 * 64, 16), (1, 6000, 16), (70, 2049, 128), (70, 6000, 128)])
def test_joins_of_few_and_of_many_runs(new, kv, per, D):
    batch = Batch([new], [kv], seed=5)
    runs = part_rows(batch, 2, 1, D) // (per * -(-2 * new // per))
    assert runs > 8 if kv == 6000 else 2 <= runs <= 8    # four waves a row, or one
    check(batch, random_cache(batch.n_pages, 1, D, 6, spread=0), 2, torch.bfloat16, True)
