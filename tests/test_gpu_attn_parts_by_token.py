"""cr_attn_kv8 where the parts of a split cache lie by token and head: a long run of queries among
short ones, so that blocks of the longest run would be many times the rows that there are.  Against
attention in 64 bits under the tolerance of the other plans."""
import random

import pytest
import torch

import rotated_bit_linear_amd as rbl
from helpers import dev, say
from kv8_ref import Batch, random_cache
from test_gpu_attn_kv8_plans import check

pytestmark = pytest.mark.gpu


def by_token(batch, Hq, Hkv, D):
    """Whether the parts' rows are a multiple of the batch's, more than 16 MiB of blocks otherwise."""
    rows = rbl.cr_attn_kv8_workspace_bytes(batch.T, batch.B, batch.max_q, batch.max_kv, Hq, Hkv, D) // ((D + 2) * 4)
    return rows > 0 and rows % (batch.T * Hq) == 0


def lengths(singles, new, kv, seed, empty=0):
    r = random.Random(seed)
    n = [1] * singles + [0] * empty
    k = [r.randint(1, kv) for _ in n]
    at = r.randrange(len(n) + 1)
    return n[:at] + [new] + n[at:], k[:at] + [kv] + k[at:]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("singles,new,kv,Hq,Hkv,D", [(23, 1500, 3000, 8, 2, 128), (40, 700, 2500, 3, 3, 64),
                                                     (150, 900, 1500, 2, 1, 64), (70, 400, 9000, 4, 1, 128)])
def test_prompt_among_single_tokens(singles, new, kv, Hq, Hkv, D, causal):
    n, k = lengths(singles, new, kv, singles, empty=5)
    batch = Batch(n, k, seed=60)
    assert by_token(batch, Hq, Hkv, D)
    check(batch, random_cache(batch.n_pages, Hkv, D, 61, spread=0), Hq, torch.bfloat16, causal)


def test_single_tokens_of_many_heads():
    """The kernel of few rows: 16 rows a block, of which each sequence has one."""
    r = random.Random(2)
    k = [r.randint(1, 6000) for _ in range(50)] + [6000]
    batch = Batch([1] * 51, k, seed=62)
    assert by_token(batch, 12, 12, 128)
    check(batch, random_cache(batch.n_pages, 12, 128, 63, spread=0), 12, torch.float16, True)


def test_tokens_of_no_sequence_and_bounds_out_of_order():
    """Rows that belong to no sequence keep what they hold; a sequence whose bounds are out of order
    counts as empty, and those after it still get their results."""
    n, k = lengths(23, 1500, 3000, 5)
    batch = Batch(n, k, seed=64)
    Hq, Hkv, D = 8, 2, 128
    cache = random_cache(batch.n_pages, Hkv, D, 65, spread=0)
    T = batch.T + 9                                       # rows past the last sequence
    q = torch.randn(T, Hq * D, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).to(dev())
    def run(cu):
        out = torch.full_like(q, 77.0)
        say("parts by token, rows of no sequence")
        rbl.attn_kv8(q, cache, cu, batch.kv_lens, batch.table, batch.max_q, batch.max_kv, Hq, out=out)
        torch.cuda.synchronize()
        return out
    whole = run(batch.cu)
    assert (whole[batch.T:] == 77.0).all().item() and not (whole[: batch.T] == 77.0).any().item()
    # a sequence of one token, of those before the last: its end is put before its start
    bad = next(b for b in range(3, batch.B - 2) if n[b] == n[b - 1] == n[b + 1] == 1)
    cu = batch.cu.clone()
    cu[bad] = -7                                          # ends sequence bad - 1, begins sequence bad
    got = run(cu)
    lost = [batch.start[bad - 1], batch.start[bad]]
    kept = [t for t in range(T) if t not in lost]
    assert (got[lost] == 77.0).all().item()
    assert torch.equal(got[kept], whole[kept])


def test_graph_and_repeats():
    n, k = lengths(23, 1500, 3000, 6)
    batch = Batch(n, k, seed=66)
    Hq, Hkv, D = 8, 2, 128
    cache = random_cache(batch.n_pages, Hkv, D, 67, spread=0)
    q = torch.randn(batch.T, Hq * D, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).to(dev())
    ws = torch.empty(rbl.cr_attn_kv8_workspace_bytes(batch.T, batch.B, batch.max_q, batch.max_kv, Hq, Hkv, D),
                     dtype=torch.uint8, device=dev())
    out = torch.empty_like(q)
    call = lambda: rbl.attn_kv8(q, cache, batch.cu, batch.kv_lens, batch.table, batch.max_q, batch.max_kv, Hq,  # noqa: E731
                                out=out, workspace=ws)
    say("parts by token, eager")
    call()
    torch.cuda.synchronize()
    ref = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(3):
        out.fill_(7.0)
        ws.fill_(0x5A)
        torch.cuda.synchronize()
        say(f"parts by token, replay {i}")
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
