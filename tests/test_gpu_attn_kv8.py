"""cr_attn_kv8 against attention in 64 bits, row by row.

Tolerance of one output, from the kernel's roundings (u = finfo(dtype).eps / 2, half a step):
  u * A          P is rounded to the type: each p is off by at most u, A = mean of |v| under p;
  u * |o|        the output's own rounding;
  2^-12 * A      FP32: the products' accumulation over up to 4096 keys (4096 * 2^-24), the
                 scores' (64-term sums, arguments up to 2^6: 2^-17 of p) and exp2's last bit;
  fp16 only: N * 2^-25 * 2^4 * max|v|, what p below 2^-14 loses (its spacing is 2^-24; the
                 value scales of a test differ by up to 2^4 from one another's)."""
import math

import pytest
import torch

import rotated_bit_linear_amd as rbl
from helpers import dev, say
from kv8_ref import DT, F8, PAGE, Batch, attention, dense, random_cache

pytestmark = pytest.mark.gpu


def tolerance(dtype, out, mag, top, kv):
    u = torch.finfo(dtype).eps / 2
    t = u * mag * (1 + 2 * u) + u * out.abs() + 2.0 ** -12 * mag
    return t + (max(kv + [0]) * 2.0 ** -21 * top if dtype == torch.float16 else 0) + 1e-30


def queries(T, Hq, D, dtype, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    t = torch.full((T, Hq * D + 8 * pad), float("nan"), dtype=dtype)
    t[:, : Hq * D] = torch.randn(T, Hq * D, generator=g).to(dtype)
    return t.to(dev())[:, : Hq * D]


def run(batch, cache, Hq, dtype, causal, seed=5, pad=0, sm=None, max_kv=None, max_q=None, q=None):
    q = queries(batch.T, Hq, cache.D, dtype, seed, pad) if q is None else q
    say(f"attn new={batch.new[:8]} kv={batch.kv[:8]} Hq={Hq} Hkv={cache.Hkv} D={cache.D} {dtype} causal={causal}")
    out = torch.full((batch.T, Hq * cache.D + 8 * pad), 77.0, dtype=dtype, device=dev())
    view = out[:, : Hq * cache.D]
    rbl.attn_kv8(q, cache, batch.cu, batch.kv_lens, batch.table, max_q or batch.max_q, max_kv or max(1, batch.max_kv),
                 Hq, sm_scale=sm, causal=causal, out=view)
    torch.cuda.synchronize()
    if pad:
        assert (out[:, Hq * cache.D:] == 77.0).all().item()
    return q, view


def check(batch, cache, Hq, dtype, causal, **kw):
    q, got = run(batch, cache, Hq, dtype, causal, **kw)
    ref, mag, top = attention(q, cache, batch, Hq, kw.get("sm") or cache.D ** -0.5, causal)
    err = (got.double().cpu().view_as(ref) - ref).abs()
    tol = tolerance(dtype, ref, mag, top, batch.kv)
    assert torch.isfinite(got).all().item()
    assert (err <= tol).all().item(), (err / tol).max().item()
    return got


HEADS = [(1, 1), (4, 4), (8, 2), (7, 1), (16, 1), (40, 2)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_single_tokens(dtype, D, Hq, Hkv):
    kv = [1, 2, 63, 64, 65, 127, 128, 129, 700, 0]
    batch = Batch([1] * len(kv), kv, seed=Hq + D)
    check(batch, random_cache(batch.n_pages, Hkv, D, 1), Hq, DT[dtype], True, pad=1)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("Hq,Hkv", [(2, 2), (6, 2), (7, 1)])
def test_prompts(dtype, D, causal, Hq, Hkv):
    """Ragged prompts; lengths around tiles and pages; rows that see nothing (more new tokens
    than cached ones, an empty cache); an empty sequence."""
    new, kv = [1, 37, 64, 130, 0, 65, 20, 9], [1, 37, 100, 130, 50, 400, 7, 0]
    batch = Batch(new, kv, seed=3)
    got = check(batch, random_cache(batch.n_pages, Hkv, D, 2), Hq, DT[dtype], causal, pad=2)
    if causal:
        at = batch.start[6]
        assert (got[at:at + 13] == 0).all().item()       # 20 new tokens, 7 cached: 13 rows see no key
    assert (got[batch.start[7]:] == 0).all().item()


@pytest.mark.parametrize("few", [True, False])
def test_long_cache_split(few):
    """One sequence over many pages: the cache is split into runs and joined."""
    new, kv, Hq, Hkv = (1, 4001, 4, 1) if few else (70, 4001, 2, 1)
    batch = Batch([new], [kv], seed=4)
    cache = random_cache(batch.n_pages, Hkv, 128, 3)
    assert rbl.cr_attn_kv8_workspace_bytes(new, 1, new, kv, Hq, Hkv, 128) > 0
    check(batch, cache, Hq, torch.bfloat16, True)
    # a workspace that holds anything, and a hint that is too short: the last run takes the rest
    check(batch, cache, Hq, torch.bfloat16, False, max_kv=1500)


@pytest.mark.parametrize("new", [1, 5, 16, 17, 32, 33, 100])
def test_row_counts_around_the_kernels_border(new):
    batch = Batch([new, max(1, new // 2)], [300 + new, new], seed=new)
    check(batch, random_cache(batch.n_pages, 1, 64, 4), 1, torch.float16, True)


def test_splits_change_nothing_visible():
    """Ragged lengths under one plan: sequences that end in the first run, in a middle one, in none."""
    kv = [4000, 10, 0, 2049, 64 * 20]
    batch = Batch([1] * 5, kv, seed=6)
    check(batch, random_cache(batch.n_pages, 2, 128, 5), 8, torch.bfloat16, True)
    batch = Batch([40, 3, 2, 1, 40], kv, seed=6)
    check(batch, random_cache(batch.n_pages, 1, 128, 5), 1, torch.bfloat16, True)


@pytest.mark.parametrize("new", [1, 50])
def test_large_scores(new):
    """Scores far apart: the running maximum moves by hundreds, and one key takes all."""
    batch = Batch([new], [500], seed=7)
    cache = random_cache(batch.n_pages, 1, 64, 6, spread=6)
    check(batch, cache, 2, torch.bfloat16, False, sm=2.0)


@pytest.mark.parametrize("new", [1, 50])
def test_value_scales_far_apart(new):
    batch = Batch([new], [700], seed=8)
    cache = random_cache(batch.n_pages, 1, 64, 7, spread=0)
    cache.v_scale.copy_(cache.v_scale * torch.exp2(torch.arange(batch.n_pages, device=dev()).float() * 7 - 40)[:, None])
    check(batch, cache, 2, torch.bfloat16, False)
    cache.v_scale.fill_(0.3)                              # any positive scale, not only powers of two
    cache.k_scale.fill_(0.007)
    check(batch, cache, 2, torch.bfloat16, False)


@pytest.mark.parametrize("new", [1, 3, 50])
@pytest.mark.parametrize("dtype", list(DT))
def test_garbage_beyond_the_cache(new, dtype):
    """Everything that no row may see is NaN: unused pages, and tokens past kv_len of the last pages."""
    batch = Batch([new, new], [130, 65 + new], seed=9)
    cache = random_cache(batch.n_pages, 2, 64, 8)
    cache.k[batch.unused.to(dev())] = 0x7F
    cache.v[batch.unused.to(dev())] = 0xFF
    for b in range(2):
        i, left = batch.page(b, (batch.kv[b] - 1) // PAGE), (batch.kv[b] - 1) % PAGE + 1
        cache.k[i, :, left:] = 0x7F
        cache.v[i, :, :, left:] = 0xFF
    check(batch, cache, 4, DT[dtype], True)


@pytest.mark.parametrize("new,Hq", [(6, 2), (40, 2), (150, 1)])
@pytest.mark.parametrize("where", ["k", "v"])
def test_nan_reaches_only_rows_that_see_it(new, Hq, where):
    """A NaN in one token: causal rows before it are exact, rows from it on are NaN."""
    batch = Batch([new], [100 + new], seed=10)
    cache = random_cache(batch.n_pages, 1, 64, 9)
    clean = attention(queries(new, Hq, 64, torch.bfloat16, 5), cache, batch, Hq, 0.125, True)
    bad = 100 + new - max(2, new // 3)                    # a position among the new tokens
    i, off = batch.page(0, bad // PAGE), bad % PAGE
    if where == "k":
        cache.k[i, 0, off, 7] = 0x7F
    else:
        cache.v[i, 0, 7, off] = 0xFF
    q, got = run(batch, cache, Hq, torch.bfloat16, True)
    got = got.double().cpu().view(new, Hq, 64)
    first = bad - 100                                     # index of the first row that sees it
    tol = tolerance(torch.bfloat16, *clean, batch.kv)
    assert ((got[:first] - clean[0][:first]).abs() <= tol[:first]).all().item()
    seen = got[first:] if where == "k" else got[first:, :, 7]
    assert torch.isnan(seen).all().item()


@pytest.mark.parametrize("new", [1, 70])
def test_bad_page_ids_are_seen_by_nobody(new):
    batch = Batch([new, new], [400, 300], seed=11)
    for b, p, v in ((0, 2, -1), (0, 4, batch.n_pages), (1, 0, 2 ** 31 - 1), (1, 4, -2 ** 31)):
        batch.table_cpu[b, p] = v
    batch.table = batch.table_cpu.to(dev())
    check(batch, random_cache(batch.n_pages, 2, 128, 10), 4, torch.bfloat16, False)


def test_lengths_beyond_the_table_and_bad_bounds():
    """kv_lens past the page table end at the table; sequences whose rows are out of order or
    past T get no output and read nothing."""
    batch = Batch([1, 1, 1], [128, 128, 128], seed=12, extra_columns=0)
    cache = random_cache(batch.n_pages, 1, 64, 11)
    q = queries(3, 2, 64, torch.bfloat16, 5)
    ref = attention(q, cache, batch, 2, 0.125, True)[0]
    batch.kv_lens = torch.tensor([2 ** 31 - 1, 128, -5], dtype=torch.int32, device=dev())
    _, got = run(batch, cache, 2, torch.bfloat16, True, q=q, max_kv=128)
    err = (got.double().cpu().view_as(ref) - ref).abs()
    assert (err[:2] <= 2 ** -6 * ref.abs().max()).all().item()
    assert (got[2] == 0).all().item()
    batch.kv_lens = torch.tensor([128, 128, 128], dtype=torch.int32, device=dev())
    batch.cu = torch.tensor([0, 1, 99, 3], dtype=torch.int32, device=dev())
    _, got = run(batch, cache, 2, torch.bfloat16, True, q=q)
    assert (got[1:] == 77.0).all().item()


def test_shared_pages_and_scales_of_zero():
    """Two sequences read the same pages (a shared prefix); a page of zeros with scale zero."""
    batch = Batch([1, 1], [128, 128], seed=13)
    batch.table_cpu[1] = batch.table_cpu[0]
    batch.table = batch.table_cpu.to(dev())
    cache = random_cache(batch.n_pages, 1, 64, 12)
    i = batch.page(0, 1)
    cache.k[i] = 0
    cache.v[i] = 0
    cache.k_scale[i] = 0
    cache.v_scale[i] = 0
    q = queries(1, 2, 64, torch.bfloat16, 5).repeat(2, 1)
    got = check(batch, cache, 2, torch.bfloat16, True, q=q)
    assert torch.equal(got[0], got[1])


def test_offsets_beyond_32_bits():
    """Pages whose bytes lie beyond 4 GiB of the cache."""
    Hkv, D = 8, 128
    n_pages = (1 << 32) // (Hkv * PAGE * D) + 64
    cache = rbl.Kv8Cache.empty(n_pages, Hkv, D)
    small = random_cache(4, Hkv, D, 13)
    batch = Batch([1], [200], seed=14)
    batch.table_cpu = torch.tensor([[n_pages - 1, 0, n_pages - 7, n_pages - 2]], dtype=torch.int32)
    batch.table = batch.table_cpu.to(dev())
    for j in range(4):
        i = batch.page(0, j)
        for name in ("k", "v", "k_scale", "v_scale"):
            getattr(cache, name)[i] = getattr(small, name)[j]
    check(batch, cache, 16, torch.bfloat16, True)


def test_another_stream_and_graph_replay():
    batch = Batch([1, 1], [3000, 500], seed=15)
    cache = random_cache(batch.n_pages, 2, 128, 14)
    q = queries(2, 8, 128, torch.bfloat16, 5)
    ref = run(batch, cache, 8, torch.bfloat16, True, q=q)[1].clone()
    ws = torch.empty(rbl.cr_attn_kv8_workspace_bytes(2, 2, 1, 3000, 8, 2, 128), dtype=torch.uint8, device=dev())
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call = lambda st=None: rbl.cr_attn_kv8(q, batch.cu, batch.kv_lens, 1, 3000, 8, cache, batch.table, 128 ** -0.5,  # noqa: E731
                                           out, ws, rbl.CR_FLAG_CAUSAL, stream=st)
    say("attn on another stream")
    call(side)
    side.synchronize()
    assert torch.equal(out, ref)
    g = torch.cuda.CUDAGraph()
    say("attn capture")
    with torch.cuda.graph(g):
        call()
    for i in range(3):
        out.fill_(7.0)
        ws.fill_(0x5A)
        torch.cuda.synchronize()
        say(f"attn replay {i}")
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


def test_repeats_bit_for_bit():
    batch = Batch([33, 200], [2000, 2200], seed=16)
    cache = random_cache(batch.n_pages, 1, 128, 15)
    outs = [run(batch, cache, 4, torch.bfloat16, True)[1].clone() for _ in range(3)]
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
