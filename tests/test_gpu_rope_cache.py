"""cr_rope_append_kv8 against 64-bit norm, rotation and coding.

Tolerances (e32 = 2^-24): a rotated FP32 value carries the roundings of the norm (sum of D squares,
root, reciprocal, two products: below 16 e32 of the value in all), of cosine and sine (2 ulp and
the angle's 2^-25 turns: 8 e32 of the pair's length) and of the combination (2 e32): 32 e32 of the
pair's length.  Queries: that and u |q|.  Codes: half a step of E4M3 (2^-4 of the value, or 2^-10
of the page's scale below its normal range) and that, a value next to a border counts either way.
Scales are powers of two: equal.  Older codes after a growth: equal to decoding, dividing, coding."""
import pytest
import torch

import rotated_bit_linear_amd as rbl
from helpers import dev, say
from kv8_ref import DT, F8, PAGE, Batch, norm, random_cache, rotate, scale_for

pytestmark = pytest.mark.gpu

E32 = 2.0 ** -24


def inputs(batch, Hq, Hkv, D, dtype, axes, seed, pad=0, weights=True, far=False):
    g = torch.Generator().manual_seed(seed)
    W = (Hq + 2 * Hkv) * D
    x = torch.full((batch.T, W + 8 * pad), float("nan"), dtype=dtype)
    x[:, :W] = (torch.randn(batch.T, W, generator=g) * torch.exp2(torch.randint(-3, 4, (batch.T, 1), generator=g).float())).to(dtype)
    top = 2 ** 31 - 1 if far else 5000
    pos = torch.randint(0, top, (batch.T, axes + 1), generator=g).int()
    w = [(1 + 0.2 * torch.randn(D, generator=g)) if weights else None for _ in range(2)]
    sections = {1: [D // 2], 2: [D // 8, D // 4], 3: [D // 8, 3 * D // 16, 3 * D // 16], 4: [D // 8] * 4}[axes]
    freq, axis = rbl.rope_table(D, sections, device="cpu")
    return x.to(dev())[:, :W], pos.to(dev())[:, :axes], [None if t is None else t.to(dev()) for t in w], freq, axis


def reference(x, pos, w, freq, axis, Hq, Hkv, D, eps, il):
    y = x.double().cpu().view(x.shape[0], Hq + 2 * Hkv, D)
    cw = [None if t is None else t.cpu() for t in w]
    q, k, v = y[:, :Hq], y[:, Hq:Hq + Hkv], y[:, Hq + Hkv:]
    p = pos.cpu()
    q, k = norm(q, cw[0], eps), norm(k, cw[1], eps)
    def length(z):                                       # of each element's pair
        s = (z[..., 0::2] ** 2 + z[..., 1::2] ** 2).sqrt().repeat_interleave(2, -1) if il else \
            (z[..., : D // 2] ** 2 + z[..., D // 2:] ** 2).sqrt().repeat(1, 1, 2)
        return s
    return rotate(q, p, freq, axis, il), length(q), rotate(k, p, freq, axis, il), length(k), v


def check_codes(codes, scale, want, slack, what):
    """codes (E4M3 values), their scale, the exact values and how far FP32 may be off."""
    half = torch.maximum(2.0 ** -4 * want.abs(), 2.0 ** -10 * scale)
    err = (codes * scale - want).abs()
    assert (err <= half + slack * (1 + 2.0 ** -3)).all().item(), \
        (what, (err - half).max().item())


def check(batch, Hq, Hkv, D, dtype, axes=3, il=False, weights=True, seed=1, pad=0, far=False, eps=1e-6, cache=None,
          in_place=False, max_new=None):
    x, pos, w, freq, axis = inputs(batch, Hq, Hkv, D, dtype, axes, seed, pad, weights, far)
    cache = cache or random_cache(batch.n_pages, Hkv, D, seed + 50)
    before = [t.clone().cpu() for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    q, ql, k, kl, v = reference(x, pos, w, freq, axis, Hq, Hkv, D, eps, il)
    say(f"rope new={batch.new[:8]} kv={batch.kv[:8]} Hq={Hq} Hkv={Hkv} D={D} {dtype} axes={axes} il={il} far={far}")
    kept = x.clone()
    out = x[:, : Hq * D] if in_place else None
    got = rbl.rope_append_kv8(x, cache, batch.cu, batch.kv_lens, batch.table, max_new or batch.max_q, Hq, pos, freq.to(dev()),
                              axis.to(dev()), q_weight=w[0], k_weight=w[1], eps=eps, interleaved=il, out=out)
    torch.cuda.synchronize()
    if not in_place:
        assert torch.equal(x, kept)
    else:
        assert torch.equal(x[:, Hq * D:], kept[:, Hq * D:])
    u = torch.finfo(dtype).eps / 2
    err = (got.double().cpu().view_as(q) - q).abs()
    tiny = torch.finfo(dtype).smallest_normal * 2 * u
    assert (err <= u * q.abs() + 32 * E32 * ql * (1 + 2 * u) + tiny).all().item(), (err - u * q.abs()).max().item()
    # the cache
    ck, cv = cache.k.cpu(), cache.v.cpu()
    sk, sv = cache.k_scale.cpu(), cache.v_scale.cpu()
    touched = torch.zeros(batch.n_pages, PAGE, dtype=torch.bool)
    pages = torch.zeros(batch.n_pages, dtype=torch.bool)
    for b in range(batch.B):
        first, end, at = batch.kv[b] - batch.new[b], batch.kv[b], batch.start[b]
        if first < 0:
            continue
        while first < end:
            i, lo = batch.page(b, first // PAGE), first % PAGE
            m = min(PAGE - lo, end - first)
            if 0 <= i < batch.n_pages:
                touched[i, :lo + m] = True
                pages[i] = True
                for new, slack, codes, scale, old, old_scale, key in (
                        (k[at:at + m], 32 * E32 * kl[at:at + m], ck, sk, before[0], before[2], True),
                        (v[at:at + m], torch.zeros(m, Hkv, D), cv, sv, before[1], before[3], False)):
                    want = scale_for(torch.nan_to_num(new, 0.0, 0.0, 0.0).abs().amax((0, 2)))
                    if lo:
                        want = torch.maximum(want, old_scale[i].double())
                    assert torch.equal(scale[i].double(), want), (b, first)
                    c = codes[i].view(F8).double()
                    c = c if key else c.transpose(1, 2)              # [Hkv, token, D]
                    check_codes(c[:, lo:lo + m].transpose(0, 1), want[None, :, None], new.double(), slack, "new")
                    if lo:
                        o = old[i].view(F8).float()
                        o = o if key else o.transpose(1, 2)
                        o = (o[:, :lo] * (old_scale[i].double() / want).float()[:, None, None]).to(F8).double()
                        assert torch.equal(c[:, :lo], o)
            first, at = first + m, at + m
    # everything else is as it was
    assert torch.equal(ck.transpose(1, 2)[~touched], before[0].transpose(1, 2)[~touched])
    assert torch.equal(cv.permute(0, 3, 1, 2)[~touched], before[1].permute(0, 3, 1, 2)[~touched])
    assert torch.equal(sk[~pages], before[2][~pages]) and torch.equal(sv[~pages], before[3][~pages])
    return cache


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("il", [False, True])
@pytest.mark.parametrize("axes", [1, 2, 3, 4])
def test_prompts(dtype, D, il, axes):
    new, kv = [1, 64, 130, 0, 33, 200, 5], [1, 64, 130, 77, 100, 500, 128]
    check(Batch(new, kv, seed=axes), 5, 2, D, DT[dtype], axes, il, weights=axes % 2 == 1, pad=axes % 2)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (32, 8), (70, 2), (0, 2), (4, 40)])
def test_single_tokens(dtype, D, Hq, Hkv):
    kv = [1, 2, 63, 64, 65, 128, 129, 1000]
    check(Batch([1] * len(kv), kv, seed=2), Hq, Hkv, D, DT[dtype], 3, D == 64)


@pytest.mark.parametrize("new", [2, 3, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127])
def test_run_lengths(new):
    """Every number of tokens at a time, and runs that start inside a page."""
    check(Batch([new, 1, new], [new, 40, new + 37], seed=new), 3, 2, 128, torch.bfloat16)
    check(Batch([new, new - 1], [new + 63, new + 1], seed=new), 3, 2, 64, torch.bfloat16, max_new=new + 9)


def test_far_positions():
    check(Batch([70], [70], seed=3), 2, 1, 128, torch.float16, 2, far=True)


def test_queries_in_place():
    check(Batch([70, 3], [70, 66], seed=4), 4, 2, 128, torch.bfloat16, in_place=True)


@pytest.mark.parametrize("il", [False, True])
def test_append_grows_the_scale_and_repeats(il):
    """One token at a time, each larger: old codes are divided; a repeated call changes nothing."""
    Hq, Hkv, D = 2, 2, 64
    cache = None
    for t in range(1, 12):
        batch = Batch([1], [t], seed=5)
        if cache is None:
            cache = random_cache(batch.n_pages, Hkv, D, 3)
            cache.k_scale.fill_(2.0 ** -20)
            cache.v_scale.fill_(2.0 ** -20)
        check(batch, Hq, Hkv, D, torch.bfloat16, 1, il, weights=False, seed=20 + t, cache=cache)
    state = [x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    batch = Batch([1], [11], seed=5)
    x, pos, w, freq, axis = inputs(batch, Hq, Hkv, D, torch.bfloat16, 1, 31, weights=False)
    for _ in range(2):
        rbl.rope_append_kv8(x, cache, batch.cu, batch.kv_lens, batch.table, 1, Hq, pos, freq.to(dev()), axis.to(dev()),
                            interleaved=il)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(state, (cache.k, cache.v, cache.k_scale, cache.v_scale)))


def test_every_code_and_tie():
    """Values that are E4M3 numbers, midpoints between two and their neighbours, at scale 1 (448 is
    among them): the codes of round to nearest even, from torch's conversion."""
    grid = torch.arange(127, dtype=torch.uint8).view(F8).float()
    mid = (grid[1:] + grid[:-1]) / 2
    vals = torch.cat((grid, mid, mid * (1 + 2 ** -7), mid * (1 - 2 ** -8)))
    vals = torch.cat((vals, -vals)).to(torch.bfloat16)
    n = -(-vals.numel() // 64)
    rows = torch.full((n, 64), 448.0, dtype=torch.bfloat16)
    rows.view(-1)[: vals.numel()] = vals
    batch = Batch([n], [n], seed=6)
    cache = random_cache(batch.n_pages, 1, 64, 4)
    x = torch.cat((rows, rows, rows), 1).to(dev())
    freq, axis = torch.zeros(32, dtype=torch.float64, device=dev()), torch.zeros(32, dtype=torch.int32, device=dev())
    say("every code and tie")
    q = rbl.rope_append_kv8(x, cache, batch.cu, batch.kv_lens, batch.table, n, 1,
                            torch.ones(n, 1, dtype=torch.int32, device=dev()), freq, axis)
    torch.cuda.synchronize()
    assert torch.equal(q.cpu(), rows)                    # frequency 0 turns nothing
    want = rows.float().to(F8).view(torch.uint8)
    i = batch.page(0, 0)
    assert cache.k_scale[i, 0].item() == 1.0 and cache.v_scale[i, 0].item() == 1.0
    assert torch.equal(cache.k[i, 0, :n].cpu().view(F8).float(), want.view(F8).float())
    assert torch.equal(cache.v[i, 0, :, :n].cpu().t().contiguous().view(F8).float(), want.view(F8).float())


@pytest.mark.parametrize("amax,scale", [(448.0, 1.0), (450.0, 2.0), (224.0, 0.5), (0.0, 2.0 ** -126), (1e-38, 2.0 ** -126),
                                        (3e38, 2.0 ** 120)])
def test_page_scales(amax, scale):
    batch = Batch([3], [3], seed=7)
    cache = random_cache(batch.n_pages, 1, 64, 5)
    x = torch.zeros(3, 192, dtype=torch.bfloat16)
    x[1, 150] = -amax
    x[2, 70] = amax
    freq, axis = torch.zeros(32, dtype=torch.float64, device=dev()), torch.zeros(32, dtype=torch.int32, device=dev())
    say(f"page scale of {amax}")
    rbl.rope_append_kv8(x.to(dev()), cache, batch.cu, batch.kv_lens, batch.table, 3, 1,
                        torch.ones(3, 1, dtype=torch.int32, device=dev()), freq, axis)
    torch.cuda.synchronize()
    i = batch.page(0, 0)
    assert cache.k_scale[i, 0].item() == scale and cache.v_scale[i, 0].item() == scale
    for codes in (cache.k[i, 0, :3].cpu(), cache.v[i, 0, :, :3].cpu().t().contiguous()):
        got = codes.view(F8).double() * scale
        assert (got.abs().max() - float(x.double().abs().max())).abs().item() <= 2.0 ** -4 * float(x.double().abs().max()) + 2.0 ** -10 * scale


def test_non_finite_values_leave_the_others():
    batch = Batch([70], [70], seed=8)
    Hq, Hkv, D = 1, 2, 64
    x, pos, w, freq, axis = inputs(batch, Hq, Hkv, D, torch.bfloat16, 1, 9, weights=False)
    clean = random_cache(batch.n_pages, Hkv, D, 6)
    dirty = rbl.Kv8Cache(*(t.clone() for t in (clean.k, clean.v, clean.k_scale, clean.v_scale)))
    args = (batch.cu, batch.kv_lens, batch.table, 70, Hq, pos, freq.to(dev()), axis.to(dev()))
    say("non-finite values")
    rbl.rope_append_kv8(x, clean, *args)
    y = x.clone()
    y[5, Hq * D + 3] = float("inf")                       # key head 0, token 5
    y[66, (Hq + Hkv) * D + D + 9] = float("nan")          # value head 1, token 66
    rbl.rope_append_kv8(y, dirty, *args)
    torch.cuda.synchronize()
    i, j = batch.page(0, 0), batch.page(0, 1)
    a, b = clean.k.cpu().clone(), dirty.k.cpu()
    pair = [3, 3 + D // 2]
    bad = b[i, 0, 5].view(F8).float()
    assert torch.isnan(bad[pair]).any().item() and torch.isfinite(bad[[d for d in range(D) if d not in pair]]).all().item()
    a[i, 0, 5] = b[i, 0, 5]
    if clean.k_scale[i, 0] == dirty.k_scale[i, 0]:        # unless token 5 held the page's largest value
        assert torch.equal(a, b)
    av, bv = clean.v.cpu().clone(), dirty.v.cpu()
    assert torch.isnan(bv[j, 1, 9, 2].view(1).view(F8).float()).item()
    av[j, 1, 9, 2] = bv[j, 1, 9, 2]
    if clean.v_scale[j, 1] == dirty.v_scale[j, 1]:
        assert torch.equal(av, bv)


def test_infinite_values_are_nan_codes():
    """Infinities of both signs in a key and in values: NaN codes there, the page's scale from the rest."""
    batch = Batch([3], [3], seed=18)
    cache = random_cache(batch.n_pages, 1, 64, 16)
    x = torch.full((3, 192), 0.5, dtype=torch.float16)
    x[1, 64 + 5], x[2, 128 + 7], x[0, 128 + 63] = float("inf"), float("-inf"), float("inf")
    freq, axis = torch.zeros(32, dtype=torch.float64, device=dev()), torch.zeros(32, dtype=torch.int32, device=dev())
    say("infinite values")
    rbl.rope_append_kv8(x.to(dev()), cache, batch.cu, batch.kv_lens, batch.table, 3, 1,
                        torch.ones(3, 1, dtype=torch.int32, device=dev()), freq, axis)
    torch.cuda.synchronize()
    i = batch.page(0, 0)
    for codes, scale, bad in ((cache.k[i, 0, :3], cache.k_scale[i, 0], {(1, 5), (1, 37)}),
                              (cache.v[i, 0, :, :3].t().contiguous(), cache.v_scale[i, 0], {(2, 7), (0, 63)})):
        assert scale.item() == 2.0 ** -9                  # 0.5 / 2^-9 = 256, and 512 would exceed 448
        got = codes.cpu().view(F8).float() * scale.item()
        nan = {tuple(t) for t in torch.isnan(got).nonzero().tolist()}
        assert nan and nan <= bad and (got[~torch.isnan(got)] == 0.5).all().item()


def test_bad_pages_and_bounds_store_nothing():
    batch = Batch([70, 70, 5, 3], [70, 70, 5, 3], seed=10)
    batch.table_cpu[0, 1] = -1
    batch.table_cpu[1, 0] = batch.n_pages
    batch.table = batch.table_cpu.to(dev())
    batch.kv[2] = 4                                       # fewer cached than new tokens: nothing is stored
    batch.kv_lens = torch.tensor(batch.kv, dtype=torch.int32, device=dev())
    check(batch, 2, 2, 64, torch.bfloat16, 1)
    # tokens past the end of the table
    batch = Batch([200], [200], seed=11, extra_columns=0)
    batch.table_cpu = batch.table_cpu[:, :2].contiguous()
    batch.table = batch.table_cpu.to(dev())
    cache = random_cache(batch.n_pages, 1, 64, 7)
    before = cache.k.clone()
    x, pos, w, freq, axis = inputs(batch, 1, 1, 64, torch.bfloat16, 1, 12)
    say("tokens past the table")
    rbl.rope_append_kv8(x, cache, batch.cu, batch.kv_lens, batch.table, 200, 1, pos, freq.to(dev()), axis.to(dev()))
    torch.cuda.synchronize()
    changed = (cache.k != before).flatten(1).any(1).nonzero().flatten().tolist()
    assert sorted(changed) == sorted(batch.table_cpu[0].tolist())


def test_another_stream_and_graph_replay():
    batch = Batch([1, 1, 1], [10, 64, 65], seed=13)
    Hq, Hkv, D = 4, 2, 128
    x, pos, w, freq, axis = inputs(batch, Hq, Hkv, D, torch.bfloat16, 3, 14)
    freq, axis = freq.to(dev()), axis.to(dev())
    start = random_cache(batch.n_pages, Hkv, D, 8)
    caches = [rbl.Kv8Cache(*(t.clone() for t in (start.k, start.v, start.k_scale, start.v_scale))) for _ in range(2)]
    outs = [torch.empty(3, Hq * D, dtype=torch.bfloat16, device=dev()) for _ in range(2)]
    call = lambda i, st=None: rbl.cr_rope_append_kv8(x, batch.cu, batch.kv_lens, 1, Hq, w[0], w[1], 1e-6, pos, freq, axis,  # noqa: E731
                                                     outs[i], caches[i], batch.table, stream=st)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    say("rope eager, another stream")
    call(0)
    call(1, side)
    torch.cuda.synchronize()
    same = lambda: torch.equal(outs[0], outs[1]) and torch.equal(caches[0].k, caches[1].k) and \
        torch.equal(caches[0].v, caches[1].v) and torch.equal(caches[0].k_scale, caches[1].k_scale)  # noqa: E731
    assert same()
    g = torch.cuda.CUDAGraph()
    say("rope capture")
    with torch.cuda.graph(g):
        call(1)
    for i in range(3):
        for name in ("k", "v", "k_scale", "v_scale"):
            getattr(caches[1], name).copy_(getattr(start, name))
        outs[1].fill_(3.0)
        torch.cuda.synchronize()
        say(f"rope replay {i}")
        g.replay()
        torch.cuda.synchronize()
        assert same()
