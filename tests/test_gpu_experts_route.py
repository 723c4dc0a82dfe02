"""The router and the plan against plain references.

Choices are whole numbers and have to be equal.  The references compute scores in float64 as the kernel
does; the test's keys differ by far more than float64's roundings, or are equal.  Weights are computed
in float64 and rounded once: half a step of FP32 (2^-24 of the value, 2^-150 below its normal range),
and 2^-44 for the roundings before (fewer than 2^9 of them, of 2^-53 each)."""
import pytest
import torch

import experts_ref as ref
import rotated_bit_linear_amd as rbl
from helpers import dev, say

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def check(logits, **kw):
    k, bias = kw["k"], kw.get("bias")
    say(f"route {tuple(logits.shape)} {logits.dtype} " + " ".join(f"{a}={b}" for a, b in kw.items() if a != "bias") + f" bias={bias is not None}")
    ids, w = rbl.route_experts(logits.to(dev()) if not logits.is_cuda else logits, k,
                               bias=None if bias is None else bias.to(dev()), n_groups=kw.get("G", 1),
                               top_groups=kw.get("top_groups", 1), group_sum=kw.get("group_sum", 2),
                               sigmoid=kw.get("sigmoid", False), renorm=kw.get("renorm", True), scale=kw.get("scale", 1.0))
    torch.cuda.synchronize()
    want_ids, want_w = ref.route(logits, **kw)
    assert torch.equal(ids.cpu(), torch.from_numpy(want_ids)), (ids.cpu()[(ids.cpu() != torch.from_numpy(want_ids)).any(1)][:3])
    want = torch.from_numpy(want_w)
    off = (w.cpu().double() - want).abs() - (want.abs() * (2.0 ** -24 + 2.0 ** -44) + 2.0 ** -150)
    assert not w.isnan().any() and off.max().item() <= 0, off.max().item()


def logits(T, E, seed, dtype=torch.float32, coarse=False):
    g = torch.Generator().manual_seed(seed)
    x = 2 * torch.randn(T, E, generator=g)
    return (torch.round(x) / 2 if coarse else x).to(dtype)   # coarse: many equal


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (5, 60, 4), (3, 65, 32), (130, 256, 8), (7, 257, 6), (4, 512, 32),
                                   (33, 8, 8), (2001, 128, 1)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_sizes(T, E, k, sigmoid):
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(3))
    for i, dt in enumerate((torch.bfloat16, torch.float16, torch.float32)):
        check(logits(T, E, 10 * E + i, dt), k=k, sigmoid=sigmoid, renorm=i != 1, scale=1.0 if i else 2.5)
        check(logits(T, E, 11 * E + i, dt), k=k, sigmoid=sigmoid, renorm=i == 1, bias=bias, scale=-0.3)


@pytest.mark.parametrize("E,G,top,k", [(256, 8, 4, 8), (60, 4, 1, 15), (64, 64, 9, 9), (512, 2, 1, 8), (12, 3, 2, 5),
                                       (510, 51, 7, 32)])
@pytest.mark.parametrize("sigmoid", [False, True])
def test_groups(E, G, top, k, sigmoid):
    bias = 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(4))
    for m in (1, 2):
        for b in (None, bias):
            check(logits(70, E, E + m), k=k, G=G, top_groups=top, group_sum=m, sigmoid=sigmoid, bias=b)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_ties_go_to_the_lower_index(sigmoid):
    flat = torch.zeros(3, 64)
    flat[1, ::2] = -0.0
    for G, top in ((1, 1), (8, 3)):
        check(flat, k=8, G=G, top_groups=top, sigmoid=sigmoid)
        check(flat, k=8, G=G, top_groups=top, sigmoid=sigmoid, bias=torch.zeros(64))
        check(logits(200, 64, 5, torch.bfloat16, coarse=True), k=8, G=G, top_groups=top, group_sum=1, sigmoid=sigmoid)
        check(logits(200, 256, 6, torch.float16, coarse=True), k=8, G=G, top_groups=top, group_sum=1, sigmoid=sigmoid)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_masked_infinite_and_extreme_logits(sigmoid):
    x = logits(12, 64, 7)
    x[0] = -INF                                        # nothing to choose
    x[1] = NAN
    x[2, 3:] = -INF                                    # fewer than k
    x[3, ::3] = NAN
    x[4, 10:20] = INF
    x[5] = torch.finfo(torch.float32).min              # the type's lowest value is a number
    x[6, :] = torch.finfo(torch.float32).min
    x[6, 17] = 1.0
    x[7] = 1000 * x[7]
    x[8, 5] = torch.finfo(torch.float32).max
    x[9] = 200 + torch.arange(64.0)                    # sigmoid: all scores round to 1
    x[10] = -800 - torch.arange(64.0)                  # sigmoid: all scores 0 in float64
    x[11, 8:16] = -INF                                 # a whole group
    bias = 0.1 * torch.randn(64, generator=torch.Generator().manual_seed(8))
    bias[40] = -INF
    bias[41] = NAN
    for kw in (dict(), dict(renorm=False), dict(G=8, top_groups=2), dict(G=8, top_groups=2, group_sum=1)):
        check(x, k=8, sigmoid=sigmoid, **kw)
    for kw in (dict(), dict(renorm=False), dict(G=8, top_groups=2), dict(G=8, top_groups=8)):
        check(x, k=8, sigmoid=sigmoid, bias=bias, **kw)
    for dt in (torch.bfloat16, torch.float16):
        y = logits(4, 64, 9, dt)
        y[0, 2:] = torch.finfo(dt).min
        y[1, 5] = torch.finfo(dt).max
        check(y, k=8, sigmoid=sigmoid)


@pytest.mark.parametrize("sigmoid", [False, True])
def test_groups_whose_sum_cancels_or_overflows(sigmoid):
    """Biases against which FP32 loses the scores in a group's sum, or the sum itself.  Groups' values are apart
    by the scores' differences: far more than float64's roundings of 2^20 (2^-32) and of 1e38 (biases alone)."""
    steps = torch.randint(0, 4, (8,), generator=torch.Generator().manual_seed(21)) / 16
    cancel = torch.stack([torch.full((8,), 2.0 ** 20), -2.0 ** 20 + steps, torch.full((8,), -2.0 ** 21)], 1).flatten()
    over = torch.tensor([[3.0, 2.0], [2.9, 2.9], [3.1, 0.5], [2.2, 2.1], [3.3, -1.0], [1.0, 1.0], [2.8, 2.7], [0.0, 3.2]]).flatten() * 1e38
    for k, top in ((2, 1), (4, 3)):
        check(logits(70, 24, 22), k=k, G=8, top_groups=top, sigmoid=sigmoid, bias=cancel)
        check(logits(70, 16, 23), k=k, G=8, top_groups=top, sigmoid=sigmoid, bias=over)


def test_strides_and_unaligned_rows():
    x = logits(9, 80, 12, torch.bfloat16).to(dev())
    check(x[:, 3:67], k=8)
    check(x[1:, :61], k=5, sigmoid=True)


# ------------------------------------------------------------------------------------- plan ----

@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (63, 1, 5), (13, 5, 60), (128, 8, 512), (129, 8, 512), (512, 8, 64), (1024, 8, 64),
                                   (1025, 8, 64), (4097, 1, 9), (8193, 1, 511), (2500, 32, 256), (20000, 8, 64), (100000, 6, 8)])
def test_plan(T, k, E):
    for seed, none, first, local in ((1, 0.0, 0, E), (2, 0.3, E // 3, max(1, E // 2))):
        ids, _ = ref.random_choices(T, k, E, seed, dev(), none=none, repeats=True)
        say(f"plan T={T} k={k} E={E} experts {first}..{first + local - 1}")
        offsets, rows = rbl.experts_plan(ids, local, first=first)
        torch.cuda.synchronize()
        flat = ids.flatten().cpu() - first
        flat = torch.where((flat < 0) | (flat >= local), local, flat)
        order = flat.sort(stable=True).indices.int()
        n = torch.bincount(flat, minlength=local + 1)[:local].cumsum(0)
        assert offsets.tolist() == [0] + n.tolist()
        order[int(n[-1]):] = -1
        assert torch.equal(rows.cpu(), order)


def test_plan_of_odd_ids():
    ids = torch.tensor([[-2 ** 31, 2 ** 31 - 1, 5, 5], [7, 4, 12, 5], [-1, 100, 11, 4]], dtype=torch.int32, device=dev())
    say("plan of ids out of range and repeated")
    offsets, rows = rbl.experts_plan(ids, 8, first=4)
    want = ref.plan(ids, 8, first=4)
    assert offsets.tolist() == want[0] and rows.tolist() == want[1]
    offsets, rows = rbl.experts_plan(ids, 3, first=200)
    assert offsets.tolist() == [0] * 4 and rows.tolist() == [-1] * 12
    offsets, rows = rbl.experts_plan(ids[:0], 3)
    assert offsets.tolist() == [0] * 4 and rows.numel() == 0
