"""The experts' products and the weighted sum against 64-bit references, and against the dense W4A8 GEMM.

Sums of codes (CR_I32) are exact.  Otherwise the FP32 value is off by the rounding of the sum to FP32, of
two products and of the bias' addition: at most 4 half steps, 2^-22 of the magnitudes that are added; the
output type adds half a step (bf16 2^-8, fp16 2^-11 and 2^-25 below its normal range, FP32 none that is
not counted).  SwiGLU a sigma(a) b: a's error moves a sigma(a) by at most (1 + |a|) times its relative
error, the exponential and the four operations after it add at most 2^-21 (a degree-7 polynomial on
[-0.35, 0.35]: 6e-9; nine roundings), b's error comes on top.
The same bits as the dense GEMM's: no tolerance."""
import pytest
import torch

import experts_ref as ref
import rotated_bit_linear_amd as rbl
from helpers import dev, say

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 0.0}
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -149}


class Case:
    def __init__(self, T, k, E, N, K, seed=0, gather=True, bias=False, none=0.0, skew=1.0):
        self.k, self.E, self.N, self.K = k, E, N, K
        self.ids, self.weights = ref.random_choices(T, k, E, seed, dev(), none=none, skew=skew)
        self.S = T * k
        self.gather = k if gather else 0
        self.a, self.sa = ref.random_rows(T if gather else self.S, K, seed + 1, dev())
        self.w, self.sw = ref.random_weight(E, N, K, seed + 2, dev())
        self.bias = torch.randn(E, N, generator=torch.Generator().manual_seed(seed + 3)).to(dev()) if bias else None
        self.offsets, self.rows = ref.plan(self.ids, E)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev())  # noqa: E731
        self.d_offsets, self.d_rows = i32(self.offsets), i32(self.rows)

    def run(self, dtype, scatter=False, swiglu=False, out=None):
        say(f"product S={self.S} E={self.E} N={self.N} K={self.K} gather={self.gather} scatter={scatter} swiglu={swiglu} "
            f"bias={self.bias is not None} {dtype}")
        cols = self.N // 2 if swiglu else self.N
        if out is None:
            out = torch.full((self.S, cols), 7, dtype=dtype, device=dev())
        rbl.gemm_s8s4_experts(self.a, self.sa, self.w, self.sw, self.d_offsets, self.d_rows, self.k, bias=self.bias,
                              gather=self.gather > 0, scatter=scatter, swiglu=swiglu, out=out)
        torch.cuda.synchronize()
        return out

    def places(self, scatter):
        n = self.offsets[-1]
        return torch.tensor(self.rows[:n], dtype=torch.long) if scatter else torch.arange(n)

    def check(self, dtype, scatter=False, swiglu=False):
        got = self.run(dtype, scatter, swiglu).cpu()
        at = self.places(scatter)
        left = torch.ones(self.S, dtype=torch.bool)
        left[at] = False
        assert (got[left] == 7).all(), "rows of no expert were written"
        acc = ref.sums(self.a, self.w, self.offsets, self.rows, self.gather)
        if dtype == torch.int32:
            assert torch.equal(got[at].long(), acc)
            return
        v, size = ref.scaled(acc, self.sa, self.sw, self.bias, self.offsets, self.rows, self.gather)
        err = 2.0 ** -22 * size
        if swiglu:
            a, b, ea, eb = *v.chunk(2, 1), *err.chunk(2, 1)
            v = a * torch.sigmoid(a) * b
            # |d(a sigma)| <= (1 + |a|) sigma(a) |da|, of which sigma(a) may itself move by |da|
            err = ((1 + a.abs()) * torch.sigmoid(a + ea) * ea + 2.0 ** -21 * (a * torch.sigmoid(a)).abs()) * (b.abs() + eb) \
                + (a * torch.sigmoid(a)).abs() * eb + 2.0 ** -120
        err = err + (v.abs() + err) * HALF[dtype] + TINY[dtype]
        off = (got[at].double() - v).abs()
        assert got[at].isfinite().all() and (off <= err).all(), ((off - err).max().item(), (off / err).max().item())


SIZES = [(1, 1, 1, 1, 1), (1, 8, 64, 96, 512), (2, 3, 5, 33, 300), (17, 2, 4, 130, 1000), (64, 4, 16, 64, 256),
         (40, 6, 7, 47, 2900), (300, 2, 3, 272, 520), (1000, 1, 2, 300, 256), (700, 4, 8, 516, 768), (90, 32, 40, 20, 257), (2100, 4, 16, 1030, 512), (515, 1, 1, 4200, 256), (77, 8, 8, 768, 1280)]


@pytest.mark.parametrize("T,k,E,N,K", SIZES)
def test_sums_are_exact(T, k, E, N, K):
    Case(T, k, E, N, K).check(torch.int32)
    Case(T, k, E, N, K, seed=5, gather=False, none=0.2).check(torch.int32, scatter=True)


@pytest.mark.parametrize("T,k,E,N,K", SIZES)
def test_values(T, k, E, N, K):
    for i, dt in enumerate((torch.bfloat16, torch.float16, torch.float32)):
        Case(T, k, E, N, K, seed=10 * i, bias=i == 1, none=0.1 * i).check(dt, scatter=i == 2)
        Case(T, k, E, N, K, seed=10 * i + 5, bias=i != 1, gather=False).check(dt, scatter=i != 2)
        Case(T, k, E, 2 * N, K, seed=10 * i + 7, bias=i == 0).check(dt, swiglu=True, scatter=i == 1)


@pytest.mark.parametrize("steps", range(1, 10))
def test_every_length_and_number_of_rows(steps):
    """K of 1 to 9 blocks of 256 (the rings' depths and their ends) for experts of 1 to 150 rows."""
    for rows in ((1, 16, 17, 32), (33, 64, 65, 150), (0, 129, 3, 200)):
        c = Case(sum(rows), 1, 4, 150, 256 * steps, seed=60 + steps)
        ids = torch.repeat_interleave(torch.arange(4), torch.tensor(rows))
        ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(steps))].int()[:, None]
        c.ids = ids.to(dev())
        c.offsets, c.rows = ref.plan(c.ids, 4)
        c.d_offsets = torch.tensor(c.offsets, dtype=torch.int32, device=dev())
        c.d_rows = torch.tensor(c.rows, dtype=torch.int32, device=dev())
        c.check(torch.int32, scatter=True)
        c.check(torch.bfloat16, swiglu=True)


def test_uneven_experts():
    """One expert has nearly all rows, several have none, one has a single row."""
    for skew, T in ((0.0, 500), (4.0, 500), (12.0, 300)):
        c = Case(T, 2, 24, 160, 512, seed=21, skew=skew)
        say(f"rows of the experts: {torch.tensor(c.offsets).diff().tolist()}")
        c.check(torch.float32)
        c.check(torch.bfloat16, scatter=True)
        c.check(torch.bfloat16, swiglu=True)
    c = Case(30, 4, 9, 64, 256, none=1.0)               # nobody chose anybody
    assert c.offsets[-1] == 0
    c.check(torch.bfloat16)


@pytest.mark.parametrize("T,k", [(3, 4), (40, 4), (150, 4), (900, 4)])
def test_same_bits_as_the_dense_gemm(T, k):
    E, N, K = 6, 200, 1100
    c = Case(T, k, E, N, K, seed=31, bias=True)
    for dt in (torch.bfloat16, torch.float16, torch.float32):
        got, halves = c.run(dt), c.run(dt, swiglu=True)
        for e in range(E):
            lo, hi = c.offsets[e], c.offsets[e + 1]
            if lo == hi:
                continue
            at = torch.tensor(c.rows[lo:hi], device=dev()) // k
            want = torch.empty(hi - lo, N, dtype=torch.float32, device=dev())
            rbl.cr_gemm_s8s4_rowscale(c.a[at].contiguous(), c.sa[at].contiguous(), c.w[e], c.sw[e], want, bias=c.bias[e])
            assert torch.equal(got[lo:hi], want.to(dt))
            act = torch.empty(hi - lo, N // 2, dtype=torch.float32, device=dev())
            rbl.cr_swiglu(want, N // 2, act)
            assert torch.equal(halves[lo:hi], act.to(dt))


def test_strides_and_neighbouring_memory():
    """Padded rows of every operand; outputs whose rows and base are only element-aligned."""
    c = Case(45, 3, 5, 70, 600, seed=41)
    a = torch.full((45, 800), 99, dtype=torch.int8, device=dev())
    a[:, :768] = c.a
    w = torch.full((5, 75, 400), 0x77, dtype=torch.uint8, device=dev())
    w[:, :70, :384] = c.w
    want = c.run(torch.bfloat16, scatter=True)
    for shift, wide in ((0, 72), (1, 71), (3, 90), (2, 76)):
        full = torch.full((135 * wide + 8,), 7, dtype=torch.bfloat16, device=dev())
        out = full[shift:shift + 135 * wide].view(135, wide)[:, :70]
        say(f"product with padded operands, output rows of {wide} from element {shift}")
        rbl.gemm_s8s4_experts(a[:, :768], c.sa, w[:, :70, :384], c.sw, c.d_offsets, c.d_rows, 3, gather=True, scatter=True, out=out)
        assert torch.equal(out, want)
        assert (full[:shift] == 7).all() and (full[shift + 135 * wide:] == 7).all()
        assert (full[shift:shift + 135 * wide].view(135, wide)[:, 70:] == 7).all()


def test_plans_that_are_none():
    """Offsets and rows that no plan writes are not followed: nothing outside C's rows is touched, and places
    that do name rows still get them.  (The bounds are also walked on the CPU, test_abi_experts.py.)"""
    c = Case(16, 2, 4, 40, 256, seed=51)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=dev())  # noqa: E731
    want = c.run(torch.float32, scatter=True)
    rows = list(c.rows)
    rows[0], rows[5], rows[9] = -7, 2 ** 31 - 1, 32
    full = torch.full((34, 40), 7.0, device=dev())
    say("product with rows out of range")
    rbl.gemm_s8s4_experts(c.a, c.sa, c.w, c.sw, c.d_offsets, i32(rows), 2, gather=True, scatter=True, out=full[1:33])
    torch.cuda.synchronize()
    assert (full[0] == 7).all() and (full[33] == 7).all()
    for i, r in enumerate(c.rows):
        good = i not in (0, 5, 9)
        assert torch.equal(full[1 + r], want[r]) if good else (full[1 + r] == 7).all()
    for bad in ([0, 10, 5, 40, 32], [-3, 8, 16, 24, 2 ** 31 - 1], [32, 24, 16, 8, 0], [-2 ** 31, 0, 0, 0, 0]):
        full = torch.full((34, 40), 7.0, device=dev())
        say(f"product with offsets {bad}")
        rbl.gemm_s8s4_experts(c.a, c.sa, c.w, c.sw, i32(bad), c.d_rows, 2, gather=True, scatter=True, out=full[1:33])
        torch.cuda.synchronize()
        assert (full[0] == 7).all() and (full[33] == 7).all()


# ----------------------------------------------------------------------------- weighted sum ----

@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (1, 8, 5376), (64, 8, 96), (7, 5, 2101), (333, 9, 514), (3, 32, 4099)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_combine(T, k, N, dtype):
    """k fused multiply-adds, each off by at most half a step of FP32 of a partial sum, and the residual's
    addition: (k + 1) 2^-24 of the magnitudes' sum; then half a step of the output's type."""
    E = max(40, k)
    for seed, none, first, local, res in ((1, 0.0, 0, E, False), (2, 0.3, 10, 20, True)):
        ids, w = ref.random_choices(T, k, E, seed, dev(), none=none)
        g = torch.Generator().manual_seed(seed + 5)
        y = torch.randn(T * k, N, generator=g).to(dtype).to(dev())
        r = torch.randn(T, N, generator=g).to(dtype).to(dev()) if res else None
        here = (ids >= first) & (ids < first + local)
        y[~here.flatten()] = float("nan")               # not read
        say(f"combine T={T} k={k} N={N} {dtype} experts {first}..{first + local - 1}")
        out = rbl.experts_combine(y, w, ids, local, first=first, residual=r)
        torch.cuda.synchronize()
        wh = torch.where(here, w, 0.0).cpu().double()
        yh = torch.where(here.flatten()[:, None], y, 0.0).cpu().double().view(T, k, N)
        terms = [wh[:, j, None] * yh[:, j] for j in range(k)] + ([r.cpu().double()] if res else [])
        v, size = sum(terms), sum(t.abs() for t in terms)
        err = (k + 1) * 2.0 ** -24 * size
        err = err + (v.abs() + err) * max(HALF[dtype], 2.0 ** -24) + TINY[dtype]
        assert ((out.cpu().double() - v).abs() <= err).all()
        if res:
            inplace = rbl.experts_combine(y, w, ids, local, first=first, residual=r, out=r)
            assert torch.equal(inplace, out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_combine_strides(dtype):
    """Rows that allow accesses of 16, 8, 4 and 2 bytes give the same values and touch nothing else."""
    ids, w = ref.random_choices(11, 3, 8, 3, dev())
    src = torch.randn(33, 530, generator=torch.Generator().manual_seed(4)).to(dtype).to(dev())
    want = rbl.experts_combine(src[:, :520].contiguous(), w, ids, 8)
    for shift, wide in ((0, 528), (4, 524), (2, 522), (1, 523)):
        buf = torch.zeros(33 * wide + 8, dtype=dtype, device=dev())
        y = buf[shift:shift + 33 * wide].view(33, wide)[:, :520]
        y.copy_(src[:, :520])
        full = torch.full((11 * wide + 8,), 7, dtype=dtype, device=dev())
        out = full[shift:shift + 11 * wide].view(11, wide)[:, :520]
        say(f"combine with rows of {wide} from element {shift}, {dtype}")
        rbl.experts_combine(y, w, ids, 8, out=out)
        assert torch.equal(out, want)
        rest = full.clone()
        rest[shift:shift + 11 * wide].view(11, wide)[:, :520] = 7
        assert (rest == 7).all()


def test_infinities_and_nan_reach_their_own_element():
    ids, w = ref.random_choices(4, 2, 4, 9, dev())
    y = torch.randn(8, 64, generator=torch.Generator().manual_seed(1)).to(dev())
    clean = rbl.experts_combine(y, w, ids, 4)
    y[3, 5], y[4, 9] = float("nan"), float("inf")
    got = rbl.experts_combine(y, w, ids, 4)
    assert got[1, 5].isnan() and got[2, 9].isinf()
    same = got == clean
    same[1, 5] = same[2, 9] = True
    assert same.all()


def test_strides_of_one_expert_and_of_one_row():
    """Views in which the stride of the axis of one says nothing: one expert of rows that lie by row first, and
    experts of a single row each."""
    c = Case(20, 1, 1, 64, 512, seed=90, skew=0.0)
    by_row = torch.zeros(64, 3, 256, dtype=torch.uint8, device=dev())
    by_row[:, 1] = c.w[0]
    want = c.run(torch.bfloat16)
    c.w = by_row.transpose(0, 1)[1:2]
    assert torch.equal(c.run(torch.bfloat16), want)
    c = Case(20, 2, 6, 1, 512, seed=91)
    want = c.run(torch.bfloat16)
    c.w = c.w.as_strided((6, 1, 256), (256, 16, 1))
    assert torch.equal(c.run(torch.bfloat16), want)


@pytest.mark.parametrize("steps", range(1, 10))
def test_tiles_of_every_length(steps):
    """As above for more rows an expert on average than 88: tiles that end after 1, 64, 65 and 128 rows."""
    for rows in ((300, 0, 193, 64), (1, 513, 128, 320)):
        c = Case(sum(rows), 1, 4, 150, 256 * steps, seed=160 + steps, bias=True)
        ids = torch.repeat_interleave(torch.arange(4), torch.tensor(rows))
        c.ids = ids[torch.randperm(len(ids), generator=torch.Generator().manual_seed(steps))].int()[:, None].to(dev())
        c.offsets, c.rows = ref.plan(c.ids, 4)
        c.d_offsets = torch.tensor(c.offsets, dtype=torch.int32, device=dev())
        c.d_rows = torch.tensor(c.rows, dtype=torch.int32, device=dev())
        bias, c.bias = c.bias, None
        c.check(torch.int32, scatter=True)
        c.bias = bias
        c.check(torch.bfloat16, swiglu=True)


@pytest.mark.parametrize("swiglu", [False, True])
def test_more_tiles_than_run_at_once(swiglu):
    """Each XCD has more than 64 tiles (it walks K from the end for every second 64); the dense GEMM's bits."""
    T, k, E, N, K = 1700, 2, 3, 8300, 700
    c = Case(T, k, E, N, K, seed=95, skew=0.5)
    got = c.run(torch.float32, swiglu=swiglu)
    for e in range(E):
        at = torch.arange(c.offsets[e], c.offsets[e + 1], device=dev())
        t = c.d_rows[at].long() // k
        want = torch.empty(len(at), N, dtype=torch.float32, device=dev())
        rbl.cr_gemm_s8s4_rowscale(c.a[t].contiguous(), c.sa[t].contiguous(), c.w[e], c.sw[e], want)
        if swiglu:
            act = torch.empty(len(at), N // 2, dtype=torch.float32, device=dev())
            rbl.cr_swiglu(want, N // 2, act)
            want = act
        assert torch.equal(got[at], want)
