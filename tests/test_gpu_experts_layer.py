"""The layer of experts: its parts one after another give the same bits; the whole against 64 bits; captured,
on other streams, two at once, and with the experts dealt out.

Against 64 bits the middle rows' codes matter: where FP32 and float64 fall on two sides of a rounding, a row
of the middle moves by half a step of 16 bits, or a code by one.  The reference takes the same rounding
points in float64.  A middle element whose FP32 value is off by 2^-20 of itself lies that near a border of
its type's steps (2^-7 of itself apart in bf16) with a chance of 2^-12; it then moves its block of 256 by
2^-7 / 16 of itself, a fraction of a code step (a row's largest / 127).  So a small share of the rows has a
few codes off by one: a code's step is 1/127 of the row's largest, against which a row's output of K codes
is off by at most the flipped codes' number over the sum of all: below 2^-7 of the row's norm for fewer than
a tenth of the codes.  Tolerance: 2^-7 of each row's norm (each expert's row), and the output's rounding."""
import pytest
import torch

import experts_ref as ref
import rotated_bit_linear_amd as rbl
from helpers import dev, say

pytestmark = pytest.mark.gpu


class Layer:
    def __init__(self, T, k, E, K, F, N, dtype=torch.bfloat16, seed=0, bias=False, residual=True, none=0.0, local=None):
        self.T, self.k, self.E, self.K, self.F, self.N, self.dtype = T, k, E, K, F, N, dtype
        self.ids, self.weights = ref.random_choices(T, k, E, seed, dev(), none=none)
        self.a, self.sa = ref.random_rows(T, K, seed + 1, dev())
        self.w1, self.s1 = ref.random_weight(E, 2 * F, K, seed + 2, dev())
        self.w2, self.s2 = ref.random_weight(E, N, F, seed + 3, dev())
        g = torch.Generator().manual_seed(seed + 4)
        self.b1 = torch.randn(E, 2 * F, generator=g).to(dev()) if bias else None
        self.b2 = torch.randn(E, N, generator=g).to(dev()) if bias else None
        self.residual = torch.randn(T, N, generator=g).to(dtype).to(dev()) if residual else None

    def __call__(self, first=0, local=None, **kw):
        at = slice(first, first + (self.E if local is None else local))
        part = lambda x: None if x is None else x[at]  # noqa: E731
        kw = dict(dict(residual=self.residual), **kw)
        return rbl.mlp_experts_w4a8(self.a, self.sa, self.ids, self.weights, self.w1[at], self.s1[at], self.w2[at], self.s2[at],
                                    first=first, bias1=part(self.b1), bias2=part(self.b2), out_dtype=self.dtype, **kw)

    def parts(self):
        offsets, rows = rbl.experts_plan(self.ids, self.E)
        h = rbl.gemm_s8s4_experts(self.a, self.sa, self.w1, self.s1, offsets, rows, self.k, self.dtype, bias=self.b1, gather=True,
                                  swiglu=True, out=torch.zeros(self.T * self.k, -(-self.F // 8) * 8, dtype=self.dtype,
                                                               device=dev())[:, :self.F])
        q, s = rbl.quant_act(h, self.F)
        y = rbl.gemm_s8s4_experts(q, s, self.w2, self.s2, offsets, rows, self.k, self.dtype, bias=self.b2, scatter=True)
        return rbl.experts_combine(y, self.weights, self.ids, self.E, residual=self.residual)

    def exact(self):
        """(values, tolerance) in float64."""
        offsets, rows = ref.plan(self.ids, self.E)
        n = offsets[-1]
        v, _ = ref.scaled(ref.sums(self.a, self.w1, offsets, rows, self.k), self.sa, self.s1, self.b1, offsets, rows, self.k)
        a, b = v.chunk(2, 1)
        h = (a * torch.sigmoid(a) * b).to(self.dtype).double()
        z = torch.zeros(n, ref.pad(self.F), dtype=torch.float64)
        z[:, :self.F] = h
        z = (z.view(-1, 256) @ ref.hadamard()).view(n, -1)
        top = z.abs().amax(1)
        q = torch.round(z / torch.where(top > 0, top, 1)[:, None] * 127)
        y, _ = ref.scaled(ref.sums(q, self.w2, offsets, rows, 0), top / 127, self.s2, self.b2, offsets, rows, 0)
        y = y.to(self.dtype).double()
        t = torch.tensor(rows[:n], dtype=torch.long)
        w = self.weights.cpu().double().flatten()[t][:, None]
        out = torch.zeros(self.T, self.N, dtype=torch.float64) if self.residual is None else self.residual.cpu().double()
        out.index_add_(0, t // self.k, w * y)
        slack = torch.zeros(self.T, dtype=torch.float64).index_add_(0, t // self.k, (w * y).norm(dim=1))
        half = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}[self.dtype]
        return out, 2.0 ** -7 * slack + half * out.norm(dim=1)


SIZES = [(1, 1, 1, 1, 1, 1), (1, 8, 64, 512, 256, 300), (5, 2, 6, 700, 333, 90), (64, 1, 3, 256, 130, 70), (2, 32, 40, 300, 64, 33),
         (1, 4, 6, 700, 1793, 90), (1, 3, 5, 1300, 4096, 140), (1, 2, 5, 256, 4100, 130), (1, 2, 3, 16500, 300, 70), (64, 4, 8, 256, 520, 257), (300, 3, 5, 300, 200, 64),
         (1100, 2, 4, 512, 256, 128)]


@pytest.mark.parametrize("T,k,E,K,F,N", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_parts_and_exact(T, k, E, K, F, N, dtype):
    for seed, bias, residual, none in ((1, False, True, 0.0), (2, True, False, 0.2)):
        c = Layer(T, k, E, K, F, N, dtype, seed, bias, residual, none)
        say(f"layer T={T} k={k} E={E} K={K} F={F} N={N} {dtype} bias={bias} residual={residual} none={none}")
        got = c()
        assert torch.equal(got, c.parts())
        v, tol = c.exact()
        off = (got.cpu().double() - v).norm(dim=1)
        assert got.isfinite().all() and (off <= tol).all(), (off / tol).max().item()


def test_transposed_order_of_the_second_weight():
    g = torch.Generator().manual_seed(3)
    w2 = torch.randn(4, 96, 500, generator=g).to(torch.bfloat16).to(dev())
    outs = []
    for flags in (0, rbl.CR_FLAG_BLOCK_TRANSPOSED):
        c = Layer(33, 2, 4, 300, 500, 96, seed=4)
        c.w2, c.s2 = rbl.quant_experts_w4(w2, flags)
        say(f"layer, flags {flags}")
        outs.append(c(flags=flags))
    assert torch.equal(*outs)                           # the same codes in another order: the same sums


@pytest.mark.parametrize("T", [1, 3])
def test_rows_between_the_products_of_every_size(T):
    """Zero, tiny (below the codes' usual range) and large rows; one token prepares them in the second product."""
    for scale in (0.0, 1e-38, 1e-33, 1e-20, 1.0, 1e12):
        for dt in (torch.float32, torch.bfloat16):
            c = Layer(T, 4, 6, 512, 700, 100, dt, seed=12, residual=False)
            c.sa = torch.full_like(c.sa, 1e-4)
            c.s1 = c.s1 * scale ** 0.5
            say(f"layer T={T}, first product scaled by {scale}, {dt}")
            assert torch.equal(c(), c.parts())


def test_experts_dealt_out():
    """Two halves of the experts, the second adding to the first's output: the residual's place in the sum moves
    (FP32 additions in another order and one rounding more, 2^-8 of each row's parts)."""
    c = Layer(50, 4, 12, 256, 300, 200, seed=6)
    say("layer, experts dealt out")
    whole, part = c(), c(first=0, local=5)
    both = c(first=5, local=7, residual=part)
    norm = whole.double().norm(dim=1) + part.double().norm(dim=1)
    assert ((both.double() - whole.double()).norm(dim=1) <= 2.0 ** -8 * norm).all()
    out = rbl.mlp_experts_w4a8(c.a, c.sa, c.ids, c.weights, c.w1, c.s1, c.w2, c.s2, first=100, residual=c.residual)
    assert torch.equal(out, c.residual)                 # no choice falls here
    out = rbl.mlp_experts_w4a8(c.a, c.sa, c.ids, c.weights, c.w1, c.s1, c.w2, c.s2, first=100)
    assert (out == 0).all()


def test_in_place_and_empty():
    c = Layer(20, 3, 6, 256, 256, 128, seed=7)
    want = c()
    r = c.residual.clone()
    assert c(residual=r, out=r) is r and torch.equal(r, want)
    e = Layer(1, 3, 6, 256, 256, 128, seed=7)
    out = rbl.mlp_experts_w4a8(e.a[:0], e.sa[:0], e.ids[:0], e.weights[:0], e.w1, e.s1, e.w2, e.s2)
    assert out.shape == (0, 128)


def test_a_dirty_workspace_changes_nothing():
    c = Layer(70, 4, 9, 512, 300, 140, seed=8, none=0.3)
    need = rbl.cr_mlp_experts_w4a8_workspace_bytes(70, 4, 9, 300, 140, c.dtype)
    want = c()
    for fill in (0, 0xFF, 0x7F):
        ws = torch.full((need + 256,), fill, dtype=torch.uint8, device=dev())
        say(f"layer, workspace of {fill:#x}")
        assert torch.equal(c(workspace=ws[:need]), want)
        assert (ws[need:] == fill).all()


def test_graph_follows_new_choices():
    """One captured launch serves steps with other choices: counts live on the device.  Several replays, eager
    work between them, every replay against the eager call."""
    for T in (1, 40, 1200):
        c = Layer(T, 4, 16, 512, 256, 192, seed=9)
        x = torch.randn(T, 16, generator=torch.Generator().manual_seed(1)).to(dev())
        ids, weights = rbl.route_experts(x, 4)
        offsets_ws = torch.empty(max(1, rbl.cr_experts_plan_workspace_bytes(T, 4, 16)), dtype=torch.uint8, device=dev())
        ws = torch.empty(rbl.cr_mlp_experts_w4a8_workspace_bytes(T, 4, 16, 256, 192, c.dtype), dtype=torch.uint8, device=dev())
        out = torch.empty(T, 192, dtype=c.dtype, device=dev())

        def step():
            rbl.cr_route_experts(x, None, 1, 1, 2, 4, 1.0, ids, weights, rbl.CR_FLAG_ROUTE_RENORM)
            rbl.mlp_experts_w4a8(c.a, c.sa, ids, weights, c.w1, c.s1, c.w2, c.s2, residual=c.residual, out=out, workspace=ws)
            return rbl.experts_plan(ids, 16, workspace=offsets_ws)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            offsets, rows = step()
        for i in range(4):
            x.copy_(torch.randn(T, 16, generator=torch.Generator().manual_seed(20 + i)))
            say(f"layer, T={T}, replay {i}")
            graph.replay()
            torch.cuda.synchronize()
            got = out.clone(), ids.clone(), weights.clone(), offsets.clone(), rows.clone()
            c.ids, c.weights = rbl.route_experts(x, 4)
            want = (c(), c.ids, c.weights, *rbl.experts_plan(c.ids, 16))
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert torch.equal(a, b)


def test_two_streams_at_once():
    cases = [Layer(T, 4, 16, 1024, 512, 512, seed=30 + T) for T in (3, 700)]
    want = [c() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    say("two layers on two streams")
    outs = [[], []]
    for _ in range(10):
        for i, (c, s) in enumerate(zip(cases, streams)):
            with torch.cuda.stream(s):
                outs[i].append(c())
    torch.cuda.synchronize()
    for got, w in zip(outs, want):
        assert all(torch.equal(g, w) for g in got)


def test_norm_route_layer():
    """A block's second half as it is used: the residual stream's norm into INT8 rows, the router on the same
    stream, the layer, its sum added to the stream."""
    g = torch.Generator().manual_seed(11)
    T, K, E, k, F = 50, 512, 16, 4, 256
    x, r = (torch.randn(T, K, generator=g).to(torch.bfloat16).to(dev()) for _ in range(2))
    gain = (1 + 0.1 * torch.randn(K, generator=g)).to(dev())
    gate = (torch.randn(E, K, generator=g) * K ** -0.5).to(dev())
    w1 = rbl.quant_experts_w4((torch.randn(E, 2 * F, K, generator=g) * K ** -0.5).to(dev()))
    w2 = rbl.quant_experts_w4((torch.randn(E, K, F, generator=g) * F ** -0.5).to(dev()))
    say("norm, router, layer")
    q, s, h = rbl.quant_act_rmsnorm(x, gain, residual=r)
    ids, weights = rbl.route_experts((h.float() * gain) @ gate.t(), k)
    out = rbl.mlp_experts_w4a8(q, s, ids, weights, *w1, *w2, residual=h)
    # against the dense layers, expert by expert: the same codes and sums; 16-bit roundings of each part
    total = h.double()
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if len(t) == 0:
            continue
        up = torch.empty(len(t), 2 * F, dtype=torch.float32, device=dev())
        rbl.cr_gemm_s8s4_rowscale(q[t].contiguous(), s[t].contiguous(), w1[0][e], w1[1][e], up)
        act = torch.empty(len(t), F, dtype=torch.float32, device=dev())
        rbl.cr_swiglu(up, F, act)
        y = rbl.linear_w4a8(act.to(torch.bfloat16), w2[0][e], w2[1][e], F)
        total.index_add_(0, t, weights[t, j].double()[:, None] * y.double())
    off = (out.double() - total).abs()
    # FP32 sums of five terms, then half a step of bf16
    assert (off <= 2.0 ** -8 * total.abs() + 2.0 ** -20 * total.abs().max()).all(), off.max().item()


def test_odd_choices():
    """Repeated, negative and far choices, on a device that holds some of the experts; as the parts."""
    for T, k in ((7, 9), (13, 5), (1, 32), (64, 1)):
        c = Layer(T, k, 32, 256, 130, 70, seed=70 + T)
        g = torch.Generator().manual_seed(T)
        ids = torch.randint(-3, 42, (T, k), generator=g).int()
        ids[0, 0], ids[-1, -1] = 2 ** 31 - 1, -2 ** 31
        c.ids = ids.to(dev())
        say(f"layer, odd choices, T={T} k={k}")
        got = rbl.mlp_experts_w4a8(c.a, c.sa, c.ids, c.weights, c.w1, c.s1, c.w2, c.s2, first=4, residual=c.residual)
        offsets, rows = rbl.experts_plan(c.ids, 32, first=4)
        h = rbl.gemm_s8s4_experts(c.a, c.sa, c.w1, c.s1, offsets, rows, k, c.dtype, gather=True, swiglu=True,
                                  out=torch.zeros(T * k, 136, dtype=c.dtype, device=dev())[:, :130])
        q, s = rbl.quant_act(h, 130)
        y = rbl.gemm_s8s4_experts(q, s, c.w2, c.s2, offsets, rows, k, c.dtype, scatter=True)
        want = rbl.experts_combine(y, c.weights, c.ids, 32, first=4, residual=c.residual)
        assert torch.equal(got, want)
