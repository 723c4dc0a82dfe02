"""The layer of experts on a device that holds some of them, with other experts' slots among its own, in both
forms of the products (by streams up to 88 slots an expert here, by tiles above); uneven and few wide experts;
and calls that repeat themselves bit for bit.

Codes and sums are whole numbers, and FP32 roundings the same for the same row: bits are compared, but for sums
of several devices' parts, where the residual and the partial sums are rounded in another order (half a step of
bf16, 2^-8, for each part of each row)."""
import pytest
import torch

import experts_ref as ref
import rotated_bit_linear_amd as rbl
from helpers import dev, say

pytestmark = pytest.mark.gpu


def choices(T, k, total, seed, none=0.05, repeats=False):
    return ref.random_choices(T, k, total, seed, dev(), none=none, repeats=repeats)


def dense(a, sa, w, sw, bias, dtype, swiglu):
    """One expert's rows by the dense GEMM."""
    out = torch.empty(len(a), len(w), dtype=torch.float32 if swiglu else dtype, device=dev())
    rbl.cr_gemm_s8s4_rowscale(a.contiguous(), sa.contiguous(), w, sw, out, bias=bias)
    if not swiglu:
        return out
    act = torch.empty(len(a), len(w) // 2, dtype=torch.float32, device=dev())
    rbl.cr_swiglu(out, len(w) // 2, act)
    return act.to(dtype)


@pytest.mark.parametrize("T,k,total,first,local", [(1500, 4, 16, 5, 3), (700, 2, 8, 7, 1), (130, 8, 12, 0, 9), (60, 4, 64, 40, 20)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_products_with_slots_elsewhere(T, k, total, first, local, dtype):
    N, K = 270, 700
    ids, _ = choices(T, k, total, T, repeats=True)
    offsets, rows = rbl.experts_plan(ids, local, first=first)
    want_offsets, want_rows = ref.plan(ids, local, first)
    assert offsets.tolist() == want_offsets and rows.tolist() == want_rows
    w, sw = ref.random_weight(local, N, K, 1, dev())
    listed = rows[:want_offsets[-1]].long()
    for gather, scatter, swiglu, with_bias in ((True, False, True, False), (True, True, False, False), (False, True, False, True),
                                               (False, False, True, True)):
        a, sa = ref.random_rows(T if gather else T * k, K, 2, dev())
        bias = torch.randn(local, N, generator=torch.Generator().manual_seed(3)).to(dev()) if with_bias else None
        say(f"product of experts {first}..{first + local - 1} of {total}, {T} x {k} slots ({T * k / local:.0f} an expert here, "
            f"{len(listed)} fall here), gather={gather} scatter={scatter} swiglu={swiglu} bias={with_bias} {dtype}")
        out = torch.full((T * k, N // 2 if swiglu else N), 7, dtype=dtype, device=dev())
        rbl.gemm_s8s4_experts(a, sa, w, sw, offsets, rows, k, bias=bias, gather=gather, scatter=scatter, swiglu=swiglu, out=out)
        at = listed if scatter else torch.arange(len(listed), device=dev())
        left = torch.ones(T * k, dtype=torch.bool, device=dev())
        left[at] = False
        assert (out[left] == 7).all()
        for e in range(local):
            i = torch.arange(want_offsets[e], want_offsets[e + 1], device=dev())
            if len(i):
                src = listed[i] // k if gather else i
                want = dense(a[src], sa[src], w[e], sw[e], None if bias is None else bias[e], torch.float32, swiglu)
                # with a bias the dense GEMM rounds the same FP32 value
                assert torch.equal(out[at[i]], want.to(dtype))
                if not swiglu:
                    assert torch.equal(out[at[i]], dense(a[src], sa[src], w[e], sw[e], None if bias is None else bias[e], dtype, False))


class Layer:
    def __init__(self, T, k, E, K, F, N, seed, dtype=torch.bfloat16, none=0.05, skew=1.0):
        self.k, self.F, self.N, self.dtype = k, F, N, dtype
        self.ids, self.weights = ref.random_choices(T, k, E, seed, dev(), none=none, skew=skew)
        self.a, self.sa = ref.random_rows(T, K, seed + 1, dev())
        self.w1, self.s1 = ref.random_weight(E, 2 * F, K, seed + 2, dev())
        self.w2, self.s2 = ref.random_weight(E, N, F, seed + 3, dev())
        self.residual = torch.randn(T, N, generator=torch.Generator().manual_seed(seed)).to(dtype).to(dev())

    def here(self, first, local):
        at = slice(first, first + local)
        return self.w1[at], self.s1[at], self.w2[at], self.s2[at]

    def __call__(self, first, local, **kw):
        kw = dict(dict(residual=self.residual), **kw)
        return rbl.mlp_experts_w4a8(self.a, self.sa, self.ids, self.weights, *self.here(first, local), first=first,
                                    out_dtype=self.dtype, **kw)

    def parts(self, first, local):
        w1, s1, w2, s2 = self.here(first, local)
        offsets, rows = rbl.experts_plan(self.ids, local, first=first)
        wide = torch.zeros(rows.numel(), -(-self.F // 8) * 8, dtype=self.dtype, device=dev())
        h = rbl.gemm_s8s4_experts(self.a, self.sa, w1, s1, offsets, rows, self.k, self.dtype, gather=True, swiglu=True,
                                  out=wide[:, :self.F])
        q, s = rbl.quant_act(h, self.F)
        y = rbl.gemm_s8s4_experts(q, s, w2, s2, offsets, rows, self.k, self.dtype, scatter=True)
        return rbl.experts_combine(y, self.weights, self.ids, local, first=first, residual=self.residual)


@pytest.mark.parametrize("T,k,E,bounds", [(1500, 4, 16, (0, 5, 8, 16)), (400, 2, 6, (0, 1, 6)), (90, 8, 32, (0, 4, 32))])
def test_layer_dealt_out(T, k, E, bounds):
    c = Layer(T, k, E, 512, 300, 200, seed=T)
    say(f"layer, {T} x {k} slots, {E} experts dealt out at {bounds}")
    whole, total, norm = c(0, E), None, 0
    assert torch.equal(whole, c.parts(0, E))
    for lo, hi in zip(bounds, bounds[1:]):
        part = c(lo, hi - lo)
        assert torch.equal(part, c.parts(lo, hi - lo))
        total = c(lo, hi - lo, residual=c.residual if total is None else total)
        norm = norm + part.double().norm(dim=1)
    assert ((total.double() - whole.double()).norm(dim=1) <= 2.0 ** -8 * (norm + whole.double().norm(dim=1))).all()
    none = rbl.mlp_experts_w4a8(c.a, c.sa, c.ids, c.weights, c.w1, c.s1, c.w2, c.s2, first=E, residual=c.residual)
    assert torch.equal(none, c.residual)


def test_a_workspace_of_nan_reaches_nothing():
    """Rows between the products that no slot here fills hold what the workspace held."""
    for T, local in ((1500, 3), (60, 3), (1, 3)):
        c = Layer(T, 4, 16, 512, 300, 200, seed=5)
        need = rbl.cr_mlp_experts_w4a8_workspace_bytes(T, 4, local, 300, 200, c.dtype)
        want = c.parts(5, local)
        for fill in (0xFF, 0x7F, 0):
            ws = torch.full((need,), fill, dtype=torch.uint8, device=dev())
            say(f"layer of {local} of 16 experts, T={T}, workspace of {fill:#x}")
            assert torch.equal(c(5, local, workspace=ws), want)


@pytest.mark.parametrize("T,skew", [(60, 12.0), (900, 12.0), (900, 4.0)])
def test_uneven_layer(T, skew):
    c = Layer(T, 2, 24, 512, 300, 200, seed=9, skew=skew)
    say(f"layer, T={T}, rows of the experts {torch.bincount(c.ids[c.ids >= 0].flatten(), minlength=24).tolist()}")
    assert torch.equal(c(0, 24), c.parts(0, 24))


@pytest.mark.parametrize("T", [1, 5, 70])
def test_few_wide_experts(T):
    c = Layer(T, 2, 8, 512, 14336, 520, seed=13)
    say(f"layer, 8 experts of 14336, T={T}")
    assert torch.equal(c(0, 8), c.parts(0, 8))


@pytest.mark.parametrize("T", [1, 64, 3000])
def test_repeats_itself(T):
    """The same call again, other calls between, gives the same bits."""
    cases = [Layer(T, 8, 64, 1024, 448, 1100, seed=s) for s in (1, 2)]
    say(f"layer, T={T}, twenty times on two inputs in turn")
    first = [c(0, 64).clone() for c in cases]
    for _ in range(20):
        for c, f in zip(cases, first):
            assert torch.equal(c(0, 64), f)
