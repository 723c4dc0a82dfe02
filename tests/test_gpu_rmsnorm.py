"""cr_quant_act_rmsnorm against the definition: the sum in the stream's type, the codes of the
CPU oracle's preparation of that sum with the weights as pre-scale (bit for bit: the row's
factor does not touch them), and the scale against FP64.

Scale tolerance: the oracle's FP32 scale (max |z| / 16 / 127, bit-exact here) times the FP32
rounding of the FP64 root.  Two right roots differ by at most one rounding (half a step each,
2 * 2^-24) and the product adds a rounding on each side (2 * 2^-24): 2^-22 relative."""
import numpy as np
import pytest
import torch

import oracle
import rotated_bit_linear_amd as rbl
from helpers import assert_bits_equal, dev, say

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
TP, BT = rbl.CR_FLAG_FORCE_TWO_PASS, rbl.CR_FLAG_BLOCK_TRANSPOSED
NAT_SCALE_TOL = 2.0 ** -22


def rows(M, K, dtype, seed, pad=0, gain=1.0):
    """[M, K] on the device with garbage (NaN) past K in every row's stride."""
    g = torch.Generator().manual_seed(seed)
    n = 16 // torch.empty(0, dtype=dtype).element_size()
    ld = (K + n - 1) // n * n + pad * n
    t = torch.full((M, ld), float("nan"), dtype=dtype)
    t[:, :K] = (torch.randn(M, K, generator=g) * gain).to(dtype)
    return t.to(dev())[:, :K]


def reference(x, r, w, eps):
    """(sum as FP32, codes, scale) on the CPU."""
    h = x.cpu().float() if r is None else (x.cpu().float() + r.cpu().float()).to(x.dtype).float()
    K = h.shape[1]
    pre = np.ones(K, np.float32) if w is None else w.cpu().numpy()
    q, s = oracle.quant_act(h.numpy(), oracle.DT_FP32, K, pre_scale=pre)
    ms = h.double().square().mean(1) + float(np.float32(eps))
    s = torch.from_numpy(s)
    return h, q, torch.where(s > 0, s.double() / ms.sqrt(), 0.0)


def untranspose(q):
    """Codes in block-transposed order back to natural order."""
    M, kp = q.shape
    return q.reshape(M, kp // 256, 16, 16).swapaxes(2, 3).reshape(M, kp)


def check(x, r, w, eps, flags=0, sum_to=None, what=""):
    h, q, s = reference(x, r, w, eps)
    say(f"rmsnorm {what} M={x.shape[0]} K={x.shape[1]} {x.dtype} residual={r is not None} flags={flags}")
    gq, gs, gh = rbl.quant_act_rmsnorm(x, w, eps, residual=r, sum=sum_to, flags=flags)
    torch.cuda.synchronize()
    got = gq.cpu().numpy()
    assert_bits_equal(untranspose(got) if flags & BT else got, q, "codes")
    err = ((gs.cpu().double() - s).abs() / s.clamp(min=1e-300)).max().item() if s.numel() else 0.0
    assert err <= NAT_SCALE_TOL, err
    assert torch.equal(gs.cpu() == 0, s == 0)
    if r is None:
        assert gh is None
    else:
        assert torch.equal(gh.cpu().float(), h)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("M,K", [(1, 1), (1, 5376), (3, 17), (5, 256), (7, 300), (2, 4111), (300, 1000), (601, 513),
                                 (2, 16384), (3, 16385), (2, 33000)])
def test_sizes(dtype, M, K):
    x, r = rows(M, K, DT[dtype], 1), rows(M, K, DT[dtype], 2, pad=1)
    w = (1 + 0.3 * torch.randn(K, generator=torch.Generator().manual_seed(3))).to(dev())
    check(x, r, w, 1e-6)
    check(x, None, None, 1e-6, flags=BT)


@pytest.mark.parametrize("nb", range(1, 65, 3))
def test_every_row_form(nb):
    K = 256 * nb - 7
    x, r = rows(270, K, torch.bfloat16, nb), rows(270, K, torch.bfloat16, nb + 100)
    check(x, r, None, 1e-5, flags=BT if nb % 2 else 0)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("K", [700, 5376, 20000])
def test_two_pass_and_in_place(dtype, K):
    x, r = rows(9, K, DT[dtype], 4), rows(9, K, DT[dtype], 5, pad=2)
    w = torch.rand(K, generator=torch.Generator().manual_seed(6)).to(dev())
    check(x, r, w, 1e-6, flags=TP, what="two-pass")
    keep_x, keep_r = x.clone(), r.clone()
    for flags in (0, TP):
        for to in (x, r):                        # the sum replaces an operand
            h, q, s = reference(keep_x, keep_r, w, 1e-6)
            x.copy_(keep_x)
            r.copy_(keep_r)
            say(f"in place K={K} {dtype} flags={flags} to {'x' if to is x else 'residual'}")
            gq, gs, gh = rbl.quant_act_rmsnorm(x, w, 1e-6, residual=r, sum=to, flags=flags)
            torch.cuda.synchronize()
            assert gh is to and torch.equal(to.cpu().float(), h)
            assert_bits_equal(gq.cpu().numpy(), q, "codes")
            other, kept = (r, keep_r) if to is x else (x, keep_x)
            assert torch.equal(other.cpu(), kept.cpu())


@pytest.mark.parametrize("flags", [0, TP])
def test_sum_not_kept(flags):
    x, r = rows(5, 900, torch.float16, 7), rows(5, 900, torch.float16, 8)
    h, q, s = reference(x, r, None, 1e-6)
    gq = torch.empty(5, 1024, dtype=torch.int8, device=dev())
    gs = torch.empty(5, device=dev())
    say(f"sum not kept flags={flags}")
    rbl.cr_quant_act_rmsnorm(x, r, None, None, 1e-6, 900, gq, gs, flags)
    torch.cuda.synchronize()
    assert_bits_equal(gq.cpu().numpy(), q, "codes")


@pytest.mark.parametrize("eps", [0.0, 1e-6, 1.0])
@pytest.mark.parametrize("flags", [0, TP])
def test_extreme_rows(eps, flags):
    """Zero rows, rows whose squares overflow or vanish in FP32, a lone element, tiny rows."""
    K = 1000
    x = rows(8, K, torch.float32, 9)
    x[0] = 0
    x[1] *= 1e25
    x[2] *= 1e-25
    x[3] = 0
    x[3, 999] = 1e-30
    x[4] *= 1e-38
    x[5] *= 1e30
    check(x, None, None, eps, flags=flags, what="extreme")
    check(x, torch.zeros_like(x), None, eps, flags=flags, what="extreme, zero residual")
    y = rows(2, K, torch.bfloat16, 10)
    check(y, -y, None, eps, flags=flags, what="cancelling residual")


def test_non_finite_rows_leave_others_exact():
    x = rows(300, 700, torch.bfloat16, 11)
    h, q, s = reference(x, None, None, 1e-6)
    bad = rows(300, 700, torch.bfloat16, 11)
    bad[7, 3], bad[200, 699] = float("nan"), float("inf")
    say("non-finite rows")
    gq, gs, _ = rbl.quant_act_rmsnorm(bad, None, 1e-6)
    torch.cuda.synchronize()
    keep = [i for i in range(300) if i not in (7, 200)]
    assert_bits_equal(gq.cpu().numpy()[keep], q[keep], "codes")
    assert torch.isfinite(gs.cpu()[keep]).all()


def test_output_strides_and_stream():
    """Codes into a wider buffer (the rest untouched), launched on another stream."""
    x = rows(40, 600, torch.float16, 12)
    h, q, s = reference(x, None, None, 1e-6)
    buf = torch.full((40, 1024), 77, dtype=torch.int8, device=dev())
    gs = torch.empty(40, device=dev())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    say("another stream, wider output")
    rbl.cr_quant_act_rmsnorm(x, None, None, None, 1e-6, 600, buf, gs, stream=side)
    side.synchronize()
    assert_bits_equal(buf[:, :768].cpu().numpy(), q, "codes")
    assert (buf[:, 768:] == 77).all().item()


def test_feeds_the_int8_gemm():
    """Norm, INT8 GEMM: close to the FP64 product.  Each operand is rounded to half a step of
    max/127 an element; for normal data the products' error stays below 2 percent."""
    M, N, K = 64, 96, 512
    x, r = rows(M, K, torch.bfloat16, 13), rows(M, K, torch.bfloat16, 14)
    wt = torch.randn(N, K, generator=torch.Generator().manual_seed(15)).to(dev())
    say("norm, then the GEMM")
    q, s, h = rbl.quant_act_rmsnorm(x, None, 1e-6, residual=r)
    qw, sw = rbl.quant_act(wt, K)
    y = rbl.gemm_s8_rowscale(q, s, qw, sw, out_dtype=torch.float32)
    torch.cuda.synchronize()
    hd = h.cpu().double()
    ref = (hd / (hd.square().mean(1, keepdim=True) + 1e-6).sqrt()) @ wt.cpu().double().T
    assert ((y.cpu().double() - ref).norm() / ref.norm()).item() < 0.02
