"""Argument checks of the layer of experts (no kernel runs: every case is rejected, or is empty, before
anything is enqueued), and the bounds that its kernels keep over device data that holds anything."""
import os
import subprocess

import pytest
import torch

import rotated_bit_linear_amd as rbl

OK, INV, DT, MIS, BIG = 0, 1, 2, 3, 4
A16 = 0x10000          # fake, aligned device address (never dereferenced)


def route(x=A16, dt=0, ld=64, T=4, E=64, bias=A16, G=8, top=4, m=2, k=8, scale=1.0, ids=A16, w=A16, flags=0):
    return rbl.lib().cr_route_experts(x, dt, ld, T, E, bias, G, top, m, k, scale, ids, w, flags, None)


def test_route_validation():
    for name in ("x", "ids", "w"):
        assert route(**{name: None}) == INV, name
    assert route(dt=3) == DT and route(dt=-1) == DT
    assert route(T=-1) == INV and route(E=0) == INV and route(E=513, ld=513, G=1, top=1) == INV
    assert route(k=0) == INV and route(k=33) == INV and route(k=33, top=8) == INV
    assert route(ld=63) == INV
    assert route(G=0) == INV and route(G=7) == INV and route(E=128, ld=128, G=128, top=64) == INV
    assert route(top=0) == INV and route(top=9) == INV
    assert route(top=1, k=9) == INV                   # fewer experts than choices in the chosen groups
    assert route(m=0) == INV and route(m=3) == INV
    assert route(scale=float("nan")) == INV and route(scale=float("inf")) == INV
    assert route(flags=1) == INV and route(flags=256) == INV
    assert route(x=A16 + 1) == MIS and route(x=A16 + 2, dt=2) == MIS
    assert route(bias=A16 + 2) == MIS and route(ids=A16 + 2) == MIS and route(w=A16 + 1) == MIS
    assert route(T=1 << 26, k=32, E=64, top=8) == INV  # slots beyond 32 bits
    assert route(T=0) == OK and route(T=0, x=None, ids=None, w=None, bias=None) == OK
    assert route(T=0, k=0) == INV


def plan(ids=A16, T=4, k=8, first=0, E=64, off=A16, rows=A16, ws=None, wsb=0):
    return rbl.lib().cr_experts_plan(ids, T, k, first, E, off, rows, ws, wsb, None)


def test_plan_validation_and_workspace():
    L = rbl.lib()
    for name in ("ids", "off", "rows"):
        assert plan(**{name: None}) == INV, name
    assert plan(T=-1) == INV and plan(k=0) == INV and plan(k=33) == INV and plan(E=0) == INV and plan(E=513) == INV
    assert plan(first=-1) == INV and plan(first=(1 << 31) - 64) == INV
    assert plan(T=1 << 28) == INV
    assert plan(ids=A16 + 2) == MIS and plan(off=A16 + 2) == MIS and plan(rows=A16 + 2) == MIS
    assert L.cr_experts_plan_workspace_bytes(512, 8, 64) == 0
    need = L.cr_experts_plan_workspace_bytes(513, 8, 64)
    assert need > 0 and need % 256 == 0
    assert plan(T=513) == INV and plan(T=513, ws=0x100010, wsb=1 << 30) == MIS
    assert plan(T=513, ws=0x100000, wsb=need - 1) == BIG
    assert L.cr_experts_plan_workspace_bytes(0, 8, 64) == 0 and L.cr_experts_plan_workspace_bytes(-1, 8, 64) == 0
    assert L.cr_experts_plan_workspace_bytes((1 << 31) // 8 - 1, 8, 512) <= 257 * 513 * 4
    assert L.cr_experts_plan_workspace_bytes(1 << 28, 8, 64) == 0


def product(a=A16, lda=512, sa=A16, M=4, b=A16, ldb=256, stride=256 * 96, sb=A16, bias=None, off=A16, rows=A16, S=32, E=64,
            N=96, Kp=512, gather=8, c=A16, dt=0, ldc=96, flags=0):
    return rbl.lib().cr_gemm_s8s4_experts(a, lda, sa, M, b, ldb, stride, sb, bias, off, rows, S, E, N, Kp, gather, c, dt, ldc,
                                          flags, None)


def test_product_validation():
    for name in ("a", "sa", "b", "sb", "off", "rows", "c"):
        assert product(**{name: None}) == INV, name
    assert product(rows=None, gather=0, flags=256) == INV
    assert product(dt=4) == DT and product(dt=-1) == DT
    assert product(M=-1) == INV and product(S=-1) == INV and product(N=-1) == INV and product(E=0) == INV
    assert product(E=513) == INV and product(M=1 << 31) == INV and product(S=1 << 31) == INV
    assert product(Kp=300) == INV and product(Kp=0) == INV
    big = rbl.CR_MAX_K_PAD + 256
    assert product(Kp=big, lda=big, ldb=big // 2, stride=96 * big // 2) == BIG
    assert product(gather=-1) == INV and product(gather=33) == INV
    assert product(lda=496) == INV and product(ldb=240) == INV and product(stride=256 * 96 - 16) == INV
    assert product(ldc=95) == INV and product(ldc=47, flags=512) == INV
    assert product(N=95, ldc=95, flags=512) == INV     # gates and values
    assert product(dt=3, bias=A16) == INV and product(dt=3, flags=512) == INV
    assert product(flags=2) == INV and product(flags=64) == INV
    assert product(a=A16 + 8) == MIS and product(lda=520) == MIS and product(b=A16 + 8) == MIS
    assert product(ldb=264, stride=264 * 96) == MIS and product(stride=256 * 96 + 8) == MIS
    assert product(sa=A16 + 2) == MIS and product(sb=A16 + 2) == MIS and product(bias=A16 + 2) == MIS
    assert product(off=A16 + 2) == MIS and product(rows=A16 + 2) == MIS and product(c=A16 + 1) == MIS
    n = 1 << 30
    assert product(S=1 << 30, M=1 << 30, N=n, ldc=n, stride=256 * n) == BIG
    assert product(S=0) == OK and product(N=0) == OK and product(M=0) == OK
    assert product(S=0, a=None, sa=None, off=None, rows=None, c=None) == OK
    assert product(S=0, flags=2) == INV


def combine(y=A16, dt=0, ld_y=96, w=A16, ids=A16, T=4, k=8, first=0, E=64, N=96, r=None, ld_r=96, o=A16, ld_o=96):
    return rbl.lib().cr_experts_combine(y, dt, ld_y, w, ids, T, k, first, E, N, r, ld_r, o, ld_o, None)


def test_combine_validation():
    for name in ("y", "w", "ids", "o"):
        assert combine(**{name: None}) == INV, name
    assert combine(dt=3) == DT and combine(dt=-1) == DT
    assert combine(T=-1) == INV and combine(k=0) == INV and combine(E=0) == INV and combine(first=-1) == INV
    assert combine(N=-1) == INV and combine(ld_y=95) == INV and combine(ld_o=95) == INV
    assert combine(r=A16 * 2, ld_r=95) == INV
    assert combine(r=A16, ld_r=104) == INV             # in place with another row stride
    assert combine(y=A16 + 1) == MIS and combine(o=A16 + 1) == MIS and combine(r=A16 + 1) == MIS
    assert combine(dt=2, y=A16 + 2) == MIS and combine(w=A16 + 2) == MIS and combine(ids=A16 + 2) == MIS
    n = (1 << 31) - 1
    assert combine(T=1 << 26, N=n, ld_y=n, ld_o=n) == BIG
    assert combine(T=0) == OK and combine(N=0) == OK and combine(T=0, y=None, w=None, ids=None, o=None) == OK


def layer(a=A16, lda=512, sa=A16, T=4, Kp=512, ids=A16, w=A16, k=8, first=0, E=64, w1=A16, ld1=256, st1=256 * 400, s1=A16,
          b1=None, F=200, w2=A16, ld2=128, st2=128 * 96, s2=A16, b2=None, N=96, r=None, ld_r=96, o=A16, dt=0, ld_o=96,
          ws=0x100000, wsb=1 << 40, flags=0):
    return rbl.lib().cr_mlp_experts_w4a8(a, lda, sa, T, Kp, ids, w, k, first, E, w1, ld1, st1, s1, b1, F, w2, ld2, st2, s2, b2,
                                         N, r, ld_r, o, dt, ld_o, ws, wsb, flags, None)


def test_layer_validation_and_workspace():
    for name in ("a", "sa", "ids", "w", "w1", "s1", "w2", "s2", "o", "ws"):
        assert layer(**{name: None}) == INV, name
    assert layer(dt=3) == DT and layer(dt=-1) == DT
    assert layer(T=-1) == INV and layer(k=0) == INV and layer(E=513) == INV and layer(first=-1) == INV and layer(F=0) == INV
    assert layer(N=-1) == INV and layer(Kp=300) == INV and layer(lda=496) == INV and layer(ld1=240) == INV
    assert layer(ld2=112) == INV and layer(st1=256 * 400 - 16) == INV and layer(st2=128 * 96 - 16) == INV
    assert layer(ld_o=95) == INV and layer(r=A16, ld_r=95) == INV
    assert layer(flags=4) == INV and layer(flags=512) == INV
    assert layer(F=rbl.CR_MAX_K_PAD + 1) == BIG and layer(N=(1 << 28) + 1) == BIG
    assert layer(a=A16 + 8) == MIS and layer(w1=A16 + 8) == MIS and layer(w2=A16 + 8) == MIS and layer(o=A16 + 1) == MIS
    assert layer(s1=A16 + 2) == MIS and layer(s2=A16 + 2) == MIS and layer(b1=A16 + 2) == MIS and layer(b2=A16 + 2) == MIS
    assert layer(ids=A16 + 2) == MIS and layer(w=A16 + 2) == MIS and layer(ws=0x100010) == MIS
    need = rbl.cr_mlp_experts_w4a8_workspace_bytes(4, 8, 64, 200, 96, torch.bfloat16)
    assert need >= 32 * (200 * 2 + 256 + 4 + 96 * 2) and need % 256 == 0
    assert layer(wsb=need - 1) == BIG
    assert layer(T=0) == OK and layer(N=0) == OK
    assert layer(T=0, a=None, sa=None, ids=None, w=None, o=None, ws=None) == OK
    assert layer(T=0, F=0) == INV and layer(T=0, lda=496) == INV
    L = rbl.lib()
    for bad in ((0, 8, 64, 200, 96, 0), (4, 0, 64, 200, 96, 0), (4, 8, 0, 200, 96, 0), (4, 8, 64, 0, 96, 0),
                (4, 8, 64, 200, 0, 0), (4, 8, 64, 200, 96, 3), (1 << 29, 8, 64, 200, 96, 0)):
        assert L.cr_mlp_experts_w4a8_workspace_bytes(*bad) == 0, bad


def test_binding_checks():
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    ids, w = torch.zeros(2, 3, dtype=i32), torch.zeros(2, 3)
    q, s = torch.zeros(2, 512, dtype=torch.int8), torch.zeros(2)
    off, rows = torch.zeros(5, dtype=i32), torch.zeros(6, dtype=i32)
    b, sb = torch.zeros(4, 8, 256, dtype=u8), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="ids"):
        rbl.experts_plan(ids.long(), 4)
    with pytest.raises(ValueError, match="ids"):
        rbl.experts_plan(ids.flatten(), 4)
    with pytest.raises(ValueError, match="ids"):
        rbl.experts_combine(torch.zeros(6, 8), w, ids.t().contiguous().t(), 4)
    with pytest.raises(ValueError, match="weights"):
        rbl.experts_combine(torch.zeros(6, 8), w.double(), ids, 4)
    with pytest.raises(ValueError, match="y must"):
        rbl.experts_combine(torch.zeros(5, 8), w, ids, 4)
    with pytest.raises(ValueError, match="residual"):
        rbl.experts_combine(torch.zeros(6, 8), w, ids, 4, residual=torch.zeros(2, 8, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="bias"):
        rbl.route_experts(torch.zeros(2, 4), 1, bias=torch.zeros(3))
    with pytest.raises(ValueError, match="offsets"):
        rbl.gemm_s8s4_experts(q, s, b, sb, off[:4], rows, 3, gather=True)
    with pytest.raises(ValueError, match="scales"):
        rbl.gemm_s8s4_experts(q, s, b, sb[:3], off, rows, 3, gather=True)
    with pytest.raises(ValueError, match="a_scale"):
        rbl.gemm_s8s4_experts(q, s[:1], b, sb, off, rows, 3, gather=True)
    with pytest.raises(ValueError, match="b_s4"):
        rbl.gemm_s8s4_experts(q, s, b.view(torch.int8), sb, off, rows, 3, gather=True)
    with pytest.raises(ValueError, match="c must"):
        rbl.gemm_s8s4_experts(q, s, b, sb, off, rows, 3, gather=True, out=torch.zeros(5, 8))
    w2, s2 = torch.zeros(4, 16, 128, dtype=u8), torch.zeros(4, 16)
    with pytest.raises(ValueError, match="same experts"):
        rbl.mlp_experts_w4a8(q, s, ids, w, b, sb, w2[:3], s2[:3])
    with pytest.raises(ValueError, match="out"):
        rbl.mlp_experts_w4a8(q, s, ids, w, b, sb, w2, s2, out=torch.zeros(2, 15))
    with pytest.raises(rbl.CrError, match="UNSUPPORTED_DTYPE"):
        rbl.cr_route_experts(torch.zeros(2, 4, dtype=torch.float64), None, 1, 1, 1, 3, 1.0, ids, w, stream=0)


def test_bounds_taken_from_device_data(tmp_path):
    hipcc = "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    here = os.path.dirname(os.path.abspath(__file__))
    exe = str(tmp_path / "experts_bounds")
    subprocess.run([hipcc, "-x", "hip", "--offload-host-only", "-std=c++17", "-O1",
                    os.path.join(here, "native", "experts_bounds.cpp"), "-o", exe], check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout
