"""Argument checks of the operators around the linear layers (no kernel runs: every case is
rejected, or is empty, before anything is enqueued)."""
import pytest
import torch

import rotated_bit_linear_amd as rbl

OK, INV, DT, MIS, BIG = 0, 1, 2, 3, 4
A16 = 0x10000          # fake, 16-byte aligned device address (never dereferenced)


def norm(x=A16, dt=0, ld_x=512, r=A16, ld_r=512, h=A16 * 2, ld_h=512, w=A16, eps=1e-6, M=4, K=512, q=A16, ld_q=512,
         s=A16, flags=0):
    return rbl.lib().cr_quant_act_rmsnorm(x, dt, ld_x, r, ld_r, h, ld_h, w, eps, M, K, q, ld_q, s, flags, None)


def test_rmsnorm_validation():
    assert norm(x=None) == INV
    assert norm(q=None) == INV
    assert norm(s=None) == INV
    assert norm(M=-1) == INV
    assert norm(K=0) == INV
    assert norm(dt=3) == DT and norm(dt=-1) == DT
    assert norm(ld_x=500) == INV and norm(ld_r=500) == INV and norm(ld_h=500) == INV
    assert norm(ld_q=256) == INV
    assert norm(eps=-1e-6) == INV and norm(eps=float("nan")) == INV and norm(eps=float("inf")) == INV
    assert norm(r=None) == INV                       # a sum without a residual
    assert norm(h=A16, ld_h=520) == INV              # in place with another row stride
    assert norm(x=A16 + 2) == MIS and norm(r=A16 + 8) == MIS and norm(h=A16 + 4) == MIS
    assert norm(ld_r=516) == MIS and norm(ld_h=516) == MIS
    assert norm(w=A16 + 2) == MIS
    assert norm(flags=4) == INV and norm(flags=16) == INV
    big = rbl.CR_MAX_K_PAD + 256
    assert norm(K=big, ld_x=big, ld_r=big, ld_h=big, ld_q=big) == BIG
    assert norm(M=0) == OK
    assert norm(M=0, x=None, r=None, h=None, q=None, s=None) == OK
    assert norm(M=0, eps=-1.0) == INV


def test_rmsnorm_binding_checks():
    x = torch.zeros(2, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="residual"):
        rbl.quant_act_rmsnorm(x, residual=torch.zeros(2, 512))
    with pytest.raises(ValueError, match="sum"):
        rbl.quant_act_rmsnorm(x, residual=x, sum=torch.zeros(2, 256, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="weight"):
        rbl.quant_act_rmsnorm(x, torch.ones(511))
    with pytest.raises(ValueError, match="weight"):
        rbl.quant_act_rmsnorm(x, torch.ones(512, dtype=torch.bfloat16))
    with pytest.raises(rbl.CrError, match="UNSUPPORTED_DTYPE"):
        rbl.cr_quant_act_rmsnorm(torch.zeros(2, 512, dtype=torch.float64), None, None, None, 1e-6, 512,
                                 torch.zeros(2, 512, dtype=torch.int8), torch.zeros(2),
                                 stream=0)


def cache(k=A16, v=A16, ks=A16, vs=A16, n=8, table=A16, ld=4):
    return rbl._Kv8(k, v, ks, vs, n, table, ld)


def rope(qkv=A16, dt=0, ld=1024, T=4, B=2, cu=A16, kv=A16, max_new=4, Hq=4, Hkv=2, D=128, qw=A16, kw=A16, eps=1e-6,
         pos=A16, ld_pos=3, axes=3, freq=A16, axis=A16, q=A16 * 2, ld_q=512, c=None, flags=0):
    c = cache() if c is None else c
    return rbl.lib().cr_rope_append_kv8(qkv, dt, ld, T, B, cu, kv, max_new, Hq, Hkv, D, qw, kw, eps, pos, ld_pos, axes,
                                        freq, axis, q, ld_q, None if c is False else c, flags, None)


def test_rope_append_validation():
    for name in ("qkv", "cu", "kv", "pos", "freq", "axis", "q"):
        assert rope(**{name: None}) == INV, name
    for name in ("k", "v", "ks", "vs", "table"):
        assert rope(c=cache(**{name: None})) == INV, name
    assert rope(c=False) == INV
    assert rope(c=cache(n=0)) == INV and rope(c=cache(ld=0)) == INV and rope(c=cache(n=-1)) == INV
    assert rope(c=cache(ld=(1 << 24) + 1)) == BIG and rope(c=cache(n=1 << 31)) == BIG
    assert rope(dt=2) == DT and rope(dt=3) == DT and rope(dt=-1) == DT
    assert rope(T=-1) == INV and rope(B=-1) == INV and rope(max_new=-1) == INV
    assert rope(D=96) == INV and rope(D=0) == INV and rope(Hq=-1) == INV and rope(Hkv=-1) == INV
    assert rope(ld=1016) == INV and rope(ld_q=504) == INV
    assert rope(ld=1028) == MIS and rope(ld_q=516) == MIS
    assert rope(qkv=A16 + 8) == MIS and rope(q=A16 + 8) == MIS and rope(freq=A16 + 4) == MIS and rope(pos=A16 + 2) == MIS
    assert rope(qw=A16 + 2) == MIS and rope(kw=A16 + 1) == MIS and rope(c=cache(k=A16 + 8)) == MIS
    assert rope(c=cache(v=A16 + 8)) == MIS and rope(c=cache(ks=A16 + 2)) == MIS and rope(c=cache(table=A16 + 2)) == MIS
    assert rope(axes=0) == INV and rope(axes=5, ld_pos=5) == INV and rope(ld_pos=2) == INV
    assert rope(eps=-1.0) == INV and rope(eps=float("nan")) == INV
    assert rope(flags=16) == INV and rope(flags=1) == INV
    assert rope(q=A16, ld_q=512) == INV                   # in place with another row stride
    assert rope(T=1 << 30, B=1 << 30, max_new=1 << 30) == BIG
    assert rope(T=0) == OK and rope(B=0) == OK and rope(max_new=0) == OK
    assert rope(T=0, qkv=None, cu=None, kv=None, pos=None, freq=None, axis=None, q=None,
                c=cache(None, None, None, None, 0, None, 0)) == OK
    assert rope(T=0, D=96) == INV


def attn(q=A16, dt=0, ld_q=512, T=4, B=2, cu=A16, kv=A16, max_q=4, max_kv=100, Hq=4, Hkv=2, D=128, c=None, sm=0.1,
         out=A16 * 2, ld_o=512, ws=0x100000, wsb=1 << 40, flags=0):
    c = cache() if c is None else c
    return rbl.lib().cr_attn_kv8(q, dt, ld_q, T, B, cu, kv, max_q, max_kv, Hq, Hkv, D, None if c is False else c, sm, out,
                                 ld_o, ws, wsb, flags, None)


def test_attn_validation_and_workspace():
    L = rbl.lib()
    for name in ("q", "out", "cu", "kv"):
        assert attn(**{name: None}) == INV, name
    for name in ("k", "v", "ks", "vs", "table"):
        assert attn(c=cache(**{name: None})) == INV, name
    assert attn(c=False) == INV and attn(c=cache(n=0)) == INV
    assert attn(dt=2) == DT and attn(dt=-1) == DT
    assert attn(Hq=5) == INV and attn(Hq=0) == INV and attn(Hkv=0) == INV and attn(D=32) == INV
    assert attn(T=-1) == INV and attn(max_q=-1) == INV and attn(max_kv=-1) == INV
    assert attn(sm=0.0) == INV and attn(sm=-1.0) == INV and attn(sm=float("nan")) == INV and attn(sm=float("inf")) == INV
    assert attn(ld_q=504) == INV and attn(ld_o=504) == INV and attn(ld_q=516) == MIS and attn(ld_o=516) == MIS
    assert attn(q=A16 + 8) == MIS and attn(out=A16 + 8) == MIS and attn(cu=A16 + 2) == MIS and attn(c=cache(v=A16 + 4)) == MIS
    assert attn(flags=1) == INV and attn(flags=32) == INV
    assert attn(T=0) == OK and attn(B=0) == OK and attn(max_q=0) == OK
    assert attn(T=0, q=None, out=None, cu=None, kv=None, c=cache(None, None, None, None, 0, None, 0), ws=None, wsb=0) == OK
    assert attn(T=1 << 30, B=1 << 30, max_q=1 << 30, max_kv=64) == BIG
    need = L.cr_attn_kv8_workspace_bytes(1, 1, 1, 100000, 8, 1, 128)
    assert need > 8 * 128 * 4                            # a long cache is split
    long = dict(T=1, B=1, max_q=1, max_kv=100000, Hq=8, Hkv=1, ld_q=1024, ld_o=1024)
    assert attn(**long, wsb=need - 1) == BIG
    assert attn(**long, ws=None) == INV and attn(**long, ws=0x100010) == MIS
    assert L.cr_attn_kv8_workspace_bytes(8192, 2, 4096, 4096, 32, 8, 128) == 0
    assert L.cr_attn_kv8_workspace_bytes(-1, 1, 1, 1, 1, 1, 64) == 0
    assert L.cr_attn_kv8_workspace_bytes(1, 1, 1, 1, 3, 2, 64) == 0


def test_cache_binding_checks():
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    ok = rbl.Kv8Cache.empty(3, 2, 64, device="cpu")
    with pytest.raises(ValueError):
        rbl.Kv8Cache(u8(3, 2, 32, 64), ok.v, ok.k_scale, ok.v_scale)
    with pytest.raises(ValueError):
        rbl.Kv8Cache(ok.k, ok.k.new_zeros(3, 2, 64, 32), ok.k_scale, ok.v_scale)
    with pytest.raises(ValueError):
        rbl.Kv8Cache(ok.k, ok.v, ok.k_scale.double(), ok.v_scale)
    with pytest.raises(ValueError):
        rbl.Kv8Cache(ok.k, ok.v, ok.k_scale[:2], ok.v_scale)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    q = torch.zeros(2, 256, dtype=torch.bfloat16)
    args = dict(cu_seqlens=i32(2), kv_lens=i32(1), page_table=i32(1, 3), max_q=2, max_kv=2, Hq=4)
    for change in (dict(cu_seqlens=i32(3)), dict(kv_lens=torch.zeros(1)), dict(page_table=i32(2, 3)),
                   dict(page_table=torch.zeros(1, 3)), dict(Hq=3), dict(page_table=i32(1, 6)[:, ::2])):
        with pytest.raises(ValueError):
            rbl.attn_kv8(q, ok, **dict(args, **change))
    qkv = torch.zeros(2, 512, dtype=torch.bfloat16)
    freq, axis = rbl.rope_table(64, [8, 12, 12], device="cpu")
    assert freq.shape == (32,) and axis.tolist() == [0] * 8 + [1] * 12 + [2] * 12
    args = dict(cu_seqlens=i32(2), kv_lens=i32(1), page_table=i32(1, 3), max_new=2, Hq=4, pos=i32(2, 3), freq=freq, axis=axis)
    for change in (dict(Hq=5), dict(pos=i32(3, 3)), dict(pos=torch.zeros(2, 3)), dict(freq=freq.float()),
                   dict(axis=axis[:31].clone()), dict(q_weight=torch.ones(63)), dict(out=torch.zeros(2, 256)),
                   dict(page_table=i32(2, 3))):
        with pytest.raises(ValueError):
            rbl.rope_append_kv8(qkv, ok, **dict(args, **change))
    with pytest.raises(ValueError):
        rbl.rope_table(64, [20, 20])
    freq, axis = rbl.rope_table(64, [4, 4], base=100.0, device="cpu")
    assert freq[8:].abs().max().item() == 0 and freq[1].item() == pytest.approx(100 ** -0.25, rel=1e-15)


def test_bounds_taken_from_device_data(tmp_path):
    """kv8.hpp's bounds on the host, for arrays that hold anything."""
    import os
    import subprocess
    hipcc = "/opt/rocm/bin/hipcc"
    if not os.path.exists(hipcc):
        pytest.skip("hipcc not available")
    here = os.path.dirname(os.path.abspath(__file__))
    exe = str(tmp_path / "kv8_bounds")
    subprocess.run([hipcc, "-x", "hip", "--offload-host-only", "-std=c++17", "-O1",
                    os.path.join(here, "native", "kv8_bounds.cpp"), "-o", exe], check=True, capture_output=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.startswith("ok"), r.stdout
