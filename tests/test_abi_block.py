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
