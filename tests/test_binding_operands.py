"""What the binding refuses before the library is called: rows that are no codes, weights that do not fit."""
import pytest
import torch

import rotated_bit_linear_amd as rbl

i32, s8, u8 = torch.int32, torch.int8, torch.uint8
T, k, E, K, F, N = 2, 3, 4, 512, 300, 16
IDS, WEIGHTS = torch.zeros(T, k, dtype=i32), torch.zeros(T, k)
OFFSETS, ROWS = torch.zeros(E + 1, dtype=i32), torch.zeros(T * k, dtype=i32)
A, SA = torch.zeros(T, K, dtype=s8), torch.zeros(T)


@pytest.fixture(autouse=True)
def no_stream(monkeypatch):
    monkeypatch.setattr(rbl, "_stream", lambda stream: 0)


def packed(rows, columns):
    return torch.zeros(E, rows, columns // 2, dtype=u8), torch.zeros(E, rows)


def product(a, w, s):
    return rbl.gemm_s8s4_experts(a, SA, w, s, OFFSETS, ROWS, k, gather=True)


def layer(a, w1, w2):
    return rbl.mlp_experts_w4a8(a, SA, IDS, WEIGHTS, *w1, *w2)


@pytest.mark.parametrize("columns", [256, 768, 1024])
def test_weights_of_another_length(columns):
    """Longer rows would give sums over their first columns, shorter ones are read past their end where the
    rows lie apart."""
    w, s = packed(8, columns)
    with pytest.raises(ValueError, match="b_s4 must hold 512"):
        product(A, w, s)
    with pytest.raises(ValueError, match="w1 must hold 512"):
        layer(A, packed(2 * F, columns), packed(N, 512))
    with pytest.raises(ValueError, match="w2 must hold 512"):
        layer(A, packed(2 * F, K), packed(N, columns))


def test_columns_cut_from_a_longer_weight():
    """Rows 400 bytes apart that end 128 bytes after they begin."""
    base = torch.zeros(E, 8, 400, dtype=u8)
    a = torch.zeros(T, 768, dtype=s8)
    with pytest.raises(ValueError, match="b_s4 must hold 768"):
        product(a, base[:, :, 272:], torch.zeros(E, 8))


@pytest.mark.parametrize("dtype", [torch.int16, torch.bfloat16, torch.float8_e4m3fn, u8])
def test_rows_that_are_no_int8_codes(dtype):
    a = torch.zeros(T, K).to(dtype)
    with pytest.raises(ValueError, match="a_s8 must be int8"):
        product(a, *packed(8, K))
    with pytest.raises(ValueError, match="a_s8 must be int8"):
        layer(a, packed(2 * F, K), packed(N, 512))


@pytest.mark.parametrize("dtype", [torch.int16, torch.float16, torch.float8_e4m3fn])
def test_dense_rows_that_are_no_int8_codes(dtype):
    """Rows of other types were read, and written, as codes."""
    bad, q, s, x = torch.zeros(T, K).to(dtype), torch.zeros(T, K, dtype=s8), torch.zeros(T), torch.zeros(T, K)
    c, bytes_ = torch.zeros(T, T), torch.zeros(T, K, dtype=u8)
    for name, call in [
        ("a_s8", lambda: rbl.cr_gemm_s8_rowscale(bad, s, q, s, c)),
        ("b_s8", lambda: rbl.cr_gemm_s8_rowscale_bias(q, s, bad, s, s, c)),
        ("a_s8", lambda: rbl.cr_gemm_s8s4_rowscale(bad, s, bytes_[:, :K // 2], s, c)),
        ("a_s8", lambda: rbl.cr_gemm_nvfp4_fused(bad, s, bytes_, bytes_, s, s, K, c)),
        ("x_s8", lambda: rbl.cr_quant_act(x, K, bad, s)),
        ("x_s8", lambda: rbl.cr_quant_act_swiglu(x, K // 2, bad, s)),
        ("x_s8", lambda: rbl.cr_quant_act_ex(x, K, False, None, bad, s)),
        ("x_s8", lambda: rbl.cr_quant_act_rmsnorm(x, None, None, s, 1e-6, K, bad, s)),
        ("w_s8", lambda: rbl.cr_prep_weight_nvfp4(bytes_, bytes_, s, K, bad, s)),
    ]:
        with pytest.raises(ValueError, match=f"{name} must be int8"):
            call()
