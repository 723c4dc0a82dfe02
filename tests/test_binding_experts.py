"""What the binding of the layer of experts refuses before the library is called."""
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
