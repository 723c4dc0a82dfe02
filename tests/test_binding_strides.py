"""Row strides that the binding hands to the library: those of expanded and overlapping rows as they are, so
that the library refuses them (it would read or write past the tensor); of a single row, whose stride may be
anything, at least its columns."""
import pytest
import torch

import rotated_bit_linear_amd as rbl

INVALID = 1
i32, s8, u8 = torch.int32, torch.int8, torch.uint8


class Recorder:
    """Stands for the library: takes every call and enqueues nothing."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or 0


@pytest.fixture(autouse=True)
def no_stream(monkeypatch):
    monkeypatch.setattr(rbl, "_stream", lambda stream: 0)


@pytest.fixture
def recorder(monkeypatch):
    r = Recorder()
    monkeypatch.setattr(rbl, "lib", lambda: r)
    return r


def overlapping(rows, cols, dtype=torch.float32):
    """Rows that begin 16 elements apart."""
    return torch.zeros(16 * rows + cols, dtype=dtype).as_strided((rows, cols), (16, 1))


def expanded(rows, cols, dtype=torch.float32):
    return torch.zeros(1, cols, dtype=dtype).expand(rows, cols)


def refused(call):
    with pytest.raises(rbl.CrError) as e:
        call()
    assert e.value.status == INVALID


T, K, E, k, N = 4, 512, 6, 2, 96
IDS, WEIGHTS = torch.zeros(T, k, dtype=i32), torch.zeros(T, k)
OFFSETS, ROWS = torch.zeros(E + 1, dtype=i32), torch.zeros(T * k, dtype=i32)
W1, S1 = torch.zeros(E, N, K // 2, dtype=u8), torch.zeros(E, N)
W2, S2 = torch.zeros(E, N, 128, dtype=u8), torch.zeros(E, N)
A, SA = torch.zeros(T, K, dtype=s8), torch.zeros(T)
WORKSPACE = torch.zeros(1 << 20, dtype=u8)
WORKSPACE = WORKSPACE[-WORKSPACE.data_ptr() % 256:]


@pytest.mark.parametrize("rows", [expanded, overlapping])
def test_experts_refuse_rows_that_overlap(rows):
    refused(lambda: rbl.route_experts(rows(T, 64), k))
    refused(lambda: rbl.gemm_s8s4_experts(rows(T, K, s8), SA, W1, S1, OFFSETS, ROWS, k, gather=True))
    refused(lambda: rbl.gemm_s8s4_experts(A, SA, W1, S1, OFFSETS, ROWS, k, gather=True, out=rows(T * k, N)))
    refused(lambda: rbl.experts_combine(rows(T * k, N), WEIGHTS, IDS, E))
    refused(lambda: rbl.experts_combine(torch.zeros(T * k, N), WEIGHTS, IDS, E, residual=rows(T, N)))
    refused(lambda: rbl.experts_combine(torch.zeros(T * k, N), WEIGHTS, IDS, E, out=rows(T, N)))

    def layer(a=A, **kw):
        return rbl.mlp_experts_w4a8(a, SA, IDS, WEIGHTS, W1, S1, W2, S2, workspace=WORKSPACE, **kw)

    refused(lambda: layer(rows(T, K, s8)))
    refused(lambda: layer(residual=rows(T, N, torch.bfloat16)))
    refused(lambda: layer(out=rows(T, N, torch.bfloat16)))


def test_experts_take_the_rows_as_they_lie(recorder):
    one = lambda n, dtype=torch.float32: torch.zeros(n, dtype=dtype).as_strided((1, n), (1, 1))  # noqa: E731
    ids, weights = IDS[:1, :1].contiguous(), WEIGHTS[:1, :1].contiguous()
    rbl.experts_combine(one(N), weights, ids, E, residual=one(N), out=one(N))
    rbl.route_experts(one(64), 1)
    rbl.gemm_s8s4_experts(one(K, s8), SA, W1, S1, OFFSETS, ROWS[:1], 1, gather=True, out=one(N))
    rbl.mlp_experts_w4a8(one(K, s8), SA, ids, weights, W1, S1, W2, S2, residual=one(N, torch.bfloat16),
                         out=one(N, torch.bfloat16), workspace=WORKSPACE)
    combine, route, product, layer = (args for _, args in recorder.calls)
    assert combine[2] == N and combine[11] == N and combine[13] == N
    assert route[2] == 64
    assert product[1] == K and product[18] == N
    assert layer[1] == K and layer[23] == N and layer[26] == N
    del recorder.calls[:]
    wide = torch.zeros(T * k, N + 16)[:, :N]           # rows apart
    rbl.experts_combine(wide, WEIGHTS, IDS, E, residual=wide[:T], out=torch.zeros(T, N))
    (combine,) = (args for _, args in recorder.calls)
    assert combine[2] == N + 16 and combine[11] == N + 16 and combine[13] == N


# ----------------------------------------------------------------------------- the cache's calls ----

Hq, Hkv, D = 4, 2, 64
CU, LENS, TABLE = torch.tensor([0, T], dtype=i32), torch.tensor([T], dtype=i32), torch.zeros(1, 1, dtype=i32)
POS, FREQ, AXIS = torch.zeros(T, 1, dtype=i32), torch.zeros(D // 2, dtype=torch.float64), torch.zeros(D // 2, dtype=i32)
b16 = torch.bfloat16


def append(qkv, pos=POS, **kw):
    cache = rbl.Kv8Cache.empty(1, Hkv, D, "cpu")
    return rbl.rope_append_kv8(qkv, cache, CU, LENS, TABLE, T, Hq, pos, FREQ, AXIS, **kw)


def attention(q, **kw):
    return rbl.attn_kv8(q, rbl.Kv8Cache.empty(1, Hkv, D, "cpu"), CU, LENS, TABLE, T, T, Hq, workspace=WORKSPACE, **kw)


@pytest.mark.parametrize("rows", [expanded, overlapping])
def test_cache_calls_refuse_rows_that_overlap(rows):
    qkv, q = torch.zeros(T, (Hq + 2 * Hkv) * D, dtype=b16), torch.zeros(T, Hq * D, dtype=b16)
    refused(lambda: append(rows(T, (Hq + 2 * Hkv) * D, b16)))
    refused(lambda: append(qkv, out=rows(T, Hq * D, b16)))
    refused(lambda: append(qkv, pos=expanded(T, 1, i32)))
    refused(lambda: attention(rows(T, Hq * D, b16)))
    refused(lambda: attention(q, out=rows(T, Hq * D, b16)))


def test_cache_calls_take_a_single_row_of_any_stride(recorder):
    one = lambda n, dtype=b16: torch.zeros(n, dtype=dtype).as_strided((1, n), (1, 1))  # noqa: E731
    append(one((Hq + 2 * Hkv) * D), pos=one(3, i32), out=one(Hq * D))
    attention(one(Hq * D), out=one(Hq * D))
    rope, attn = (args for _, args in recorder.calls)
    assert rope[2] == (Hq + 2 * Hkv) * D and rope[15] == 3 and rope[20] == Hq * D
    assert attn[2] == Hq * D and attn[15] == Hq * D
