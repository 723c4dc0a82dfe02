"""The workspace of cr_attn_kv8 follows the rows that a batch has, not its longest run times its
sequences (sizes only: nothing is launched)."""
import random

import rotated_bit_linear_amd as rbl


def need(T, B, max_q, max_kv, Hq, Hkv, D):
    return rbl.cr_attn_kv8_workspace_bytes(T, B, max_q, max_kv, Hq, Hkv, D)


def bound(T, Hq, D):
    return max(64 * T * Hq * (D + 2) * 4, 40 << 20)


def test_one_prompt_among_single_tokens():
    """A few hundred megabytes at most for what was gigabytes by blocks of the longest run."""
    assert 0 < need(2111, 64, 2048, 32768, 32, 8, 128) <= 8 * 2111 * 32 * 130 * 4
    assert 0 < need(2111, 64, 2048, 131072, 32, 8, 128) <= 16 * 2111 * 32 * 130 * 4
    assert need(13072, 256, 12817, 32768, 32, 8, 128) <= 16 * 13072 * 32 * 130 * 4


def test_bound_over_many_sizes():
    r = random.Random(1)
    for _ in range(20000):
        Hkv = r.choice([1, 2, 3, 8, 12])
        Hq, D, B = Hkv * r.choice([1, 2, 4, 7]), r.choice([64, 128]), int(2 ** r.uniform(0, 14))
        max_q = int(2 ** r.uniform(0, 15))
        T = max_q + r.randint(0, B - 1) * r.choice([0, 1, max_q])
        got = need(T, B, max_q, int(2 ** r.uniform(0, 20)), Hq, Hkv, D)
        assert got <= bound(T, Hq, D), (T, B, max_q, Hq, Hkv, D, got)
        assert got % ((D + 2) * 4) == 0
