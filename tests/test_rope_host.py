"""Host-only checks of rope_apply and rope_inv_freq beyond those of test_kv8_host.py
(no GPU needed: only refused calls are made)."""
import math

import pytest

import split_kv_merge_attn_b200 as skv
from tests.test_kv8_host import INVALID, addr, rope

Q_BYTES, K_BYTES = 4 * 8 * 128 * 2, 2 * 8 * 128 * 2  # of rope()'s q (4 heads) and k (2), S = 8, D = 128
POS_BYTES, F_BYTES = 8 * 4, 32 * 8                   # its positions and frequencies


@pytest.mark.parametrize("kw", [
    dict(pos=addr(2)), dict(pos=addr(2) + Q_BYTES - 4), dict(pos=addr(2) - POS_BYTES + 4), dict(pos=addr(3) + 64),
    dict(f=addr(2) + 64), dict(f=addr(3)), dict(f=addr(3) + K_BYTES - 8), dict(f=addr(3) - F_BYTES + 8),
    dict(qo=addr(0), pos=addr(0) + 128), dict(ko=addr(1), f=addr(1) + 128),  # in place
    dict(k=None, ko=None, Hkv=0, pos=addr(2) + 64),
])
def test_outputs_over_positions_or_frequencies_are_refused(kw):
    assert rope(**kw) == INVALID


@pytest.mark.parametrize("R,base,L,fast,slow", [
    (128, 1e4, 2048, 32.0, 1.0), (128, 1e4, 32768, 32.0, 1.0), (128, 1e4, 65536, 32.0, 1.0),
    (128, 1e4, 131072, 32.0, 1.0), (128, 1e4, 1 << 20, 32.0, 1.0), (64, 1e4, 131072, 32.0, 1.0),
    (128, 5e5, 131072, 32.0, 1.0), (32, 100.0, 4096, 8.0, 2.0), (16, 1e4, 1 << 30, 64.0, 4.0),
    (2, 1e4, 131072, 32.0, 1.0),
])
@pytest.mark.parametrize("factor", [1.0, 4.0, 40.0])
def test_yarn_against_its_definition(R, base, L, fast, slow, factor):
    """Pair i turns L base^(-2i/R) / (2 pi) times over L positions; the (real) pair that
    turns n times is found by bisection.  The ramp runs between the pairs of `fast` and
    `slow` turns, rounded outwards and held to [0, R - 1], also where the second lies behind
    the last pair (base^(1 - 2/R) < L / (2 pi slow))."""
    def pair(n):
        lo, hi = -1000.0, 1000.0  # turns fall with the pair
        for _ in range(200):
            mid = (lo + hi) / 2
            turns = math.log(L / (2 * math.pi)) - 2 * mid / R * math.log(base)
            lo, hi = (mid, hi) if turns > math.log(n) else (lo, mid)
        return lo
    first, last = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), R - 1)
    got, m = skv.rope_inv_freq(R, base, "yarn", factor, original_len=L, beta_fast=fast, beta_slow=slow, device="cpu")
    for i in range(R // 2):
        f = base ** (-2.0 * i / R)
        g = 0.0 if i <= first else 1.0 if i >= last else (i - first) / (last - first)
        want = f * (1 - g) + f / factor * g
        assert abs(got[i].item() - want) <= 1e-13 * want
    assert m == pytest.approx(0.1 * math.log(factor) + 1.0, rel=1e-15)


def test_yarn_leaves_pairs_that_turn_often_enough():
    """Where even the slowest pair turns 19 times over original_len (more than beta_slow),
    none is interpolated fully."""
    f, _ = skv.rope_inv_freq(128, 1e4, "yarn", 4.0, original_len=1 << 20, device="cpu")
    ratio = f[-1].item() * 1e4 ** (126 / 128)
    assert ratio > 0.8
