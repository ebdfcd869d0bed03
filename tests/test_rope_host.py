"""Host-only checks of rope_apply and rope_inv_freq beyond those of test_kv8_host.py
(no GPU needed: only refused calls are made)."""
import pytest

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
