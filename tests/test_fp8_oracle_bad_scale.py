"""The float64 reference where a block's older tokens have no valid scale (CPU)."""
import numpy as np
import pytest

from oracle import fp8_ref as R


@pytest.mark.parametrize("bad", [0.0, -2.0, np.nan, np.inf, 2.0 ** 65, 2.0 ** -65])
def test_older_rows_are_given_up(bad):
    kc = np.full((1, 2, 8, 64), 0x38, dtype=np.uint8)           # 1.0 everywhere
    sc = np.array([[bad, 0.5]], dtype=np.float32)
    x = np.full((1, 2, 64), 448.0)
    k, v, ks, vs, _ = R.append_fp8(x, x, kc, kc, sc, np.ones_like(sc), [[0]], [4], [0, 1])
    assert np.all(k[0, 0, :3] == 0x7F) and np.all(k[0, 0, 3] == 0x7E) and ks[0, 0] == 1.0
    assert np.all(k[0, 0, 4:] == 0x38)                          # behind the new row: as it was
    assert np.all(k[0, 1, :3] == 0x30) and ks[0, 1] == 1.0      # the other head's: 0.5 in the new steps
    assert np.all(v[0, :, :3] == 0x38) and np.all(vs == 1.0)


def test_a_block_whose_first_token_is_new_takes_any():
    kc = np.full((1, 1, 8, 64), 0x38, dtype=np.uint8)
    sc = np.array([[np.nan]], dtype=np.float32)
    k, _, ks, _, _ = R.append_fp8(np.full((2, 1, 64), 224.0), np.zeros((2, 1, 64)), kc, kc, sc, sc, [[0]], [2], [0, 2])
    assert ks[0, 0] == 0.5 and np.all(k[0, 0, :2] == 0x7E) and np.all(k[0, 0, 2:] == 0x38)
