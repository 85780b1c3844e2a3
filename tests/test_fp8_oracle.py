"""The float64 reference of the 8-bit cache against torch's own e4m3 and
against the definitions, on the CPU."""
import numpy as np
import pytest
import torch

from oracle import fp8_ref as R


def test_every_byte_decodes_as_e4m3():
    b = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(b).view(torch.float8_e4m3fn).double().numpy()
    got = R.e4m3_decode(b)
    assert np.array_equal(np.isnan(t), np.isnan(got)) and np.array_equal(t[~np.isnan(t)], got[~np.isnan(t)])


def test_encode_rounds_to_nearest_even_and_stops_at_448():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * s for s in (1e-3, 0.02, 1.0, 90.0, 500.0)])
    ties = (R.E4M3[:126] + R.E4M3[1:127]) / 2                 # halfway between neighbours
    x = np.concatenate([x, ties, -ties, R.E4M3[:127], [0.0, 448.0, 1e9, -1e9]]).astype(np.float32)
    want = torch.from_numpy(np.clip(x, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(R.e4m3_encode(x), want)
    assert list(R.e4m3_encode(np.array([np.nan, np.inf, -np.inf]))) == [0x7F] * 3


@pytest.mark.parametrize("m2,e", [(0.0, -64), (12.25, -7), (np.nextafter(np.float32(12.25), np.float32(20)), -6),
                                  (448.0 ** 2, 0), (448.0 ** 2 * 4, 1), (3e38, 56), (1e-45, -64)])
def test_needed_scale_at_its_borders(m2, e):
    assert R.needed_scale(m2) == 2.0 ** e


def test_pair_norm_bounds_every_rotation():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((6, 2, 64))
    f = (10000.0 ** (-np.arange(0, 48, 2) / 48)).astype(np.float32)
    for inter in (False, True):
        m = np.sqrt(R.largest_square(x, 48, inter, 1.5).astype(np.float64))
        for pos in (0, 1, 7, 1000, 123457):
            y = R.rope(x, [pos] * 6, f, inter, 1.5)
            assert np.all(np.abs(y[..., :48]).max(axis=(0, 2)) <= m * (1 + 1e-6))
            # A rotation keeps each pair's length.
            assert np.allclose(np.sum(y[..., :48] ** 2), 1.5 ** 2 * np.sum(x[..., :48] ** 2))
            assert np.array_equal(y[..., 48:], x[..., 48:])


def test_not_finite_values_are_left_out_of_the_largest():
    x = np.zeros((1, 1, 32))
    x[0, 0, :5] = [np.inf, np.nan, 3.0, -5.0, 1e38]
    assert R.largest_square(x[..., :4], 0, False, 1.0)[0] == 25.0
    assert R.largest_square(x, 0, False, 1.0)[0] == np.finfo(np.float32).max      # the square overflows


def test_append_by_hand():
    # A block of 8 with three older rows at scale 2^-3; one new row that needs 2^0.
    kc = np.zeros((2, 1, 8, 64), dtype=np.uint8)
    kc[1, 0, :3] = R.e4m3_encode(np.array([[1.0], [0.0625], [-448.0]]) * np.ones((3, 64)))
    kc[1, 0, 5] = 0x55                                          # behind the new row: left as it is
    sc = np.full((2, 1), 0.125, dtype=np.float32)
    x = np.full((1, 1, 64), 300.0)
    k, v, ks, vs, _ = R.append_fp8(x, x * 0, kc, kc, sc, sc, [[1]], [4], [0, 1])
    assert ks[1, 0] == 1.0 and vs[1, 0] == 0.125 and ks[0, 0] == 0.125
    assert np.all(R.e4m3_decode(k[1, 0, :4]) == np.array([0.125, 0.0078125, -56.0, 288.0])[:, None])   # 300 rounds to 288
    assert np.all(k[1, 0, 5] == 0x55) and np.all(k[1, 0, 4] == 0)
    assert np.array_equal(v[1, 0, :3], kc[1, 0, :3]) and np.all(v[1, 0, 3] == 0)


def test_attention_of_equal_scores_is_the_mean():
    rng = np.random.default_rng(2)
    vb = rng.integers(0, 0x70, size=(2, 1, 8, 64), dtype=np.uint8)
    ks, vs = np.ones((2, 1), np.float32), np.array([[2.0], [0.5]], np.float32)
    out, spread, _ = R.attention_fp8(np.zeros((1, 2, 64)), vb, vb, ks, vs, [[1, 0]], [11], [0, 1], 0.125)
    rows = np.concatenate([R.e4m3_decode(vb[1, 0]) * 0.5, R.e4m3_decode(vb[0, 0, :3]) * 2.0])
    assert np.allclose(out, rows.mean(0)) and np.allclose(spread, out)
