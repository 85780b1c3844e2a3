"""The error bound of the 8-bit attention's tests sees a lost tile (CPU)."""
import numpy as np
import pytest

from fp8sharp import TILE, host_case, reference
from oracle import fp8_ref as R


def _weights(c, h):
    """p_j of the one sequence, and its values [L, D], both float64."""
    L = int(c["lens"][0])
    K, V = R.rows_fp8(c["kb"], c["ks"], c["bt"][0], L), R.rows_fp8(c["vb"], c["vs"], c["bt"][0], L)
    G = c["q64"].shape[1] // K.shape[1]
    z = c["scale"] * (K[:, h // G] @ c["q64"][0, h])
    return np.exp(z - z.max()), V[:, h // G]


@pytest.mark.parametrize("L,D,B", [(40000, 64, 8), (31000, 128, 16), (131072, 128, 32), (300, 64, 16)])
def test_one_tile_less_or_one_part_misweighted_is_out_of_bounds(L, D, B):
    c = host_case(L, [L], 2, 1, D, B)
    ref, tol = reference(c)
    rng = np.random.default_rng(1)
    tiles = -(-L // TILE)
    for h in range(2):
        p, V = _weights(c, h)
        assert np.all(np.abs(p @ V / p.sum() - ref[0, h]) <= tol[0, h])
        for t in rng.integers(0, tiles, size=12):
            at = slice(t * TILE, (t + 1) * TILE)
            for factor in (0.0, 0.5, 1.2):                      # lost, or joined with another weight
                w = p.copy()
                w[at] *= factor
                off = np.abs(w @ V / w.sum() - ref[0, h])
                assert np.any(off > 2 * tol[0, h]), (t, factor)
        # Its numerator alone, or its share of the denominator alone.
        t = int(rng.integers(0, tiles))
        w = p.copy()
        w[t * TILE:(t + 1) * TILE] = 0
        assert np.any(np.abs(w @ V / p.sum() - ref[0, h]) > 2 * tol[0, h])
