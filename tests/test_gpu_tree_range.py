"""Tree and cross attention over values at the ends of their range: sums of weights times
large values stay finite where the attention is, and small ones keep their bits."""
import numpy as np
import pytest
import torch

from treelib import DEV, Case, clean

pytestmark = pytest.mark.gpu


def _climb(c, s, first, rise):
    """Scores of sequence s that lie near 0 for its first keys and `rise` (base 2) above
    from key `first` on, for the query direction that all rows share."""
    c.q[:] = 1.0
    flat = torch.arange(c.lens[s], device=DEV)
    table = torch.as_tensor(c.tables[s].astype(np.int64), device=DEV)
    at = table[flat // c.B] * c.B + flat % c.B
    # q.k = D times the mean of k: a constant row gives rise / log2(e).
    step = rise * np.log(2.0) / (c.scale * c.D)
    rows = (torch.randn(c.lens[s], c.Hkv, c.D, generator=torch.Generator().manual_seed(s)) * 0.05).to(DEV)
    rows[first:] += step
    c.k.view(-1, c.Hkv, c.D)[at] = rows.to(torch.bfloat16)


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("rows,G,D", [(5, 4, 128), (70, 1, 64), (150, 2, 64), (200, 1, 128)])
@pytest.mark.parametrize("rise", [0.0, 9.0, 23.0, 40.0])
def test_large_values(tree, rows, G, D, rise):
    # Fewer than 2^9 keys with values below 2^117: no sum of weights of at most 1 leaves the range.
    c = Case(rows + int(rise), [300, 500, rows], [rows, rows, rows], G, 2, D, 16, tree)
    for s in range(3):
        _climb(c, s, 70 if s else 129, rise)
    c.v[:] = (c.v.float().clamp(-3.9, 3.9) * 2.0 ** 115).to(torch.bfloat16)
    c.check(c.run(), f"rise {rise}")
    c.check(c.run(torch.bfloat16), f"rise {rise}, bf16")
    clean()


@pytest.mark.parametrize("rise", [0.0, -23.0, 23.0])
def test_small_values(rise):
    # Parts that start from the reference of a sequence with other scores.
    c = Case(3, [400] * 300, [3] * 300, 2, 2, 64, 16, False)
    for s in range(0, 300, 2):
        _climb(c, s, 0, rise)
    c.v[:] = (c.v.float() * 2.0 ** -60).to(torch.bfloat16)
    c.check(c.run())
    clean()
