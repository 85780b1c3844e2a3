"""accept_tree refuses a bound beyond its trees before it allocates results for it."""
import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from treelib import DEV, clean, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bound", [8193, 2**31 - 1, 1 << 40])
def test_a_bound_beyond_the_trees_is_refused(bound):
    n = 256                                                    # (2^31 entries of each: 2 TB)
    z = torch.zeros(n, dtype=torch.int64, device=DEV)
    lens = torch.ones(n, dtype=torch.int32, device=DEV)
    rows = dev(np.arange(n + 1, dtype=np.int32))
    torch.cuda.reset_peak_memory_stats()
    held = torch.cuda.memory_allocated()
    with pytest.raises(pk.PagedKVError) as e:
        pk.accept_tree(z, lens, z, rows, bound, lens)
    assert e.value.status == -3 and torch.cuda.max_memory_allocated() == held
    acc, num, _, _ = pk.accept_tree(z, lens, z, rows, 8192, lens)
    assert acc.shape == (n, 8192) and torch.all(num == 1)
    clean()
