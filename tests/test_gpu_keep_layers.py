"""Compaction of several layers: a layer of which one pointer is bad keeps both its K and
its V as they were."""
import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from paged_kv_cache_122_gb300 import _native
from test_gpu_accept_keep import Pool
from treelib import bits, clean

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("fault", ["null", "unaligned"])
@pytest.mark.parametrize("layers,bad", [(2, 1), (5, 0), (70, 66)])
def test_a_layer_with_one_bad_pointer_is_left_alone(which, fault, layers, bad):
    p = Pool(layers, [6, 9, 1, 40], 20, 2, 64, 8, layers=layers)
    before = [[bits(c) for c in caches] for caches in (p.k, p.v)]
    want = [[p.want(c) for c in caches] for caches in (p.k, p.v)]
    ptrs = [pk.LayerPointers(p.k), pk.LayerPointers(p.v)]
    ptrs[which].ptrs[bad] = 0 if fault == "null" else int(ptrs[which].ptrs[bad]) + 8
    pk.pk_keep_tokens_layers(*ptrs, *p.lists(40))
    assert pk.pk_get_device_error() == _native.DEVERR_POINTER
    for i, caches in enumerate((p.k, p.v)):
        for l in range(layers):
            assert np.array_equal(bits(caches[l]), before[i][l] if l == bad else want[i][l]), (i, l)
    assert any(not np.array_equal(a, b) for a, b in zip(before[0], want[0]))
    clean()
