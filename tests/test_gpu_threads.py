"""Calls that share the cached workspace of one stream, made by several host threads at
once: each call's kernels stay together, so that every call joins its own parts."""
import threading

import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from paged_kv_cache_122_gb300 import workloads as W
from treelib import DEV, Case, clean, dev

pytestmark = pytest.mark.gpu


def _tree(seed, lens, rows, G, Hkv, D, tree):
    c = Case(seed, lens, rows, G, Hkv, D, 16, tree)
    cu, tb, sl, most = dev(c.cu), dev(c.tables), dev(np.asarray(c.lens, np.int32)), max(rows)
    mask = dev(c.mask.view(np.int64)) if tree else None

    def call():
        kw = dict(out_dtype=torch.float32, max_seq_len=max(lens))
        if tree:
            return pk.paged_attention_tree(c.q, cu, most, mask, c.k, c.v, tb, sl, c.scale, **kw)
        return pk.paged_attention_cross(c.q, cu, most, c.k, c.v, tb, sl, c.scale, **kw)
    return call


def _decode(seed, lens, H, Hkv, D):
    w = W.custom(seed, lens, H, Hkv, D, 16)
    t = W.make_tensors(w, torch.device(DEV))
    return lambda: pk.paged_attention_decode(t["q"], t["k_cache"], t["v_cache"], t["block_tables"], t["seq_lens"], w.scale,
                                             out_dtype=torch.float32, max_seq_len=w.max_seq_len)


@pytest.mark.parametrize("side", [False, True])
def test_threads_on_one_stream(side):
    # Blocks of one and of two query tiles, both head dims, and decode: slots of every
    # layout, and outputs of every length.
    calls = [_tree(1, [5000, 700], [20, 7], 4, 2, 128, True), _tree(2, [3000], [300], 2, 1, 64, False),
             _tree(3, [9000], [2], 1, 4, 64, False), _decode(4, [4000] * 3 + [900] * 29, 32, 8, 128)]
    want = [call() for call in calls]
    torch.cuda.synchronize()
    clean()
    stream = torch.cuda.Stream() if side else torch.cuda.default_stream()
    start = threading.Barrier(len(calls))
    wrong, failures = [None] * len(calls), []

    def work(i):
        try:
            with torch.cuda.stream(stream):
                bad = torch.zeros((), dtype=torch.int64, device=DEV)
                start.wait()
                for _ in range(150):
                    out = calls[i]()
                    bad += (out != want[i]).sum()
                wrong[i] = bad
        except Exception as e:                                 # (told by the main thread)
            failures.append(e)
            start.abort()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failures, failures
    assert [int(b) for b in wrong] == [0] * len(calls)
    clean()
