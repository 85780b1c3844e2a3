"""Tree and cross attention plan their ranges before the programmatic wait and plan again
when lengths or rows read after the wait differ.

pk_selftest_cross_stale_lengths makes the first plan come from other arrays, so that the
second one always runs where they differ.  Its output has to equal a normal call's bit
for bit (the same final plan) and report nothing.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from treelib import DEV, Case, clean, dev

pytestmark = pytest.mark.gpu

# (rows a sequence at most, heads per KV head, head dim): blocks of one query tile, one
# and two of them, two of them.
SHAPES = [(5, 4, 128), (70, 4, 128), (300, 1, 64)]


def _case(rows, G, D, n, longest, seed):
    rng = np.random.default_rng(seed)
    lens = [int(x) for x in rng.integers(1, longest, n)]
    lens[n // 2] = 0
    return Case(seed, lens, [int(x) for x in rng.integers(0, rows + 1, n - 1)] + [rows], G, 2, D, 16, False)


def _check(c, stale_lens, stale_cu, most, cap):
    args = (c.q, dev(c.cu), most, c.k, c.v, dev(c.tables), dev(np.asarray(c.lens, np.int32)), c.scale)
    ws = pk.new_workspace(pk.pk_tree_workspace_bytes(c.H, c.Hkv, c.D, most, cap), DEV)
    kw = dict(max_seq_len=cap, workspace=ws)
    want = torch.full(c.q.shape, 7.0, device=DEV)
    pk.paged_attention_cross(*args, out=want, **kw)
    clean()
    out = torch.full_like(want, 7.0)
    assert pk.pk_selftest_cross_stale_lengths(*args, dev(np.asarray(stale_lens, np.int32)), dev(np.asarray(stale_cu, np.int32)),
                                              out=out, **kw) == 0
    assert torch.equal(out, want)
    clean()
    return out


@pytest.mark.parametrize("rows,G,D", SHAPES)
@pytest.mark.parametrize("n,longest", [(5, 6000), (60, 1500), (384, 400)])
@pytest.mark.parametrize("kind", ["zeros", "fewer", "more", "reversed", "out of range", "same"])
@pytest.mark.parametrize("which", ["lengths", "rows", "both"])
def test_stale_arrays_give_the_normal_result(rows, G, D, n, longest, kind, which):
    c = _case(rows, G, D, n, longest, rows + n)
    cap, T = max(c.lens), int(c.cu[-1])
    rng = np.random.default_rng(n)
    counts = np.asarray(c.rows)

    def starts(x):
        return np.concatenate([[0], np.cumsum(x)])
    lens, cu = {
        "zeros": (np.zeros(n), np.zeros(n + 1)),
        "fewer": (np.asarray(c.lens) // 3, starts(counts // 3)),
        "more": (np.minimum(np.asarray(c.lens) * 3 + 200, cap), np.minimum(np.arange(n + 1) * rows, T)),
        "reversed": (np.asarray(c.lens)[::-1], starts(counts[::-1])),
        "out of range": (rng.integers(-2**31, 2**31, n), rng.integers(-2**31, 2**31, n + 1)),
        "same": (np.asarray(c.lens), c.cu),
    }[kind]
    out = _check(c, lens if which != "rows" else c.lens, cu if which != "lengths" else c.cu, rows, cap)
    if kind == "reversed" and which == "both" and n == 5:
        c.check(out, kind)


def test_a_call_without_keys_planned_from_one_with_keys():
    c = Case(3, [0, 0, 0], [4, 0, 9], 2, 1, 64, 16, False)
    out = _check(c, [16, 16, 16], [0, 4, 8, 13], 9, 16)
    assert torch.all(out == 0)


def test_more_sequences_than_are_planned_ahead():
    c = _case(3, 1, 64, 500, 300, 9)
    _check(c, np.zeros(500), np.zeros(501), 3, max(c.lens))


def test_refusals():
    c = Case(4, [40, 50], [4, 4], 1, 2, 64, 16, False)
    args = (c.q, dev(c.cu), 4, c.k, c.v, dev(c.tables), dev(np.asarray(c.lens, np.int32)), c.scale)
    good = dev(np.asarray(c.lens, np.int32)), dev(c.cu)
    for bad in ((good[0][:1], good[1]), (good[0], good[1][:2]), (good[0].cpu(), good[1])):
        with pytest.raises(ValueError):
            pk.pk_selftest_cross_stale_lengths(*args, *bad, max_seq_len=50)
    with pytest.raises(TypeError):
        pk.pk_selftest_cross_stale_lengths(*args, good[0].long(), good[1], max_seq_len=50)
