"""Tree and cross attention against the float64 reference, at the lengths, masks and
layouts where they can go wrong; bounds are derived in oracle/tree_ref.py."""
import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from paged_kv_cache_122_gb300 import _native
from treelib import DEV, Case, clean, dev

pytestmark = pytest.mark.gpu

LENS = [1, 2, 63, 64, 65, 127, 128, 129, 191, 192, 193, 256, 700, 1500]


@pytest.mark.parametrize("D,B", [(128, 16), (64, 8), (128, 32), (64, 32), (128, 8)])
@pytest.mark.parametrize("G,Hkv,nodes", [(1, 3, 5), (2, 2, 17), (4, 2, 26), (4, 1, 33), (8, 1, 16), (8, 1, 40), (16, 1, 9),
                                         (1, 1, 130)])
def test_tree_matches_reference(G, Hkv, nodes, D, B):
    rng = np.random.default_rng(G * 1000 + nodes + D + B)
    rows = [min(n, int(rng.integers(1, nodes + 1))) for n in LENS]
    rows[-1] = rows[-3] = nodes
    c = Case(nodes + G, LENS, rows, G, Hkv, D, B, True)
    c.check(c.run(), "fp32")
    c.check(c.run(torch.bfloat16), "bf16")
    clean()


@pytest.mark.parametrize("D,B", [(128, 16), (64, 16), (128, 8), (64, 32)])
@pytest.mark.parametrize("G,Hkv,most", [(1, 2, 1), (1, 2, 129), (4, 2, 70), (8, 1, 33), (16, 1, 20), (2, 3, 300)])
def test_cross_matches_reference(G, Hkv, most, D, B):
    rng = np.random.default_rng(most + D)
    lens = [0, 5, 64, 128, 129, 0, 320, 1000, 77]
    rows = [int(x) for x in rng.integers(0, most + 1, len(lens))]
    rows[1] = rows[5] = most                                  # more rows than keys; rows without keys
    c = Case(most + B, lens, rows, G, Hkv, D, B, False)
    c.check(c.run(), "fp32")
    c.check(c.run(torch.bfloat16), "bf16")
    clean()


@pytest.mark.parametrize("off", range(0, 40, 3))
def test_trees_that_start_anywhere_in_a_tile(off):
    # The mask's words against the tile's: every shift, trees that end inside a tile and
    # that span three of them.
    lens = [90 + off, 128 + off, 250 + off]
    c = Case(off, lens, [min(lens[0], 80), 66, 200], 1, 1, 64, 8, True)
    c.check(c.run(), f"offset {off}")


def test_masks_of_any_kind():
    # Not ancestors only: random bits, rows that see nothing, bits behind the tree.
    c = Case(3, [200, 40, 64, 3, 500], [70, 40, 64, 3, 130], 2, 2, 64, 16, True, words=4)
    rng = np.random.default_rng(3)
    c.mask = rng.integers(0, 2**63, c.mask.shape, dtype=np.uint64) * 2 + rng.integers(0, 2, c.mask.shape, dtype=np.uint64)
    c.mask[::7] = 0
    out = c.run()
    c.check(out)
    for s in (1, 2, 3):                                       # no context: an empty mask is an empty row
        for r in range(c.cu[s], c.cu[s + 1]):
            if r % 7 == 0:
                assert torch.all(out[r] == 0)
    clean()


def test_a_chain_is_the_causal_call():
    c = Case(5, [300, 17, 129, 64], [16, 16, 2, 9], 1, 4, 128, 16, True)
    c.mask = np.array([[(1 << (r + 1)) - 1] for n in c.rows for r in range(n)], np.uint64)
    out = c.run()
    c.check(out)
    causal = pk.paged_attention_multi_query(c.q, dev(c.cu), 16, c.k, c.v, dev(c.tables), dev(np.asarray(c.lens, np.int32)),
                                            c.scale, out_dtype=torch.float32, max_seq_len=300)
    ref = c.reference()
    from oracle import tree_ref as R
    tol = R.bound(*ref, 300, 128, False)
    assert np.all(np.abs((out - causal).double().cpu().numpy()) <= 2 * tol)


@pytest.mark.parametrize("tree", [True, False])
@pytest.mark.parametrize("rows,G,Hkv,D", [(8, 4, 2, 128), (100, 1, 1, 64), (300, 2, 1, 128), (5, 16, 1, 64)])
def test_one_long_sequence_is_split_over_the_gpu(tree, rows, G, Hkv, D):
    c = Case(rows, [20000], [rows], G, Hkv, D, 32, tree)
    c.check(c.run())
    c.check(c.run(torch.bfloat16))
    clean()


@pytest.mark.parametrize("rows", [3, 200])
def test_many_sequences_beyond_a_thread_each(rows):
    rng = np.random.default_rng(rows)
    n = 800 if rows == 3 else 390
    lens = [int(x) for x in rng.integers(0, 200, n)]
    c = Case(rows, lens, [int(x) for x in rng.integers(0, rows + 1, n)], 1, 1, 64, 16, False)
    c.check(c.run())
    clean()


def test_strong_scores_negative_zero_and_large_scales():
    for scale in (-0.3, 0.0, 4.0, 1e-30, -1e-44):
        c = Case(11, [130, 400, 65], [65, 3, 65], 2, 1, 64, 16, True, strength=1.0)
        c.scale = scale
        c.check(c.run(), f"scale {scale}")
    c = Case(12, [1000, 300], [40, 200], 4, 1, 128, 16, False, strength=30.0)
    # Scores that climb along the keys: the reference max moves in every tile.
    ramp = torch.linspace(0, 6, c.blocks * 16, device=DEV).view(c.blocks, 16, 1, 1)
    order = torch.as_tensor(c.tables[0][:63].astype(np.int64), device=DEV)
    c.k[order] = (c.q[0, 0].float() * 0.05 * ramp[:63]).to(torch.bfloat16)
    c.check(c.run())
    clean()


@pytest.mark.parametrize("tree", [True, False])
def test_rows_behind_the_sequences_and_bad_keys_are_not_seen(tree):
    c = Case(7, [100, 257, 13], [13, 70, 13], 2, 2, 64, 16, tree)
    want = c.run()
    clean()
    # NaN and infinities in every row of the pool that no sequence owns: behind the last
    # key of a page, and in pages of nobody.
    owned = torch.zeros(c.blocks * c.B, dtype=torch.bool)
    for s, n in enumerate(c.lens):
        for j in range(n):
            owned[int(c.tables[s][j // c.B]) * c.B + j % c.B] = True
    free = ~owned.view(c.blocks, c.B).to(DEV)
    c.k[free] = float("nan")
    c.v[free] = float("inf")
    assert torch.equal(c.run(), want)
    clean()
    # A page that is not there: its keys are left out, whatever lies in the ring.
    c.tables[1, 5] = c.blocks + 3
    c.tables[1, 9] = -1
    out = c.run()
    assert pk.pk_get_device_error() == _native.DEVERR_BLOCK_ID
    assert torch.isfinite(out).all() and torch.equal(out[:13], want[:13]) and torch.equal(out[83:], want[83:])
    seen = np.ones(257, bool)
    seen[80:96] = seen[144:160] = False
    _check_with_keys(c, out, 1, seen)


def _check_with_keys(c, out, s, seen):
    """Sequence s of ``out`` against attention over the keys that are there."""
    q0, n, L = int(c.cu[s]), c.rows[s], c.lens[s]
    k, v = (x.double().cpu() for x in (c.k, c.v))
    for g in range(c.H):
        h = g // (c.H // c.Hkv)
        K = torch.stack([k[c.tables[s][j // c.B], j % c.B, h] if seen[j] else torch.zeros(c.D).double() for j in range(L)])
        V = torch.stack([v[c.tables[s][j // c.B], j % c.B, h] if seen[j] else torch.zeros(c.D).double() for j in range(L)])
        vis = torch.as_tensor(np.tile(seen, (n, 1)))
        if c.mask is not None:
            for r in range(n):
                for i in range(n):
                    vis[r, L - n + i] &= bool((int(c.mask[q0 + r, i // 64]) >> (i % 64)) & 1)
        x = (c.q[q0:q0 + n, g].double().cpu() @ K.T * c.scale).masked_fill(~vis, -np.inf)
        p = torch.nan_to_num(torch.softmax(x, -1))
        want = p @ V
        spread = (p[:, :, None] * (V[None] - want[:, None]).abs()).sum(1)
        tol = 1.01 * 2.0 ** -8 * spread + 1e-4 * (p @ V.abs()) + 1e-30      # (2^-8: half a step of a bf16 weight)
        assert torch.all((out[q0:q0 + n, g].double().cpu() - want).abs() <= tol)


def test_a_key_that_is_not_finite_shows_in_the_rows_that_see_it():
    c = Case(8, [150], [6], 1, 1, 64, 16, True)
    c.mask = np.array([[1], [3], [5], [9], [17], [33]], np.uint64)       # node 0 and itself
    want = c.run()
    j = 150 - 6 + 3
    c.k[int(c.tables[0][j // 16]), j % 16] = float("nan")
    out = c.run()
    assert torch.isnan(out[3]).all()
    keep = [0, 1, 2, 4, 5]
    assert torch.equal(out[keep], want[keep])


def test_bad_lengths_leave_their_rows_alone():
    c = Case(9, [100, 130, 64, 40], [4, 4, 4, 4], 2, 1, 64, 16, True)
    want = c.run()
    sl, cu = dev(np.asarray(c.lens, np.int32)), dev(c.cu)
    mask = dev(c.mask.view(np.int64))

    def run(lens, cu=cu, most=4, max_seq_len=130, total=16):
        out = torch.full((total, c.H, c.D), 7.0, device=DEV)
        pk.paged_attention_tree(c.q[:total], cu, most, mask[:total], c.k, c.v, dev(c.tables), lens, c.scale, out=out,
                                max_seq_len=max_seq_len)
        return out, pk.pk_get_device_error()
    for bad in (-1, 131, 3, 2**31 - 1, -2**31):
        lens = sl.clone()
        lens[1] = bad
        out, err = run(lens)
        assert err == _native.DEVERR_SEQ_LEN
        assert torch.all(out[4:8] == 7) and torch.equal(out[:4], want[:4]) and torch.equal(out[8:], want[8:])
    for rows in ([0, 4, 9, 9, 13], [0, 4, 3, 7, 11], [0, 4, 8, 12, 17], [0, 4, 8, 12, 2**31 - 1], [-4, 0, 4, 8, 12]):
        out, err = run(sl, dev(np.asarray(rows, np.int32)))
        assert err == _native.DEVERR_SEQ_LEN and torch.isfinite(out).all()
    # Rows that no sequence owns, and a batch padded with sequences of no rows.
    out, err = run(dev(np.asarray([100, 130, 0, 0], np.int32)), dev(np.asarray([0, 4, 8, 8, 8], np.int32)))
    assert err == 0 and torch.all(out[8:] == 7) and torch.equal(out[:8], want[:8])


def test_no_keys_at_all_is_zeros():
    c = Case(10, [0, 0], [3, 140], 1, 2, 64, 16, False)
    out = torch.full((143, 2, 64), 7.0, device=DEV)
    c.run(out=out, max_seq_len=0)
    assert torch.all(out == 0)
    clean()


def test_refusals_of_the_binding():
    c = Case(13, [40, 50], [4, 4], 1, 2, 64, 16, True)
    with pytest.raises(ValueError):
        c.run(out=torch.empty(8, 2, 128, device=DEV))
    with pytest.raises(TypeError):
        c.run(out_dtype=torch.float16)
    with pytest.raises(ValueError):
        c.run(out=torch.empty(8, 2, 128, device=DEV, dtype=torch.float32)[..., ::2])
    with pytest.raises(ValueError, match="workspace"):
        c.run(max_seq_len=64 if c.tables.shape[1] * 16 < 129 else 200, workspace=torch.empty(16, dtype=torch.uint8))
    c.mask = c.mask[:-1]
    with pytest.raises(ValueError, match="tree_mask"):
        c.run()
    c.mask = np.zeros((8, 0), np.uint64)
    with pytest.raises(pk.PagedKVError):
        c.run()
    with pytest.raises(ValueError):
        pk.paged_attention_cross(c.q, dev(c.cu)[:2], 4, c.k, c.v, dev(c.tables), dev(np.asarray(c.lens, np.int32)), 1.0)
    with pytest.raises(pk.PagedKVError):
        pk.paged_attention_cross(c.q, dev(c.cu), 4, c.k, c.v, dev(c.tables), dev(np.asarray(c.lens, np.int32)), 1.0,
                                 max_seq_len=1 << 33)


def test_an_output_that_starts_on_any_16_bytes():
    c = Case(14, [300, 20], [9, 9], 2, 1, 64, 16, True)
    want = c.run(torch.bfloat16)
    room = torch.zeros(want.numel() + 8, dtype=torch.bfloat16, device=DEV)
    out = room[8:].view(want.shape)
    assert out.data_ptr() % 32 == 16
    assert torch.equal(c.run(out=out), want)


def test_wide_mask_rows_and_a_larger_bound():
    c = Case(15, [400, 90], [30, 12], 4, 1, 128, 16, True)
    want = c.run()
    c.mask = np.concatenate([c.mask, np.full((len(c.mask), 3), 2**64 - 1, np.uint64)], axis=1)
    out = pk.paged_attention_tree(c.q, dev(c.cu), 200, dev(c.mask.view(np.int64)), c.k, c.v, dev(c.tables),
                                  dev(np.asarray(c.lens, np.int32)), c.scale, out_dtype=torch.float32)
    ref = c.reference()
    from oracle import tree_ref as R
    assert np.all(np.abs((out - want).double().cpu().numpy()) <= 2 * R.bound(*ref, 400, 128, False))
    clean()
