"""The accepted path of a tree and the move of its rows: exact against the
references, with their refusals."""
import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from oracle import tree_ref as R
from paged_kv_cache_122_gb300 import _native
from treelib import DEV, bits, clean, dev, parents_of

pytestmark = pytest.mark.gpu


def _trees(seed, sizes, vocab):
    rng = np.random.default_rng(seed)
    parents = [parents_of(n, rng) if n else [] for n in sizes]
    tokens = [rng.integers(0, vocab, n) for n in sizes]
    targets = [rng.integers(0, vocab, n) for n in sizes]
    return parents, tokens, targets


@pytest.mark.parametrize("vocab", [1, 2, 3, 1 << 40])
def test_accept_matches_reference(vocab):
    sizes = [1, 0, 2, 5, 64, 129, 700, 8192, 0, 33]
    parents, tokens, targets = _trees(vocab % 97, sizes, vocab)
    cu = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    lens = np.asarray([n + 11 * i for i, n in enumerate(sizes)], np.int32)

    def cat(x, dtype):
        return dev(np.concatenate([np.asarray(a, dtype) for a in x]))
    acc, num, nxt, new = pk.accept_tree(cat(tokens, np.int64), cat(parents, np.int32), cat(targets, np.int64), dev(cu), 8192,
                                        dev(lens))
    assert acc.shape == (10, 8192)
    for s, n in enumerate(sizes):
        path = R.accept(tokens[s], parents[s], targets[s])
        assert acc[s].tolist() == path + [-1] * (8192 - len(path))
        assert int(num[s]) == len(path) and int(new[s]) == lens[s] - n + len(path)
        assert int(nxt[s]) == (targets[s][path[-1]] if path else -1)
    clean()


def test_accept_ties_padding_and_bad_parents():
    tok = dev(np.asarray([1, 5, 5, 5, 6, 6, 9], np.int64))
    tgt = dev(np.asarray([5, 6, 6, 6, 0, 9, 4], np.int64))
    for parents, path in (([-1, 0, 0, 0, 2, 3, 5], [0, 1]), ([7, -1, 0, 0, 2, 3, 5], [0, 2, 4]),
                          ([0, 1, 2, 0, 3, 3, 5], [0, 3, 4]), ([-1, 9, 9, -5, 4, 2**31 - 1, -2**31], [0])):
        acc, num, nxt, new = pk.accept_tree(tok, dev(np.asarray(parents, np.int32)), tgt, dev(np.asarray([0, 7], np.int32)), 7,
                                            dev(np.asarray([7], np.int32)))
        assert acc[0, :int(num)].tolist() == path and int(new) == len(path)
    clean()


def test_accept_bad_rows_are_reported():
    tok = torch.zeros(6, dtype=torch.int64, device=DEV)
    par = torch.zeros(6, dtype=torch.int32, device=DEV)
    for cu, lens, most in (([0, 3, 2], [9, 9], 6), ([0, 3, 7], [9, 9], 6), ([-1, 3, 6], [9, 9], 6), ([0, 3, 6], [9, 2], 6),
                           ([0, 2, 6], [9, 9], 3), ([0, 3, 6], [9, -4], 6)):
        acc, num, nxt, new = pk.accept_tree(tok, par, tok, dev(np.asarray(cu, np.int32)), most, dev(np.asarray(lens, np.int32)))
        assert pk.pk_get_device_error() == _native.DEVERR_SEQ_LEN
        bad = [s for s in range(2) if not (0 <= cu[s] <= cu[s + 1] <= 6 and cu[s + 1] - cu[s] <= min(most, lens[s]))]
        for s in bad:
            assert int(num[s]) == 0 and int(nxt[s]) == -1 and int(new[s]) == lens[s] and torch.all(acc[s] == -1)
    with pytest.raises(pk.PagedKVError):
        pk.accept_tree(tok, par, tok, dev(np.asarray([0, 6], np.int32)), 8193, dev(np.asarray([9], np.int32)))
    with pytest.raises(ValueError):
        pk.accept_tree(tok, par[:5], tok, dev(np.asarray([0, 6], np.int32)), 6, dev(np.asarray([9], np.int32)))


def test_accept_into_the_lengths_themselves():
    sizes = [3, 70, 1]
    parents, tokens, targets = _trees(5, sizes, 2)
    cu = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    lens = dev(np.asarray([9, 70, 4], np.int32))
    t = [dev(np.concatenate([np.asarray(a, d) for a in x])) for x, d in ((tokens, np.int64), (parents, np.int32), (targets, np.int64))]
    rows = dev(cu)
    want = pk.accept_tree(*t, rows, 70, lens)
    acc, num, nxt = (torch.empty_like(x) for x in want[:3])
    st = _native.load().pk_accept_tree(acc.data_ptr(), num.data_ptr(), nxt.data_ptr(), lens.data_ptr(), t[0].data_ptr(),
                                       t[1].data_ptr(), t[2].data_ptr(), 74, rows.data_ptr(), 70, lens.data_ptr(), 3,
                                       torch.cuda.current_stream().cuda_stream)
    assert st == 0 and all(torch.equal(a, b) for a, b in zip((acc, num, nxt, lens), want))
    clean()


class Pool:
    def __init__(self, seed, sizes, ctx, Hkv, D, B, layers=1):
        rng = np.random.default_rng(seed)
        self.B, self.sizes = B, sizes
        self.lens = np.asarray([int(rng.integers(0, ctx + 1)) + n for n in sizes], np.int32)
        self.cu = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        need = [-(-int(n) // B) for n in self.lens]
        ids = rng.permutation(sum(need) + 3).astype(np.int32)
        self.tables = np.full((len(sizes), max(need) + 1), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.tables[s, :n] = ids[at:at + n]
            at += n
        gen = torch.Generator(device=DEV).manual_seed(seed)
        self.k, self.v = ([torch.randn(len(ids), B, Hkv, D, generator=gen, device=DEV).to(torch.bfloat16) for _ in range(layers)]
                          for _ in range(2))
        self.paths = []
        for n in sizes:
            parents, node, path = parents_of(n, rng) if n else [], int(rng.integers(n)) if n else -1, []
            while node >= 0:
                path.append(node)
                node = parents[node]
            self.paths.append(path[::-1])

    def lists(self, stride):
        acc = np.full((len(self.sizes), stride), -1, np.int32)
        for s, p in enumerate(self.paths):
            acc[s, :len(p)] = p
        return dev(self.tables), dev(self.lens), dev(self.cu), dev(acc), dev(np.asarray([len(p) for p in self.paths], np.int32))

    def want(self, cache):
        return R.keep(bits(cache), self.tables, self.lens, self.cu, self.paths, self.B)


@pytest.mark.parametrize("Hkv,D,B", [(8, 128, 16), (1, 64, 8), (3, 64, 32), (3, 128, 8), (32, 128, 16)])
def test_keep_matches_reference(Hkv, D, B):
    p = Pool(Hkv + D, [1, 7, 0, 30, 64, 200, 2], 40, Hkv, D, B, layers=3)
    want = [[p.want(c) for c in caches] for caches in (p.k, p.v)]
    one = p.k[0].clone(), p.v[0].clone()
    pk.keep_tokens(*one, *p.lists(200))
    pk.pk_keep_tokens_layers(p.k, p.v, *p.lists(200))
    for l in range(3):
        assert np.array_equal(bits(p.k[l]), want[0][l]) and np.array_equal(bits(p.v[l]), want[1][l])
    assert torch.equal(one[0], p.k[0]) and torch.equal(one[1], p.v[0])
    clean()


def test_keep_every_second_of_a_long_tree():
    # More tokens than a pass takes: rows of one pass are sources of none after it.
    p = Pool(1, [900, 901], 13, 4, 128, 16)
    p.paths = [list(range(0, 900, 2)), list(range(1, 901, 3))]
    want = p.want(p.k[0]), p.want(p.v[0])
    pk.keep_tokens(p.k[0], p.v[0], *p.lists(901))
    assert np.array_equal(bits(p.k[0]), want[0]) and np.array_equal(bits(p.v[0]), want[1])
    clean()


def test_keep_refuses_bad_lists_and_blocks():
    p = Pool(2, [8, 8, 8], 20, 2, 64, 8)
    before = p.k[0].clone(), p.v[0].clone()
    good = list(p.paths)
    for bad in ([0, 2, 2], [0, 3, 1], [0, 8], [-1, 2], [5, 2**31 - 1]):
        p.paths = [good[0], bad, good[2]]
        k, v = before[0].clone(), before[1].clone()
        pk.keep_tokens(k, v, *p.lists(8))
        assert pk.pk_get_device_error() == _native.DEVERR_DRAFT
        p.paths = [good[0], [], good[2]]
        assert np.array_equal(bits(k), p.want(before[0])) and np.array_equal(bits(v), p.want(before[1]))
    p.paths = good
    tables, lens, cu, acc, num = p.lists(8)
    for count in (-1, 9, 2**31 - 1):
        k, v = before[0].clone(), before[1].clone()
        n = num.clone()
        n[:] = count
        pk.keep_tokens(k, v, tables, lens, cu, acc, n)
        assert pk.pk_get_device_error() == _native.DEVERR_DRAFT
        assert torch.equal(k, before[0]) and torch.equal(v, before[1])
    for bad in (-1, 7, 10**6):
        k, v = before[0].clone(), before[1].clone()
        l = lens.clone()
        l[:] = bad
        pk.keep_tokens(k, v, tables, l, cu, acc, num)
        assert pk.pk_get_device_error() == _native.DEVERR_SEQ_LEN
        assert torch.equal(k, before[0]) and torch.equal(v, before[1])
    t = tables.clone()
    t[:] = 10**6
    p.paths = [[0, 3], [0, 3], [0, 3]]
    _, _, _, acc, num = p.lists(8)
    k, v = before[0].clone(), before[1].clone()
    pk.keep_tokens(k, v, t, lens, cu, acc, num)
    assert pk.pk_get_device_error() == _native.DEVERR_BLOCK_ID
    assert torch.equal(k, before[0]) and torch.equal(v, before[1])
    with pytest.raises(ValueError):
        pk.keep_tokens(k, v[:-1], tables, lens, cu, acc, num)
    with pytest.raises(ValueError):
        pk.keep_tokens(k, v, tables, lens, cu, acc[:2], num)
    with pytest.raises(ValueError):
        pk.pk_keep_tokens_layers([k], [v, v], tables, lens, cu, acc, num)


def test_keep_layers_with_a_missing_layer():
    p = Pool(3, [6, 9], 20, 2, 64, 8, layers=2)
    want = p.want(p.k[0])
    k, v = pk.LayerPointers(p.k), pk.LayerPointers(p.v)
    k.ptrs[1] = 0
    before = p.k[1].clone()
    pk.pk_keep_tokens_layers(k, v, *p.lists(9))
    assert pk.pk_get_device_error() == _native.DEVERR_POINTER
    assert np.array_equal(bits(p.k[0]), want) and torch.equal(p.k[1], before)
