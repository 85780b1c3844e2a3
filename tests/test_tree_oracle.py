"""The float64 references of tree verification, against closed forms and the causal
reference.  CPU only."""
import numpy as np

import oracle
from oracle import tree_ref as R


def _pool(seed, lens, Hkv, D, B):
    rng = np.random.default_rng(seed)
    need = [-(-n // B) for n in lens]
    ids = rng.permutation(sum(need) + 2).astype(np.int32)
    tables = np.full((len(lens), max(need)), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = ids[at:at + n]
        at += n
    def rand(*shape):
        return (rng.standard_normal(shape).astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    return rng, tables, rand(len(ids), B, Hkv, D), rand(len(ids), B, Hkv, D), rand


def test_a_chain_is_the_causal_reference():
    lens, rows = [9, 30, 4], [4, 1, 4]
    _, tables, k, v, rand = _pool(1, lens, 2, 8, 8)
    cu = [0, 4, 5, 9]
    q = rand(9, 4, 8)
    mask = np.concatenate([R.ancestors_mask([-1] + list(range(n - 1)), 1) for n in rows])
    got = R.masked_attention(q, k, v, tables, lens, cu, 0.3, 8, mask)[0]
    want = oracle.paged_multi_query_attention(q, k, v, tables, lens, cu, 0.3, 8)
    assert np.abs(got - want).max() < 1e-12


def test_cross_attention_is_every_key_and_empty_rows_are_zero():
    lens = [11, 0, 3]
    _, tables, k, v, rand = _pool(2, [11, 1, 3], 1, 4, 8)
    q = rand(5, 2, 4)
    out, spread, size, _ = R.masked_attention(q, k, v, tables, lens, [0, 2, 4, 5], 0.5, 8)
    assert np.all(out[2:4] == 0) and np.all(size[2:4] == 0)
    K = oracle.bf16_bits_to_f64(oracle.gather_sequence(k, tables[0], 11, 8, 0))
    V = oracle.bf16_bits_to_f64(oracle.gather_sequence(v, tables[0], 11, 8, 0))
    qq = oracle.bf16_bits_to_f64(q[1, 1])
    w = np.exp(0.5 * K @ qq)
    assert np.abs(out[1, 1] - w @ V / w.sum()).max() < 1e-12
    assert np.all(spread <= 2 * size + 1e-12)


def test_masks_of_siblings_and_of_nothing():
    parents = [-1, 0, 0, 1, 2]
    mask = R.ancestors_mask(parents, 1)
    assert mask[:, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0b10101]
    wide = R.ancestors_mask([-1] + list(range(69)), 2)
    assert int(wide[69, 1]) == 0b111111 and int(wide[69, 0]) == (1 << 64) - 1
    _, tables, k, v, rand = _pool(3, [5], 1, 4, 8)
    q = rand(5, 1, 4)
    mask[4, 0] = 0
    out = R.masked_attention(q, k, v, tables, [5], [0, 5], 1.0, 8, mask)[0]
    assert np.all(out[4] == 0)
    first = oracle.bf16_bits_to_f64(oracle.gather_sequence(v, tables[0], 5, 8, 0))[0]
    assert np.abs(out[0, 0] - first).max() < 1e-12            # node 0 sees itself alone


def test_accepted_path_and_rows():
    tokens, parents, targets = [9, 5, 7, 7, 3], [-1, 0, 0, 0, 2], [7, 1, 3, 3, 8]
    assert R.accept(tokens, parents, targets) == [0, 2, 4]     # the lowest of the two sevens
    assert R.accept([], [], []) == []
    _, tables, k, _, _ = _pool(4, [20], 1, 4, 8)
    out = R.keep(k, tables, [20], [0, 5], [[0, 2, 4]], 8)
    def row(c, t):
        return c[tables[0][t // 8], t % 8].tolist()
    assert [row(out, t) for t in range(15, 20)] == [row(k, t) for t in (15, 17, 19, 18, 19)]
