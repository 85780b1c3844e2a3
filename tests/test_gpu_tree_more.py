"""Tree verification where earlier cases do not reach: workspaces that do not do, masks of
more sequences than are planned ahead, paths of every node, a whole step in a graph."""
import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from oracle import tree_ref as R
from test_gpu_accept_keep import Pool
from treelib import DEV, Case, bits, clean, dev, parents_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tree", [True, False])
def test_workspaces_that_do_not_do(tree):
    c = Case(1, [300, 20], [9, 9], 2, 1, 64, 16, tree)
    want = c.run()
    need = pk.pk_tree_workspace_bytes(2, 1, 64, 9, 300)
    assert need > 0
    for size in (16, need - 1):
        with pytest.raises(ValueError, match="too small"):
            c.run(workspace=torch.empty(size, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="contiguous tensor on"):
        c.run(workspace=torch.empty(need, dtype=torch.uint8))
    room = torch.empty(need + 16, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError, match="contiguous tensor on"):
        c.run(workspace=torch.empty(2 * need, dtype=torch.uint8, device=DEV)[::2])
    with pytest.raises(pk.PagedKVError) as e:
        c.run(workspace=room[8:8 + need])
    assert e.value.status == -6
    # One that is just large enough, with a guard behind it; and none where nothing is cut.
    room[need:] = 77
    assert torch.equal(c.run(workspace=room[:need]), want) and torch.all(room[need:] == 77)
    c = Case(2, [128, 20], [9, 9], 2, 1, 64, 16, tree)
    assert pk.pk_tree_workspace_bytes(2, 1, 64, 9, 128) == 0
    c.check(c.run(workspace=room[:0]))
    clean()


@pytest.mark.parametrize("n,nodes,G", [(800, 5, 1), (385, 3, 4), (390, 40, 4)])
def test_masks_of_more_sequences_than_are_planned_ahead(n, nodes, G):
    rng = np.random.default_rng(n)
    rows = [int(x) for x in rng.integers(0, nodes + 1, n)]
    lens = [r + int(x) for r, x in zip(rows, rng.integers(0, 200, n))]
    c = Case(n, lens, rows, G, 1, 64, 16, True)
    c.mask[::5] = 0
    c.check(c.run())
    c.check(c.run(torch.bfloat16))
    clean()


@pytest.mark.parametrize("sizes", [[1], [2, 1, 3], [512, 129, 128, 127], [8192, 1000]])
def test_trees_whose_every_node_is_accepted(sizes):
    T = sum(sizes)
    rng = np.random.default_rng(T)
    tok = rng.integers(0, 1 << 40, T)
    tgt = np.empty(T, np.int64)
    cu = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    for a, b in zip(cu[:-1], cu[1:]):                         # a chain that the target agrees with
        tgt[a:b - 1], tgt[b - 1] = tok[a + 1:b], -7
    parents = np.concatenate([np.arange(-1, n - 1) for n in sizes]).astype(np.int32)
    lens = np.asarray([n + 5 for n in sizes], np.int32)
    most = max(sizes)
    acc, num, nxt, new = pk.accept_tree(dev(tok), dev(parents), dev(tgt), dev(cu), most, dev(lens))
    for s, n in enumerate(sizes):
        assert acc[s].tolist() == list(range(n)) + [-1] * (most - n)
    assert num.tolist() == sizes and nxt.tolist() == [-7] * len(sizes) and new.tolist() == lens.tolist()
    if most < 8192:                                           # nothing moves
        p = Pool(3, sizes, 20, 2, 64, 8)
        p.paths = [list(range(n)) for n in sizes]
        k, v = p.k[0].clone(), p.v[0].clone()
        pk.keep_tokens(k, v, dev(p.tables), dev(p.lens), dev(p.cu), acc, num)
        assert torch.equal(k, p.k[0]) and torch.equal(v, p.v[0])
    clean()


def test_a_long_path_moves_by_one():
    # Every node but the second of a chain of 1,000: each row goes to the place before it.
    p = Pool(4, [1000, 300], 13, 3, 64, 16)
    p.paths = [[0] + list(range(2, 1000)), list(range(1, 300))]
    want = p.want(p.k[0]), p.want(p.v[0])
    pk.keep_tokens(p.k[0], p.v[0], *p.lists(1000))
    assert np.array_equal(bits(p.k[0]), want[0]) and np.array_equal(bits(p.v[0]), want[1])
    clean()


@pytest.mark.parametrize("side", [False, True])
def test_a_step_in_a_graph(side):
    # Accepted paths, their rows in two layers, and attention to what is kept, replayed with
    # other tokens, trees and lengths in the same tensors; then the same calls on a stream.
    sizes, ctx = [20, 1, 33], [700, 13, 90]
    c = Case(5, [a + b for a, b in zip(sizes, ctx)], sizes, 4, 2, 128, 16, True)
    cu, tb, sl = dev(c.cu), dev(c.tables), dev(np.asarray(c.lens, np.int32))
    T, most = sum(sizes), max(sizes)
    tok, tgt = (torch.zeros(T, dtype=torch.int64, device=DEV) for _ in range(2))
    par = torch.zeros(T, dtype=torch.int32, device=DEV)
    k, v = [c.k.clone(), (c.k * 2).clone()], [c.v.clone(), (c.v * 2).clone()]
    layers = pk.LayerPointers(k), pk.LayerPointers(v)

    def step():
        acc, num, nxt, new = pk.accept_tree(tok, par, tgt, cu, most, sl)
        pk.pk_keep_tokens_layers(*layers, tb, sl, cu, acc, num)
        out = pk.paged_attention_cross(c.q, cu, most, k[0], v[0], tb, new, c.scale, out_dtype=torch.float32, max_seq_len=723)
        return acc, num, nxt, new, out
    stream = torch.cuda.Stream()
    if side:
        def run():
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                res = step()
            torch.cuda.current_stream().wait_stream(stream)
            return res
    else:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            held = step()

        def run():
            graph.replay()
            return held
    for trial in range(5):
        rng = np.random.default_rng(trial)
        parents = [parents_of(n, rng) for n in sizes]
        hosts = rng.integers(0, 2, T), rng.integers(0, 2, T)
        tok.copy_(dev(hosts[0]))
        tgt.copy_(dev(hosts[1]))
        par.copy_(dev(np.concatenate([np.asarray(p, np.int32) for p in parents])))
        c.lens = [a + int(rng.integers(0, b + 1)) for a, b in zip(sizes, ctx)]
        sl.copy_(dev(np.asarray(c.lens, np.int32)))
        before = [bits(x) for x in k + v]
        acc, num, nxt, new, out = run()
        paths = [R.accept(hosts[0][a:b], p, hosts[1][a:b]) for p, a, b in zip(parents, c.cu[:-1], c.cu[1:])]
        assert [acc[s, :int(num[s])].tolist() for s in range(3)] == paths
        assert nxt.tolist() == [int(hosts[1][a + p[-1]]) for a, p in zip(c.cu[:-1], paths)]
        for old, cache in zip(before, k + v):
            assert np.array_equal(bits(cache), R.keep(old, c.tables, c.lens, c.cu, paths, c.B))
        c.lens = [L - n + len(p) for L, n, p in zip(c.lens, sizes, paths)]
        assert new.tolist() == c.lens
        c.k, c.v, c.mask = k[0], v[0], None
        c.check(out, f"trial {trial}")
    clean()
