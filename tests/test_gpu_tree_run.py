"""Verification of drafted trees as a serving loop makes it: nodes appended by slots,
attended, accepted, moved together, their pages freed; in graphs, on streams, with
lengths that the call before writes; and the attention's bounded waits."""
import time

import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from oracle import tree_ref as R
from paged_kv_cache_122_gb300 import _native
from treelib import DEV, Case, bits, clean, dev, parents_of

pytestmark = pytest.mark.gpu


def test_serving_loop_keeps_the_cache_of_the_accepted_tokens():
    H, Hkv, D, B, blocks, layers = 8, 2, 64, 8, 96, 2
    rng = np.random.default_rng(0)
    gen = torch.Generator().manual_seed(0)
    bm = pk.BlockManager(blocks, B)
    kc, vc = ([torch.zeros(blocks, B, Hkv, D, dtype=torch.bfloat16, device=DEV) for _ in range(layers)] for _ in range(2))
    freq = (10000.0 ** (-torch.arange(0, D, 2) / D)).to(DEV)
    seqs, held = [3, 5, 8], {}
    for s in seqs:
        bm.add_sequence(s)
        held[s] = [[] for _ in range(layers)]                 # (k, v) rows that the cache has to hold

    def append(counts, positions):
        T = sum(counts)
        slots = dev(bm.append_slots([s for s, n in zip(seqs, counts) for _ in range(n)]))
        rows = []
        for l in range(layers):
            x = torch.randn(T, H + 2 * Hkv, D, generator=gen).to(torch.bfloat16).to(DEV)
            q = pk.rope_and_cache(x[:, :H], x[:, H:H + Hkv], x[:, H + Hkv:], kc[l], vc[l], slots, dev(np.asarray(positions)), freq)
            at = slots.cpu().numpy()
            rows.append((q, kc[l].view(-1, Hkv, D)[at].clone(), vc[l].view(-1, Hkv, D)[at].clone()))
        return rows

    def tables():
        bt, lens = bm.export(seqs, 24)
        return dev(bt), dev(lens)
    prompt = [13, 40, 7]
    rows = append(prompt, [i for n in prompt for i in range(n)])
    at = 0
    for s, n in zip(seqs, prompt):
        for l in range(layers):
            held[s][l] = [(rows[l][1][i], rows[l][2][i]) for i in range(at, at + n)]
        at += n
    for step in range(6):
        sizes = [int(x) for x in rng.integers(1, 30, len(seqs))]
        parents = [parents_of(n, rng) for n in sizes]
        depth = []
        for p in parents:
            d = []
            for r in range(len(p)):
                d.append(0 if r == 0 else d[p[r]] + 1)
            depth += d
        before = [bm.sequence_info(s)[0] for s in seqs]
        base = np.repeat(before, sizes)
        rows = append(sizes, base + np.asarray(depth))
        bt, lens = tables()
        cu_h = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
        cu = dev(cu_h)
        mask_h = np.concatenate([R.ancestors_mask(p, 1) for p in parents])
        for l in range(layers):
            out = pk.paged_attention_tree(rows[l][0], cu, max(sizes), dev(mask_h.view(np.int64)), kc[l], vc[l], bt, lens,
                                          D ** -0.5, out_dtype=torch.float32)
            ref = R.masked_attention(bits(rows[l][0]), bits(kc[l]), bits(vc[l]), bt.cpu().numpy(), lens.tolist(), cu_h, D ** -0.5,
                                     B, mask_h)
            assert np.all(np.abs(out.double().cpu().numpy() - ref[0]) <= R.bound(*ref, int(lens.max()), D, False))
        tok, tgt = (rng.integers(0, 3, sum(sizes)) for _ in range(2))
        acc, num, nxt, new = pk.accept_tree(dev(tok), dev(np.concatenate([np.asarray(p, np.int32) for p in parents])), dev(tgt),
                                            cu, max(sizes), lens)
        pk.pk_keep_tokens_layers(kc, vc, bt, lens, cu, acc, num)
        for i, s in enumerate(seqs):
            path = R.accept(tok[cu_h[i]:cu_h[i + 1]], parents[i], tgt[cu_h[i]:cu_h[i + 1]])
            assert acc[i, :int(num[i])].tolist() == path
            for l in range(layers):
                held[s][l] += [(rows[l][1][cu_h[i] + r], rows[l][2][cu_h[i] + r]) for r in path]
            bm.truncate(s, int(new[i]))
            assert int(new[i]) == before[i] + len(path)
        bt, lens = tables()
        for i, s in enumerate(seqs):
            n = int(lens[i])
            at = [int(bt[i, j // B]) * B + j % B for j in range(n)]
            for l in range(layers):
                assert torch.equal(kc[l].view(-1, Hkv, D)[at], torch.stack([a for a, _ in held[s][l]]))
                assert torch.equal(vc[l].view(-1, Hkv, D)[at], torch.stack([b for _, b in held[s][l]]))
        assert bm.blocks_in_use() == sum(-(-int(n) // B) for n in lens)
    clean()


def test_step_in_two_graphs_that_run_side_by_side():
    # Each graph's workspace is its own; replayed on two streams at once, again and again.
    cases = [Case(s, [3000, 900, 40], [20, 33, 7], 4, 2, 128, 16, True) for s in (1, 2)]
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for c in cases:
        cu, tb, sl, mk = dev(c.cu), dev(c.tables), dev(np.asarray(c.lens, np.int32)), dev(c.mask.view(np.int64))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            for _ in range(3):
                out = pk.paged_attention_tree(c.q, cu, 33, mk, c.k, c.v, tb, sl, c.scale, out_dtype=torch.float32)
        graphs.append((g, cu, tb, sl, mk))
        outs.append(out)
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(10):
        for out in outs:
            out.zero_()
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g[0].replay()
        torch.cuda.synchronize()
        for out, w in zip(outs, want):
            assert torch.equal(out, w)
    clean()


def test_calls_on_another_stream():
    c = Case(4, [2000, 100], [50, 9], 2, 1, 64, 16, False)
    want = c.run()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for _ in range(5):
        out = c.run(stream=st)
        torch.cuda.current_stream().wait_stream(st)
        assert torch.equal(out, want)
    clean()


def test_repeated_calls_give_the_same_bits():
    c = Case(5, [5000, 700, 129], [100, 40, 3], 4, 2, 64, 32, True)
    want = c.run()
    for _ in range(20):
        assert torch.equal(c.run(), want)
    clean()


@pytest.mark.parametrize("busy_mb", [0, 256])
def test_lengths_that_the_kernel_before_writes(busy_mb):
    # accept_tree writes the lengths and the attention is its programmatic dependent: what
    # it planned from the old ones must not be used.
    c = Case(6, [900, 300, 500, 64], [5, 5, 5, 5], 4, 2, 128, 16, False)
    cu, tb = dev(c.cu), dev(c.tables)
    tok = torch.zeros(20, dtype=torch.int64, device=DEV)
    lib = _native.load()
    big = torch.empty(max(1, busy_mb << 20), dtype=torch.uint8, device=DEV)
    ws = pk.new_workspace(pk.pk_tree_workspace_bytes(8, 2, 128, 5, 900), DEV)
    for trial in range(6):
        rng = np.random.default_rng(trial)
        parents = np.concatenate([[-1] + [int(rng.integers(-1, r)) for r in range(1, 5)] for _ in range(4)]).astype(np.int32)
        par = dev(parents)
        old, new = dev(np.asarray([900, 300, 500, 64], np.int32)), torch.full((4,), 17 * trial, dtype=torch.int32, device=DEV)
        acc = torch.empty(4, 5, dtype=torch.int32, device=DEV)
        num, nxt = torch.empty(4, dtype=torch.int32, device=DEV), torch.empty(4, dtype=torch.int64, device=DEV)
        out = torch.zeros(20, 8, 128, device=DEV)
        torch.cuda.synchronize()
        big.fill_(trial)
        st = torch.cuda.current_stream().cuda_stream
        assert lib.pk_accept_tree(acc.data_ptr(), num.data_ptr(), nxt.data_ptr(), new.data_ptr(), tok.data_ptr(), par.data_ptr(),
                                  tok.data_ptr(), 20, cu.data_ptr(), 5, old.data_ptr(), 4, st) == 0
        pk.paged_attention_cross(c.q, cu, 5, c.k, c.v, tb, new, c.scale, out=out, max_seq_len=900, workspace=ws)
        torch.cuda.synchronize()
        c.lens = new.tolist()
        for s in range(4):
            path = R.accept([0] * 5, parents[5 * s:5 * s + 5], [0] * 5)
            assert c.lens[s] == [900, 300, 500, 64][s] - 5 + len(path)
        c.check(out)
    clean()


def test_lengths_that_are_written_and_written_back():
    # Two calls before the attention change the lengths and change them back while it may
    # already plan: the plan has to be of the lengths that it compares afterwards.
    c = Case(16, [700, 40, 333], [4, 4, 4], 4, 2, 64, 16, False)
    cu, tb = dev(c.cu), dev(c.tables)
    want = c.run()
    lib = _native.load()
    z = torch.zeros(12, dtype=torch.int64, device=DEV)
    par = dev(np.asarray([-1, 0, 1, 2] * 3, np.int32))
    acc, num, nxt = (torch.empty(n, dtype=d, device=DEV) for n, d in ((12, torch.int32), (3, torch.int32), (3, torch.int64)))
    final, other = dev(np.asarray(c.lens, np.int32)), dev(np.asarray([64, 690, 5], np.int32))
    buf = final.clone()
    big = torch.empty(128 << 20, dtype=torch.uint8, device=DEV)
    ws = pk.new_workspace(pk.pk_tree_workspace_bytes(8, 2, 64, 4, 700), DEV)
    for trial in range(20):
        out = torch.zeros_like(want)
        big.fill_(trial)
        st = torch.cuda.current_stream().cuda_stream
        for src in (other, final):
            # (Every node is accepted: the new lengths are the old ones.)
            assert lib.pk_accept_tree(acc.data_ptr(), num.data_ptr(), nxt.data_ptr(), buf.data_ptr(), z.data_ptr(),
                                      par.data_ptr(), z.data_ptr(), 12, cu.data_ptr(), 4, src.data_ptr(), 3, st) == 0
        pk.paged_attention_cross(c.q, cu, 4, c.k, c.v, tb, buf, c.scale, out=out, max_seq_len=700, workspace=ws)
        assert torch.equal(out, want)
    clean()


def _timeout_case(rows, lens):
    c = Case(rows, lens, [rows] * len(lens), 4, 2, 128, 16, False)
    args = (c.q, dev(c.cu), rows, c.k, c.v, dev(c.tables), dev(np.asarray(c.lens, np.int32)), c.scale)
    ws = pk.new_workspace(pk.pk_tree_workspace_bytes(8, 2, 128, rows, max(lens)), DEV)
    ws.zero_()
    return args, dict(max_seq_len=max(lens), workspace=ws)


@pytest.mark.parametrize("rows,lens,stall", [(8, [60000, 90000], 1), (8, [60000, 90000], 6), (200, [6000, 9000], 2)])
def test_wait_runs_out_and_the_next_call_is_correct(rows, lens, stall):
    # CTA 0's range holds more key tiles than that: 14 of the long sequences' 2,346, 5 of
    # the wide blocks' 944.
    args, kw = _timeout_case(rows, lens)
    want = pk.paged_attention_cross(*args, **kw)
    clean()
    t0 = time.perf_counter()
    assert pk.pk_selftest_cross_wait_timeout(*args, stall, 5000, **kw) == 0
    torch.cuda.synchronize()
    assert pk.pk_get_device_error() & _native.DEVERR_TIMEOUT
    assert time.perf_counter() - t0 < 5.0
    for _ in range(2):
        assert torch.equal(pk.paged_attention_cross(*args, **kw), want)
        clean()


@pytest.mark.parametrize("stall", [1, 6])
def test_a_stall_beyond_the_range_does_nothing(stall):
    # 236 tiles of 16 and 4 segments of 38 more make 122 ranges of 32: tile 1 starts at 54,
    # so CTA 0 has tile 0 alone.
    args, kw = _timeout_case(8, [6000, 9000])
    want = pk.paged_attention_cross(*args, **kw)
    out = torch.empty_like(want)
    assert pk.pk_selftest_cross_wait_timeout(*args, stall, 5000, out=out, **kw) == 0
    clean()
    assert torch.equal(out, want)
