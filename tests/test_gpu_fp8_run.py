"""The 8-bit cache's calls together, as a serving loop makes them: prompts
appended in chunks and attended through the gather, forks cloned copy-on-write
with the block manager, decode steps, verification of drafted tokens, a swap out
and in; in graphs, and on several streams."""
import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from fp8lib import DEV, attend, attention_case, bf16, cache_bytes, check_attention, to_dev
from oracle import fp8_ref as R

pytestmark = pytest.mark.gpu

H, HKV, D, B = 8, 2, 128, 16
SCALE = 1.0 / np.sqrt(D)
FREQ = (10000.0 ** (-np.arange(0, D, 2) / D)).astype(np.float32)


class Loop:
    """A cache, a block manager and the float64 attention of what was appended."""

    def __init__(self, blocks=64):
        self.bm = pk.BlockManager(blocks, B)
        self.cache = pk.new_cache_fp8(blocks, HKV, B, D, DEV)
        self.f = to_dev(FREQ)
        self.rng = np.random.default_rng(0)
        self.k, self.v = {}, {}                                 # appended rows, rotated, float64

    def tables(self, seqs):
        bt, lens = self.bm.export(seqs, 64)[:2]
        return to_dev(np.asarray(bt, np.int32)), to_dev(np.asarray(lens, np.int32))

    def append(self, seqs, counts):
        """New random tokens of each sequence; returns their rotated queries and cu."""
        T = sum(counts)
        q, q64 = bf16(self.rng, T, H, D)
        k, k64 = bf16(self.rng, T, HKV, D)
        v, v64 = bf16(self.rng, T, HKV, D)
        self.bm.append_slots([s for s, n in zip(seqs, counts) for _ in range(n)])
        pairs = self.bm.take_copies()
        if len(pairs):
            pk.copy_blocks_fp8(*self.cache, to_dev(np.asarray(pairs, np.int64).reshape(-1, 2)))
        bt, lens = self.tables(seqs)
        cu = to_dev(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32))
        out = pk.rope_and_cache_fp8(q, k, v, *self.cache, bt, lens, self.f, cu_q_lens=cu, max_q_len=max(counts))
        r = 0
        for s, n in zip(seqs, counts):
            at = len(self.k[s])
            self.k[s] = np.concatenate([self.k[s], R.rope(k64[r:r + n], np.arange(at, at + n), FREQ)])
            self.v[s] = np.concatenate([self.v[s], v64[r:r + n]])
            r += n
        return out, cu, bt, lens

    def check(self, seqs, counts, q, out):
        """Against float64 attention of the UNQUANTISED rows.  An e4m3 value is
        within 2^-4 of itself, so a score moves by at most 2^-4 of sum |q||k| (in
        practice by its root mean square), which these inputs keep below 0.5."""
        q64, got, r = q.double().cpu().numpy(), out.double().cpu().numpy(), 0
        err, norm = 0.0, 0.0
        for s, n in zip(seqs, counts):
            for i in range(n):
                m = len(self.k[s]) - n + i + 1
                for h in range(H):
                    z = SCALE * self.k[s][:m, h // (H // HKV)] @ q64[r, h]
                    p = np.exp(z - z.max())
                    ref = p @ self.v[s][:m, h // (H // HKV)] / p.sum()
                    err += np.sum((got[r, h] - ref) ** 2)
                    norm += np.sum(ref ** 2)
                r += 1
        assert np.sqrt(err / norm) < 2.0 ** -4                  # values to 2^-4 each at worst, errors independent


def test_a_serving_loop():
    x = Loop()
    for s in (0, 1):
        x.bm.add_sequence(s)
        x.k[s], x.v[s] = np.zeros((0, HKV, D)), np.zeros((0, HKV, D))
    # Prompts in chunks: each chunk attends through the gathered bf16 pages.
    for counts in ([37, 150], [60, 3]):
        q, cu, bt, lens = x.append([0, 1], counts)
        pages = [-(-int(n) // B) for n in lens.tolist()]
        start = np.concatenate([[0], np.cumsum(pages)])
        ok, ov = (torch.zeros(int(start[-1]) * B, HKV, D, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        pk.gather_kv_fp8(*x.cache, bt, lens, to_dev((start[:-1] * B).astype(np.int64)), ok, ov)
        flat = np.full((2, max(pages)), -1, np.int32)
        for s in (0, 1):
            flat[s, :pages[s]] = np.arange(start[s], start[s + 1])
        out = pk.paged_attention_multi_query(q, cu, max(counts), ok.view(-1, B, HKV, D), ov.view(-1, B, HKV, D),
                                             to_dev(flat), lens, SCALE)
        x.check([0, 1], counts, q, out)
    # Fork: both write the shared last block; the clone takes the scales along.
    x.bm.fork(0, 2)
    x.k[2], x.v[2] = x.k[0].copy(), x.v[0].copy()
    seqs = [0, 1, 2]
    for _ in range(5):
        q, cu, bt, lens = x.append(seqs, [1, 1, 1])
        x.check(seqs, [1, 1, 1], q, pk.paged_attention_decode_fp8(q, *x.cache, bt, lens, SCALE))
    # Two drafted tokens each, verified in one call.
    q, cu, bt, lens = x.append(seqs, [2, 2, 2])
    x.check(seqs, [2, 2, 2], q, pk.paged_attention_multi_query_fp8(q, cu, 2, *x.cache, bt, lens, SCALE))
    # Swap everything out and in again.
    host = [torch.empty(t.shape, dtype=torch.uint8 if t.dtype == torch.float8_e4m3fn else t.dtype,
                        pin_memory=True).view(t.dtype) for t in x.cache]
    all_blocks = torch.arange(x.cache[0].shape[0], device=DEV)[:, None].repeat(1, 2)
    before = pk.paged_attention_decode_fp8(q[::2].contiguous(), *x.cache, bt, lens, SCALE)
    pk.swap_blocks_fp8(host, x.cache, all_blocks)
    again = pk.new_cache_fp8(x.cache[0].shape[0], HKV, B, D, DEV)
    pk.swap_blocks_fp8(again, host, all_blocks)
    assert torch.equal(pk.paged_attention_decode_fp8(q[::2].contiguous(), *again, bt, lens, SCALE), before)
    assert pk.pk_get_device_error() == 0


def _graph(fn):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fn()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fn()
    return g


def test_a_step_replays_in_a_graph_with_new_lengths():
    c = attention_case(1, [40, 700, 1500], [1] * 3, 8, 2, 128, 16)
    d = c["dev"]
    lens = d["sl"].clone()
    k, _ = bf16(np.random.default_rng(3), 3, 2, 128)
    keep = {}

    def step():
        q = pk.rope_and_cache_fp8(c["q"], k, k, d["k"], d["v"], d["ks"], d["vs"], d["bt"], d["sl"], to_dev_freq)
        keep["out"] = pk.paged_attention_decode_fp8(q, d["k"], d["v"], d["ks"], d["vs"], d["bt"], d["sl"], c["scale"])
    to_dev_freq = to_dev(FREQ)
    g = _graph(step)
    for new in (lens, lens - 5, lens - 13):
        d["sl"].copy_(new)
        g.replay()
        torch.cuda.synchronize()
        got, state = keep["out"].clone(), [cache_bytes(d["k"]), d["ks"].clone()]
        step()
        torch.cuda.synchronize()
        assert torch.equal(keep["out"], got)
        assert np.array_equal(cache_bytes(d["k"]), state[0]) and torch.equal(d["ks"], state[1])
        g = _graph(step)
    assert pk.pk_get_device_error() == 0


def test_two_graphs_replayed_at_once_do_not_share_scratch():
    cases = [attention_case(s, lens, [1] * len(lens), 8, 2, 128, 16) for s, lens in ((1, [9000, 700]), (2, [300, 12000, 4000]))]
    want = [attend(c) for c in cases]
    got = [None, None]
    graphs = []
    for i, c in enumerate(cases):
        def run(i=i, c=c):
            for _ in range(20):
                got[i] = attend(c)
        graphs.append(_graph(run))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for w, o, c in zip(want, got, cases):
        assert torch.equal(w, o)
    assert pk.pk_get_device_error() == 0


def test_calls_on_two_streams_at_once():
    cases = [attention_case(s, [5000, 300, 64], [1] * 3, 4, 2, 128, 16) for s in (5, 6)]
    want = [attend(c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for c, s in zip(cases, streams):
            got.append(attend(c, stream=s))
    torch.cuda.synchronize()
    for i, o in enumerate(got):
        assert torch.equal(o, want[i % 2])
    for c, w in zip(cases, want):
        check_attention(c, w)
    assert pk.pk_get_device_error() == 0


def test_lengths_written_just_before_the_call():
    # The kernel plans from the lengths before the previous kernel has ended,
    # and again if they changed.
    c = attention_case(7, [900, 30, 2500, 129], [1] * 4, 8, 2, 128, 16)
    d = c["dev"]
    want = attend(c)
    stale = torch.tensor([1, 2500, 0, 700], dtype=torch.int32, device=DEV).clamp(max=d["bt"].shape[1] * 16)
    real = d["sl"].clone()
    hold = torch.empty(1 << 28, dtype=torch.uint8, device=DEV)
    for _ in range(3):
        d["sl"].copy_(stale)
        torch.cuda.synchronize()
        hold.fill_(1)
        d["sl"].copy_(real)
        out = attend(c)
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    pk.pk_get_device_error()


def test_memory_of_a_call_on_another_stream():
    # What a call on a side stream allocates is the side stream's: it is handed
    # out again only behind the call, eager (a workspace that a larger one
    # replaces) and captured (one of the graph's pool, on a forked branch).
    from paged_kv_cache_122_gb300 import api, fp8
    c = attention_case(11, [9000, 700], [1, 1], 8, 2, 128, 16)
    want = attend(c)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)                           # about 30 ms
    old = api.workspace_for(DEV, 3 << 20, side).data_ptr()
    api.workspace_for(DEV, 5 << 20, side)                       # the first is free now
    assert torch.empty(3 << 20, dtype=torch.uint8, device=DEV).data_ptr() != old
    out = attend(c, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want)

    made = []
    new_workspace, fp8.new_workspace = fp8.new_workspace, lambda n, dev: made.append(new_workspace(n, dev)) or made[-1]
    try:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            side.wait_stream(torch.cuda.current_stream())
            out = attend(c, stream=side)
            ptr, size = made.pop().data_ptr(), 1 << 20
            other = [torch.full((size,), 7, dtype=torch.uint8, device=DEV) for _ in range(40)]
            torch.cuda.current_stream().wait_stream(side)
    finally:
        fp8.new_workspace = new_workspace
    assert all(not o.data_ptr() <= ptr < o.data_ptr() + size for o in other)
    for _ in range(3):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert pk.pk_get_device_error() == 0
