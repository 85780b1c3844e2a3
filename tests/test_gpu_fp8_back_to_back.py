"""Steps of the 8-bit cache's calls back to back, as in a serving loop's graph.

Each kernel starts while the one before it still runs and waits inside: an
attention call may share its SMs with the previous step's, which read the same
tables and scales before the append between them changed them.  Every step's
result must be that of the same step with nothing else on the GPU.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from fp8lib import DEV, attention_case, to_dev

pytestmark = pytest.mark.gpu

STEPS = 40


def _case(lens, G, Hkv, D, B):
    """Sequences with room for STEPS tokens; new tokens grow, so that a block's scale grows with every step."""
    c = attention_case(1, [n + STEPS for n in lens], [1] * len(lens), G, Hkv, D, B)
    rng = np.random.default_rng(2)
    N = len(lens)
    x = rng.standard_normal((STEPS, N, (G + 2) * Hkv, D)) * 1.3 ** np.arange(STEPS)[:, None, None, None]
    c["x"] = torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).to(DEV)
    c["at"] = [torch.tensor([n + t + 1 for n in lens], dtype=torch.int32, device=DEV) for t in range(STEPS)]
    c["f"] = to_dev((10000.0 ** (-np.arange(0, D, 2) / D)).astype(np.float32))
    return c


def _steps(c, state, G, Hkv, outs, sync, lens=None):
    """Every step, with its lengths copied to `lens` or, without it, in memory of their own
    (then nothing stands between the calls)."""
    own = lens is None
    for t in range(STEPS):
        x = c["x"][t]
        if own:
            lens = c["at"][t]
        else:
            lens.copy_(c["at"][t])
        q = pk.rope_and_cache_fp8(x[:, :G * Hkv], x[:, G * Hkv:(G + 1) * Hkv], x[:, (G + 1) * Hkv:], *state, c["dev"]["bt"], lens, c["f"])
        if sync:
            torch.cuda.synchronize()
        pk.paged_attention_decode_fp8(q, *state, c["dev"]["bt"], lens, c["scale"], out=outs[t], max_seq_len=c["cap"])
        if sync:
            torch.cuda.synchronize()


@pytest.mark.parametrize("lens,G,Hkv,D,B", [([100, 40, 7, 90], 4, 2, 128, 16), ([1000, 500], 8, 2, 64, 8),
                                            ([300] * 64, 4, 8, 128, 16), ([3000, 20], 16, 2, 128, 32), ([60] * 8, 1, 8, 64, 32)])
@pytest.mark.parametrize("own_lens", [False, True])
def test_every_step_of_a_graph_is_the_step_alone(lens, G, Hkv, D, B, own_lens):
    c = _case(lens, G, Hkv, D, B)
    c["cap"] = c["dev"]["bt"].shape[1] * B
    d = c["dev"]

    def fresh():
        return [d["k"].view(torch.uint8).clone().view(d["k"].dtype), d["v"].view(torch.uint8).clone().view(d["v"].dtype),
                d["ks"].clone(), d["vs"].clone()]
    shape = (STEPS, len(lens), G * Hkv, D)
    want, got = (torch.zeros(shape, device=DEV) for _ in range(2))
    sl = None if own_lens else torch.zeros(len(lens), dtype=torch.int32, device=DEV)
    ref = fresh()
    _steps(c, ref, G, Hkv, want, True, sl)
    state = fresh()
    _steps(c, state, G, Hkv, got, False, sl)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    start, state = fresh(), fresh()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _steps(c, state, G, Hkv, got, False, sl)
    for _ in range(3):
        for x, y in zip(state, start):
            x.view(torch.uint8).copy_(y.view(torch.uint8))
        got.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        for x, y in zip(state, ref):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert pk.pk_get_device_error() == 0


def test_a_padded_batch_in_a_graph():
    # Rows for 6 sequences of which 4 live: the others have length 0 and no rows
    # (cu_q_lens stays at its last value).  Nothing of them is written or reported.
    G, Hkv, D, B = 4, 2, 128, 16
    c = attention_case(5, [40, 700, 1, 129], [1] * 4, G, Hkv, D, B)
    d = c["dev"]
    bt = torch.full((6, d["bt"].shape[1]), -1, dtype=torch.int32, device=DEV)
    bt[:4] = d["bt"]
    sl = torch.tensor([40, 700, 1, 129, 0, 0], dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, 1, 2, 3, 4, 4, 4], dtype=torch.int32, device=DEV)
    x = torch.randn(6, (G + 2) * Hkv, D, device=DEV).to(torch.bfloat16)
    f = to_dev((10000.0 ** (-np.arange(0, D, 2) / D)).astype(np.float32))
    state = [d["k"], d["v"], d["ks"], d["vs"]]
    q = torch.full((6, G * Hkv, D), 5.0, dtype=torch.bfloat16, device=DEV)
    out = torch.empty(6, G * Hkv, D, device=DEV)

    def step():
        pk.rope_and_cache_fp8(x[:, :G * Hkv], x[:, G * Hkv:(G + 1) * Hkv], x[:, (G + 1) * Hkv:], *state, bt, sl, f, cu_q_lens=cu,
                              max_q_len=1, q_out=q)
        pk.paged_attention_decode_fp8(q, *state, bt, sl, c["scale"], out=out)
    step()
    torch.cuda.synchronize()
    want = out.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    out.fill_(9.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.all(out[4:] == 0) and torch.all(q[4:] == 5.0)
    assert torch.any(q[:4] != 5.0) and pk.pk_get_device_error() == 0
