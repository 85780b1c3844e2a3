"""Rotary positions and the append to the bf16 cache in one pass, against the
float64 rotation.

Tolerance: the result is rounded once to bf16 (half a step, 2^-8 of the value);
before that the cosine and sine are off by at most 2^-22 each (32-bit values of
an angle exact to 2^-33 turns) and the two products and their sum by 2^-24
each, so the unrounded result is within 2^-21 of the pair's length.
"""
import numpy as np
import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from fp8lib import DEV, bf16, to_dev
from oracle import fp8_ref as R

pytestmark = pytest.mark.gpu


def _freq(rot, base=500000.0):
    return (base ** (-np.arange(0, rot, 2) / rot)).astype(np.float32)


def _check(got, x64, y, factor=1.0):
    got = got.double().cpu().numpy()
    length = np.sqrt(np.sum(x64 ** 2, axis=-1, keepdims=True)) * factor      # bounds every pair's
    tol = 2.0 ** -8 * np.abs(y) + 2.0 ** -21 * length
    assert np.all(np.abs(got - y) <= tol), np.max(np.abs(got - y) - tol)


def _pool(T, B, Hkv, D, spare=2):
    P = -(-T // B) + spare
    return torch.full((P, B, Hkv, D), 7.0, dtype=torch.bfloat16, device=DEV)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot,H,Hkv,B", [(64, 64, 8, 8, 16), (64, 16, 3, 1, 8), (128, 128, 16, 2, 32),
                                           (128, 64, 5, 5, 16), (128, 48, 64, 8, 8), (64, 48, 7, 3, 16)])
def test_rotation_and_append(D, rot, H, Hkv, B, interleaved):
    rng = np.random.default_rng(D + rot + H)
    T = 37
    q, q64 = bf16(rng, T, H, D)
    k, k64 = bf16(rng, T, Hkv, D)
    v, v64 = bf16(rng, T, Hkv, D)
    kc, vc = _pool(T, B, Hkv, D), _pool(T, B, Hkv, D)
    slots = rng.permutation(kc.shape[0] * B)[:T].astype(np.int64)
    pos = rng.integers(0, 1 << 20, size=T).astype(np.int64)
    pos[:4] = [0, 1, -5, 2 ** 31 - 1]
    f = _freq(rot)
    out = pk.rope_and_cache(q, k, v, kc, vc, to_dev(slots), to_dev(pos), to_dev(f), interleaved=interleaved, factor=1.25)
    _check(out, q64, R.rope(q64, pos, f, interleaved, 1.25), 1.25)
    rows = kc.view(-1, Hkv, D)[to_dev(slots)]
    _check(rows, k64, R.rope(k64, pos, f, interleaved, 1.25), 1.25)
    assert torch.equal(vc.view(-1, Hkv, D)[to_dev(slots)], v)
    untouched = torch.ones(kc.shape[0] * B, dtype=torch.bool, device=DEV)
    untouched[to_dev(slots)] = False
    assert torch.all(kc.view(-1, Hkv, D)[untouched] == 7.0) and torch.all(vc.view(-1, Hkv, D)[untouched] == 7.0)
    assert pk.pk_get_device_error() == 0


@pytest.mark.parametrize("T", [1, 2, 255, 1000])
def test_strided_views_of_a_fused_projection_and_in_place(T):
    rng = np.random.default_rng(T)
    H, Hkv, D, B = 8, 2, 128, 16
    qkv, x64 = bf16(rng, T, H + 2 * Hkv, D)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    kc, vc = _pool(T, B, Hkv, D), _pool(T, B, Hkv, D)
    slots = torch.arange(T, device=DEV)
    pos = torch.arange(T, device=DEV) + 100000
    f = to_dev(_freq(D))
    want = pk.rope_and_cache(q.contiguous(), k.contiguous(), v.contiguous(), kc, vc, slots, pos, f)
    kc2, vc2 = _pool(T, B, Hkv, D), _pool(T, B, Hkv, D)
    out = pk.rope_and_cache(q, k, v, kc2, vc2, slots, pos, f)
    assert out.is_contiguous() and torch.equal(out, want) and torch.equal(kc, kc2) and torch.equal(vc, vc2)
    same = pk.rope_and_cache(q, k, v, kc2, vc2, slots, pos, f, q_out=q)       # in place, in the projection
    assert same is q and torch.equal(q, want)
    assert torch.equal(qkv[:, H:].double().cpu(), torch.from_numpy(x64[:, H:]))  # k and v as they were
    _check(out, x64[:, :H], R.rope(x64[:, :H], pos.cpu().numpy(), _freq(D)))


def test_without_rotation_is_the_plain_append():
    rng = np.random.default_rng(5)
    T, Hkv, D, B = 70, 3, 64, 8
    k, _ = bf16(rng, T, Hkv, D)
    v, _ = bf16(rng, T, Hkv, D)
    slots = to_dev(np.concatenate([rng.permutation(80)[:69], [-1]]).astype(np.int64))
    a, b, c, d = (_pool(T, B, Hkv, D) for _ in range(4))
    pk.reshape_and_cache(k, v, a, b, slots)
    assert pk.rope_and_cache(None, k, v, c, d, slots, None, None) is None
    assert torch.equal(a, c) and torch.equal(b, d)


def test_padding_tokens_and_slots_outside_the_pool():
    rng = np.random.default_rng(6)
    T, H, Hkv, D, B = 5, 4, 2, 64, 16
    q, q64 = bf16(rng, T, H, D)
    k, _ = bf16(rng, T, Hkv, D)
    kc, vc = _pool(0, B, Hkv, D), _pool(0, B, Hkv, D)
    slots = torch.tensor([0, -1, 2 * B, 5, 2 ** 40], dtype=torch.int64, device=DEV)
    pos = np.arange(T)
    out = pk.rope_and_cache(q, k, k, kc, vc, slots, to_dev(pos), to_dev(_freq(D)))
    assert pk.pk_get_device_error() == pk._native.DEVERR_SLOT
    _check(out, q64, R.rope(q64, pos, _freq(D)))              # every query is rotated
    hit = (vc.view(-1, Hkv * D) != 7.0).any(1).nonzero().flatten().tolist()
    assert hit == [0, 5]


def test_not_finite_values_stay_in_their_pair_and_odd_frequencies():
    T, D = 1, 64
    q = torch.zeros(T, 1, D, dtype=torch.bfloat16, device=DEV)
    q[0, 0, :] = 1.0
    q[0, 0, 3] = float("nan")
    q[0, 0, 7] = float("inf")
    kc = _pool(1, 8, 1, D)
    f = _freq(D)
    f[5:9] = [0.0, np.inf, 3.0, -0.25]                          # no turn, no turn, more than a half turn, backwards
    out = pk.rope_and_cache(q, q, q, kc, kc.clone(), torch.zeros(1, dtype=torch.int64, device=DEV),
                            torch.tensor([11], device=DEV), to_dev(f)).double().cpu().numpy()[0, 0]
    bad = {3, 35, 7, 39}
    assert set(np.nonzero(~np.isfinite(out))[0]) == bad
    f[6] = 0.0
    ref = R.rope(np.ones((1, 1, D)), [11], f)[0, 0]
    good = [i for i in range(D) if i not in bad]
    assert np.all(np.abs(out[good] - ref[good]) <= 2.0 ** -8 * np.abs(ref[good]) + 2.0 ** -20)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 16), (128, 64), (128, 80), (64, 32), (64, 48)])
def test_elements_that_are_not_rotated_keep_their_bits(D, rot, interleaved):
    # Every 16-bit pattern, NaNs with their payloads among them.
    T, H, Hkv, B = 9, 6, 2, 16
    rng = np.random.default_rng(rot)
    bits = [torch.from_numpy(rng.integers(-2 ** 15, 2 ** 15, size=(T, n, D)).astype(np.int16)).to(DEV) for n in (H, Hkv, Hkv)]
    q, k, v = (b.view(torch.bfloat16) for b in bits)
    kc, vc = _pool(T, B, Hkv, D), _pool(T, B, Hkv, D)
    slots = torch.arange(T, device=DEV)
    out = pk.rope_and_cache(q, k, v, kc, vc, slots, slots + 100, to_dev(_freq(rot)), interleaved=interleaved)
    assert torch.equal(out.view(torch.int16)[..., rot:], bits[0][..., rot:])
    assert torch.equal(kc.view(torch.int16).view(-1, Hkv, D)[:T, :, rot:], bits[1][..., rot:])
    assert torch.equal(vc.view(torch.int16).view(-1, Hkv, D)[:T], bits[2])
    cache = pk.new_cache_fp8(1, Hkv, B, D, DEV)
    bt, sl = torch.zeros(1, 1, dtype=torch.int32, device=DEV), torch.full((1,), T, dtype=torch.int32, device=DEV)
    cu = torch.tensor([0, T], dtype=torch.int32, device=DEV)
    out8 = pk.rope_and_cache_fp8(q, k, v, *cache, bt, sl, to_dev(_freq(rot)), cu_q_lens=cu, positions=slots + 100,
                                 interleaved=interleaved)
    assert torch.equal(out8.view(torch.int16)[..., rot:], bits[0][..., rot:])
    assert pk.pk_get_device_error() == 0


def test_other_stream_and_refusals():
    rng = np.random.default_rng(8)
    T, H, D, B = 64, 4, 128, 16
    q, _ = bf16(rng, T, H, D)
    kc, vc = _pool(T, B, H, D), _pool(T, B, H, D)
    slots, pos, f = torch.arange(T, device=DEV), torch.arange(T, device=DEV), to_dev(_freq(D))
    want = pk.rope_and_cache(q, q, q, kc, vc, slots, pos, f)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = pk.rope_and_cache(q, q, q, kc, vc, slots, pos, f, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    call = pk.rope_and_cache
    with pytest.raises(ValueError, match="positions"):
        call(q, q, q, kc, vc, slots, None, f)
    with pytest.raises(TypeError):
        call(q, q, q, kc, vc, slots.int(), pos, f)
    with pytest.raises(TypeError):
        call(q.float(), q, q, kc, vc, slots, pos, f)
    with pytest.raises(ValueError):
        call(q, q[:, :3], q, kc, vc, slots, pos, f)
    with pytest.raises(ValueError, match="contiguous"):
        call(q.transpose(0, 1), q, q, kc, vc, slots, pos, f)
    with pytest.raises(ValueError):
        call(q, q, q, kc, vc, slots, pos, to_dev(np.ones(65, np.float32)))
    with pytest.raises(pk.PagedKVError, match="UNSUPPORTED"):
        call(q, q, q, kc, vc, slots, pos, to_dev(np.ones(12, np.float32)))
    wide = torch.zeros(T, H * D + 4, dtype=torch.bfloat16, device=DEV)[:, :H * D].view(T, H, D)
    with pytest.raises(pk.PagedKVError, match="ALIGNMENT"):
        call(wide, q, q, kc, vc, slots, pos, f)
    assert pk.pk_get_device_error() == 0
