"""Host checks of the rotary append and of the 8-bit cache's calls.  CPU only:
every call fails validation, is a no-op, or finds no device."""
import ctypes

import pytest
import torch

from paged_kv_cache_122_gb300 import _native, build

NULL = None


@pytest.fixture(scope="module")
def lib():
    if not build.up_to_date():
        build.build()
    return _native.load()


def _fake(offset=0):
    buf = (ctypes.c_uint8 * 64)()
    _fake.keep = buf
    return ctypes.c_void_p(((ctypes.addressof(buf) + 15) & ~15) + offset)


def _call(fn, names, base, **kw):
    a = dict(base)
    a.update(kw)
    return fn(*[_fake() if a[n] == "p" else _fake(a[n][1]) if isinstance(a[n], tuple) else a[n] for n in names])


ROPE = ["q_out", "q", "k", "v", "qos", "qs", "ks", "vs", "kc", "vc", "slots", "pos", "freq", "rot", "inter", "factor", "t",
        "h", "hkv", "d", "nb", "b", "st"]
ROPE_OK = dict(q_out="p", q="p", k="p", v="p", qos=1024, qs=1024, ks=256, vs=256, kc="p", vc="p", slots="p", pos="p",
               freq="p", rot=64, inter=0, factor=1.0, t=4, h=8, hkv=2, d=128, nb=16, b=16, st=None)


def _rope_faults(call):
    assert call(d=96) == -3 and call(b=12) == -3                  # head dim, block size
    assert call(rot=24) == -3                                     # not a multiple of 16
    assert call(rot=144) == -2 and call(rot=-16) == -2
    assert call(factor=0.0) == -2 and call(factor=float("nan")) == -2 and call(factor=float("inf")) == -2
    assert call(t=-1) == -2 and call(h=-1) == -2 and call(hkv=0) == -2 and call(nb=-1) == -2
    assert call(qs=1016) == -2 and call(ks=248) == -2             # tokens would overlap
    assert call(qs=1028) == -6 and call(vs=260) == -6             # not whole vectors
    assert call(k=NULL) == -1 and call(q=NULL) == -1 and call(freq=NULL) == -1 and call(kc=NULL) == -1
    assert call(v=("o", 8)) == -6 and call(q_out=("o", 2)) == -6
    if not torch.cuda.is_available():
        assert call() == -7                                       # valid, but no device here
        assert call(h=0, q=NULL, q_out=NULL, qs=0, qos=0) == -7   # no queries
        assert call(rot=0, freq=NULL) == -7                       # no rotation


def test_rope_and_cache_host_validation(lib):
    def call(**kw):
        return _call(lib.pk_rope_and_cache, ROPE, ROPE_OK, **kw)
    _rope_faults(call)
    assert call(t=0) == 0
    assert call(pos=NULL) == -1 and call(slots=NULL) == -1
    if not torch.cuda.is_available():
        assert call(rot=0, pos=NULL) == -7


APPEND = ["q_out", "q", "k", "v", "qos", "qs", "ks", "vs", "kc", "vc", "ksc", "vsc", "bt", "mb", "sl", "cu", "mq", "n", "pos",
          "freq", "rot", "inter", "factor", "t", "h", "hkv", "d", "nb", "b", "st"]
APPEND_OK = dict(ROPE_OK, ksc="p", vsc="p", bt="p", mb=4, sl="p", cu="p", mq=4, n=2)


def test_rope_and_cache_fp8_host_validation(lib):
    def call(**kw):
        return _call(lib.pk_rope_and_cache_fp8, APPEND, APPEND_OK, **kw)
    _rope_faults(call)
    assert call(t=0) == 0 and call(n=0) == 0
    assert call(n=-1) == -2 and call(n=65536) == -2 and call(mb=-1) == -2 and call(mq=-1) == -2
    assert call(cu=NULL) == -2                                    # 4 rows for 2 sequences
    assert call(ksc=NULL) == -1 and call(bt=NULL) == -1 and call(sl=NULL) == -1
    if not torch.cuda.is_available():
        assert call(cu=NULL, n=4) == -7 and call(pos=NULL) == -7


DECODE = ["out", "dt", "q", "kc", "vc", "ksc", "vsc", "bt", "mb", "sl", "msl", "n", "h", "hkv", "d", "nb", "b", "scale", "ws",
          "wsb", "st"]
DECODE_OK = dict(out="p", dt=0, q="p", kc="p", vc="p", ksc="p", vsc="p", bt="p", mb=4, sl="p", msl=64, n=2, h=8, hkv=2, d=128,
                 nb=16, b=16, scale=0.088, ws="p", wsb=1 << 30, st=None)
MULTI = ["out", "dt", "q", "tq", "cu", "mq"] + DECODE[3:]
MULTI_OK = dict(DECODE_OK, tq=4, cu="p", mq=2)


@pytest.mark.parametrize("name,names,ok", [("pk_paged_attention_decode_fp8", DECODE, DECODE_OK),
                                           ("pk_paged_attention_multi_query_fp8", MULTI, MULTI_OK)])
def test_attention_fp8_host_validation(lib, name, names, ok):
    def call(**kw):
        return _call(getattr(lib, name), names, ok, **kw)
    assert call(h=6, hkv=4) == -2 and call(msl=65) == -2 and call(n=-1) == -2 and call(n=65536) == -2
    assert call(scale=float("nan")) == -2 and call(mb=-1, msl=0) == -2
    assert call(d=96) == -3 and call(b=64) == -3 and call(dt=7) == -3
    assert call(h=24, hkv=8) == -3 and call(h=64, hkv=2) == -3    # groups of 3 and 32
    assert call(nb=2 ** 31 - 1, hkv=2) == -2                      # pieces beyond a TMA coordinate
    assert call(n=0) == 0
    for p in ("out", "q", "kc", "vc", "ksc", "vsc", "bt", "sl"):
        assert call(**{p: NULL}) == -1, p
    assert call(q=("o", 2)) == -6 and call(kc=("o", 8)) == -6 and call(out=("o", 4)) == -6
    if not torch.cuda.is_available():
        assert call() == -7
        assert call(mb=64, msl=1024, ws=NULL) == -4 and call(mb=64, msl=1024, wsb=100) == -4
        assert call(ws=NULL, wsb=0) == -7                         # no sequence longer than a tile: none needed


def test_multi_query_fp8_widths(lib):
    def call(**kw):
        return _call(lib.pk_paged_attention_multi_query_fp8, MULTI, MULTI_OK, **kw)
    assert call(tq=0) == 0 and call(tq=-1) == -2 and call(mq=-1) == -2 and call(cu=NULL) == -1
    assert call(mq=5) == -3                                       # 4 heads x 8 columns
    assert call(mq=2 ** 31 - 1) == -3
    if not torch.cuda.is_available():
        assert call(mq=4) == -7 and call(mq=3) == -7


def test_workspace_bytes(lib):
    f = lib.pk_decode_fp8_workspace_bytes
    assert f(4, 8, 8, 64, 128) == 0 and f(4, 8, 8, 64, 129) == 2 * 1024 * 8384
    assert f(8, 32, 8, 128, 131072) == 2 * 1024 * 8384
    assert f(1, 6, 4, 128, 4096) == 0 and f(1, 8, 8, 96, 4096) == 0 and f(-1, 8, 8, 64, 10) == 0


def test_gather_and_block_moves_host_validation(lib):
    names = ["ok", "ov", "kc", "vc", "ksc", "vsc", "bt", "mb", "sl", "cu", "rows", "msl", "n", "hkv", "d", "nb", "b", "st"]
    ok = dict(ok="p", ov="p", kc="p", vc="p", ksc="p", vsc="p", bt="p", mb=4, sl="p", cu="p", rows=100, msl=64, n=2, hkv=2,
              d=128, nb=16, b=16, st=None)

    def gather(**kw):
        return _call(lib.pk_gather_kv_fp8, names, ok, **kw)
    assert gather(msl=65) == -2 and gather(n=-1) == -2 and gather(hkv=0) == -2 and gather(rows=-1) == -2
    assert gather(d=32) == -3 and gather(b=24) == -3
    assert gather(n=0) == 0 and gather(msl=0) == 0 and gather(rows=0) == 0
    assert gather(ok=NULL) == -1 and gather(cu=NULL) == -1 and gather(ov=("o", 8)) == -6
    copy = ["kc", "vc", "ksc", "vsc", "pairs", "n", "hkv", "d", "nb", "b", "st"]

    def cp(**kw):
        return _call(lib.pk_copy_blocks_fp8, copy, dict(ok, pairs="p"), **kw)
    assert cp(n=-1) == -2 and cp(hkv=0) == -2 and cp(nb=-1) == -2 and cp(d=96) == -3 and cp(b=12) == -3
    assert cp(n=0) == 0 and cp(pairs=NULL) == -1 and cp(vsc=NULL) == -1 and cp(kc=("o", 8)) == -6
    assert cp(hkv=2 ** 30) == -2                                  # a block of more chunks than a grid has
    swap = ["dk", "dv", "dks", "dvs", "sk", "sv", "sks", "svs", "pairs", "n", "hkv", "d", "b", "snb", "dnb", "st"]
    sok = dict(ok, dk="p", dv="p", dks="p", dvs="p", sk="p", sv="p", sks="p", svs="p", pairs="p", snb=8, dnb=8)

    def sw(**kw):
        return _call(lib.pk_swap_blocks_fp8, swap, sok, **kw)
    assert sw(n=-1) == -2 and sw(snb=-1) == -2 and sw(d=96) == -3 and sw(n=0) == 0
    assert sw(dks=NULL) == -1 and sw(sv=NULL) == -1 and sw(sk=("o", 4)) == -6
    if not torch.cuda.is_available():
        assert gather() == -7 and cp() == -7 and sw() == -7


def test_binding_refuses_cpu_tensors_and_wrong_types():
    import paged_kv_cache_122_gb300 as pk
    k, v, ks, vs = pk.new_cache_fp8(4, 2, 16, 64, "cpu")
    assert k.dtype == torch.float8_e4m3fn and tuple(ks.shape) == (4, 2)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    bt, sl = torch.zeros(1, 1, dtype=torch.int32), torch.ones(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pk.paged_attention_decode_fp8(q, k, v, ks, vs, bt, sl, 0.125)
    with pytest.raises(TypeError, match="float8"):
        pk.copy_blocks_fp8(k.view(torch.uint8), v, ks, vs, torch.zeros(1, 2, dtype=torch.int64))
    with pytest.raises(TypeError):
        pk.paged_attention_multi_query_fp8(q, None, 1, k, v, ks, vs, bt, sl, 0.125)
    with pytest.raises(ValueError, match="CUDA"):
        pk.swap_blocks_fp8((k, v, ks, vs), (k, v, ks, vs), torch.zeros(1, 2, dtype=torch.int64))
    cache = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        pk.rope_and_cache(q, q[:, :2], q[:, :2], cache, cache, torch.zeros(1, dtype=torch.int64),
                          torch.zeros(1, dtype=torch.int64), None)
