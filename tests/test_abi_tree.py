"""Host checks of tree verification and cross attention.  CPU only: every call fails
validation, is a no-op, or finds no device."""
import ctypes
import os
import re

import pytest
import torch

import paged_kv_cache_122_gb300 as pk
from conftest import ROOT
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


def test_every_declared_call_is_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "pagedkv_tree.h")).read(), flags=re.S)
    names = set(re.findall(r"\b(pk_[a-z_0-9]+)\s*\(", text))
    assert {"pk_paged_attention_tree", "pk_paged_attention_cross", "pk_accept_tree", "pk_keep_tokens_layers"} <= names
    for n in names:
        assert hasattr(lib, n) and n in _native.SIGNATURES


CROSS = ["out", "dt", "q", "tq", "cu", "mq", "k", "v", "bt", "mb", "sl", "ms", "n", "h", "hkv", "d", "nb", "b", "scale", "ws",
         "wb", "st"]
OK = dict(out="p", dt=0, q="p", tq=8, cu="p", mq=4, k="p", v="p", bt="p", mb=32, sl="p", ms=512, n=2, h=8, hkv=2, d=128, nb=64,
          b=16, scale=0.1, ws="p", wb=1 << 30, st=None, mask="p", mw=1, stall=1, limit=1000)
TREE = CROSS[:6] + ["mask", "mw"] + CROSS[6:]


def _attention_faults(call):
    assert call(d=96) == -3 and call(b=12, ms=64) == -3 and call(dt=7) == -3 and call(h=6, hkv=2) == -3
    assert call(h=7) == -2 and call(n=-1) == -2 and call(tq=-1) == -2 and call(mq=-1) == -2 and call(ms=-1) == -2
    assert call(ms=513) == -2 and call(n=65536) == -2 and call(nb=-1) == -2 and call(hkv=0) == -2
    assert call(scale=float("nan")) == -2 and call(scale=float("inf")) == -2
    for name in ("out", "q", "cu", "k", "v", "bt", "sl"):
        assert call(**{name: NULL}) == -1, name
    for name in ("out", "q", "k", "v"):
        assert call(**{name: ("o", 8)}) == -6, name
    assert call(ws=NULL) == -4 and call(wb=1000) == -4 and call(ws=("o", 8)) == -6
    assert call(n=0) == 0 and call(tq=0) == 0 and call(mq=0) == 0
    if not torch.cuda.is_available():
        assert call() == -7
        assert call(ms=128, ws=NULL, wb=0) == -7              # one tile: nothing is cut
        assert call(ms=0, k=NULL, v=NULL, bt=NULL, ws=NULL, wb=0) == -7


def test_attention_host_validation(lib):
    _attention_faults(lambda **kw: _call(lib.pk_paged_attention_cross, CROSS, OK, **kw))

    def tree(**kw):
        return _call(lib.pk_paged_attention_tree, TREE, OK, **kw)
    _attention_faults(tree)
    assert tree(mask=NULL) == -1 and tree(mask=("o", 4)) == -6
    assert tree(mw=0) == -2 and tree(mq=65) == -2 and tree(mw=-1) == -2 and tree(mw=1 << 30) == -2
    if not torch.cuda.is_available():
        assert tree(mq=65, mw=2) == -7 and tree(mask=("o", 8)) == -7
    test = CROSS[:-1] + ["stall", "limit", "st"]
    for bad in (dict(stall=0), dict(limit=99), dict(limit=1000001)):
        assert _call(lib.pk_selftest_cross_wait_timeout, test, OK, **bad) == -2


def test_workspace_bytes(lib):
    f = lib.pk_tree_workspace_bytes
    one, two = f(32, 8, 128, 32, 4096), f(32, 8, 128, 33, 4096)
    assert one == 2 * 160 * (64 + 4 * 128 * (2 + 128)) and two == 2 * 160 * (64 + 2 * 4 * 128 * (2 + 128))
    assert f(8, 8, 64, 128, 129) == 2 * 160 * (64 + 4 * 128 * (2 + 64))
    assert f(32, 8, 128, 32, 128) == 0 and f(32, 8, 96, 32, 4096) == 0 and f(32, 7, 128, 32, 4096) == 0
    assert f(24, 8, 128, 32, 4096) == 0 and f(32, 8, 128, 0, 4096) == 0 and f(0, 0, 128, 1, 4096) == 0


ACC = ["acc", "num", "next", "lens", "tok", "par", "tgt", "tq", "cu", "mq", "sl", "n", "st"]
ACC_OK = dict(acc="p", num="p", next="p", lens="p", tok="p", par="p", tgt="p", tq=8, cu="p", mq=4, sl="p", n=2, st=None)
KEEP = ["k", "v", "bt", "mb", "sl", "cu", "acc", "stride", "num", "n", "hkv", "d", "nb", "b", "st"]
KEEP_OK = dict(k="p", v="p", bt="p", mb=4, sl="p", cu="p", acc="p", stride=4, num="p", n=2, hkv=2, d=64, nb=9, b=8, st=None, l=3)


def test_accept_and_keep_host_validation(lib):
    def acc(**kw):
        return _call(lib.pk_accept_tree, ACC, ACC_OK, **kw)
    assert acc(mq=8193) == -3 and acc(tq=-1) == -2 and acc(mq=-1) == -2 and acc(n=-1) == -2 and acc(n=0) == 0
    for name in ("acc", "num", "next", "lens", "tok", "par", "tgt", "cu", "sl"):
        assert acc(**{name: NULL}) == -1, name

    def keep(**kw):
        return _call(lib.pk_keep_tokens, KEEP, KEEP_OK, **kw)
    layers = KEEP[:10] + ["l"] + KEEP[10:]

    def keep_layers(**kw):
        return _call(lib.pk_keep_tokens_layers, layers, KEEP_OK, **kw)
    for call in (keep, keep_layers):
        assert call(d=96) == -3 and call(b=4) == -3 and call(n=-1) == -2 and call(n=65536) == -2 and call(hkv=0) == -2
        assert call(stride=-1) == -2 and call(mb=-1) == -2 and call(nb=-1) == -2
        for name in ("k", "v", "bt", "sl", "cu", "acc", "num"):
            assert call(**{name: NULL}) == -1, name
        assert call(n=0) == 0 and call(stride=0) == 0
        if not torch.cuda.is_available():
            assert call() == -7
    assert keep(k=("o", 8)) == -6
    assert keep_layers(l=-1) == -2 and keep_layers(l=32768) == -2 and keep_layers(l=0) == 0
    if not torch.cuda.is_available():
        assert acc() == -7


def test_binding_wants_cuda_tensors_of_the_right_types():
    q = torch.zeros(4, 4, 64, dtype=torch.bfloat16)
    kc = torch.zeros(4, 8, 2, 64, dtype=torch.bfloat16)
    i32 = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pk.paged_attention_cross(q, i32, 2, kc, kc, torch.zeros(1, 4, dtype=torch.int32), i32[:1], 1.0)
    with pytest.raises(TypeError):
        pk.paged_attention_tree(q.float(), i32, 2, torch.zeros(4, 1, dtype=torch.int64), kc, kc,
                                torch.zeros(1, 4, dtype=torch.int32), i32[:1], 1.0)
    with pytest.raises(ValueError, match="CUDA"):
        pk.accept_tree(torch.zeros(4, dtype=torch.int64), torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int64),
                       i32, 2, i32[:1])
    with pytest.raises(TypeError):
        pk.accept_tree(None, None, None, None, 2, None)
    with pytest.raises(ValueError, match="CUDA"):
        pk.keep_tokens(kc, kc, torch.zeros(1, 4, dtype=torch.int32), i32[:1], i32, torch.zeros(1, 2, dtype=torch.int32), i32[:1])
