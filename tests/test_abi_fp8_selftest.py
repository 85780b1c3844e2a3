"""Host checks of the 8-bit decode's self-tests (CPU: nothing is launched)."""
import torch

from test_abi_fp8 import DECODE, DECODE_OK, NULL, _call, lib  # noqa: F401


def test_wait_timeout_host_validation(lib):  # noqa: F811
    names = DECODE[:-1] + ["stall", "limit", "st"]

    def call(**kw):
        return _call(lib.pk_selftest_decode_fp8_wait_timeout, names, dict(DECODE_OK, stall=1, limit=5000), **kw)
    assert call(stall=0) == -2 and call(stall=-3) == -2
    assert call(limit=50) == -2 and call(limit=2000000) == -2
    assert call(d=96) == -3 and call(ksc=NULL) == -1            # then the decode call's own checks
    assert call(n=0) == 0
    if not torch.cuda.is_available():
        assert call() == -7


def test_stale_lengths_host_validation(lib):  # noqa: F811
    names = DECODE[:-3] + ["stale"] + DECODE[-3:]

    def call(**kw):
        return _call(lib.pk_selftest_decode_fp8_stale_lengths, names, dict(DECODE_OK, stale="p"), **kw)
    assert call(stale=NULL) == -1
    assert call(d=96) == -3 and call(q=("o", 2)) == -6
    assert call(n=0) == 0
    if not torch.cuda.is_available():
        assert call() == -7
