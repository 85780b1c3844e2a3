"""Host checks of the self-test of the second look at the lengths.  CPU only."""
import torch

from test_abi_tree import CROSS, NULL, OK, _attention_faults, _call, lib  # noqa: F401  (lib: a fixture)


def test_stale_lengths_host_validation(lib):  # noqa: F811
    names = CROSS[:-3] + ["stale", "stale_cu"] + CROSS[-3:]
    base = dict(OK, stale="p", stale_cu="p")

    def call(**kw):
        return _call(lib.pk_selftest_cross_stale_lengths, names, base, **kw)
    _attention_faults(call)
    assert call(stale=NULL) == -1 and call(stale_cu=NULL) == -1 and call(stale=NULL, n=0) == -1
    if not torch.cuda.is_available():
        assert call() == -7
