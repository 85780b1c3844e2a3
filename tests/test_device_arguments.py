"""Devices named without an index, or by a string, wherever a call takes a device."""
import subprocess
import sys

import pytest
import torch

from conftest import ROOT
from paged_kv_cache_122_gb300 import api


class _Stream:
    cuda_stream = 77


def test_a_device_without_an_index_means_the_current_one(monkeypatch):
    asked = []

    def raw(index):
        assert type(index) is int, f"invalid argument {index!r}"
        asked.append(index)
        return 40 + index
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", raw, raising=False)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 2)
    assert api._raw_stream(torch.device("cuda", 1)) == 41
    assert api._raw_stream(torch.device("cuda")) == 42
    assert api._raw_stream("cuda:3") == 43 and api._raw_stream("cuda") == 42
    assert api._raw_stream(torch.device("cuda"), _Stream()) == 77
    assert asked == [1, 2, 3, 2]


@pytest.mark.gpu
@pytest.mark.parametrize("device", [None, "cuda", "cuda:0", torch.device("cuda"), torch.device("cuda", 0), 0])
def test_the_error_word_of_any_spelling(device):
    import paged_kv_cache_122_gb300 as pk
    assert pk.pk_get_device_error(device) == 0
    k = torch.zeros(2, 8, 1, 64, dtype=torch.bfloat16, device="cuda:0")
    pk.copy_blocks(k, k.clone(), torch.tensor([[0, 9]], device="cuda:0"))
    assert pk.pk_get_device_error(device) == pk._native.DEVERR_PAIR
    assert pk.pk_get_device_error(device) == 0


@pytest.mark.gpu
def test_workspaces_of_any_spelling():
    for device in ("cuda", "cuda:0", torch.device("cuda"), torch.device("cuda", 0)):
        ws = api.workspace_for(device, 1000)
        assert ws.device == torch.device("cuda", 0) and ws.numel() >= 1000
        assert api.workspace_for(device, 10) is ws


@pytest.mark.gpu
@pytest.mark.parametrize("device", ["cuda", "cuda:0"])
def test_as_the_first_call_of_a_process(device):
    code = f"import paged_kv_cache_122_gb300 as pk; print(pk.pk_get_device_error({device!r}))"
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert out.returncode == 0 and out.stdout.split() == ["0"], out.stderr
