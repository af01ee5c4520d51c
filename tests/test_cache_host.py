"""Refusals of KVCache, whatever GPUs are there: its tensors are stood in for."""
import types

import pytest
import torch

from block_diffusion_speculative_draft_gb300 import api

SHAPE = types.SimpleNamespace(L=1, nkv=2, d=64)


@pytest.fixture(autouse=True)
def no_gpu(monkeypatch):
    """Allocations on a CUDA device become shapes without memory; cuda:0 is current."""
    zeros = torch.zeros

    def shape_only(*size, dtype=None, device=None):
        t = zeros(*size, dtype=dtype, device="meta")
        return types.SimpleNamespace(dtype=t.dtype, shape=t.shape, device=torch.device(device), data_ptr=lambda: 256)

    monkeypatch.setattr(api, "_torch_module", torch)
    monkeypatch.setattr(torch, "zeros", shape_only)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)


def _len(device, dtype=torch.int32, b=2):
    return types.SimpleNamespace(dtype=dtype, shape=(b,), is_contiguous=lambda: True, device=torch.device(device),
                                 is_cuda=torch.device(device).type == "cuda", data_ptr=lambda: 256)


@pytest.mark.parametrize("device,where", [("cuda:1", "cuda:0"), ("cuda:0", "cuda:1"), ("cuda", "cuda:1"), (1, "cuda:0"),
                                          (torch.device("cuda", 1), "cuda:0"), ("cuda", "cpu")])
def test_lengths_on_another_device_than_the_cache(device, where):
    with pytest.raises(ValueError, match="len"):
        api.KVCache(SHAPE, 2, 16, device, len=_len(where))


@pytest.mark.parametrize("device,where", [("cuda:1", "cuda:1"), ("cuda", "cuda:0"), (1, "cuda:1"),
                                          (torch.device("cuda"), "cuda:0")])
def test_lengths_on_the_cache_s_device(device, where):
    given = _len(where)
    assert api.KVCache(SHAPE, 2, 16, device, len=given).len is given


def test_lengths_of_another_type_or_shape():
    for bad in (_len("cuda:0", dtype=torch.int64), _len("cuda:0", b=3)):
        with pytest.raises(ValueError, match="len"):
            api.KVCache(SHAPE, 2, 16, "cuda:0", len=bad)
