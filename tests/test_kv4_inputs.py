"""Inputs of the 4-bit cache's calls: taken as they are where they fit the ABI, copied where they do not (no GPU)."""
import pytest
import torch

from head_dim_flash_gb300 import api


def at(shape, off):
    """A contiguous tensor that begins `off` elements into an aligned allocation."""
    n = 1
    for s in shape:
        n *= s
    x = torch.arange(n + 16, dtype=torch.float32).to(torch.bfloat16)
    assert x.data_ptr() % 16 == 0
    return x[off:off + n].view(shape)


@pytest.mark.parametrize("off", [0, 1, 4, 8])
def test_dense_inputs(off):
    x = at((2, 2, 5, 64), off)
    y, view = api._in_view(x)
    assert torch.equal(x, y) and view.data == y.data_ptr() and y.data_ptr() % 16 == 0
    assert (y is x) == (off % 8 == 0)
    t = x.transpose(1, 2)
    y, view = api._in_view(t)
    assert torch.equal(t, y) and y.data_ptr() % 16 == 0
    assert (y is t) == (off % 8 == 0)


@pytest.mark.parametrize("off", [0, 1, 4, 8])
def test_packed_inputs(off):
    x = at((7, 2, 64), off)
    y = api._in_packed(x)
    assert torch.equal(x, y) and y.is_contiguous() and y.data_ptr() % 16 == 0
    assert (y is x) == (off % 8 == 0)
    t = at((7, 4, 64), off)[:, 1:3]   # heads of a wider tensor
    y = api._in_packed(t)
    assert torch.equal(t, y) and y.is_contiguous() and y.data_ptr() % 16 == 0


def test_the_decode_workspace_is_in_the_package():
    import head_dim_flash_gb300 as ffpa

    assert ffpa.decode_kv4_workspace is api.decode_kv4_workspace and "decode_kv4_workspace" in ffpa.__all__
    for name in ffpa.__all__:
        assert hasattr(ffpa, name)


def test_the_current_stream_without_torchs_private_name(monkeypatch):
    import importlib.util
    import types

    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device: types.SimpleNamespace(cuda_stream=100 + device))
    spec = importlib.util.spec_from_file_location("head_dim_flash_gb300.api_again", api.__file__)
    again = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(again)
    assert again._raw_stream(torch.device("cuda", 3)) == 103
