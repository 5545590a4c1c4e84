"""Host side of the Python binding, with CUDA's calls replaced: runs on a machine without a GPU."""
from types import SimpleNamespace

import pytest


@pytest.fixture(scope="module")
def api():
    from chunk_sparse_moe_b200 import build
    build.build()
    from chunk_sparse_moe_b200 import api
    return api


def test_current_stream_with_and_without_the_raw_handle(api, monkeypatch):
    import torch
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: SimpleNamespace(cuda_stream=100 + d))
    monkeypatch.setattr(api, "_raw_stream", lambda d: 200 + d)
    assert api._stream() == 203
    monkeypatch.setattr(api, "_raw_stream", None)
    assert api._stream() == 103
