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


def test_device_status_goes_to_the_workspace_s_device(api, monkeypatch):
    """A workspace on another device than the current one: its device is current for the call, and the stream
    that is waited for is that device's."""
    import torch
    now, seen = [0], []

    class On:
        def __init__(self, device):
            self.device = device

        def __enter__(self):
            self.before, now[0] = now[0], self.device.index

        def __exit__(self, *a):
            now[0] = self.before

    def status(ptr, stream, detail):
        seen.append((ptr, stream, now[0]))
        return 4

    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", On)
    monkeypatch.setattr(api, "_raw_stream", lambda d: 200 + d)
    monkeypatch.setattr(api, "lib", SimpleNamespace(blockffn_get_device_status=status))
    ws = lambda i: SimpleNamespace(buf=SimpleNamespace(device=SimpleNamespace(index=i), data_ptr=lambda: 256))  # noqa: E731
    assert api.device_status(ws(0)) == (4, 0) and api.device_status(ws(1)) == (4, 0)
    assert seen == [(256, 200, 0), (256, 201, 1)] and now == [0]
