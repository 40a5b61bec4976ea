"""Which stream's memory a workspace that the binding allocates comes from, without a GPU: torch's allocator is
replaced by one that notes the stream it is called under."""
import contextlib
import types

import pytest
import torch

from causal_prefix_scan_hla2_amd import hla2 as H


@pytest.fixture
def taken(monkeypatch):
    """The streams under which torch.empty was called (None: the current one)."""
    now, seen, empty = [None], [], torch.empty

    @contextlib.contextmanager
    def under(s):
        now.append(s)
        yield
        now.pop()

    def fake_empty(n, dtype, device):
        seen.append(now[-1])
        return empty(n, dtype=dtype)

    monkeypatch.setattr(torch.cuda, "stream", under)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda ptr, device: ("external", ptr, device))
    monkeypatch.setattr(torch, "empty", fake_empty)
    return seen


LIKE = types.SimpleNamespace(device=torch.device("cuda", 0), is_cuda=True, get_device=lambda: 0)
STREAM = types.SimpleNamespace(cuda_stream=4096, device_index=0)


def test_the_workspace_belongs_to_the_calls_stream(taken):
    for stream in (None, STREAM, 4096, 0):
        ws, n = H._workspace(None, 512, LIKE, stream)
        assert n == 512 == ws.numel()
    assert taken == [None] + [("external", ptr, LIKE.device) for ptr in (4096, 4096, 0)]


def test_no_workspace_is_taken_where_none_is_needed(taken):
    assert H._workspace(None, 0, LIKE, STREAM) == (None, 0) and not taken


def test_a_stream_of_another_device_is_refused():
    with pytest.raises(ValueError, match="stream"):
        H._launch("hla2_gated_scan_step", True, LIKE, types.SimpleNamespace(cuda_stream=4096, device_index=1))


class Stub:
    """A library whose every call succeeds and whose every workspace is 64 bytes (or floats)."""

    def __getattr__(self, name):
        return lambda *args: 64 if name.endswith("_bytes") or name.endswith("_floats") else 0


X = torch.zeros(1, 1, 4, 8)
CALLS = {
    "forward": lambda s: H.hla2_forward(X, X, X, X, stream=s),
    "state": lambda s: H.hla2_forward_state(X, X, X, X, torch.zeros(64), stream=s),
    "backward": lambda s: H.hla2_backward(X, X, X, X, X, X, X, stream=s),
    "ahla": lambda s: H.hla2_ahla_forward(X, X, X, X, stream=s),
    "ho3": lambda s: H.hla2_ho3_forward(X, X, X, X, stream=s),
}


@pytest.mark.parametrize("call", CALLS)
def test_every_call_takes_its_workspace_so(call, monkeypatch):
    seen = []
    monkeypatch.setattr(H, "lib", Stub)
    monkeypatch.setattr(H, "_scratch", lambda need, like, stream: seen.append((need, stream)) or torch.zeros(need, dtype=torch.uint8))
    assert CALLS[call](STREAM) == 0
    assert seen == [(64, STREAM)]
