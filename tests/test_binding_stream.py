"""The binding's look-up of the current stream, on any machine (torch's side is a stand-in)."""
import types

import pytest

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("missing", ["_cuda_getCurrentRawStream", "_cuda_getDevice"])
def test_without_torchs_private_calls_the_public_one_serves(monkeypatch, missing):
    import zero_sharded_mixed_shard_gb300 as z
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 55, raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: types.SimpleNamespace(cuda_stream=77))
    assert z._stream(None) == 55
    monkeypatch.delattr(torch._C, missing)
    assert z._stream(None) == 77


def test_a_stream_that_is_given_is_taken(monkeypatch):
    import zero_sharded_mixed_shard_gb300 as z
    monkeypatch.setattr(torch.cuda, "current_stream", None)
    assert z._stream(12) == 12 and z._stream(types.SimpleNamespace(cuda_stream=34)) == 34
