"""A call without a stream runs on torch's current one."""

import pytest
import torch

pytestmark = pytest.mark.gpu


def test_the_current_stream_is_followed(cuda, monkeypatch):
    from attention_kv_cache_gb300 import kvsel as K
    for raw in (None, lambda device: 0):                 # torch's own getter, and one that answers 0 always
        with monkeypatch.context() as m:
            if raw is not None:
                m.setattr(torch._C, "_cuda_getCurrentRawStream", raw, raising=False)
            m.setattr(K, "_current_stream", None)
            for s in (torch.cuda.default_stream(), torch.cuda.Stream(), torch.cuda.Stream()):
                with torch.cuda.stream(s):
                    assert K._stream(None) == K._stream(None) == s.cuda_stream
            assert K._stream(None) == torch.cuda.current_stream().cuda_stream


def test_a_first_call_within_a_capture(cuda, monkeypatch):
    from attention_kv_cache_gb300 import kvsel as K
    torch.cuda.synchronize()
    x, g = torch.zeros(4, device=cuda), torch.cuda.CUDAGraph()
    with monkeypatch.context() as m:
        m.setattr(K, "_current_stream", None)
        with torch.cuda.graph(g):
            assert K._stream(None) == torch.cuda.current_stream().cuda_stream
            x += 1
        assert K._current_stream is None
    g.replay()
    assert x.tolist() == [1.0] * 4
