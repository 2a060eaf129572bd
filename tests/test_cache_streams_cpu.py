"""Streams that the cache's calls refuse, without a GPU."""
import types

import pytest
import torch

from tests.test_cache_cpu import _Fake, _fake_cache


def queries():
    q = _Fake((3, 2, 1, 64), torch.bfloat16)
    q.requires_grad = False
    return q


CALLS = [lambda c, s: c.attention(queries(), stream=s), lambda c, s: c.write(queries(), queries(), stream=s),
         lambda c, s: c.read(4, stream=s)]


@pytest.mark.parametrize("call", CALLS)
def test_streams_of_another_device_are_refused(call):
    with pytest.raises(ValueError, match="stream is on cuda:1"):
        call(_fake_cache(), types.SimpleNamespace(device=torch.device("cuda", 1), cuda_stream=77))


@pytest.mark.parametrize("call", CALLS)
def test_the_per_thread_default_stream_is_refused(call):
    """Its handle, 2, is the same in every thread: their calls would share a workspace on different streams."""
    for stream in (2, types.SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=2)):
        with pytest.raises(ValueError, match="per-thread"):
            call(_fake_cache(), stream)
