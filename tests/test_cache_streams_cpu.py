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
