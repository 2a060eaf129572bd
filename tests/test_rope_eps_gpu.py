"""Norms whose eps is as large as the rows: every finite eps counts, also beside rows whose squares pass fp32."""
import numpy as np
import pytest
import torch

from causal_scaled_dot_gb300.kv_cache import KVCache
from causal_scaled_dot_gb300.rotary import Rotary
from tests import rope_util
from tests.cache_util import rows, scale_of
from tests.rope_util import to_f64
from tests.test_rope_gpu import split, weights

pytestmark = pytest.mark.gpu
B, S, HQ, HKV = 2, 37, 3, 2
LARGEST = float(torch.finfo(torch.float32).max)


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def projected(D, sigma):
    """Rows of magnitudes about sigma, sequence by sequence and token by token from 2^-8 to 2^2 of it."""
    x = rows((B, S, (HQ + 2 * HKV) * D), D, sigma)
    return (x.float() * torch.logspace(-8, 2, B * S, base=2).round(decimals=3).view(B, S, 1)).to(torch.bfloat16)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("sigma", [1.0, 2.0 ** 60, 2.0 ** 63])
@pytest.mark.parametrize("eps", [1e-6, 2.0 ** 100, 2.0 ** 121, 2.0 ** 126, LARGEST])
def test_large_eps(D, interleaved, sigma, eps):
    r, x = Rotary.from_base(D, interleaved=interleaved), projected(D, sigma)
    w = weights(D, torch.float32)
    more = dict(q_norm=w[0].cuda(), k_norm=w[1].cuda(), eps=eps)
    qkv, at = x.cuda(), np.broadcast_to(np.arange(S), (B, S))
    q, k, v = r.heads(qkv, HQ, HKV, **more)
    up = [rows(t.shape, 7 + i).cuda() for i, t in enumerate((q, k, v))]
    dx, dwq, dwk = r.heads_backward(*up, qkv, HQ, HKV, **more)
    eps = float(np.float32(eps))
    for got, g, dy, dw, one, wt in zip((q, k), split(dx.cpu(), HQ, HKV), up, (dwq, dwk), split(x, HQ, HKV), w):
        want, tol, _ = rope_util.forward(one, at, r, to_f64(wt), eps)
        assert (np.abs(to_f64(got) - want) <= tol).all()
        want, tol, want_w, tol_w = rope_util.backward(to_f64(dy), one, at, r, to_f64(wt), eps)
        assert (np.abs(g - want) <= tol).all()
        assert (np.abs(to_f64(dw) - want_w) <= tol_w).all()
    # and on the way into the cache
    cache = KVCache.empty(B, HKV, D, S, block_size=16)
    cache.seq_lens.add_(S)
    h = qkv.unflatten(2, (HQ + 2 * HKV, D)).transpose(1, 2)
    cq = cache.append(h[:, HQ:HQ + HKV], h[:, HQ + HKV:], r, q=h[:, :HQ], check_status=True, **more)
    assert torch.equal(cq, q)
    y, _, fp32 = rope_util.forward(split(x, HQ, HKV)[1], at, r, to_f64(w[1]), eps)
    held = to_f64(cache.read(S)[0])
    for b in range(B):
        for head in range(HKV):
            for first in range(0, S, 16):
                one = (b, head, slice(first, first + 16))
                tol = np.maximum(2.0 ** -4 * np.abs(y[one]), 2.0 ** -10 * scale_of(y[one])) + fp32[one]
                assert (np.abs(held[one] - y[one]) <= tol).all()
