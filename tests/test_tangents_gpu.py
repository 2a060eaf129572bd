"""Forward-mode tangents: no call carries them, so a dual tensor is refused instead of losing its own."""
import pytest
import torch
from torch.autograd import forward_ad

from causal_scaled_dot_gb300.kv_cache import KVCache
from causal_scaled_dot_gb300.rotary import Rotary
from tests.cache_util import rows

pytestmark = pytest.mark.gpu
D = 64


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def dual(t):
    return forward_ad.make_dual(t, torch.ones_like(t))


@pytest.mark.parametrize("which", ["q", "k", "q_norm", "k_norm"])
@pytest.mark.parametrize("recorded", [False, True])
def test_rotation_refuses_them(which, recorded):
    r, x = Rotary.from_base(D), rows((1, 9, 4 * D), 2).cuda()
    h = x.unflatten(2, (4, D)).transpose(1, 2)
    given = dict(q=h[:, :2], k=h[:, 2:3], q_norm=torch.ones(D, device="cuda"), k_norm=torch.ones(D, device="cuda"))
    if recorded:
        given["q_norm"].requires_grad_()
    want = r.rotate(**given)
    with forward_ad.dual_level():
        with pytest.raises(ValueError, match="tangent"):
            r.rotate(**{**given, which: dual(given[which])})
        with pytest.raises(ValueError, match="tangent"):
            norms = {n: dual(t) if n == which else t for n, t in given.items() if n in ("q_norm", "k_norm")}
            r.heads(x if which.endswith("norm") else dual(x), 2, 1, **norms)
        for a, b in zip(r.rotate(**given), want):  # a level alone is no matter
            assert torch.equal(a, b)


@pytest.mark.parametrize("which", ["q", "k", "v", "q_norm", "k_norm"])
def test_the_append_refuses_them(which):
    cache, r = KVCache.empty(1, 1, D, 64), Rotary.from_base(D)
    cache.seq_lens.add_(9)
    h = rows((1, 9, 4 * D), 2).cuda().unflatten(2, (4, D)).transpose(1, 2)
    given = dict(q=h[:, :2], k=h[:, 2:3], v=h[:, 3:], q_norm=torch.ones(D, device="cuda"), k_norm=torch.ones(D, device="cuda"))
    before = cache.k.view(torch.uint8).clone()
    with forward_ad.dual_level():
        with pytest.raises(ValueError, match="tangent"):
            cache.append(rotary=r, **{**given, which: dual(given[which])})
        assert torch.equal(cache.k.view(torch.uint8), before)
        cache.append(rotary=r, **given)


def test_the_caches_other_calls_refuse_them():
    cache = KVCache.empty(1, 1, D, 64)
    cache.seq_lens.add_(9)
    q, k = (rows((1, H, 9, D), 2 + H).cuda() for H in (2, 1))
    with forward_ad.dual_level():
        for call in (lambda: cache.write(dual(k), k), lambda: cache.write(k, dual(k)), lambda: cache.attention(dual(q))):
            with pytest.raises(ValueError, match="tangent"):
                call()
        cache.write(k, k)
        cache.attention(q)
