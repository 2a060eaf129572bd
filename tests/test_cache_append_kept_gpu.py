"""What an append writes of V and of both scales, bit for bit, and that everything else in the cache keeps its bits."""
import numpy as np
import pytest
import torch

from causal_scaled_dot_gb300.rotary import Rotary
from tests.cache_util import PlainCache, make, to_f64
from tests.test_cache_append_gpu import CACHES, projected
from tests.test_cache_gpu import ints, set_lens
from tests.test_rope_gpu import weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def bits(cache):
    """Copies of k, v, k_scale and v_scale as whole numbers."""
    return [t.view(torch.uint8 if t.element_size() == 1 else torch.int32).cpu().numpy().copy()
            for t in (cache.k, cache.v, cache.k_scale, cache.v_scale)]


@pytest.mark.parametrize("D,block", CACHES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [None, torch.bfloat16])
def test_written_and_kept(D, block, interleaved, norm):
    """Uneven prompts, a padded chunk, single tokens; one slot idle, spare blocks, codes and scales of NaN before."""
    B, Hq, Hkv = 3, 4, 2
    r = Rotary.from_base(D, interleaved=interleaved)
    w = [t.cuda() for t in weights(D, norm)] if norm else (None, None)
    cache, table = make(B, Hkv, D, block, 400, seed=2 * D + block)
    plain, lens = PlainCache(cache.k.shape[0], Hkv, block, D), [0] * B
    for step, new in enumerate(([150, 0, 37], [70, 0, 101], [1, 0, 1], [1, 0, 1], [3, 0, 2])):
        lens = [t + n for t, n in zip(lens, new)]
        set_lens(cache, lens)
        before = bits(cache)
        q, k, v = projected(B, max(new), Hq, Hkv, D, 50 + step)
        v = v * 4.0 ** step  # the blocks' scales rise
        cache.append(k, v, r, q=q, new_lens=ints(new), q_norm=w[0], k_norm=w[1], check_status=True)
        after = bits(cache)
        plain.write(np.zeros(v.shape), to_f64(v), table, lens, new)
        rows, pages = np.zeros(cache.k.shape[:1] + (block,), bool), np.zeros(cache.k.shape[0], bool)
        for b, (t, n) in enumerate(zip(lens, new)):
            for i in range((t - n) // block, -(-t // block)) if n else ():
                pages[table[b][i]] = True
                rows[table[b][i], :min(block, t - i * block)] = True
        for x, y in zip(before[:2], after[:2]):
            assert np.array_equal(x.transpose(0, 2, 1, 3)[~rows], y.transpose(0, 2, 1, 3)[~rows])
        for x, y in zip(before[2:], after[2:]):
            assert np.array_equal(x[~pages], y[~pages])
        assert np.array_equal(to_f64(cache.v_scale)[pages], plain.v_scale[pages])
        got, want = to_f64(cache.v.float()).transpose(0, 2, 1, 3)[rows], plain.v.transpose(0, 2, 1, 3)[rows]
        assert np.array_equal(got, want, equal_nan=True)
        assert np.isfinite(to_f64(cache.k_scale)[pages]).all()
