"""Writes into blocks whose scale the caller has set: any positive number, not only the powers of two that a
write itself chooses."""
import numpy as np
import pytest
import torch

from tests.cache_util import codes_of, make, to_f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("scale", [0.75, 3.0, 1.0, 0.625, 7 * 2.0 ** -9, 1.3])
@pytest.mark.parametrize("D,n", [(64, 1), (128, 3), (128, 60)])
def test_codes_under_a_scale_of_the_caller(scale, D, n):
    """code = x / s to nearest even, ties among them: x = s (m + 1/2) steps wherever bf16 holds it."""
    cache, table = make(1, 2, D, 64, 64, seed=5)
    first = 4  # tokens that stand in the block, codes of 0 under `scale`
    scale = float(np.float32(scale))
    page = table[0][0]
    for name in ("k", "v"):
        getattr(cache, name).view(torch.uint8)[page, :, :first] = 0
        getattr(cache, name + "_scale")[page] = scale
    g = torch.Generator().manual_seed(3)
    odd = 2 * torch.randint(8, 16, (1, 2, n, D), generator=g) + 1  # 17 .. 31: halfway between two codes
    x = (odd * 2.0 ** torch.randint(-4, 4, odd.shape, generator=g).double() * scale * torch.sign(torch.randn(odd.shape, generator=g)))
    x = x.bfloat16()
    cache.seq_lens.fill_(first + n)
    cache.write(x.cuda(), -x.cuda(), check_status=True)
    for name, sign in (("k", 1), ("v", -1)):
        assert (getattr(cache, name + "_scale")[page] == scale).all()
        got = to_f64(getattr(cache, name)[page].float())
        assert (got[:, :first] == 0).all()
        assert np.array_equal(got[:, first:first + n], codes_of(sign * to_f64(x)[0] / scale))
